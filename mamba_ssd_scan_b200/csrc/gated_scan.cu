// gated_scan.cu -- the gated linear recurrence, its gradient and its decode
// step (the formulas stand in include/ssd.h).
//
// A step h <- a h + u is an affine map, and maps compose: (A, H) after (A', H')
// is (A A', A H' + H).  So a sequence is cut into groups of 8 consecutive
// tokens (4 in the fp32 forward), each thread composes its group's maps, and the
// groups' maps are composed in turn.  The forward keeps the maps from the group's
// start up to each token in registers: a token's state is then one packed operation
// on the state that enters the group.  The gradient replays its group from there.
// The gates (about 4 special-function results per element) are formed once and the
// inputs are read once.
//
// A compute warp takes one group of tokens of 64 channels (a pair per lane);
// the 8 compute warps of a CTA take consecutive groups (a tile of 64 tokens; 32 in
// the fp32 forward), and the CTAs of a cluster consecutive tiles.  A ninth warp
// composes the tile's map, sends it to the cluster's CTAs through distributed shared memory
// (asynchronous stores that complete on the receiver's mbarrier), and hands
// each group its entering state.  The order of composition is fixed, so
// results do not depend on timing; there is no workspace and no wait on another
// cluster.  Every mbarrier wait is bounded: on expiry the CTA raises its abort
// flag, finishes without waiting, and the call's status reads SSD_ERR_TIMEOUT.
//
// Measured (B200, L2 flushed; share of the measured copy bandwidth over the
// call's least bytes).  Forward, bf16: b6 L4096 C4736 174 us (83 %), b8 L4096
// C2048 127 us (66 %), with eight restarts a row 150; b1 L65536 C1536 227 us (55
// %); fp32: b8 L4096 C2048 199 us (84 %).  Gradient, bf16: b4 L4096 C4736 226 us (75
// %), b8 L4096 C2048 224 us (65 %), with eight restarts a row 263; b1 L65536 C1536
// 421 us (52 %); fp32: b8 L4096 C2048 390 us (75 %).  These have the usual decays,
// 0.9 to 0.999 at the open gate.  Where a warp's channels reach decays below e^-1/4
// (drawn from 0.3 to 0.999) its other code runs: b8 L4096 C2048 bf16 145 us, with
// restarts 172, the gradient 276 and 314; b1 L65536 C1536 262 and 511; fp32 213 and
// 421.  Groups of 16 tokens at two CTAs per SM measured 220 us at b6 C4736, groups of
// four at four CTAs 203 (172 then).  Where the CTAs fill the SMs evenly the forward
// is bound by its instructions (55 per channel pair and token; issue slots 54 % busy,
// the special-function pipe 63 %) as much as by its bytes.  Neither binds the
// gradient: at b8 C2048 its bytes take 146 us and its instructions 120 (issue 54 %);
// it waits, with 14.7 warps on an SM, which its 96 registers a thread allow (9
// warps, two CTAs; it spills 8 to 16 bytes there, the forward with restarts 16 at
// 72).  b8 C2048 is 256 CTAs on 148 SMs, a third of which take one where the others
// take two; halves of the sequence in clusters of two cost more than they even out.
// Long sequences of few channels wait for the exchange, once per round.
#include <atomic>
#include <type_traits>
#include <utility>
#include "mixers.h"
#include "tcgen05.cuh"
#include "rows_tma.cuh"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int kInterval = SSD_GATED_SCAN_INTERVAL;
constexpr int NW = 8;                   // groups per CTA, a warp each
constexpr int kThreads = (NW + 1) * 32;  // and the warp that moves tiles and composes maps
constexpr int TPT = 8;           // the gradient's tokens per group
constexpr int TILE = NW * TPT;   // and per CTA and round
static_assert(TILE == kInterval, "a tile starts where a state is kept");
constexpr int CPB = 64;          // channels per CTA
constexpr int kMaxCluster = 16;

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

__device__ __forceinline__ float ex2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sqrt_approx(float v) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// min and max that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 2^(k v) for a constant k = hi + lo in two parts.  For fp32 inputs (EXACT) it is
// cut off at 2^top and the rounding of k v (up to 2^-24 |k v| in the exponent)
// is carried along; for bf16 inputs that rounding stays well inside their own
// 2^-9, and the gates are cut off as they are read.
template <bool EXACT>
__device__ __forceinline__ float2 exp2_scaled(float2 v, float hi, float lo, float top = 126.0f) {
    if constexpr (EXACT) {  // (no infinite products)
        v = make_float2(min_nan(max_nan(v.x, -200.0f), 200.0f), min_nan(max_nan(v.y, -200.0f), 200.0f));
        const float2 t = mul2(v, dup(hi));
        const float2 e = make_float2(ex2_approx(min_nan(t.x, top)), ex2_approx(min_nan(t.y, top)));
        const float2 d = fma2(v, dup(lo), fma2(v, dup(hi), make_float2(-t.x, -t.y)));  // what t lost
        return fma2(e, mul2(d, dup(0.69314718f)), e);
    }
    const float2 t = mul2(v, dup(hi));
    return make_float2(ex2_approx(t.x), ex2_approx(t.y));
}
// log2(e) in two parts
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266174e-8f;

// A pair of gates as it lies in memory; bf16 gates no lower than `least` (two
// equal halves; NaN stays), which bounds e^-gate.
__device__ __forceinline__ float2 read_gates(float2 raw, uint32_t) { return raw; }
__device__ __forceinline__ float2 read_gates(uint32_t raw, uint32_t least) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(raw) : "r"(least));
    return Pair<__nv_bfloat16>::widen(raw);
}
// widened gates, cut off alike
template <bool EXACT> __device__ __forceinline__ float2 least_gates(float2 v, float least) {
    return EXACT ? v : make_float2(max_nan(v.x, least), max_nan(v.y, least));
}
constexpr uint32_t kLeastA = 0xC2AEC2AEu;  // -87: e^87 < 2^126
constexpr uint32_t kLeastX = 0xC226C226u;  // -41.5: e^41.5 < 2^60

// sigma of a pair of gates with one reciprocal per channel:
// 1 / ((1 + e^-a)(1 + e^-x)) times the other factor (a reciprocal each would
// make five special-function results per element, close to what the pipe
// gives in the time the bytes take).  e^-x is cut off at 2^60 (i is then off by
// 2^-60).  Where the product passes 2^126 its reciprocal is 0 and r = i = 0: the token
// counts as shut, where sqrt(r) i, the size of what it adds, is below 2^-62.
template <bool EXACT>
__device__ __forceinline__ void sigmas(float2 ga, float2 gx, float2& r, float2& i) {
    const float2 one = dup(1.0f);
    const float2 ea = add2(exp2_scaled<EXACT>(ga, -kLog2eHi, -kLog2eLo), one);
    const float2 ex = add2(exp2_scaled<EXACT>(gx, -kLog2eHi, -kLog2eLo, 60.0f), one);
    const float2 d = mul2(ea, ex);
    const float2 inv = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    r = mul2(inv, ex);
    i = mul2(inv, ea);
}

// What a token keeps of the state, as the multiplier m of two step forms.  Down to
// la = -1/4 (la = log a <= 0) m = a - 1 <= 0 and the step is h + m h: a decay near 1
// keeps its relative accuracy in la, and 1 - a^2 = -m (2 + m) is formed without
// cancellation.  Beyond, m = a > 0 and the step is m h: the little that such a
// token keeps is not rounded at the size of the whole (h + (a - 1) h was off by 6 % of
// a h at la = -16, and lost it at -20).  A decay below 2^-126 counts as 2^-149, so that m
// stays positive.  m = a - 1 is la + la^2 q, q the cubic that is nearest to
// (e^la - 1 - la) / la^2 there by m's relative error (fitted: off by 2^-28 of m; the
// series needs another term).  la never falls below the channel's own -scale
// softplus(decay), so where that is above -1/4 (SLOW; the usual decays of 0.9 to
// 0.999 at the open gate) the second form is not evaluated.  The choice is made
// once per group, not per token: a branch between the tokens kept them from
// overlapping (220 cycles per token and warp).
template <bool EXACT, bool SLOW> __device__ __forceinline__ float2 decays(float2 la) {
    float2 q = dup(0.0075347102f);
    q = fma2(q, la, dup(0.041502319f));
    q = fma2(q, la, dup(0.16665322f));
    q = fma2(q, la, dup(0.49999964f));
    float2 m = fma2(mul2(q, la), la, la);
    if constexpr (!SLOW) {
        const float2 e = exp2_scaled<EXACT>(la, kLog2eHi, kLog2eLo);
        const float least = __int_as_float(1);
        m = make_float2(la.x >= -0.25f ? m.x : max_nan(e.x, least), la.y >= -0.25f ? m.y : max_nan(e.y, least));
    }
    return m;
}
// where m is a itself (SLOW: nowhere)
struct Far {
    bool x, y;
};
template <bool SLOW> __device__ __forceinline__ Far far_of(float2 m) {
    return SLOW ? Far{false, false} : Far{m.x > 0.0f, m.y > 0.0f};
}
__device__ __forceinline__ float2 choose(Far far, float2 yes, float2 no) {
    return make_float2(far.x ? yes.x : no.x, far.y ? yes.y : no.y);
}
// a h + u, a h and a
__device__ __forceinline__ float2 step(Far far, float2 m, float2 h, float2 u) {
    return add2(choose(far, dup(0.0f), h), fma2(m, h, u));
}
__device__ __forceinline__ float2 keep(Far far, float2 m, float2 h) { return fma2(m, h, choose(far, dup(0.0f), h)); }
__device__ __forceinline__ float2 decay_of(Far far, float2 m) { return add2(m, choose(far, dup(0.0f), dup(1.0f))); }
// A multiplier that changes no state and no adjoint, infinite ones included: a = 1, or
// a - 1 = 2^-149, which adds nothing to a finite h (0 would be 0 times infinity).
template <bool SLOW> constexpr float kNothing = SLOW ? 1.401298464e-45f : 1.0f;
// 1 - a^2: of m = a - 1 as -m (2 + m), of m = a by one of two ways that cost alike.
// The forward takes 1 - m m, by other constants in the same two operations (b8 L4096
// C2048 bf16, decays from 0.3 on: 141 us, by the other way 143), the gradient goes
// through m - 1 (214 us at the usual decays, whose own code is the same but for the
// registers that it is left; by the other way 218).
template <bool SLOW, bool DIRECT> __device__ __forceinline__ float2 one_less_square(Far far, float2 m) {
    if constexpr (!SLOW && DIRECT)
        return fma2(m, fma2(m, dup(-1.0f), choose(far, dup(0.0f), dup(-2.0f))), choose(far, dup(1.0f), dup(0.0f)));
    if constexpr (!SLOW) m = add2(m, choose(far, dup(-1.0f), dup(0.0f)));
    return mul2(m, fma2(m, dup(-1.0f), dup(-2.0f)));
}
// sqrt(1 - a^2)
template <bool SLOW, bool DIRECT> __device__ __forceinline__ float2 input_weight(Far far, float2 m) {
    const float2 n2 = one_less_square<SLOW, DIRECT>(far, m);
    return make_float2(sqrt_approx(n2.x), sqrt_approx(n2.y));
}
// the least 1 - a^2 whose root is formed, 2^-126
constexpr float kLeastSquare = 1.17549435e-38f;
// -scale * softplus(decay) of a pair of channels (0 outside them)
__device__ __forceinline__ float2 decay_rates(const GatedScanParams& p, int64_t c, bool active) {
    return active ? make_float2(-p.scale * softplus_f32(p.decay[c]), -p.scale * softplus_f32(p.decay[c + 1]))
                  : dup(0.0f);
}
__device__ __forceinline__ float sigma_f32(float v) { return 1.0f / (1.0f + expf(-v)); }

// ---- clusters ----
// (the barrier is an aligned one: a warp that parted before it joins first)
__device__ __forceinline__ void cluster_sync_all() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the shared::cluster address of this CTA's shared variable in CTA `rank`
__device__ __forceinline__ uint32_t in_rank(const void* mine, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(mine)), "r"(rank));
    return r;
}
// asynchronous stores into a CTA of the cluster that complete on its mbarrier
__device__ __forceinline__ void store_async(uint32_t dst, float4 v, uint32_t mbar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 :
                 : "r"(dst), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(mbar)
                 : "memory");
}
__device__ __forceinline__ void store_async(uint32_t dst, int v, uint32_t mbar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.s32 [%0], %1, [%2];"
                 :
                 : "r"(dst), "r"(v), "r"(mbar)
                 : "memory");
}
// Bounded wait on an mbarrier of this CTA (that peers of the cluster may
// complete).  A probe suspends the warp until the phase completes or 2 us have
// passed.  On expiry the CTA's abort flag is raised.  Waits on a peer give up
// after about a second, those on the CTA's own warps and loads after four, so
// that they outlast it.
constexpr uint32_t kPeerProbes = 1u << 19, kOwnProbes = 1u << 21, kProbeNs = 2000;
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity, uint32_t probes, volatile int* abort) {
    for (uint32_t i = 0; i < probes; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(mbar), "r"(parity), "r"(kProbeNs)
            : "memory");
        if (ok) return true;
    }
    *abort = 1;
    return false;
}

// CTAs of the scan and its gradient that gave up on a wait (ssd_gated_scan_check_status).
__device__ uint32_t g_gated_gave_up;

// restarts among the group's tokens: lane j's flag of token t0 + j
template <int N>
__device__ __forceinline__ bool reset_flag(const uint8_t* reset, int64_t row, int64_t t0, int64_t L, int lane) {
    return lane < N && t0 + lane < L && reset[row * L + t0 + lane] != 0;
}

// the composition of a map with a state; a map with a restart inside forgets
// the state without multiplying it (0 times an infinite state is not 0)
__device__ __forceinline__ float2 apply(float4 m, bool restart, float2 h) {
    const float2 H = make_float2(m.z, m.w);
    return restart ? H : fma2(make_float2(m.x, m.y), h, H);
}

// f(restarts): a group without one takes code without its selects
template <bool RESET, typename F> __device__ __forceinline__ void by_restarts(uint32_t rst, F f) {
    if (RESET && rst != 0) f(std::true_type());
    else f(std::false_type());
}
// f(slow, restarts) for the two properties of a group that change its code
template <bool RESET, typename F> __device__ __forceinline__ void by_group(bool slow, uint32_t rst, F f) {
    by_restarts<RESET>(rst, [&](auto restarts) {
        if (slow) f(std::true_type(), restarts);
        else f(std::false_type(), restarts);
    });
}

struct Exchange {
    float4 group_map[NW][32];             // this CTA's groups
    float4 tile_map[2][kMaxCluster][32];  // the cluster's tiles, two rounds
    float2 entering[NW][32];              // the state entering each group
    int group_rst[NW], tile_rst[2][kMaxCluster];
    // the input tiles of a slot have landed; the groups' maps are written (and x
    // and gate_x read); their entering states are; their outputs are
    uint64_t loaded[2], maps_ready, states_ready, outputs_ready, tiles_ready[2];
    int abort;
};

template <typename E> __device__ __forceinline__ void init_exchange(E& ex) {
    if (threadIdx.x == 0) {
        tc::mbar_init(tc::smem_u32(&ex.maps_ready), NW);
        tc::mbar_init(tc::smem_u32(&ex.outputs_ready), NW);
        tc::mbar_init(tc::smem_u32(&ex.states_ready), 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(tc::smem_u32(&ex.tiles_ready[i]), 1);
            tc::mbar_init(tc::smem_u32(&ex.loaded[i]), 1);
        }
        tc::fence_mbar_init();
        ex.abort = 0;
    }
    __syncthreads();
}

// (one warp) This CTA's tile map m to every CTA of the cluster, and the wait for
// all of theirs; false once it has given up.
template <bool RESET, typename E>
__device__ __forceinline__ bool exchange_tiles(E& ex, float4 m, bool rst, int it, int rank, int cl, bool withhold,
                                               uint32_t tile_bytes, int lane) {
    const int buf = it & 1;
    const uint32_t bar = tc::smem_u32(&ex.tiles_ready[buf]);
    if (lane == 0) tc::mbar_expect_tx(bar, tile_bytes);
    __syncwarp();
    if (!withhold) {
        for (int to = 0; to < cl; ++to)
            store_async(in_rank(&ex.tile_map[buf][rank][lane], to), m, in_rank(&ex.tiles_ready[buf], to));
        if (RESET && lane < cl)
            store_async(in_rank(&ex.tile_rst[buf][rank], lane), static_cast<int>(rst),
                        in_rank(&ex.tiles_ready[buf], lane));
    }
    return __all_sync(0xffffffffu, wait_phase(bar, (it >> 1) & 1, kPeerProbes, &ex.abort));
}

// The forward's tokens per group: 8 (tiles of 64 rows) for bf16, 4 for fp32,
// whose tiles are twice as large, so that three CTAs with two rounds of input
// tiles each share an SM.
template <typename T> constexpr int kFwdTokens = sizeof(T) == 2 ? 8 : 4;
template <typename T> constexpr int kRowBytes = CPB * sizeof(T);

struct ScanMaps {
    CUtensorMap x, gate_a, gate_x, y;
};

template <typename T> constexpr int kRingBytes = 2 * 3 * NW * kFwdTokens<T> * kRowBytes<T>;

// A compute warp's groups, one per round: t is its first, reset the batch row's
// restarts, states the kept states of the lane's channels (or null).
template <typename T, bool RESET, bool SLOW>
__device__ __forceinline__ void scan_groups(float2 k, const uint8_t* reset, float* states, int64_t L, int64_t C,
                                            int64_t t, int64_t round, int rounds) {
    constexpr bool EXACT = sizeof(T) == 4;
    constexpr int ST = 2, TPT = kFwdTokens<T>, TB = TPT * kRowBytes<T>, CB = NW * TB;
    using Raw = typename Pair<T>::Raw;
    extern __shared__ __align__(128) uint8_t ring[];
    Exchange& ex = *reinterpret_cast<Exchange*>(ring + kRingBytes<T>);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool flag = RESET && reset_flag<TPT>(reset, 0, t, L, lane);
    uint8_t* const mine = ring + warp * TB + lane * sizeof(Raw);
    for (int it = 0; it < rounds; ++it, t += round) {
        const int slot = it % ST;
        uint8_t* src = mine + slot * 3 * CB;
        auto at = [&](int tile, int j) { return reinterpret_cast<Raw*>(src + tile * CB + j * kRowBytes<T>); };
        uint32_t rst = 0;
        if constexpr (RESET) {
            rst = __ballot_sync(0xffffffffu, flag);
            flag = reset_flag<TPT>(reset, 0, t + round, L, lane);
        }
        wait_phase(tc::smem_u32(&ex.loaded[slot]), (it / ST) & 1, kOwnProbes, &ex.abort);
        // the gates and the maps from the group's start up to each token
        float2 As[TPT], Hs[TPT];
        float2 A = dup(1.0f), H = dup(0.0f);
        by_restarts<RESET>(rst, [&](auto restarts) {
#pragma unroll
            for (int j = 0; j < TPT; ++j) {
                const bool rs = decltype(restarts)::value && ((rst >> j) & 1);
                float2 r, i, ga = read_gates(*at(2, j), kLeastA);
                if (rs) ga = dup(0.0f);  // not used: whatever it holds
                sigmas<EXACT>(ga, read_gates(*at(1, j), kLeastX), r, i);
                As[j] = decays<EXACT, SLOW>(mul2(k, r));  // (the token's multiplier, then its map)
                float2 n = input_weight<SLOW, true>(far_of<SLOW>(As[j]), As[j]);
                if (rs) n = dup(1.0f);
                Hs[j] = mul2(mul2(n, i), Pair<T>::widen(*at(0, j)));
            }
#pragma unroll
            for (int j = 0; j < TPT; ++j) {
                const bool rs = decltype(restarts)::value && ((rst >> j) & 1);
                const Far far = far_of<SLOW>(As[j]);
                H = rs ? Hs[j] : step(far, As[j], H, Hs[j]);
                A = rs ? dup(0.0f) : keep(far, As[j], A);
                As[j] = A;
                Hs[j] = H;
            }
        });
        if (t + TPT > L) {  // the group's map is its last token's
            A = dup(1.0f);
            H = dup(0.0f);
#pragma unroll
            for (int j = 0; j < TPT; ++j) {
                A = t + j < L ? As[j] : A;
                H = t + j < L ? Hs[j] : H;
            }
        }
        ex.group_map[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        if (RESET && lane == 0) ex.group_rst[warp] = rst != 0;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.maps_ready));
        // the outputs, over gate_a's tile; the ninth warp's wait on its cluster is
        // bounded and it always arrives
        wait_phase(tc::smem_u32(&ex.states_ready), it & 1, kOwnProbes, &ex.abort);
        const float2 h = ex.entering[warp][lane];
        // (a kept state's token starts a group)
        if (states && t < L && t % kInterval == 0)
            *reinterpret_cast<float2*>(states + t / kInterval * C) = h;
        if (RESET && rst != 0) {
            const int from = __ffs(static_cast<int>(rst)) - 1;  // where h is dropped
#pragma unroll
            for (int j = 0; j < TPT; ++j)
                *at(2, j) = Pair<T>::narrow(j >= from ? Hs[j] : fma2(As[j], h, Hs[j]));
        } else {
#pragma unroll
            for (int j = 0; j < TPT; ++j) *at(2, j) = Pair<T>::narrow(fma2(As[j], h, Hs[j]));
        }
        tc::fence_smem_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.outputs_ready));
    }
}
// The same as a function that is called: next to the other decays' code the compiler
// found worse schedules for either (b1 L65536 C1536 bf16 227 us, by calls 221; b6
// L4096 C4736 at decays from 0.3 on 199, by calls 193).  With restarts it is the
// other way round (b8 L4096 C2048 149 us by calls, 145 without).
template <typename T, bool SLOW, typename... Args> __device__ __noinline__ void call_scan_groups(Args... args) {
    scan_groups<T, false, SLOW>(args...);
}

template <typename T, bool RESET>
__global__ void __launch_bounds__(kThreads, 3)
    gated_scan_kernel(GatedScanParams p, const __grid_constant__ ScanMaps maps, int cl, int withhold) {
    constexpr int ST = 2, TPT = kFwdTokens<T>, TILE = NW * TPT, TB = TPT * kRowBytes<T>, CB = NW * TB;
    using Raw = typename Pair<T>::Raw;
    extern __shared__ __align__(128) uint8_t ring[];    // [ST][3] tiles: x, gate_x, gate_a (then y)
    Exchange& ex = *reinterpret_cast<Exchange*>(ring + kRingBytes<T>);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t C = p.channels, L = p.seqlen, b = blockIdx.y;
    const int rank = static_cast<int>(blockIdx.x) % cl;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x / cl) * CPB, c = c0 + 2 * lane;
    const bool active = c < C;
    const int64_t round = static_cast<int64_t>(cl) * TILE;
    const int rounds = static_cast<int>((L + round - 1) / round);
    init_exchange(ex);
    if (cl > 1) cluster_sync_all();  // every CTA's barriers exist before a peer completes on them
    const int64_t first = static_cast<int64_t>(rank) * TILE;  // the tile's first token, round 0

    if (warp == NW) {
        // The ninth warp: the tiles' loads and stores (lane 0), and the maps.
        // x and gate_x of round n arm the slot's barrier for all three; gate_a's
        // place holds y until its store has read it.
        const uint32_t tiles = tc::smem_u32(ring);
        const int ci = static_cast<int>(c0), bi = static_cast<int>(b);
        auto load_x = [&](int n) {
            const uint32_t dst = tiles + (n % ST) * 3 * CB, bar = tc::smem_u32(&ex.loaded[n % ST]);
            const int t = static_cast<int>(first + n * round);
            tc::mbar_expect_tx(bar, 3 * CB);
            tc::tma_load_rows(dst, &maps.x, bar, ci, t, bi);
            tc::tma_load_rows(dst + CB, &maps.gate_x, bar, ci, t, bi);
        };
        auto load_a = [&](int n) {
            tc::tma_load_rows(tiles + (n % ST) * 3 * CB + 2 * CB, &maps.gate_a, tc::smem_u32(&ex.loaded[n % ST]), ci,
                              static_cast<int>(first + n * round), bi);
        };
        if (lane == 0) {
            for (int n = 0; n < ST && n < rounds; ++n) {
                load_x(n);
                load_a(n);
            }
        }
        float2 carry = (active && p.init_state) ? *reinterpret_cast<const float2*>(p.init_state + b * C + c)
                                                : dup(0.0f);
        const uint32_t tile_bytes = static_cast<uint32_t>(cl) * (32 * sizeof(float4) + (RESET ? sizeof(int) : 0));
        bool ok = true;  // (whole-warp: no map is sent, received or waited for after a timeout)
        for (int it = 0; it < rounds; ++it) {
            const int buf = it & 1;
            // the compute warps' arrivals depend on no other CTA: waited for in any case
            wait_phase(tc::smem_u32(&ex.maps_ready), it & 1, kOwnProbes, &ex.abort);
            if (lane == 0 && it + ST < rounds) load_x(it + ST);
            float4 g[NW];
            uint32_t rst = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                g[w] = ex.group_map[w][lane];
                if (RESET && ex.group_rst[w]) rst |= 1u << w;
            }
            float2 h = carry;
            if (cl > 1 && ok) {
                float4 m = g[0];
#pragma unroll
                for (int w = 1; w < NW; ++w) {
                    const bool gr = RESET && ((rst >> w) & 1);
                    const float2 hh = apply(g[w], gr, make_float2(m.z, m.w));
                    const float2 aa = gr ? dup(0.0f) : mul2(make_float2(g[w].x, g[w].y), make_float2(m.x, m.y));
                    m = make_float4(aa.x, aa.y, hh.x, hh.y);
                }
                ok = exchange_tiles<RESET>(ex, m, rst != 0, it, rank, cl, rank == 0 && it == withhold, tile_bytes,
                                           lane);
                for (int q = 0; q < cl; ++q) {
                    if (q == rank) h = carry;
                    carry = apply(ex.tile_map[buf][q][lane], RESET && ex.tile_rst[buf][q], carry);
                }
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                ex.entering[w][lane] = h;
                h = apply(g[w], RESET && ((rst >> w) & 1), h);
            }
            if (cl == 1) carry = h;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.states_ready));
            wait_phase(tc::smem_u32(&ex.outputs_ready), it & 1, kOwnProbes, &ex.abort);
            if (lane == 0) {
                const int64_t t = first + it * round;
                if (t < L) {
                    tc::tma_store_rows(&maps.y, tiles + (it % ST) * 3 * CB + 2 * CB, ci, static_cast<int>(t), bi);
                    tc::bulk_commit_group();
                }
                if (it + ST < rounds) {
                    tc::bulk_wait_read_all();  // y has left its place
                    load_a(it + ST);
                }
            }
        }
        if (p.final_state && active && rank == 0)
            *reinterpret_cast<float2*>(p.final_state + b * C + c) = carry;
        if (lane == 0) tc::bulk_wait_all();
    } else {
        const int64_t nst = (L + kInterval - 1) / kInterval;
        const float2 k = decay_rates(p, c, active);
        const bool slow = __all_sync(0xffffffffu, k.x >= -0.25f && k.y >= -0.25f);
        const uint8_t* reset = RESET ? p.reset + b * L : nullptr;
        float* states = p.states && active ? p.states + b * nst * C + c : nullptr;
        const int64_t t = first + warp * TPT;
        if constexpr (RESET) {
            if (slow) scan_groups<T, true, true>(k, reset, states, L, C, t, round, rounds);
            else scan_groups<T, true, false>(k, reset, states, L, C, t, round, rounds);
        } else {
            if (slow) call_scan_groups<T, true>(k, reset, states, L, C, t, round, rounds);
            else call_scan_groups<T, false>(k, reset, states, L, C, t, round, rounds);
        }
    }
    __syncthreads();
    if (cl > 1) cluster_sync_all();  // no peer's map arrives after a CTA has left
    if (threadIdx.x == 0 && ex.abort) atomicAdd(&g_gated_gave_up, 1u);
}

// The gradient, the same way from the last token to the first: a group also has
// the map of the adjoint it passes on, c <- a (dy + c) token by token backwards,
// whose factor is the same A.  The state entering a tile is the forward's (a
// tile is one interval), so only the adjoint crosses tiles.  The warps form
// both maps, the ninth hands each group its entering state and adjoint, and the
// group is replayed, forwards for the states and backwards for the
// outputs, which take the places of x, gate_x and gate_a in shared memory.
struct ExchangeBwd {
    float4 group_map[NW][32];             // A, H
    float2 group_rev[NW][32];             // G: c out = A c in + G
    float4 tile_map[2][kMaxCluster][32];  // A, G of the cluster's tiles, two rounds
    float4 entering[NW][32];              // the state and the adjoint entering each group
    int group_rst[NW], tile_rst[2][kMaxCluster];
    uint64_t loaded[2], maps_ready, states_ready, outputs_ready, tiles_ready[2];
    int abort;
};

// The places of a token's gates, once they are read, hold its u and then the state
// before it.
__device__ __forceinline__ void park(uint32_t* gx, uint32_t* ga, float2 h) {
    *gx = __float_as_uint(h.x);
    *ga = __float_as_uint(h.y);
}
__device__ __forceinline__ float2 unpark(const uint32_t* gx, const uint32_t* ga) {
    return make_float2(__uint_as_float(*gx), __uint_as_float(*ga));
}
__device__ __forceinline__ void park(float2* gx, float2*, float2 h) { *gx = h; }
__device__ __forceinline__ float2 unpark(const float2* gx, const float2*) { return *gx; }

// rounds of input tiles in shared memory (one for fp32, so that two CTAs share an SM)
template <typename T> constexpr int kStagesBwd = sizeof(T) == 2 ? 2 : 1;

struct ScanBwdMaps {
    CUtensorMap x, gate_a, gate_x, dy, dx, dgate_a, dgate_x;
};

template <typename T, bool RESET>
__global__ void __launch_bounds__(kThreads, 2)
    gated_scan_bwd_kernel(GatedScanParams p, const __grid_constant__ ScanBwdMaps maps, int cl, int withhold) {
    constexpr bool EXACT = sizeof(T) == 4;
    constexpr int ST = kStagesBwd<T>, TB = TPT * kRowBytes<T>, CB = NW * TB;
    using Raw = typename Pair<T>::Raw;
    extern __shared__ __align__(128) uint8_t ring[];    // [ST][4] tiles: x, gate_x, gate_a, dy; dx, dgate_x, dgate_a
    __shared__ ExchangeBwd ex;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t C = p.channels, L = p.seqlen, b = blockIdx.y;
    const int rank = static_cast<int>(blockIdx.x) % cl;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x / cl) * CPB, c = c0 + 2 * lane;
    const bool active = c < C;
    const int64_t round = static_cast<int64_t>(cl) * TILE;
    const int rounds = static_cast<int>((L + round - 1) / round);
    init_exchange(ex);
    if (cl > 1) cluster_sync_all();
    // rounds run backwards: the first token of this CTA's tile
    auto first = [&](int it) {
        return static_cast<int64_t>(rounds - 1 - it) * round + static_cast<int64_t>(rank) * TILE;
    };
    float2 sum = dup(0.0f);

    if (warp == NW) {
        const uint32_t tiles = tc::smem_u32(ring);
        const int ci = static_cast<int>(c0), bi = static_cast<int>(b);
        auto load = [&](int n) {
            const uint32_t dst = tiles + (n % ST) * 4 * CB, bar = tc::smem_u32(&ex.loaded[n % ST]);
            const int t = static_cast<int>(first(n));
            tc::mbar_expect_tx(bar, 4 * CB);
            tc::tma_load_rows(dst, &maps.x, bar, ci, t, bi);
            tc::tma_load_rows(dst + CB, &maps.gate_x, bar, ci, t, bi);
            tc::tma_load_rows(dst + 2 * CB, &maps.gate_a, bar, ci, t, bi);
            tc::tma_load_rows(dst + 3 * CB, &maps.dy, bar, ci, t, bi);
        };
        if (lane == 0)
            for (int n = 0; n < ST && n < rounds; ++n) load(n);
        const int64_t nst = (L + kInterval - 1) / kInterval;
        // the kept state entering this CTA's tile of a round
        auto kept = [&](int it) {
            const int64_t t = it < rounds ? first(it) : L;
            return active && t < L ? *reinterpret_cast<const float2*>(p.states + (b * nst + t / kInterval) * C + c)
                                   : dup(0.0f);
        };
        // the adjoint entering the round from the right
        float2 carry = (active && p.d_final) ? *reinterpret_cast<const float2*>(p.d_final + b * C + c) : dup(0.0f);
        float2 next = kept(0);
        const uint32_t tile_bytes = static_cast<uint32_t>(cl) * (32 * sizeof(float4) + (RESET ? sizeof(int) : 0));
        bool ok = true;
        for (int it = 0; it < rounds; ++it) {
            const int buf = it & 1;
            float2 h = next;
            next = kept(it + 1);
            wait_phase(tc::smem_u32(&ex.maps_ready), it & 1, kOwnProbes, &ex.abort);
            auto factor = [&](int w) { return *reinterpret_cast<const float2*>(&ex.group_map[w][lane]); };
            auto step = [&](int w, float2 v) {
                const float2 G = ex.group_rev[w][lane];
                return RESET && ex.group_rst[w] ? G : fma2(factor(w), v, G);
            };
            float2 cin = carry;
            if (cl > 1 && ok) {
                float2 a = factor(NW - 1), g = ex.group_rev[NW - 1][lane];
                bool rst = RESET && ex.group_rst[NW - 1];
#pragma unroll
                for (int w = NW - 2; w >= 0; --w) {
                    g = step(w, g);
                    a = RESET && ex.group_rst[w] ? dup(0.0f) : mul2(factor(w), a);
                    rst |= RESET && ex.group_rst[w];
                }
                ok = exchange_tiles<RESET>(ex, make_float4(a.x, a.y, g.x, g.y), rst, it, rank, cl,
                                           rank == 0 && it == withhold, tile_bytes, lane);
                for (int q = cl - 1; q >= 0; --q) {
                    if (q == rank) cin = carry;
                    carry = apply(ex.tile_map[buf][q][lane], RESET && ex.tile_rst[buf][q], carry);
                }
            }
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                *reinterpret_cast<float2*>(&ex.entering[w][lane]) = h;
                h = apply(ex.group_map[w][lane], RESET && ex.group_rst[w], h);
            }
#pragma unroll
            for (int w = NW - 1; w >= 0; --w) {
                *(reinterpret_cast<float2*>(&ex.entering[w][lane]) + 1) = cin;
                cin = step(w, cin);
            }
            if (cl == 1) carry = cin;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.states_ready));
            wait_phase(tc::smem_u32(&ex.outputs_ready), it & 1, kOwnProbes, &ex.abort);
            if (lane == 0) {
                const int64_t t = first(it);
                if (t < L) {
                    const uint32_t out = tiles + (it % ST) * 4 * CB;
                    tc::tma_store_rows(&maps.dx, out, ci, static_cast<int>(t), bi);
                    tc::tma_store_rows(&maps.dgate_x, out + CB, ci, static_cast<int>(t), bi);
                    tc::tma_store_rows(&maps.dgate_a, out + 2 * CB, ci, static_cast<int>(t), bi);
                    tc::bulk_commit_group();
                }
                if (it + ST < rounds) {
                    tc::bulk_wait_read_all();
                    load(it + ST);
                }
            }
        }
        if (p.d_init && active && rank == 0) *reinterpret_cast<float2*>(p.d_init + b * C + c) = carry;
        if (lane == 0) tc::bulk_wait_all();
    } else {
        const float2 k = decay_rates(p, c, active);
        const bool slow = __all_sync(0xffffffffu, k.x >= -0.25f && k.y >= -0.25f);
        bool flag = RESET && reset_flag<TPT>(p.reset, b, first(0) + warp * TPT, L, lane);
        uint8_t* const mine = ring + warp * TB + lane * sizeof(Raw);
        for (int it = 0; it < rounds; ++it) {
            const int64_t t = first(it) + warp * TPT;
            const int slot = it % ST;
            uint8_t* src = mine + slot * 4 * CB;
            auto at = [&](int tile, int j) { return reinterpret_cast<Raw*>(src + tile * CB + j * kRowBytes<T>); };
            uint32_t rst = 0;
            if constexpr (RESET) {
                rst = __ballot_sync(0xffffffffu, flag);
                flag = it + 1 < rounds && reset_flag<TPT>(p.reset, b, t - round, L, lane);
            }
            const int left = t + TPT <= L ? TPT : static_cast<int>(L - t < 0 ? 0 : L - t);
            wait_phase(tc::smem_u32(&ex.loaded[slot]), (it / ST) & 1, kOwnProbes, &ex.abort);
            float2 r[TPT], i[TPT], m[TPT];
            float2 A = dup(1.0f), H = dup(0.0f), G = dup(0.0f);
            by_group<RESET>(slow, rst, [&](auto is_slow, auto restarts) {
                constexpr bool SLOW = decltype(is_slow)::value;
#pragma unroll
                for (int j = 0; j < TPT; ++j) {
                    const bool rs = decltype(restarts)::value && ((rst >> j) & 1);
                    float2 ga = read_gates(*at(2, j), kLeastA);
                    if (rs) ga = dup(0.0f);
                    sigmas<EXACT>(ga, read_gates(*at(1, j), kLeastX), r[j], i[j]);
                    m[j] = decays<EXACT, SLOW>(mul2(k, r[j]));
                    float2 n = input_weight<SLOW, false>(far_of<SLOW>(m[j]), m[j]);
                    if (rs) n = dup(1.0f);
                    float2 u = mul2(n, mul2(i[j], Pair<T>::widen(*at(0, j))));
                    if (j >= left) {  // tokens past the end change nothing
                        m[j] = dup(kNothing<SLOW>);
                        u = dup(0.0f);
                    }
                    park(at(1, j), at(2, j), u);
                    const Far far = far_of<SLOW>(m[j]);
                    A = rs ? dup(0.0f) : keep(far, m[j], A);
                    H = rs ? u : step(far, m[j], H, u);
                }
#pragma unroll
                for (int j = TPT - 1; j >= 0; --j) {  // (dy reads as zero past the end)
                    G = add2(G, Pair<T>::widen(*at(3, j)));
                    G = decltype(restarts)::value && ((rst >> j) & 1) ? dup(0.0f) : keep(far_of<SLOW>(m[j]), m[j], G);
                }
            });
            ex.group_map[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
            ex.group_rev[warp][lane] = G;
            if (RESET && lane == 0) ex.group_rst[warp] = rst != 0;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.maps_ready));
            wait_phase(tc::smem_u32(&ex.states_ready), it & 1, kOwnProbes, &ex.abort);
            const float4 in = ex.entering[warp][lane];
            float2 h = make_float2(in.x, in.y), g = make_float2(in.z, in.w);
            // What follows is formed again from r, i and m: kept over the wait, n of the
            // group would cost 16 more registers.
#pragma unroll
            for (int j = 0; j < TPT; ++j)
                asm volatile(""
                             : "+f"(m[j].x), "+f"(m[j].y), "+f"(r[j].x), "+f"(r[j].y), "+f"(i[j].x), "+f"(i[j].y));
            by_group<RESET>(slow, rst, [&](auto is_slow, auto restarts) {
                constexpr bool SLOW = decltype(is_slow)::value;
                // forwards: the state before each token
#pragma unroll
                for (int j = 0; j < TPT; ++j) {
                    const float2 u = unpark(at(1, j), at(2, j));
                    park(at(1, j), at(2, j), h);
                    const bool rs = decltype(restarts)::value && ((rst >> j) & 1);
                    h = rs ? u : step(far_of<SLOW>(m[j]), m[j], h, u);
                }
                // backwards: the outputs
#pragma unroll
                for (int j = TPT - 1; j >= 0; --j) {
                    const bool rs = decltype(restarts)::value && ((rst >> j) & 1);
                    const float2 x = Pair<T>::widen(*at(0, j)), hp = unpark(at(1, j), at(2, j));
                    g = add2(g, Pair<T>::widen(*at(3, j)));
                    const float2 ix = mul2(i[j], x), la = mul2(k, r[j]);
                    const Far far = far_of<SLOW>(m[j]);
                    const float2 a = decay_of(far, m[j]);
                    // n and 1 / n from one reciprocal root; a decay of exactly 1 (n = 0)
                    // gives a finite dla, times la = 0
                    const float2 n2 = one_less_square<SLOW, false>(far, m[j]);
                    const float2 rn = make_float2(rsqrt_approx(max_nan(n2.x, kLeastSquare)),
                                                  rsqrt_approx(max_nan(n2.y, kLeastSquare)));
                    const float2 n = rs ? dup(1.0f) : mul2(n2, rn);
                    const float2 dx = mul2(mul2(g, n), i[j]);
                    const float2 dgx = mul2(dx, fma2(ix, dup(-1.0f), x));
                    float2 dla = mul2(mul2(g, a), fma2(mul2(a, rn), mul2(ix, dup(-1.0f)), hp));
                    if (rs) dla = dup(0.0f);
                    const float2 dga = mul2(dla, fma2(la, mul2(r[j], dup(-1.0f)), la));
                    if (j < left) sum = fma2(dla, r[j], sum);
                    g = rs ? dup(0.0f) : keep(far, m[j], g);
                    *at(0, j) = Pair<T>::narrow(dx);
                    *at(1, j) = Pair<T>::narrow(dgx);
                    *at(2, j) = Pair<T>::narrow(dga);
                    // two tokens at a time: all eight at once spill (388 us instead of 226)
                    if ((j & 1) == 0) asm volatile("" ::: "memory");
                }
            });
            tc::fence_smem_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.outputs_ready));
        }
    }
    // the CTA's sums of dla r, group after group
    __syncthreads();
    if (warp < NW) ex.group_rev[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && active) {
        float2 s = dup(0.0f);
#pragma unroll
        for (int w = 0; w < NW; ++w) s = add2(s, ex.group_rev[w][lane]);
        *reinterpret_cast<float2*>(p.partial + (b * cl + rank) * C + c) = s;
    }
    if (cl > 1) cluster_sync_all();
    if (threadIdx.x == 0 && ex.abort) atomicAdd(&g_gated_gave_up, 1u);
}

// ddecay = -scale * sigma(decay) * the sum of dla * r over batch and time
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(kSumWarps * 32) gated_scan_finish_kernel(GatedScanParams p, int64_t rows) {
    grid_dep_wait();
    column_sums<kSumWarps>(p.partial, rows, p.channels, [&](int64_t c, float s) {
        p.ddecay[c] = -p.scale * sigma_f32(p.decay[c]) * s;
    });
}

// The decode step: a thread takes 4 channels of R batch rows, so that the
// channels' softplus is formed once for all of them and R rows' loads are in
// flight together.  Bandwidth-bound at large batches (the state in and out, four
// inputs and outputs; fp32 b512 C5120 17 to 18 us between events after an L2 flush, 7.8
// back to back from L2, its 63 MB 9.7); a small one is its launch, and consecutive steps overlap theirs
// by programmatic dependent launch (bf16 b256 C5120 8 us a step, one row of
// 1536 channels the same).
constexpr int kUpdateThreads = 128;
template <typename T> struct Quad4;
template <> struct Quad4<float> {
    using Raw = float4;
    static __device__ __forceinline__ void widen(Raw r, float2& a, float2& b) {
        a = make_float2(r.x, r.y);
        b = make_float2(r.z, r.w);
    }
    static __device__ __forceinline__ Raw narrow(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
};
template <> struct Quad4<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void widen(Raw r, float2& a, float2& b) {
        a = Pair<__nv_bfloat16>::widen(r.x);
        b = Pair<__nv_bfloat16>::widen(r.y);
    }
    static __device__ __forceinline__ Raw narrow(float2 a, float2 b) {
        return make_uint2(Pair<__nv_bfloat16>::narrow(a), Pair<__nv_bfloat16>::narrow(b));
    }
};

template <typename T, int R>
__global__ void __launch_bounds__(kUpdateThreads) gated_update_kernel(GatedUpdateParams p) {
    constexpr bool EXACT = sizeof(T) == 4;
    using Q = Quad4<T>;
    using Raw = typename Q::Raw;
    const int64_t quads = p.channels / 4, quad = static_cast<int64_t>(blockIdx.x) * kUpdateThreads + threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.y) * R;
    grid_dep_wait();
    grid_dep_launch();
    if (quad >= quads) return;
    float4 st[R];
    Raw x[R], ga[R], gx[R];
    bool rs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = row0 + r < p.batch ? row0 + r : p.batch - 1, i = row * quads + quad;
        st[r] = reinterpret_cast<const float4*>(p.state)[i];
        x[r] = static_cast<const Raw*>(p.x)[i];
        ga[r] = static_cast<const Raw*>(p.gate_a)[i];
        gx[r] = static_cast<const Raw*>(p.gate_x)[i];
        rs[r] = p.reset && p.reset[row];
    }
    const float4 d = reinterpret_cast<const float4*>(p.decay)[quad];
    const float2 k[2] = {make_float2(-p.scale * softplus_f32(d.x), -p.scale * softplus_f32(d.y)),
                         make_float2(-p.scale * softplus_f32(d.z), -p.scale * softplus_f32(d.w))};
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (row0 + r >= p.batch) break;
        float2 xv[2], av[2], iv[2];
        Q::widen(x[r], xv[0], xv[1]);
        Q::widen(ga[r], av[0], av[1]);
        Q::widen(gx[r], iv[0], iv[1]);
        float2 h[2] = {make_float2(st[r].x, st[r].y), make_float2(st[r].z, st[r].w)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float2 rg, ig;
            if (rs[r]) av[j] = dup(0.0f);
            sigmas<EXACT>(least_gates<EXACT>(av[j], -87.0f), least_gates<EXACT>(iv[j], -41.5f), rg, ig);
            const float2 la = mul2(k[j], rg), m = decays<EXACT, false>(la);
            const Far far{!(la.x >= -0.25f), !(la.y >= -0.25f)};  // (the choice that decays makes)
            const float2 n = rs[r] ? dup(1.0f) : input_weight<false, true>(far, m);
            const float2 u = mul2(mul2(n, ig), xv[j]);
            h[j] = rs[r] ? u : step(far, m, h[j], u);
        }
        const int64_t i = (row0 + r) * quads + quad;
        reinterpret_cast<float4*>(p.new_state)[i] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
        static_cast<Raw*>(p.y)[i] = Q::narrow(h[0], h[1]);
    }
}

int device_sms() {
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        n = 148;
    }
    return n;
}

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute* attr, int64_t blocks, int64_t batch, int cl,
                                  size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * cl), static_cast<unsigned>(batch));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = static_cast<unsigned>(cl);
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cl > 1 ? 1 : 0;
    return cfg;
}

// CTAs per cluster.  More of them cut the rounds a sequence takes, but share the
// SMs, add an exchange per round and, beyond what the device holds at once
// (asked of the runtime, once per device), run in waves.  A round measured
// about 1.3 + 0.5 k us with k CTAs on an SM, 0.7 us more in a cluster, and the
// start of a wave about one and a half rounds; the size with the least sum is
// taken.  (bf16 b1 L65536 C1536: 15, 232 us; 10, 255; 8, 302.  bf16 gradient
// b8 L4096 C2048: 1, 226 us; 2, 247; b1 L65536 C1536: 10, 425; 8, 488.  fp32
// gradient b2 L777 C1536: 5, 36 us; 13, 42; 1, 73.)
constexpr int kMaxDevices = 64;
template <typename Kern>
int cluster_size(std::atomic<int> (&held)[kMaxDevices][kMaxCluster + 1], Kern kern, size_t smem,
                 int64_t blocks, int64_t batch, int64_t tiles) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) {
        cudaGetLastError();
        return 1;
    }
    const double sms = device_sms();
    const int64_t clusters = blocks * batch;
    int best = 1;
    double least = 0.0;
    for (int cl = 1; cl <= kMaxCluster && cl <= tiles; ++cl) {
        int n = held[dev][cl].load(std::memory_order_relaxed);  // clusters at once; 0 = not asked, -1 = none
        if (n == 0) {
            cudaLaunchAttribute attr;
            cudaLaunchConfig_t cfg = cluster_config(&attr, 1, 1, cl, smem, nullptr);
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
                cudaGetLastError();
                n = -1;
            }
            held[dev][cl].store(n, std::memory_order_relaxed);
        }
        if (n < 1) continue;
        const int64_t waves = (clusters + n - 1) / n, rounds = (tiles + cl - 1) / cl;
        const double share = static_cast<double>(clusters < n ? clusters : n) * cl / sms;
        const double cost = static_cast<double>(waves) * (static_cast<double>(rounds) + 1.5) *
                            (1.3 + 0.5 * (share < 1.0 ? 1.0 : share) + (cl > 1 ? 0.7 : 0.0));
        if (least == 0.0 || cost < least) {
            least = cost;
            best = cl;
        }
    }
    return best;
}

template <auto Kern, typename... Args>
cudaError_t launch_clusters(const GatedScanParams& p, int tile, size_t smem, cudaStream_t s, int* cluster,
                            const Args&... args) {
    static std::atomic<int> held[kMaxDevices][kMaxCluster + 1];
    const cudaError_t e = prepare_kernel<Kern>(static_cast<int>(smem), true);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.channels + CPB - 1) / CPB;
    const int cl = cluster_size(held, Kern, smem, blocks, p.batch, (p.seqlen + tile - 1) / tile);
    *cluster = cl;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_config(&attr, blocks, p.batch, cl, smem, s);
    return cudaLaunchKernelEx(&cfg, Kern, p, args..., cl, static_cast<int>(debug_withhold(SSD_DEBUG_GATED_MAP)));
}

}  // namespace

size_t gated_scan_bwd_partial_bytes(int64_t batch, int64_t, int64_t channels) {
    return static_cast<size_t>(batch) * kMaxCluster * channels * sizeof(float);
}

template <typename T> cudaError_t launch_gated_scan(const GatedScanParams& p, cudaStream_t s) {
    constexpr int tile = NW * kFwdTokens<T>;
    const size_t smem = kRingBytes<T> + sizeof(Exchange);
    ScanMaps m;
    const std::pair<CUtensorMap*, const void*> arrays[] = {
        {&m.x, p.x}, {&m.gate_a, p.gate_a}, {&m.gate_x, p.gate_x}, {&m.y, p.y}};
    for (const auto& a : arrays)
        if (!make_tmap_rows(a.first, a.second, sizeof(T) == 2, p.channels, p.seqlen, p.batch, tile))
            return cudaErrorInvalidValue;
    int cl = 1;
    return p.reset ? launch_clusters<gated_scan_kernel<T, true>>(p, tile, smem, s, &cl, m)
                   : launch_clusters<gated_scan_kernel<T, false>>(p, tile, smem, s, &cl, m);
}

template <typename T> cudaError_t launch_gated_scan_bwd(const GatedScanParams& p, cudaStream_t s) {
    const size_t smem = kStagesBwd<T> * 4 * TILE * kRowBytes<T>;
    ScanBwdMaps m;
    const std::pair<CUtensorMap*, const void*> arrays[] = {
        {&m.x, p.x}, {&m.gate_a, p.gate_a}, {&m.gate_x, p.gate_x}, {&m.dy, p.dy},
        {&m.dx, p.dx}, {&m.dgate_a, p.dgate_a}, {&m.dgate_x, p.dgate_x}};
    for (const auto& a : arrays)
        if (!make_tmap_rows(a.first, a.second, sizeof(T) == 2, p.channels, p.seqlen, p.batch, TILE))
            return cudaErrorInvalidValue;
    int cl = 1;
    const cudaError_t e =
        p.reset ? launch_clusters<gated_scan_bwd_kernel<T, true>>(p, TILE, smem, s, &cl, m)
                : launch_clusters<gated_scan_bwd_kernel<T, false>>(p, TILE, smem, s, &cl, m);
    if (e != cudaSuccess) return e;
    return launch_kernel(gated_scan_finish_kernel, dim3(static_cast<unsigned>((p.channels + 31) / 32)),
                         dim3(kSumWarps * 32), 0, s, true, p, p.batch * cl);
}

template <typename T, int R> cudaError_t launch_update_rows(const GatedUpdateParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.channels / 4 + kUpdateThreads - 1) / kUpdateThreads),
                    static_cast<unsigned>((p.batch + R - 1) / R));
    return launch_kernel(gated_update_kernel<T, R>, grid, dim3(kUpdateThreads), 0, s, true, p);
}
template <typename T> cudaError_t launch_gated_update(const GatedUpdateParams& p, cudaStream_t s) {
    // four rows per thread where that still gives every SM four CTAs
    const int64_t ctas = (p.channels / 4 + kUpdateThreads - 1) / kUpdateThreads * ((p.batch + 3) / 4);
    return ctas >= 4 * device_sms() ? launch_update_rows<T, 4>(p, s) : launch_update_rows<T, 1>(p, s);
}

cudaError_t gated_scan_take_status(int* v, cudaStream_t s) {
    static GaveUp gave_up;
    return gave_up.take(g_gated_gave_up, v, s);
}

template cudaError_t launch_gated_scan<float>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan<__nv_bfloat16>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan_bwd<float>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan_bwd<__nv_bfloat16>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_update<float>(const GatedUpdateParams&, cudaStream_t);
template cudaError_t launch_gated_update<__nv_bfloat16>(const GatedUpdateParams&, cudaStream_t);

}  // namespace ssd
