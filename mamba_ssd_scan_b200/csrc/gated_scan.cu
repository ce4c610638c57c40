// gated_scan.cu -- the gated linear recurrence, its gradient and its decode
// step (the formulas stand in include/ssd.h).
//
// A step h <- a h + u is an affine map, and maps compose: (A, H) after (A', H')
// is (A A', A H' + H).  So a sequence is cut into groups of 8 consecutive
// tokens, each thread runs its group from zero, the groups' maps are composed,
// and each thread then replays its group from the state that enters it.  The
// replay costs two packed operations per token on values that are still in
// registers, while the gates (about 4 special-function results per element)
// are formed once and the inputs are read once.
//
// A compute warp takes one group of tokens of 64 channels (a pair per lane);
// the 8 compute warps of a CTA take consecutive groups (a tile of 64 tokens),
// and the CTAs of a cluster consecutive tiles.  A ninth warp composes the
// tile's map, sends it to the cluster's CTAs through distributed shared memory
// (asynchronous stores that complete on the receiver's mbarrier), and hands
// each group its entering state.  The order of composition is fixed, so
// results do not depend on timing; there is no workspace and no wait on another
// cluster.  Every mbarrier wait is bounded: on expiry the CTA raises its abort
// flag, finishes without waiting, and the call's status reads SSD_ERR_TIMEOUT.
#include <stdlib.h>
#include "mixers.h"
#include "tcgen05.cuh"
#include "tma.cuh"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int kInterval = SSD_GATED_SCAN_INTERVAL;
constexpr int NW = 8;            // compute warps (groups) per CTA
constexpr int TPB = (NW + 1) * 32;
constexpr int TPT = 8;           // tokens per group
constexpr int TILE = NW * TPT;   // tokens per CTA and round
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

// 2^(k v) for a constant k = hi + lo in two parts, cut off at 2^top.  For fp32
// inputs the rounding of k v (up to 2^-24 |k v| in the exponent) is carried
// along; for bf16 inputs it stays well inside their own 2^-9.
template <bool EXACT>
__device__ __forceinline__ float2 exp2_scaled(float2 v, float hi, float lo, float top = 126.0f) {
    if constexpr (EXACT)  // no infinite products below
        v = make_float2(min_nan(max_nan(v.x, -200.0f), 200.0f), min_nan(max_nan(v.y, -200.0f), 200.0f));
    const float2 t = mul2(v, dup(hi));
    float2 e = make_float2(ex2_approx(min_nan(t.x, top)), ex2_approx(min_nan(t.y, top)));
    if constexpr (EXACT) {
        const float2 d = fma2(v, dup(lo), fma2(v, dup(hi), make_float2(-t.x, -t.y)));  // what t lost
        e = fma2(e, mul2(d, dup(0.69314718f)), e);
    }
    return e;
}
// log2(e) in two parts
constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266174e-8f;

// sigma of a pair of gates with one reciprocal per channel:
// 1 / ((1 + e^-a)(1 + e^-x)) times the other factor (a reciprocal each would
// make five special-function results per element, close to what the pipe
// gives in the time the bytes take).  e^-x is cut off at 2^60 (i is then off by
// 2^-60); with a below about -46 the product may overflow, its reciprocal is 0
// and r = i = 0: the gate counts as shut, where r < 2^-66.
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

// em1 = a - 1 = e^la - 1 (la <= 0) and a.  a = 1 + em1 enters the recurrence as
// h + em1 h, so that a decay near 1 keeps its relative accuracy in la, and
// 1 - a^2 = -em1 (2 + em1) without cancellation.  Down to -1/4 from the Taylor
// series to the sixth power (what it leaves out is below 2^-24 of em1), beyond
// from e^la.  la never falls below the channel's own -scale softplus(decay),
// so where that is above -1/4 (`slow`, the same for a whole warp; the usual
// decays of 0.9 to 0.999 at the open gate) the second form is not evaluated.
template <bool EXACT>
__device__ __forceinline__ void decays(float2 la, bool slow, float2& em1, float2& a) {
    float2 q = dup(1.0f / 720.0f);
    q = fma2(q, la, dup(1.0f / 120.0f));
    q = fma2(q, la, dup(1.0f / 24.0f));
    q = fma2(q, la, dup(1.0f / 6.0f));
    q = fma2(q, la, dup(0.5f));
    em1 = fma2(mul2(q, la), la, la);
    a = add2(em1, dup(1.0f));
    if (!slow) {
        const float2 e = exp2_scaled<EXACT>(la, kLog2eHi, kLog2eLo);
        if (!(la.x >= -0.25f)) {
            a.x = e.x;
            em1.x = e.x - 1.0f;
        }
        if (!(la.y >= -0.25f)) {
            a.y = e.y;
            em1.y = e.y - 1.0f;
        }
    }
}
// sqrt(1 - a^2)
__device__ __forceinline__ float2 input_weight(float2 em1) {
    const float2 n2 = mul2(em1, fma2(em1, dup(-1.0f), dup(-2.0f)));
    return make_float2(sqrt_approx(n2.x), sqrt_approx(n2.y));
}
// -scale * softplus(decay) of a pair of channels (0 outside them)
__device__ __forceinline__ float2 decay_rates(const GatedScanParams& p, int64_t c, bool active) {
    return active ? make_float2(-p.scale * softplus_f32(p.decay[c]), -p.scale * softplus_f32(p.decay[c + 1]))
                  : dup(0.0f);
}
__device__ __forceinline__ float sigma_f32(float v) { return 1.0f / (1.0f + expf(-v)); }

// ---- clusters ----
__device__ __forceinline__ void cluster_sync_all() {
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
// bounded wait on a local mbarrier that peers complete; false once aborted
__device__ __forceinline__ bool wait_cluster(uint32_t mbar, uint32_t parity, volatile int* abort) {
    for (uint32_t i = 0; i < tc::kSpinLimit; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(mbar), "r"(parity), "r"(200)
            : "memory");
        if (ok) return true;
        if ((i & 63) == 63 && *abort) return false;
    }
    *abort = 1;
    return false;
}

// SSD_ERR_TIMEOUT once a scan or its gradient gave up on a wait; read and
// cleared by ssd_gated_scan_check_status.
__device__ int g_gated_status;

// ---- a warp's tile of one array: TPT rows of 64 channels, by 16-byte copies ----
template <typename T, int TPT> struct Tile {
    static constexpr int kRowBytes = CPB * sizeof(T);
    static constexpr int kBytes = TPT * kRowBytes;
    static constexpr int kChunks = kRowBytes / 16;          // per row
    static constexpr int kRows = 32 / kChunks;              // rows per copy instruction
    static constexpr int kElems = 16 / static_cast<int>(sizeof(T));
    // rows 0 .. TPT - 1 of the array whose row 0 the lane's own chunk starts at src (row
    // stride C elements); rows from `left` on and, without `in`, all of the lane's chunks read as zero
    static __device__ __forceinline__ void load(uint8_t* dst, const T* src, int left, bool in, int64_t C, int lane) {
        uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + lane * 16;
        const int n = in ? left - lane / kChunks : 0;  // rows of this lane's column of chunks
#pragma unroll
        for (int k = 0; k < TPT / kRows; ++k) {
            const bool on = k * kRows < n;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         :
                         : "r"(s + k * 512), "l"(on ? src + k * kRows * C : nullptr), "r"(on ? 16 : 0)
                         : "memory");
        }
    }
    static __device__ __forceinline__ float2 read(const uint8_t* t, int row, int lane) {
        using Raw = typename Pair<T>::Raw;
        return Pair<T>::widen(*reinterpret_cast<const Raw*>(t + row * kRowBytes + lane * sizeof(Raw)));
    }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" : : "n"(N) : "memory");
}

// restarts among the group's tokens, bit j = token t0 + j
template <int TPT>
__device__ __forceinline__ uint32_t reset_mask(const uint8_t* reset, int64_t row, int64_t t0, int64_t L, int lane) {
    const bool on = lane < TPT && t0 + lane < L && reset[row * L + t0 + lane] != 0;
    return __ballot_sync(0xffffffffu, on);
}

// the composition of a map with a state; a map with a restart inside forgets
// the state without multiplying it (0 times an infinite state is not 0)
__device__ __forceinline__ float2 apply(float4 m, bool restart, float2 h) {
    const float2 H = make_float2(m.z, m.w);
    return restart ? H : fma2(make_float2(m.x, m.y), h, H);
}

struct Exchange {
    float4 group_map[NW][32];             // this CTA's groups
    float4 tile_map[2][kMaxCluster][32];  // the cluster's tiles, two rounds
    float2 entering[NW][32];              // the state entering each group
    int group_rst[NW], tile_rst[2][kMaxCluster];
    uint64_t maps_ready, states_ready, tiles_ready[2];
    int abort;
};

// 16-byte copies in flight ahead of the arithmetic, in groups of tokens
constexpr int kStages = 2;

template <typename T, bool RESET>
__global__ void __launch_bounds__(TPB, 3) gated_scan_kernel(GatedScanParams p, int cl, int withhold) {
    constexpr bool EXACT = sizeof(T) == 4;
    using TL = Tile<T, TPT>;
    extern __shared__ __align__(16) uint8_t ring[];    // [NW][kStages][3] tiles
    __shared__ Exchange ex;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t C = p.channels, L = p.seqlen, b = blockIdx.y;
    const int rank = static_cast<int>(blockIdx.x) % cl;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x / cl) * CPB, c = c0 + 2 * lane;
    const bool active = c < C;
    const int64_t round = static_cast<int64_t>(cl) * TILE;
    const int rounds = static_cast<int>((L + round - 1) / round);
    if (threadIdx.x == 0) {
        tc::mbar_init(tc::smem_u32(&ex.maps_ready), NW);
        tc::mbar_init(tc::smem_u32(&ex.states_ready), 1);
        tc::mbar_init(tc::smem_u32(&ex.tiles_ready[0]), 1);
        tc::mbar_init(tc::smem_u32(&ex.tiles_ready[1]), 1);
        tc::fence_mbar_init();
        ex.abort = 0;
    }
    __syncthreads();
    if (cl > 1) cluster_sync_all();  // every CTA's barriers exist before a peer completes on them

    if (warp == NW) {
        float2 carry = (active && p.init_state) ? *reinterpret_cast<const float2*>(p.init_state + b * C + c)
                                                : dup(0.0f);
        const uint32_t tile_bytes = static_cast<uint32_t>(cl) * (32 * sizeof(float4) + (RESET ? sizeof(int) : 0));
        bool ok = true;  // (whole-warp: no map is sent, received or waited for after a timeout)
        for (int it = 0; it < rounds; ++it) {
            const int buf = it & 1;
            if (ok) ok = tc::wait_or_abort(tc::smem_u32(&ex.maps_ready), it & 1, &ex.abort);
            ok = __all_sync(0xffffffffu, ok);
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
                const uint32_t bar = tc::smem_u32(&ex.tiles_ready[buf]);
                if (lane == 0) tc::mbar_expect_tx(bar, tile_bytes);
                __syncwarp();
                if (!(rank == 0 && it == withhold)) {
                    for (int to = 0; to < cl; ++to)
                        store_async(in_rank(&ex.tile_map[buf][rank][lane], to), m, in_rank(&ex.tiles_ready[buf], to));
                    if (RESET && lane < cl)
                        store_async(in_rank(&ex.tile_rst[buf][rank], lane), rst != 0, in_rank(&ex.tiles_ready[buf], lane));
                }
                ok = __all_sync(0xffffffffu, wait_cluster(bar, (it >> 1) & 1, &ex.abort));
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
        }
        if (p.final_state && active && rank == 0)
            *reinterpret_cast<float2*>(p.final_state + b * C + c) = carry;
    } else {
        int64_t t0 = static_cast<int64_t>(rank) * TILE + warp * TPT;  // the group's first token
        const int64_t nst = (L + kInterval - 1) / kInterval;
        T* y = static_cast<T*>(p.y) + (b * L + t0) * C + c;
        uint8_t* tiles = ring + warp * kStages * 3 * TL::kBytes;
        // the lane's own 16-byte chunk of the group's first row
        const int64_t cc = c0 + (lane % TL::kChunks) * TL::kElems;
        const bool in = cc < C;
        int64_t next = (b * L + t0 + lane / TL::kChunks) * C + cc;  // ... of the next round to fetch
        auto rows_left = [&](int64_t t) { return t + TPT <= L ? TPT : static_cast<int>(L - t < 0 ? 0 : L - t); };
        // (an empty group of copies past the last round keeps the count)
        auto fetch = [&](int it, int slot) {
            if (it < rounds) {
                const int left = rows_left(static_cast<int64_t>(it) * round + rank * TILE + warp * TPT);
                uint8_t* dst = tiles + slot * 3 * TL::kBytes;
                TL::load(dst, static_cast<const T*>(p.x) + next, left, in, C, lane);
                TL::load(dst + TL::kBytes, static_cast<const T*>(p.gate_a) + next, left, in, C, lane);
                TL::load(dst + 2 * TL::kBytes, static_cast<const T*>(p.gate_x) + next, left, in, C, lane);
                next += round * C;
            }
            copies_commit();
        };
#pragma unroll
        for (int s = 0; s < kStages; ++s) fetch(s, s);
        const float2 k = decay_rates(p, c, active);
        const bool slow = __all_sync(0xffffffffu, k.x >= -0.25f && k.y >= -0.25f);
        bool ok = true;
        for (int it = 0; it < rounds; ++it, t0 += round, y += round * C) {
            const int slot = it % kStages;
            uint32_t rst = 0;
            if constexpr (RESET) rst = reset_mask<TPT>(p.reset, b, t0, L, lane);
            copies_wait<kStages - 1>();
            __syncwarp();
            // the gates and the group's map
            const uint8_t* src = tiles + slot * 3 * TL::kBytes;
            float2 em1[TPT], u[TPT];
#pragma unroll
            for (int j = 0; j < TPT; ++j) {
                float2 r, i, a;
                sigmas<EXACT>(TL::read(src + TL::kBytes, j, lane), TL::read(src + 2 * TL::kBytes, j, lane), r, i);
                decays<EXACT>(mul2(k, r), slow, em1[j], a);
                float2 n = input_weight(em1[j]);
                if (RESET && ((rst >> j) & 1)) n = dup(1.0f);
                u[j] = mul2(mul2(n, i), TL::read(src, j, lane));
            }
            __syncwarp();
            fetch(it + kStages, slot);
            const int left = rows_left(t0);
            if (left < TPT) {  // tokens past the end change nothing
#pragma unroll
                for (int j = 0; j < TPT; ++j)
                    if (j >= left) em1[j] = u[j] = dup(0.0f);
            }
            float2 A = dup(1.0f), H = dup(0.0f);
#pragma unroll
            for (int j = 0; j < TPT; ++j) {
                if (RESET && ((rst >> j) & 1)) {
                    A = dup(0.0f);
                    H = u[j];
                } else {
                    A = fma2(em1[j], A, A);
                    H = add2(H, fma2(em1[j], H, u[j]));
                }
            }
            ex.group_map[warp][lane] = make_float4(A.x, A.y, H.x, H.y);
            if (RESET && lane == 0) ex.group_rst[warp] = rst != 0;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ex.maps_ready));
            // the outputs
            if (ok) ok = tc::wait_or_abort(tc::smem_u32(&ex.states_ready), it & 1, &ex.abort);
            float2 h = ex.entering[warp][lane];
            // a tile starts at a multiple of the interval: group 0 keeps its state
            if (warp == 0 && p.states && active && left > 0)
                *reinterpret_cast<float2*>(p.states + (b * nst + t0 / kInterval) * C + c) = h;
            const int live = active ? left : 0;
            T* yt = y;
#pragma unroll
            for (int j = 0; j < TPT; ++j, yt += C) {
                if (RESET && ((rst >> j) & 1)) h = u[j];
                else h = add2(h, fma2(em1[j], h, u[j]));
                if (j < live) *reinterpret_cast<typename Pair<T>::Raw*>(yt) = Pair<T>::narrow(h);
            }
        }
    }
    __syncthreads();
    if (cl > 1) cluster_sync_all();  // no peer's map arrives after a CTA has left
    if (threadIdx.x == 0 && ex.abort) atomicExch(&g_gated_status, static_cast<int>(SSD_ERR_TIMEOUT));
}

template <typename T>
__global__ void __launch_bounds__(128) gated_scan_bwd_kernel(GatedScanParams p) {
    constexpr bool EXACT = sizeof(T) == 4;
    const int64_t C = p.channels, L = p.seqlen;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (c >= C) return;
    const float k = -p.scale * softplus_f32(p.decay[c]);
    const int64_t nst = (L + kInterval - 1) / kInterval;
    float carry = p.d_final ? p.d_final[b * C + c] : 0.0f;  // a_{t+1} g_{t+1}
    float sum = 0.0f;
    auto gate = [&](int64_t o, bool rs, float2& r, float2& i, float2& la, float2& em1, float2& a, float2& n) {
        sigmas<EXACT>(dup(to_f32(static_cast<const T*>(p.gate_a)[o])),
                      dup(to_f32(static_cast<const T*>(p.gate_x)[o])), r, i);
        la = mul2(dup(k), r);
        decays<EXACT>(la, false, em1, a);
        if (rs) {
            em1 = dup(-1.0f);
            a = dup(0.0f);
        }
        n = input_weight(em1);
    };
    for (int64_t st = nst - 1; st >= 0; --st) {
        float hp[kInterval];
        float h = p.states[(b * nst + st) * C + c];
        const int64_t t0 = st * kInterval;
        const int n = static_cast<int>(L - t0 < kInterval ? L - t0 : kInterval);
        for (int j = 0; j < n; ++j) {
            const int64_t o = (b * L + t0 + j) * C + c;
            const bool rs = p.reset && p.reset[b * L + t0 + j];
            float2 r, i, la, em1, a, nn;
            gate(o, rs, r, i, la, em1, a, nn);
            hp[j] = h;
            h = (rs ? 0.0f : fmaf(em1.x, h, h)) + nn.x * (i.x * to_f32(static_cast<const T*>(p.x)[o]));
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t o = (b * L + t0 + j) * C + c;
            const bool rs = p.reset && p.reset[b * L + t0 + j];
            float2 r, i, la, em1, a, nn;
            gate(o, rs, r, i, la, em1, a, nn);
            const float x = to_f32(static_cast<const T*>(p.x)[o]);
            const float gt = to_f32(static_cast<const T*>(p.dy)[o]) + carry;
            const float ix = i.x * x;
            static_cast<T*>(p.dx)[o] = from_f32<T>(gt * nn.x * i.x);
            static_cast<T*>(p.dgate_x)[o] = from_f32<T>(gt * nn.x * ix * (1.0f - i.x));
            // a decay of exactly 1 (n = 0) passes a finite dla times la = 0
            const float dla = rs ? 0.0f : gt * a.x * (hp[j] - a.x / fmaxf(nn.x, 1e-18f) * ix);
            static_cast<T*>(p.dgate_a)[o] = from_f32<T>(dla * la.x * (1.0f - r.x));
            sum = fmaf(dla, r.x, sum);
            carry = rs ? 0.0f : fmaf(em1.x, gt, gt);
        }
    }
    if (p.d_init) p.d_init[b * C + c] = carry;
    p.partial[b * C + c] = sum;
}

// ddecay = -scale * sigma(decay) * the sum of dla * r over batch and time
__global__ void __launch_bounds__(kColSumThreads) gated_scan_finish_kernel(GatedScanParams p, int64_t rows) {
    grid_dep_wait();
    column_sums(p.partial, rows, p.channels, [&](int64_t c, float s) {
        p.ddecay[c] = -p.scale * sigma_f32(p.decay[c]) * s;
    });
}

template <typename T>
__global__ void __launch_bounds__(256) gated_update_kernel(GatedUpdateParams p) {
    constexpr bool EXACT = sizeof(T) == 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= p.batch * p.channels) return;
    const int64_t c = i % p.channels;
    grid_dep_wait();
    grid_dep_launch();
    const bool rs = p.reset && p.reset[i / p.channels];
    float2 r, ii, em1, a;
    sigmas<EXACT>(dup(to_f32(static_cast<const T*>(p.gate_a)[i])), dup(to_f32(static_cast<const T*>(p.gate_x)[i])), r, ii);
    decays<EXACT>(mul2(dup(-p.scale * softplus_f32(p.decay[c])), r), false, em1, a);
    if (rs) em1 = dup(-1.0f);
    const float h = p.state[i];
    const float hn = (rs ? 0.0f : fmaf(em1.x, h, h)) +
                     input_weight(em1).x * (ii.x * to_f32(static_cast<const T*>(p.x)[i]));
    p.new_state[i] = hn;
    static_cast<T*>(p.y)[i] = from_f32<T>(hn);
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

// CTAs per cluster: the smallest power of two that gives every SM two CTAs, as
// long as the sequence has tiles for them.
int cluster_size(int64_t blocks, int64_t seqlen, int tile) {
    if (const char* e = getenv("DEV_CL")) return atoi(e);
    int cl = 1;
    const int64_t want = 2 * static_cast<int64_t>(device_sms());
    while (cl < kMaxCluster && blocks * cl < want && static_cast<int64_t>(cl) * tile < seqlen) cl *= 2;
    return cl;
}

template <typename Kern, typename... Args>
cudaError_t launch_clusters(Kern kern, int64_t blocks, int64_t batch, int cl, size_t smem, cudaStream_t s,
                            const Args&... args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess && cl > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * cl), static_cast<unsigned>(batch));
    cfg.blockDim = dim3(TPB);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cl);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cl > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

size_t gated_scan_bwd_partial_bytes(int64_t batch, int64_t, int64_t channels) {
    return static_cast<size_t>(batch) * channels * sizeof(float);
}

template <typename T> cudaError_t launch_gated_scan(const GatedScanParams& p, cudaStream_t s) {
    const int64_t blocks = (p.channels + CPB - 1) / CPB;
    const int cl = cluster_size(blocks * p.batch, p.seqlen, TILE);
    const size_t smem = NW * kStages * 3 * Tile<T, TPT>::kBytes;
    const int wh = static_cast<int>(debug_withhold(SSD_DEBUG_GATED_MAP));
    return p.reset ? launch_clusters(gated_scan_kernel<T, true>, blocks, p.batch, cl, smem, s, p, cl, wh)
                   : launch_clusters(gated_scan_kernel<T, false>, blocks, p.batch, cl, smem, s, p, cl, wh);
}

template <typename T> cudaError_t launch_gated_scan_bwd(const GatedScanParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.channels + 127) / 128), static_cast<unsigned>(p.batch));
    gated_scan_bwd_kernel<T><<<grid, 128, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_kernel(gated_scan_finish_kernel, dim3(static_cast<unsigned>((p.channels + 31) / 32)),
                         dim3(kColSumThreads), 0, s, true, p, p.batch);
}

template <typename T> cudaError_t launch_gated_update(const GatedUpdateParams& p, cudaStream_t s) {
    const int64_t n = p.batch * p.channels;
    return launch_kernel(gated_update_kernel<T>, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                         0, s, true, p);
}

cudaError_t gated_scan_take_status(int* v, cudaStream_t s) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(v, g_gated_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_gated_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e;
}

template cudaError_t launch_gated_scan<float>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan<__nv_bfloat16>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan_bwd<float>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan_bwd<__nv_bfloat16>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_update<float>(const GatedUpdateParams&, cudaStream_t);
template cudaError_t launch_gated_update<__nv_bfloat16>(const GatedUpdateParams&, cudaStream_t);

}  // namespace ssd
