// gated_scan.cu -- the gated linear recurrence, its gradient and its decode
// step (the formulas stand in include/ssd.h).
//
// A step h <- a h + u is an affine map, and maps compose: (A, H) after (A', H')
// is (A A', A H' + H).  So a sequence is cut into groups of consecutive
// tokens, each thread runs its group from zero, the groups' maps are composed,
// and each thread then replays its group from the state that enters it.  The
// replay costs two packed operations per token on values that are still in
// registers, while the gates (about 4 special-function results per element)
// are formed once and the inputs are read once.
//
// A warp takes one group of tokens of 64 channels (a pair per lane); the 8
// warps of a CTA take consecutive groups, and the CTAs of a cluster consecutive
// tiles, whose maps they exchange through distributed shared memory, one
// cluster barrier per round of cluster x tile tokens.  Then every CTA knows the
// state entering its tile and the one entering the next round.  The order of
// composition is fixed, so results do not depend on timing, and there is no
// workspace and no wait on another cluster.
#include "mixers.h"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int kInterval = SSD_GATED_SCAN_INTERVAL;
constexpr int NW = 8;            // warps (groups) per CTA
constexpr int TPB = NW * 32;
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
__device__ __forceinline__ float exp2_scaled(float v, float hi, float lo, float top = 126.0f) {
    if constexpr (EXACT) v = min_nan(max_nan(v, -200.0f), 200.0f);  // no infinite products below
    const float t = min_nan(v * hi, top);
    float e = ex2_approx(t);
    if constexpr (EXACT) {
        const float d = fmaf(v, lo, fmaf(v, hi, -(v * hi)));  // what t lost
        e = fmaf(e, d * 0.69314718f, e);
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
    const float2 ea = add2(make_float2(exp2_scaled<EXACT>(ga.x, -kLog2eHi, -kLog2eLo),
                                       exp2_scaled<EXACT>(ga.y, -kLog2eHi, -kLog2eLo)), one);
    const float2 ex = add2(make_float2(exp2_scaled<EXACT>(gx.x, -kLog2eHi, -kLog2eLo, 60.0f),
                                       exp2_scaled<EXACT>(gx.y, -kLog2eHi, -kLog2eLo, 60.0f)), one);
    const float2 d = mul2(ea, ex);
    const float2 inv = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    r = mul2(inv, ex);
    i = mul2(inv, ea);
}

// em1 = a - 1 = e^la - 1 (la <= 0) and a.  a = 1 + em1 enters the recurrence as
// h + em1 h, so that a decay near 1 keeps its relative accuracy in la, and
// 1 - a^2 = -em1 (2 + em1) without cancellation.  Below -1/4 from e^la, above
// from the Taylor series to the seventh power (cut off at 2^-24 of em1); the usual decays
// (a slowest one of 0.9 to 0.999 per channel) take the series only, which
// saves them a special-function result.
template <bool EXACT>
__device__ __forceinline__ void decays(float2 la, float2& em1, float2& a) {
    float2 q = dup(1.0f / 5040.0f);
    q = fma2(q, la, dup(1.0f / 720.0f));
    q = fma2(q, la, dup(1.0f / 120.0f));
    q = fma2(q, la, dup(1.0f / 24.0f));
    q = fma2(q, la, dup(1.0f / 6.0f));
    q = fma2(q, la, dup(0.5f));
    em1 = fma2(mul2(q, la), la, la);
    a = add2(em1, dup(1.0f));
    if (la.x < -0.25f) {
        a.x = exp2_scaled<EXACT>(la.x, kLog2eHi, kLog2eLo);
        em1.x = a.x - 1.0f;
    }
    if (la.y < -0.25f) {
        a.y = exp2_scaled<EXACT>(la.y, kLog2eHi, kLog2eLo);
        em1.y = a.y - 1.0f;
    }
}
// sqrt(1 - a^2)
__device__ __forceinline__ float2 input_weight(float2 em1) {
    const float2 n2 = mul2(make_float2(-em1.x, -em1.y), add2(em1, dup(2.0f)));
    return make_float2(sqrt_approx(n2.x), sqrt_approx(n2.y));
}
// -scale * softplus(decay) of a pair of channels (0 outside them)
__device__ __forceinline__ float2 decay_rates(const GatedScanParams& p, int64_t c, bool active) {
    return active ? make_float2(-p.scale * softplus_f32(p.decay[c]), -p.scale * softplus_f32(p.decay[c + 1]))
                  : dup(0.0f);
}
__device__ __forceinline__ float sigma_f32(float v) { return 1.0f / (1.0f + expf(-v)); }

// ---- clusters ----
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float4 into the same shared variable of the cluster's CTA `rank`
__device__ __forceinline__ void store_remote(const float4* mine, int rank, float4 v) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                 :
                 : "r"(r), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void store_remote(const int* mine, int rank, int v) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.s32 [%0], %1;" : : "r"(r), "r"(v) : "memory");
}

// ---- a warp's tile of one array: TPT rows of 64 channels, by 16-byte copies ----
template <typename T, int TPT> struct Tile {
    static constexpr int kRowBytes = CPB * sizeof(T);
    static constexpr int kBytes = TPT * kRowBytes;
    // rows t0 .. t0 + TPT - 1 of src [L][C], from channel c0; zeros past L and C
    static __device__ __forceinline__ void load(uint8_t* dst, const T* src, int64_t t0, int64_t L, int64_t c0,
                                                int64_t C, int lane) {
        constexpr int CH = kRowBytes / 16;  // chunks per row
#pragma unroll
        for (int k = 0; k < TPT * CH / 32; ++k) {
            const int row = (lane + 32 * k) / CH, ch = (lane + 32 * k) % CH;
            const int64_t c = c0 + ch * (16 / static_cast<int>(sizeof(T)));
            const bool in = t0 + row < L && c < C;
            const T* g = in ? src + (t0 + row) * C + c : src;
            const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(dst + row * kRowBytes + ch * 16));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         :
                         : "r"(s), "l"(g), "r"(in ? 16 : 0)
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

template <typename T> constexpr int kFwdTokens = sizeof(T) == 2 ? 16 : 8;  // tokens per thread

template <typename T, bool RESET>
__global__ void __launch_bounds__(TPB, 2) gated_scan_kernel(GatedScanParams p, int cl) {
    constexpr int TPT = kFwdTokens<T>;
    constexpr int TILE = NW * TPT;
    constexpr bool EXACT = sizeof(T) == 4;
    using TL = Tile<T, TPT>;
    extern __shared__ __align__(16) uint8_t ring[];    // [NW][3] tiles
    __shared__ float4 group_map[2][NW][32];             // this CTA's groups
    __shared__ float4 tile_map[2][kMaxCluster][32];     // the cluster's tiles
    __shared__ int group_rst[2][NW], tile_rst[2][kMaxCluster];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t C = p.channels, L = p.seqlen, b = blockIdx.y;
    const int rank = static_cast<int>(blockIdx.x) % cl;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x / cl) * CPB, c = c0 + 2 * lane;
    const bool active = c < C;
    const T* x = static_cast<const T*>(p.x) + b * L * C;
    const T* ga = static_cast<const T*>(p.gate_a) + b * L * C;
    const T* gx = static_cast<const T*>(p.gate_x) + b * L * C;
    T* y = static_cast<T*>(p.y) + b * L * C + c;
    const int64_t nst = (L + kInterval - 1) / kInterval;
    uint8_t* tiles = ring + warp * 3 * TL::kBytes;
    auto fetch = [&](int64_t t0) {
        TL::load(tiles, x, t0, L, c0, C, lane);
        TL::load(tiles + TL::kBytes, ga, t0, L, c0, C, lane);
        TL::load(tiles + 2 * TL::kBytes, gx, t0, L, c0, C, lane);
        copies_commit();
    };
    const int64_t round = static_cast<int64_t>(cl) * TILE;
    int64_t t0 = static_cast<int64_t>(rank) * TILE + warp * TPT;
    fetch(t0);
    const float2 k = decay_rates(p, c, active);
    float2 carry = (active && p.init_state) ? *reinterpret_cast<const float2*>(p.init_state + b * C + c)
                                            : dup(0.0f);
    if (cl > 1) {  // every CTA of the cluster runs before its shared memory is written
        cluster_arrive();
        cluster_wait();
    }
    int buf = 0;
    for (int64_t tr = 0; tr < L; tr += round, t0 += round, buf ^= 1) {
        uint32_t rst = 0;
        if constexpr (RESET) rst = reset_mask<TPT>(p.reset, b, t0, L, lane);
        copies_wait<0>();
        __syncwarp();
        float2 em1[TPT], u[TPT];
#pragma unroll
        for (int j = 0; j < TPT; ++j) {
            float2 r, i, a;
            sigmas<EXACT>(TL::read(tiles + TL::kBytes, j, lane), TL::read(tiles + 2 * TL::kBytes, j, lane), r, i);
            decays<EXACT>(mul2(k, r), em1[j], a);
            float2 n = input_weight(em1[j]);
            if (RESET && ((rst >> j) & 1)) n = dup(1.0f);
            u[j] = mul2(mul2(n, i), TL::read(tiles, j, lane));
        }
        __syncwarp();
        if (tr + round < L) fetch(t0 + round);
        // tokens past the end change nothing
        if (t0 + TPT > L) {
#pragma unroll
            for (int j = 0; j < TPT; ++j)
                if (t0 + j >= L) em1[j] = u[j] = dup(0.0f);
        }
        // the group's map
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
        group_map[buf][warp][lane] = make_float4(A.x, A.y, H.x, H.y);
        if (RESET && lane == 0) group_rst[buf][warp] = rst != 0;
        __syncthreads();
        // the state entering the group: carry, the tiles before, the groups before
        float2 h = carry;
        if (cl > 1) {
            // warps 0 .. cl - 1 (twice around for clusters beyond NW) send the tile's map
            float4 m = group_map[buf][0][lane];
            int any = RESET ? group_rst[buf][0] : 0;
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                const float4 g = group_map[buf][w][lane];
                const bool gr = RESET && group_rst[buf][w];
                const float2 hh = apply(g, gr, make_float2(m.z, m.w));
                const float2 aa = gr ? dup(0.0f) : mul2(make_float2(g.x, g.y), make_float2(m.x, m.y));
                m = make_float4(aa.x, aa.y, hh.x, hh.y);
                any |= gr;
            }
            for (int to = warp; to < cl; to += NW) {
                store_remote(&tile_map[buf][rank][lane], to, m);
                if (RESET && lane == 0) store_remote(&tile_rst[buf][rank], to, any);
            }
            cluster_arrive();
            cluster_wait();
            for (int q = 0; q < cl; ++q) {
                if (q == rank) h = carry;
                carry = apply(tile_map[buf][q][lane], RESET && tile_rst[buf][q], carry);
            }
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w == warp && cl > 1) break;
            const float2 v = apply(group_map[buf][w][lane], RESET && group_rst[buf][w], cl > 1 ? h : carry);
            if (cl > 1) {
                h = v;
            } else {
                if (w == warp) h = carry;
                carry = v;
            }
        }
        if (active && p.states && t0 < L && t0 % kInterval == 0)
            *reinterpret_cast<float2*>(p.states + (b * nst + t0 / kInterval) * C + c) = h;
#pragma unroll
        for (int j = 0; j < TPT; ++j) {
            if (RESET && ((rst >> j) & 1)) h = u[j];
            else h = add2(h, fma2(em1[j], h, u[j]));
            if (active && t0 + j < L)
                *reinterpret_cast<typename Pair<T>::Raw*>(y + (t0 + j) * C) = Pair<T>::narrow(h);
        }
    }
    if (p.final_state && active && rank == 0 && warp == 0)
        *reinterpret_cast<float2*>(p.final_state + b * C + c) = carry;
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
        decays<EXACT>(la, em1, a);
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
    decays<EXACT>(mul2(dup(-p.scale * softplus_f32(p.decay[c])), r), em1, a);
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
    constexpr int TPT = kFwdTokens<T>;
    const int64_t blocks = (p.channels + CPB - 1) / CPB;
    const int cl = cluster_size(blocks * p.batch, p.seqlen, NW * TPT);
    const size_t smem = NW * 3 * Tile<T, TPT>::kBytes;
    return p.reset ? launch_clusters(gated_scan_kernel<T, true>, blocks, p.batch, cl, smem, s, p, cl)
                   : launch_clusters(gated_scan_kernel<T, false>, blocks, p.batch, cl, smem, s, p, cl);
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

template cudaError_t launch_gated_scan<float>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan<__nv_bfloat16>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan_bwd<float>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_scan_bwd<__nv_bfloat16>(const GatedScanParams&, cudaStream_t);
template cudaError_t launch_gated_update<float>(const GatedUpdateParams&, cudaStream_t);
template cudaError_t launch_gated_update<__nv_bfloat16>(const GatedUpdateParams&, cudaStream_t);

}  // namespace ssd
