// conv1d_bwd.cu -- the gradients of the causal depthwise convolution (the
// formulas stand in include/ssd.h).
//
// Bandwidth-bound: x and dy are read once and dx written once.  A warp takes 64
// channels (a pair per lane) over a segment of the sequence, in batches of 16
// tokens (8 of fp32) that TMA brings into its own ring of shared-memory tiles.
// It takes eight tokens of a batch at a time and keeps
// two windows in registers: the K inputs that feed a token's output, and the
// last K gradients before the activation, whose weighted sum is the gradient
// of the input K - 1 tokens back.  dx takes the place of x in the tile and
// leaves by a TMA store; a segment's first and last K - 1 rows, which its
// neighbours' tiles overlap, go out directly.  A segment runs K - 1 tokens past
// its end to finish its inputs' gradients (it forms those tokens' gradients
// again; their share of dweight belongs to the next segment).  Each warp
// leaves its sums of dweight and dbias in a row of the workspace, and a second
// kernel adds the rows in order.
//
// Measured (B200, L2 flushed; share of the measured copy bandwidth over the
// call's least bytes), K 4 with SiLU: bf16 b1 L65536 C5376 378 us (87 %), b8 L4096
// C2304 97 us (72 %); fp32 b8 L4096 C1536 119 us (79 %).  A call costs 0.15 us per
// token of a segment and about 17 us besides (the launch, filling the ring, the
// segments' ends, the sums' kernel); issue slots are 55 % busy (44 instructions per
// channel pair and token), the FMA pipe 53 %, the special-function pipe 41 %.
#include <type_traits>
#include "mixers.h"
#include "rows_tma.cuh"
#include "tcgen05.cuh"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int NW = 8;     // warps (segments) per CTA
constexpr int CPW = 64;   // channels per warp
constexpr int SB = 8;     // tokens at a time (at least K - 1)
// Tokens per batch: tiles of 2 KB.  Of half that (8 tokens of bf16) the TMA
// requests are twice as many, b1 L65536 C5376 K4 took 394 us instead of 372.
template <typename T> constexpr int kBatch = sizeof(T) == 2 ? 16 : 8;
constexpr int kSegUnit = 16;  // segments are whole batches of either type
// CTAs per SM: two, whose 128 registers a thread let the tokens of a batch overlap
// (b8 L4096 C2304 K4, batches of 8: 100 us; three at 80 registers 109, four at 64
// 130; windows of four tokens instead of eight, two CTAs 108, three 112)
constexpr int kPerSm = 2;
constexpr int kRing = 3;  // batches in shared memory
template <typename T> constexpr int kRowBytes = CPW * sizeof(T);
template <typename T> constexpr int kWarpBytes = kRing * 2 * kBatch<T> * kRowBytes<T>;  // x and dy tiles

// Warps that gave up on a wait (ssd_conv1d_check_status).
__device__ uint32_t g_conv_bwd_gave_up;

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
// silu'(o) = sg (1 + o (1 - sg)), sg = 1 / (1 + 2^(-o log2 e)); where the power
// overflows, sg = 0
__device__ __forceinline__ float2 dsilu2(float2 o) {
    const float2 t = mul2(o, dup(-1.4426950408889634f));
    const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), dup(1.0f));
    const float2 sg = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    return mul2(sg, fma2(o, fma2(sg, dup(-1.0f), dup(1.0f)), dup(1.0f)));
}

// Bounded wait on a batch: a probe suspends the warp until the copies have landed or 2
// us have passed, and after about a second it gives up.
__device__ __forceinline__ bool wait_loaded(uint32_t mbar, uint32_t parity) {
    for (uint32_t i = 0; i < 1u << 19; ++i)
        if (tc::mbar_try_wait_hint(mbar, parity, 2000)) return true;
    return false;
}

struct ConvBwdMaps {
    CUtensorMap x, dy, dx;
};

// segments of seg tokens (a multiple of kSegUnit), nseg per (batch, channel block).
// `withhold` = 0, 1, 2 makes the first warp leave that batch out (a test of the bounded
// wait); -1 in normal use.
template <typename T, int K, bool ACT>
__global__ void __launch_bounds__(NW * 32, kPerSm)
    conv1d_bwd_kernel(ConvBwdParams p, const __grid_constant__ ConvBwdMaps maps, int64_t seg, int nseg, int64_t warps,
                      int withhold) {
    using P = Pair<T>;
    using Raw = typename P::Raw;
    constexpr int R = kRing, KM = K - 1, TB = kBatch<T>;
    constexpr uint32_t kTile = TB * kRowBytes<T>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t loaded[NW][R];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t wi = static_cast<int64_t>(blockIdx.x) * NW + warp;
    if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) tc::mbar_init(tc::smem_u32(&loaded[warp][r]), 1);
        tc::fence_mbar_init();
    }
    __syncwarp();
    if (wi >= warps) return;  // (warps are independent: no barrier follows)
    const int64_t L = p.seqlen, Cn = p.channels;
    const int64_t nblk = (Cn + CPW - 1) / CPW;
    const int64_t s = wi / (nblk * p.batch), col = wi - s * (nblk * p.batch);  // neighbours: one row of blocks
    const int64_t b = col / nblk, c0 = (col - b * nblk) * CPW, c = c0 + 2 * lane;
    const bool active = c < Cn;
    const int64_t ta = s * seg, te = ta + seg < L ? ta + seg : L;
    const int nb = static_cast<int>((te - ta + TB - 1) / TB);  // whole batches, then one for the K - 1 tokens after
    const int total = nb + (K > 1 ? 1 : 0);

    uint8_t* ring = smem + warp * kWarpBytes<T>;
    auto load = [&](int n) {
        const uint32_t dst = tc::smem_u32(ring) + (n % R) * 2 * kTile, bar = tc::smem_u32(&loaded[warp][n % R]);
        const int t = static_cast<int>(ta + static_cast<int64_t>(n) * TB);
        tc::mbar_expect_tx(bar, 2 * kTile);
        tc::tma_load_rows(dst, &maps.x, bar, static_cast<int>(c0), t, static_cast<int>(b));
        tc::tma_load_rows(dst + kTile, &maps.dy, bar, static_cast<int>(c0), t, static_cast<int>(b));
    };
    if (lane == 0)
        for (int n = 0; n < R && n < total; ++n)
            if (n != withhold || wi > 0) load(n);

    float2 w[K], dw[K], bias = dup(0.0f), db = dup(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = active ? make_float2(p.weight[c * K + k], p.weight[(c + 1) * K + k]) : dup(0.0f);
        dw[k] = dup(0.0f);
    }
    if (active && p.bias) bias = make_float2(p.bias[c], p.bias[c + 1]);
    const T* xb = static_cast<const T*>(p.x) + b * L * Cn + c;
    T* dxb = static_cast<T*>(p.dx) + b * L * Cn + c;
    // xw[KM + j]: the input of token j of the eight; xw[0 .. KM - 1] the K - 1 before.
    // dv alike: the gradients before the activation.
    float2 xw[KM + SB], dv[KM + SB];
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        dv[k] = dup(0.0f);
        xw[k] = dup(0.0f);
        const int64_t i = ta - KM + k;
        if (active && i >= 0) xw[k] = P::widen(*reinterpret_cast<const Raw*>(xb + i * Cn));
        else if (active && p.init_state)
            xw[k] = make_float2(p.init_state[(b * Cn + c) * KM + (KM + i)],
                                p.init_state[(b * Cn + c + 1) * KM + (KM + i)]);
    }
    // token j of eight: its input and its gradient before the activation
    auto token = [&](const uint8_t* tile, int j) {
        xw[KM + j] = P::widen(*reinterpret_cast<const Raw*>(tile + j * kRowBytes<T>));
        float2 d = P::widen(*reinterpret_cast<const Raw*>(tile + kTile + j * kRowBytes<T>));
        if (ACT) {
            float2 o = bias;
#pragma unroll
            for (int k = 0; k < K; ++k) o = fma2(w[k], xw[j + k], o);
            d = mul2(d, dsilu2(o));
        }
        dv[KM + j] = d;
    };
    auto sums = [&](int j) {
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k] = fma2(dv[KM + j], xw[j + k], dw[k]);
        db = add2(db, dv[KM + j]);
    };
    // the gradient of the input K - 1 tokens before token j
    auto input_gradient = [&](int j) {
        float2 g = mul2(w[0], dv[KM + j]);
#pragma unroll
        for (int k = 1; k < K; ++k) g = fma2(w[k], dv[KM + j - k], g);
        return g;
    };
    // Eight tokens from t on of a segment's first batch or its last (the halo), or with
    // tokens past the sequence's end (`past`): these have no gradient and no share in
    // the sums, whatever the inputs before them (0 times an infinite one is not 0).
    auto edge = [&](uint8_t* tile, int64_t t, int n, auto past) {
        constexpr bool PAST = decltype(past)::value;
        const bool halo = n == nb;
#pragma unroll
        for (int j = 0; j < SB; ++j) {
            token(tile, j);
            const bool end = PAST && t + j >= L;
            if (end) dv[KM + j] = dup(0.0f);
            if (!halo && !end) sums(j);
            float2 g = input_gradient(j);
            const int64_t f = t + j - L;
            if (PAST && f >= 0 && f < KM && p.d_final && active) {  // inputs the final state repeats
                g.x += p.d_final[(b * Cn + c) * KM + f];
                g.y += p.d_final[(b * Cn + c + 1) * KM + f];
            }
            const int64_t i = t + j - KM;
            if (n > 0 && !halo) {
                *reinterpret_cast<Raw*>(tile + j * kRowBytes<T>) = P::narrow(g);
            } else if (active) {
                if (halo ? (j < KM && i < te) : i >= ta) {
                    if (i < L) *reinterpret_cast<Raw*>(dxb + i * Cn) = P::narrow(g);
                } else if (n == 0 && i < 0 && p.d_init) {
                    p.d_init[(b * Cn + c) * KM + (KM + i)] = g.x;
                    p.d_init[(b * Cn + c + 1) * KM + (KM + i)] = g.y;
                }
            }
        }
    };
    int late = total;  // the batch whose wait gave up
    for (int n = 0; n < total; ++n) {
        uint8_t* tile = ring + (n % R) * 2 * kTile + lane * sizeof(Raw);
        const int64_t t0 = ta + static_cast<int64_t>(n) * TB;
        const bool halo = n == nb;
        if (!__all_sync(0xffffffffu, wait_loaded(tc::smem_u32(&loaded[warp][n % R]), (n / R) & 1))) {
            late = n;
            break;
        }
        const bool whole = n > 0 && !halo && t0 + TB <= L;  // inside the segment, without a condition
#pragma unroll 1
        for (int o = 0; o < (halo ? SB : TB); o += SB, tile += SB * kRowBytes<T>) {
            if (whole) {
#pragma unroll
                for (int j = 0; j < SB; ++j) {
                    token(tile, j);
                    sums(j);
                    *reinterpret_cast<Raw*>(tile + j * kRowBytes<T>) = P::narrow(input_gradient(j));
                }
            } else if (t0 + o + SB <= L) {
                edge(tile, t0 + o, n, std::false_type());
            } else {
                edge(tile, t0 + o, n, std::true_type());
            }
#pragma unroll
            for (int k = 0; k < KM; ++k) {
                xw[k] = xw[SB + k];
                dv[k] = dv[SB + k];
            }
        }
        if (n > 0 && !halo) tc::fence_smem_async();
        __syncwarp();
        if (lane == 0) {
            if (n > 0 && !halo) {
                tc::tma_store_rows(&maps.dx, tc::smem_u32(ring) + (n % R) * 2 * kTile, static_cast<int>(c0),
                                   static_cast<int>(t0 - KM), static_cast<int>(b));
            }
            tc::bulk_commit_group();
            // the previous batch's store has read its tile: it takes the batch R - 1 ahead
            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            if (n > 0 && n - 1 + R < total) load(n - 1 + R);
        }
    }
    if (lane == 0) tc::bulk_wait_all();
    if (late < total) {
        // the copies in flight land (bounded) before the warp leaves its shared memory
        const int issued = late > 0 ? late - 1 + R : R;
        for (int n = late; n < issued && n < total; ++n)
            wait_loaded(tc::smem_u32(&loaded[warp][n % R]), (n / R) & 1);
        if (lane == 0) atomicAdd(&g_conv_bwd_gave_up, 1u);
        return;
    }
    if (active) {  // row [K + 1][Cn], dbias last
        float* row = p.partial + (b * nseg + s) * (K + 1) * Cn + c;
#pragma unroll
        for (int k = 0; k <= K; ++k) *reinterpret_cast<float2*>(row + k * Cn) = k < K ? dw[k < K ? k : 0] : db;
    }
}

constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(kSumWarps * 32) conv1d_bwd_finish_kernel(ConvBwdParams p, int64_t rows) {
    grid_dep_wait();
    const int64_t K = p.width, Cn = p.channels;
    column_sums<kSumWarps>(p.partial, rows, (K + 1) * Cn, [&](int64_t i, float s) {
        const int64_t k = i / Cn, c = i - k * Cn;
        if (k < K) p.dweight[c * K + k] = s;
        else if (p.dbias) p.dbias[c] = s;
    });
}

// Segments: the number, up to one per 32 tokens, with the least waves x (tokens
// of a segment + the batch it loads past its end, 16), at the warps the device
// holds at once.  The addend hardly matters, since the least is nearly always one
// full wave: 1, 16, 64 and 113 measured the same at ten sizes from b1 L1030 C64 to
// b1 L65536 C5376.
struct ConvGrid {
    int64_t seg, nseg, warps;
};
ConvGrid conv_grid(int64_t batch, int64_t seqlen, int64_t channels) {
    const int64_t cols = (channels + CPW - 1) / CPW * batch, slots = int64_t{148} * kPerSm * NW;
    ConvGrid best{};
    int64_t least = 0;
    for (int64_t n = 1; n <= 1024 && (n == 1 || (seqlen + n - 1) / n >= 32); ++n) {
        ConvGrid g;
        g.seg = ((seqlen + n - 1) / n + kSegUnit - 1) / kSegUnit * kSegUnit;
        g.nseg = (seqlen + g.seg - 1) / g.seg;
        g.warps = cols * g.nseg;
        const int64_t cost = (g.warps + slots - 1) / slots * (g.seg + 16);
        if (least == 0 || cost < least) {
            least = cost;
            best = g;
        }
    }
    return best;
}

template <typename T, int K, bool ACT>
cudaError_t launch_act(const ConvBwdParams& p, const ConvBwdMaps& m, const ConvGrid& g, cudaStream_t s) {
    constexpr int smem = NW * kWarpBytes<T>;
    const cudaError_t e = prepare_kernel<conv1d_bwd_kernel<T, K, ACT>>(smem, false);
    if (e != cudaSuccess) return e;
    const auto ctas = static_cast<unsigned>((g.warps + NW - 1) / NW);
    conv1d_bwd_kernel<T, K, ACT>
        <<<ctas, NW * 32, smem, s>>>(p, m, g.seg, static_cast<int>(g.nseg), g.warps,
                                     static_cast<int>(debug_withhold(SSD_DEBUG_CONV_TILE)));
    return cudaGetLastError();
}

template <typename T, int K> cudaError_t launch_k(const ConvBwdParams& p, cudaStream_t s) {
    const ConvGrid g = conv_grid(p.batch, p.seqlen, p.channels);
    ConvBwdMaps m;
    const bool bf16 = sizeof(T) == 2;
    if (!make_tmap_rows(&m.x, p.x, bf16, p.channels, p.seqlen, p.batch, kBatch<T>) ||
        !make_tmap_rows(&m.dy, p.dy, bf16, p.channels, p.seqlen, p.batch, kBatch<T>) ||
        !make_tmap_rows(&m.dx, p.dx, bf16, p.channels, p.seqlen, p.batch, kBatch<T>))
        return cudaErrorInvalidValue;
    const cudaError_t e = p.activation ? launch_act<T, K, true>(p, m, g, s) : launch_act<T, K, false>(p, m, g, s);
    if (e != cudaSuccess) return e;
    const int64_t cols = (p.width + 1) * p.channels;
    return launch_kernel(conv1d_bwd_finish_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)),
                         dim3(kSumWarps * 32), 0, s, true, p, p.batch * g.nseg);
}

}  // namespace

size_t conv1d_bwd_partial_bytes(int64_t batch, int64_t seqlen, int64_t channels, int64_t width) {
    return static_cast<size_t>(batch * conv_grid(batch, seqlen, channels).nseg) * (width + 1) *
           channels * sizeof(float);
}

template <typename T> cudaError_t launch_conv1d_bwd(const ConvBwdParams& p, cudaStream_t s) {
    switch (p.width) {
        case 1: return launch_k<T, 1>(p, s);
        case 2: return launch_k<T, 2>(p, s);
        case 3: return launch_k<T, 3>(p, s);
        case 4: return launch_k<T, 4>(p, s);
        case 5: return launch_k<T, 5>(p, s);
        case 6: return launch_k<T, 6>(p, s);
        case 7: return launch_k<T, 7>(p, s);
        case 8: return launch_k<T, 8>(p, s);
        default: return cudaErrorInvalidValue;
    }
}

template cudaError_t launch_conv1d_bwd<float>(const ConvBwdParams&, cudaStream_t);
template cudaError_t launch_conv1d_bwd<__nv_bfloat16>(const ConvBwdParams&, cudaStream_t);

cudaError_t conv1d_bwd_take_status(int* v, cudaStream_t s) {
    static GaveUp gave_up;
    return gave_up.take(g_conv_bwd_gave_up, v, s);
}

}  // namespace ssd
