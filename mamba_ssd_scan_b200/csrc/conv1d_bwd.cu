// conv1d_bwd.cu -- the gradients of the causal depthwise convolution (the
// formulas stand in include/ssd.h).
//
// A warp takes 64 channels (a pair per lane) over a segment of the sequence
// and walks its tokens with two sliding windows in registers: the K inputs
// that feed the token's output, and the last K gradients before the
// activation, whose weighted sum is the gradient of the input K - 1 tokens
// back.  A segment runs K - 1 tokens past its end to finish its inputs'
// gradients (it recomputes those tokens' gradients; their share of dweight
// belongs to the next segment).  The warps of a CTA take consecutive segments
// and add their dweight and dbias in shared memory; one row per CTA goes to
// the workspace, and a second kernel adds the rows in order.
#include "mixers.h"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int NW = 8;     // warps (segments) per CTA
constexpr int CPW = 64;   // channels per warp

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }

// silu'(o) = sg (1 + o (1 - sg)), sg = sigma(o)
__device__ __forceinline__ float dsilu(float o) {
    const float sg = 1.0f / (1.0f + __expf(-o));
    return sg * fmaf(o, 1.0f - sg, 1.0f);
}

template <typename T, int K, bool ACT>
__global__ void __launch_bounds__(NW * 32) conv1d_bwd_kernel(ConvBwdParams p, int64_t seg) {
    using P = Pair<T>;
    __shared__ float2 red[NW][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t L = p.seqlen, Cn = p.channels, b = blockIdx.z;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * CPW + 2 * lane;
    const bool active = c < Cn;
    const int64_t ta = (static_cast<int64_t>(blockIdx.y) * NW + warp) * seg;
    const int64_t te = ta + seg < L ? ta + seg : L;
    float2 w[K], dw[K], bias = dup(0.0f), db = dup(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = active ? make_float2(p.weight[c * K + k], p.weight[(c + 1) * K + k]) : dup(0.0f);
        dw[k] = dup(0.0f);
    }
    if (active && p.bias) bias = make_float2(p.bias[c], p.bias[c + 1]);
    const T* xb = static_cast<const T*>(p.x) + b * L * Cn + c;
    const T* yb = static_cast<const T*>(p.dy) + b * L * Cn + c;
    T* db_x = static_cast<T*>(p.dx) + b * L * Cn + c;
    if (active && ta < L) {
        float2 xw[K], dw_[K];  // xin[t-(K-1) .. t], do[t .. t-(K-1)]
#pragma unroll
        for (int k = 0; k < K; ++k) {
            dw_[k] = dup(0.0f);
            const int64_t i = ta - K + k;  // shifted by one when token ta enters
            if (k == 0) xw[k] = dup(0.0f);
            else if (i >= 0) xw[k] = P::widen(*reinterpret_cast<const typename P::Raw*>(xb + i * Cn));
            else if (p.init_state)
                xw[k] = make_float2(p.init_state[(b * Cn + c) * (K - 1) + (K - 1 + i)],
                                    p.init_state[(b * Cn + c + 1) * (K - 1) + (K - 1 + i)]);
            else xw[k] = dup(0.0f);
        }
        const int64_t tend = te + K - 1;
        for (int64_t t = ta; t < tend; ++t) {
            float2 x = dup(0.0f), d = dup(0.0f);
            if (t < L) {
                x = P::widen(*reinterpret_cast<const typename P::Raw*>(xb + t * Cn));
                d = P::widen(*reinterpret_cast<const typename P::Raw*>(yb + t * Cn));
            }
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) xw[k] = xw[k + 1];
            xw[K - 1] = x;
            if (ACT && t < L) {
                float2 o = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) o = fma2(w[k], xw[k], o);
                d.x *= dsilu(o.x);
                d.y *= dsilu(o.y);
            }
            if (t < te) {
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k] = fma2(d, xw[k], dw[k]);
                db.x += d.x;
                db.y += d.y;
            }
#pragma unroll
            for (int k = K - 1; k > 0; --k) dw_[k] = dw_[k - 1];
            dw_[0] = d;
            const int64_t i = t - (K - 1);
            if (i < ta && !(ta == 0 && i < 0)) continue;
            float2 g = dup(0.0f);
#pragma unroll
            for (int k = 0; k < K; ++k) g = fma2(w[k], dw_[k], g);
            if (t >= L && p.d_final) {
                g.x += p.d_final[(b * Cn + c) * (K - 1) + (t - L)];
                g.y += p.d_final[(b * Cn + c + 1) * (K - 1) + (t - L)];
            }
            if (i >= 0) {
                *reinterpret_cast<typename P::Raw*>(db_x + i * Cn) = P::narrow(g);
            } else if (p.d_init) {
                p.d_init[(b * Cn + c) * (K - 1) + t] = g.x;
                p.d_init[(b * Cn + c + 1) * (K - 1) + t] = g.y;
            }
        }
    }
    // the CTA's sums, segment after segment; row [K + 1][Cn], dbias last
    float* row = p.partial + (b * gridDim.y + blockIdx.y) * (K + 1) * Cn;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        __syncthreads();
        red[warp][lane] = k < K ? dw[k < K ? k : 0] : db;
        __syncthreads();
        if (warp == 0 && active) {
            float2 v = dup(0.0f);
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                v.x += red[j][lane].x;
                v.y += red[j][lane].y;
            }
            *reinterpret_cast<float2*>(row + k * Cn + c) = v;
        }
    }
}

__global__ void __launch_bounds__(kColSumThreads) conv1d_bwd_finish_kernel(ConvBwdParams p, int64_t rows) {
    grid_dep_wait();
    const int64_t K = p.width, Cn = p.channels;
    column_sums(p.partial, rows, (K + 1) * Cn, [&](int64_t i, float s) {
        const int64_t k = i / Cn, c = i - k * Cn;
        if (k < K) p.dweight[c * K + k] = s;
        else if (p.dbias) p.dbias[c] = s;
    });
}

// Segments: enough warps for about eight per SM scheduler, at least 32 tokens
// each (the K - 1 tokens past a segment's end are computed twice).
struct ConvGrid {
    int64_t seg, rows;
    unsigned gx, gy;
};
ConvGrid conv_grid(int64_t batch, int64_t seqlen, int64_t channels) {
    ConvGrid g;
    const int64_t nblk = (channels + CPW - 1) / CPW;
    const int64_t want = 148 * 32;  // warps
    int64_t nseg = want / (nblk * batch);
    if (nseg < 1) nseg = 1;
    g.seg = (seqlen + nseg - 1) / nseg;
    if (g.seg < 32) g.seg = 32;
    nseg = (seqlen + g.seg - 1) / g.seg;
    g.gx = static_cast<unsigned>(nblk);
    g.gy = static_cast<unsigned>((nseg + NW - 1) / NW);
    g.rows = batch * g.gy;
    return g;
}

template <typename T, int K> cudaError_t launch_k(const ConvBwdParams& p, cudaStream_t s) {
    const ConvGrid g = conv_grid(p.batch, p.seqlen, p.channels);
    const dim3 grid(g.gx, g.gy, static_cast<unsigned>(p.batch));
    if (p.activation) conv1d_bwd_kernel<T, K, true><<<grid, NW * 32, 0, s>>>(p, g.seg);
    else conv1d_bwd_kernel<T, K, false><<<grid, NW * 32, 0, s>>>(p, g.seg);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t cols = (p.width + 1) * p.channels;
    return launch_kernel(conv1d_bwd_finish_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)),
                         dim3(kColSumThreads), 0, s, true, p, g.rows);
}

}  // namespace

size_t conv1d_bwd_partial_bytes(int64_t batch, int64_t seqlen, int64_t channels, int64_t width) {
    return static_cast<size_t>(conv_grid(batch, seqlen, channels).rows) * (width + 1) * channels * sizeof(float);
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

}  // namespace ssd
