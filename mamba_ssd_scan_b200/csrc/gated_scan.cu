// gated_scan.cu -- the gated linear recurrence, its gradient and its decode
// step (the formulas stand in include/ssd.h).
//
// One thread per (batch, channel) walks the sequence.
#include "mixers.h"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int kInterval = SSD_GATED_SCAN_INTERVAL;

// The decay and the input weight of one element.  With la = log a, both come
// from em1 = e^la - 1, formed without cancellation: a = 1 + em1 enters the
// recurrence as h + em1 h (so a decay near 1 keeps its relative accuracy in
// la), and 1 - a^2 = -em1 (2 + em1).  a itself, where the gradient scales with
// it, is e^la once it is small (1 + em1 would lose it).
struct Gates {
    float r, i, la, em1, a, n;
};
__device__ __forceinline__ float sigma_f32(float v) { return 1.0f / (1.0f + expf(-v)); }
// c = -scale * softplus(decay)
__device__ __forceinline__ Gates gates(float ga, float gx, float c, bool reset) {
    Gates g;
    g.r = sigma_f32(ga);
    g.i = sigma_f32(gx);
    g.la = c * g.r;
    g.em1 = reset ? -1.0f : expm1f(g.la);
    g.a = reset ? 0.0f : (g.la < -0.25f ? expf(g.la) : 1.0f + g.em1);
    g.n = sqrtf(-g.em1 * (2.0f + g.em1));
    return g;
}

template <typename T>
__global__ void __launch_bounds__(128) gated_scan_kernel(GatedScanParams p) {
    const int64_t C = p.channels, L = p.seqlen;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (c >= C) return;
    const float k = -p.scale * softplus_f32(p.decay[c]);
    const int64_t nst = (L + kInterval - 1) / kInterval;
    float h = p.init_state ? p.init_state[b * C + c] : 0.0f;
    for (int64_t t = 0; t < L; ++t) {
        const int64_t o = (b * L + t) * C + c;
        if (p.states && t % kInterval == 0) p.states[(b * nst + t / kInterval) * C + c] = h;
        const bool rs = p.reset && p.reset[b * L + t];
        const Gates g = gates(to_f32(static_cast<const T*>(p.gate_a)[o]),
                              to_f32(static_cast<const T*>(p.gate_x)[o]), k, rs);
        // a select, not 0 * h: an infinite state does not outlive its sequence
        h = (rs ? 0.0f : fmaf(g.em1, h, h)) + g.n * (g.i * to_f32(static_cast<const T*>(p.x)[o]));
        static_cast<T*>(p.y)[o] = from_f32<T>(h);
    }
    if (p.final_state) p.final_state[b * C + c] = h;
}

template <typename T>
__global__ void __launch_bounds__(128) gated_scan_bwd_kernel(GatedScanParams p) {
    const int64_t C = p.channels, L = p.seqlen;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (c >= C) return;
    const float k = -p.scale * softplus_f32(p.decay[c]);
    const int64_t nst = (L + kInterval - 1) / kInterval;
    float carry = p.d_final ? p.d_final[b * C + c] : 0.0f;  // a_{t+1} g_{t+1}
    float sum = 0.0f;
    for (int64_t st = nst - 1; st >= 0; --st) {
        float hp[kInterval];
        float h = p.states[(b * nst + st) * C + c];
        const int64_t t0 = st * kInterval;
        const int n = static_cast<int>(L - t0 < kInterval ? L - t0 : kInterval);
        for (int j = 0; j < n; ++j) {
            const int64_t o = (b * L + t0 + j) * C + c;
            const bool rs = p.reset && p.reset[b * L + t0 + j];
            const Gates g = gates(to_f32(static_cast<const T*>(p.gate_a)[o]),
                                  to_f32(static_cast<const T*>(p.gate_x)[o]), k, rs);
            hp[j] = h;
            h = (rs ? 0.0f : fmaf(g.em1, h, h)) + g.n * (g.i * to_f32(static_cast<const T*>(p.x)[o]));
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t o = (b * L + t0 + j) * C + c;
            const bool rs = p.reset && p.reset[b * L + t0 + j];
            const Gates g = gates(to_f32(static_cast<const T*>(p.gate_a)[o]),
                                  to_f32(static_cast<const T*>(p.gate_x)[o]), k, rs);
            const float x = to_f32(static_cast<const T*>(p.x)[o]);
            const float gt = to_f32(static_cast<const T*>(p.dy)[o]) + carry;
            const float a = g.a;
            const float ix = g.i * x;
            static_cast<T*>(p.dx)[o] = from_f32<T>(gt * g.n * g.i);
            static_cast<T*>(p.dgate_x)[o] = from_f32<T>(gt * g.n * ix * (1.0f - g.i));
            // a decay of exactly 1 (n = 0) passes a finite dla times la = 0
            const float dla = rs ? 0.0f : gt * a * (hp[j] - a / fmaxf(g.n, 1e-18f) * ix);
            static_cast<T*>(p.dgate_a)[o] = from_f32<T>(dla * g.la * (1.0f - g.r));
            sum = fmaf(dla, g.r, sum);
            carry = rs ? 0.0f : fmaf(g.em1, gt, gt);
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
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= p.batch * p.channels) return;
    const int64_t c = i % p.channels;
    grid_dep_wait();
    grid_dep_launch();
    const bool rs = p.reset && p.reset[i / p.channels];
    const Gates g = gates(to_f32(static_cast<const T*>(p.gate_a)[i]),
                          to_f32(static_cast<const T*>(p.gate_x)[i]),
                          -p.scale * softplus_f32(p.decay[c]), rs);
    const float h = p.state[i];
    const float hn = (rs ? 0.0f : fmaf(g.em1, h, h)) + g.n * (g.i * to_f32(static_cast<const T*>(p.x)[i]));
    p.new_state[i] = hn;
    static_cast<T*>(p.y)[i] = from_f32<T>(hn);
}

}  // namespace

size_t gated_scan_bwd_partial_bytes(int64_t batch, int64_t, int64_t channels) {
    return static_cast<size_t>(batch) * channels * sizeof(float);
}

template <typename T> cudaError_t launch_gated_scan(const GatedScanParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.channels + 127) / 128), static_cast<unsigned>(p.batch));
    gated_scan_kernel<T><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
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
