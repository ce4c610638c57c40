// mixers.h -- the gated linear recurrence, the head norm with the position
// rotation and the convolution's gradient as api.cu sees them.
#pragma once

#include <atomic>

#include "internal.cuh"

namespace ssd {

// A kernel's attributes on the current device, set at its first launch there:
// dynamic shared memory up to `smem` bytes, and clusters beyond 8 CTAs.
template <auto Kern> cudaError_t prepare_kernel(int smem, bool clusters) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && clusters) e = cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// One call of the gated linear recurrence: forward (y, final_state, states
// out) or backward (states in, dy ... out).
struct GatedScanParams {
    int64_t batch, seqlen, channels;
    float scale;
    const void* x;             // [b, L, C]
    const void* gate_a;        // [b, L, C]
    const void* gate_x;        // [b, L, C]
    const float* decay;        // [C]
    const uint8_t* reset;      // [b, L]; may be null
    const float* init_state;   // [b, C]; may be null (forward)
    void* y;                   // [b, L, C] (forward)
    float* final_state;        // [b, C]; may be null (forward)
    float* states;             // [b, ceil(L / 64), C]; may be null in the forward
    const void* dy;            // [b, L, C] (backward, as the rest)
    const float* d_final;      // [b, C]; may be null
    void* dx;
    void* dgate_a;
    void* dgate_x;
    float* ddecay;             // [C]
    float* d_init;             // [b, C]; may be null
    float* partial;            // workspace: rows of [C] with sums of dla * r
};
// The decode step: seqlen 1, state -> new_state.
struct GatedUpdateParams {
    int64_t batch, channels;
    float scale;
    const float* state;        // [b, C]
    const void* x;             // [b, C]
    const void* gate_a;
    const void* gate_x;
    const float* decay;
    const uint8_t* reset;      // [b]; may be null
    float* new_state;          // may be state
    void* y;
};
template <typename T> cudaError_t launch_gated_scan(const GatedScanParams& p, cudaStream_t s);
template <typename T> cudaError_t launch_gated_scan_bwd(const GatedScanParams& p, cudaStream_t s);
template <typename T> cudaError_t launch_gated_update(const GatedUpdateParams& p, cudaStream_t s);
// *v = SSD_ERR_TIMEOUT if the scan or its gradient gave up on a wait since the last check (synchronises s).
cudaError_t gated_scan_take_status(int* v, cudaStream_t s);
// Bytes of the backward's partial sums.
size_t gated_scan_bwd_partial_bytes(int64_t batch, int64_t seqlen, int64_t channels);

// One call of the head norm with the rotation: index 0 = q, 1 = k.
struct NormRopeParams {
    int64_t batch, seqlen;
    int heads[2];              // heads[1] may be 0
    int headdim, rot_dim, adjacent;
    float eps;
    const void* in[2];
    int64_t in_stride[2];      // elements between tokens
    const float* weight[2];    // [headdim]; may be null (1)
    const float* inv_freq;     // [rot_dim / 2]
    const int64_t* positions;  // [b, L]; may be null
    void* out[2];              // forward
    int64_t out_stride[2];
    const void* dout[2];       // backward, as the rest
    int64_t dout_stride[2];
    void* din[2];
    int64_t din_stride[2];
    float* dweight[2];         // may be null
    float* partial[2];         // workspace: rows of [headdim]
};
template <typename T> cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s);
template <typename T> cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s);
// Rows of each of the backward's two partial arrays (fp32 rows of headdim).
int64_t norm_rope_bwd_rows();

struct ConvBwdParams {
    int64_t batch, seqlen, channels, width;
    int32_t activation;
    const void* x;
    const float* weight;
    const float* bias;         // may be null
    const float* init_state;   // may be null
    const void* dy;
    const float* d_final;      // may be null
    void* dx;
    float* dweight;
    float* dbias;              // may be null
    float* d_init;             // may be null
    float* partial;            // workspace: rows of [width + 1][channels]
};
template <typename T> cudaError_t launch_conv1d_bwd(const ConvBwdParams& p, cudaStream_t s);
size_t conv1d_bwd_partial_bytes(int64_t batch, int64_t seqlen, int64_t channels, int64_t width);
// *v = SSD_ERR_TIMEOUT if the gradient gave up on a wait since the last check (synchronises s).
cudaError_t conv1d_bwd_take_status(int* v, cudaStream_t s);

}  // namespace ssd
