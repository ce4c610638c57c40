// vec16.cuh -- 16-byte vectors of the two element types, widened to fp32.
#pragma once

#include "internal.cuh"

namespace ssd {

// Four fp32 or eight bf16 consecutive elements as one 16-byte word.
template <typename T> struct Vec16;
template <> struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(uint4 a, float* v) {
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
        v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    }
    static __device__ __forceinline__ uint4 narrow(const float* v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};
template <> struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(uint4 a, float* v) {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // round to nearest even, the one rounding of each output
    static __device__ __forceinline__ uint4 narrow(const float* v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Two consecutive channels of one token, widened to an fp32 pair.
template <typename T> struct Pair;
template <> struct Pair<float> {
    using Raw = float2;
    static __device__ __forceinline__ float2 widen(Raw r) { return r; }
    static __device__ __forceinline__ Raw narrow(float2 v) { return v; }
    static __device__ __forceinline__ Raw zero() { return make_float2(0.0f, 0.0f); }
};
template <> struct Pair<__nv_bfloat16> {
    using Raw = uint32_t;
    static __device__ __forceinline__ float2 widen(Raw r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    static __device__ __forceinline__ Raw narrow(float2 v) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ Raw zero() { return 0u; }
};

// Sums of the columns of partial [rows][cols] (fp32), rows in a fixed order:
// a block takes 32 columns, its W warps every W-th row each, and the warps' sums
// are added in order.  The value of column c goes to store(c, sum).
template <int W, typename Store>
__device__ __forceinline__ void column_sums(const float* partial, int64_t rows, int64_t cols, Store store) {
    __shared__ float part[W][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
        int64_t r = warp;
        for (; r + 3 * W < rows; r += 4 * W) {  // four loads in flight
            const float a = partial[r * cols + c], b = partial[(r + W) * cols + c];
            const float d = partial[(r + 2 * W) * cols + c], e = partial[(r + 3 * W) * cols + c];
            s += (a + b) + (d + e);
        }
        for (; r < rows; r += W) s += partial[r * cols + c];
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) t += part[w][lane];
        store(c, t);
    }
}

}  // namespace ssd
