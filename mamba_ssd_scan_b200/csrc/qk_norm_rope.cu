// qk_norm_rope.cu -- RMSNorm over each head of q and k and the rotation of its
// leading pairs by the token's position, and the gradient (the formulas stand
// in include/ssd.h).
//
// A unit is one head of one token.  A head is cut into slots of two 16-byte
// vectors: slot l < RS (the rotated part) holds vector l of the first half and
// vector l of the second half of the rotated elements, so that a lane holds
// both elements of each of its pairs; the slots after that hold two
// consecutive vectors of the unrotated rest.  A unit is spread over LPU lanes
// (the power of two >= its slots, one slot per lane), and its mean is a
// shuffle reduction over them.  A CTA takes a tile of tokens: it first forms
// the tile's cosines and sines in shared memory (once for all heads of q and
// k), then its lanes run through the tile's units.
#include "mixers.h"
#include "vec16.cuh"

namespace ssd {
namespace {

constexpr int TPB = 256;

// The two vector indices of slot l, -1 = none.
struct Slot {
    int v0, v1;
    bool rot;
};
template <int N> __device__ __forceinline__ Slot slot_of(int l, int headdim, int rot_dim) {
    const int rs = rot_dim / (2 * N), nv = headdim / N;
    Slot s;
    if (l < rs) {
        s.v0 = l;
        s.v1 = l + rs;
        s.rot = true;
    } else {
        s.v0 = 2 * rs + 2 * (l - rs);
        s.v1 = s.v0 + 1;
        s.rot = false;
        if (s.v0 >= nv) s.v0 = -1;
        if (s.v1 >= nv) s.v1 = -1;
    }
    return s;
}

// cos and sin of position * inv_freq for a tile of tokens, in the order the
// lanes read them: a slot's N pairs are N / 2 16-byte chunks of (cos, sin) x 2,
// chunk k of slot l of token t at ((t * N / 2) + k) * rs + l.  The angle is an
// fp64 product (positions up to 2^53 are exact; at 2^31 the turn is off by
// less than 1e-7), reduced by whole turns before the fp32 cosine and sine.
template <int N>
__device__ void fill_angles(float2* cs, const NormRopeParams& p, int64_t tok0, int ntok) {
    const int half = p.rot_dim / 2, rs = p.rot_dim / (2 * N);
    for (int e = threadIdx.x; e < ntok * half; e += blockDim.x) {
        const int t = e / half, j = e - t * half;
        const int64_t tok = tok0 + t;
        const int64_t pos = p.positions ? p.positions[tok] : tok % p.seqlen;
        const double turns = static_cast<double>(pos) * static_cast<double>(p.inv_freq[j]) *
                             0.15915494309189533577;  // 1 / (2 pi)
        float sn, cn;
        sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn, &cn);
        int l, w;  // the slot that holds pair j and its place there
        if (!p.adjacent) {
            l = j / N;
            w = j % N;
        } else {  // the first vector's N / 2 pairs, then the second's
            const int q = half / 2, jj = j < q ? j : j - q;
            l = jj / (N / 2);
            w = jj % (N / 2) + (j < q ? 0 : N / 2);
        }
        cs[(((t * (N / 2)) + w / 2) * rs + l) * 2 + (w & 1)] = make_float2(cn, sn);
    }
}

// Rotates a slot's N pairs: lo / hi are its two vectors.  `sign` -1 rotates back.
template <int N>
__device__ __forceinline__ void rotate(float* lo, float* hi, const float2* cs, int rs, int t, int l,
                                       bool adjacent, float sign) {
    const float4* c4 = reinterpret_cast<const float4*>(cs) + (t * (N / 2)) * rs + l;
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float4 c = c4[k * rs];
        const float s0 = sign * c.y, s1 = sign * c.w;
        if (!adjacent) {
            const float a0 = lo[2 * k], b0 = hi[2 * k], a1 = lo[2 * k + 1], b1 = hi[2 * k + 1];
            lo[2 * k] = fmaf(a0, c.x, -b0 * s0);
            hi[2 * k] = fmaf(a0, s0, b0 * c.x);
            lo[2 * k + 1] = fmaf(a1, c.z, -b1 * s1);
            hi[2 * k + 1] = fmaf(a1, s1, b1 * c.z);
        } else {
            float* v = (k < N / 4) ? lo + 4 * k : hi + 4 * (k - N / 4);
            const float a0 = v[0], b0 = v[1], a1 = v[2], b1 = v[3];
            v[0] = fmaf(a0, c.x, -b0 * s0);
            v[1] = fmaf(a0, s0, b0 * c.x);
            v[2] = fmaf(a1, c.z, -b1 * s1);
            v[3] = fmaf(a1, s1, b1 * c.z);
        }
    }
}

template <int N>
__device__ __forceinline__ void load_weight(const float* w, int v, float* o) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 a = (w && v >= 0) ? __ldg(reinterpret_cast<const float4*>(w + v * N + i))
                                       : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        o[i] = a.x; o[i + 1] = a.y; o[i + 2] = a.z; o[i + 3] = a.w;
    }
}

template <typename T>
__device__ __forceinline__ uint4 load16(const T* p, int v) {
    return v >= 0 ? *reinterpret_cast<const uint4*>(p + v * Vec16<T>::N) : make_uint4(0, 0, 0, 0);
}


template <typename T>
__global__ void __launch_bounds__(TPB) norm_rope_kernel(NormRopeParams p, int lpu, int tile, int64_t tokens) {
    constexpr int N = Vec16<T>::N;
    extern __shared__ __align__(16) float2 cs[];
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * tile;
    const int ntok = static_cast<int>(tokens - tok0 < tile ? tokens - tok0 : tile);
    fill_angles<N>(cs, p, tok0, ntok);
    __syncthreads();
    const int l = threadIdx.x & (lpu - 1);
    const int step = TPB / lpu;
    const Slot s = slot_of<N>(l, p.headdim, p.rot_dim);
    const int rs = p.rot_dim / (2 * N);
    const float inv_d = 1.0f / static_cast<float>(p.headdim);
    const int nq = ntok * p.heads[0], units = nq + ntok * p.heads[1];
    // whole warps run the same number of rounds (the shuffles take all lanes)
    for (int u0 = 0; u0 < units; u0 += step) {
        const int u = u0 + static_cast<int>(threadIdx.x) / lpu;
        const bool live = u < units;
        const int kind = u < nq ? 0 : 1;
        const int uu = live ? (kind ? u - nq : u) : 0;
        const int heads = live && kind ? p.heads[1] : p.heads[0];
        const int kd = live ? kind : 0;
        const int t = uu / heads, h = uu - t * heads;
        const int64_t tok = tok0 + t;
        const T* in = static_cast<const T*>(p.in[kd]) + tok * p.in_stride[kd] + static_cast<int64_t>(h) * p.headdim;
        float lo[N], hi[N], w0[N], w1[N];
        Vec16<T>::widen(load16(in, live ? s.v0 : -1), lo);
        Vec16<T>::widen(load16(in, live ? s.v1 : -1), hi);
        load_weight<N>(p.weight[kd], s.v0, w0);
        load_weight<N>(p.weight[kd], s.v1, w1);
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
        for (int o = lpu / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            lo[i] *= inv * w0[i];
            hi[i] *= inv * w1[i];
        }
        if (s.rot) rotate<N>(lo, hi, cs, rs, t, l, p.adjacent, 1.0f);
        if (live) {
            T* out = static_cast<T*>(p.out[kd]) + tok * p.out_stride[kd] + static_cast<int64_t>(h) * p.headdim;
            if (s.v0 >= 0) *reinterpret_cast<uint4*>(out + s.v0 * N) = Vec16<T>::narrow(lo);
            if (s.v1 >= 0) *reinterpret_cast<uint4*>(out + s.v1 * N) = Vec16<T>::narrow(hi);
        }
    }
}

// The gradient of q (kind 0) or k (kind 1): a CTA takes tiles tile0, tile0 +
// ctas, ... and leaves one row of the weight's gradient in partial.
template <typename T>
__global__ void __launch_bounds__(TPB) norm_rope_bwd_kernel(NormRopeParams p, int lpu, int tile, int64_t tokens,
                                                            int ctas_q) {
    constexpr int N = Vec16<T>::N;
    extern __shared__ __align__(16) float2 cs[];
    const int kd = static_cast<int>(blockIdx.x) < ctas_q ? 0 : 1;
    const int cta = kd ? blockIdx.x - ctas_q : blockIdx.x;
    const int ctas = kd ? gridDim.x - ctas_q : ctas_q;
    const int heads = p.heads[kd];
    const int l = threadIdx.x & (lpu - 1);
    const int step = TPB / lpu;
    const Slot s = slot_of<N>(l, p.headdim, p.rot_dim);
    const int rs = p.rot_dim / (2 * N);
    const float inv_d = 1.0f / static_cast<float>(p.headdim);
    float w0[N], w1[N], acc0[N] = {}, acc1[N] = {};
    load_weight<N>(p.weight[kd], s.v0, w0);
    load_weight<N>(p.weight[kd], s.v1, w1);
    const int64_t ntiles = (tokens + tile - 1) / tile;
    for (int64_t ti = cta; ti < ntiles; ti += ctas) {
        const int64_t tok0 = ti * tile;
        const int ntok = static_cast<int>(tokens - tok0 < tile ? tokens - tok0 : tile);
        __syncthreads();  // the previous tile's angles are read
        fill_angles<N>(cs, p, tok0, ntok);
        __syncthreads();
        const int units = ntok * heads;
        for (int u0 = 0; u0 < units; u0 += step) {
            const int u = u0 + static_cast<int>(threadIdx.x) / lpu;
            const bool live = u < units;
            const int uu = live ? u : 0;
            const int t = uu / heads, h = uu - t * heads;
            const int64_t tok = tok0 + t, ho = static_cast<int64_t>(h) * p.headdim;
            const T* in = static_cast<const T*>(p.in[kd]) + tok * p.in_stride[kd] + ho;
            const T* de = static_cast<const T*>(p.dout[kd]) + tok * p.dout_stride[kd] + ho;
            float lo[N], hi[N], e0[N], e1[N];
            Vec16<T>::widen(load16(in, live ? s.v0 : -1), lo);
            Vec16<T>::widen(load16(in, live ? s.v1 : -1), hi);
            Vec16<T>::widen(load16(de, live ? s.v0 : -1), e0);
            Vec16<T>::widen(load16(de, live ? s.v1 : -1), e1);
            if (s.rot) rotate<N>(e0, e1, cs, rs, t, l, p.adjacent, -1.0f);
            float ss = 0.0f, m = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
                m = fmaf(e0[i] * w0[i], lo[i], fmaf(e1[i] * w1[i], hi[i], m));
            }
            for (int o = lpu / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                m += __shfl_xor_sync(0xffffffffu, m, o);
            }
            const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
            const float k = -inv * inv * m * inv_d;
            float d0[N], d1[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                d0[i] = inv * fmaf(lo[i], k, e0[i] * w0[i]);
                d1[i] = inv * fmaf(hi[i], k, e1[i] * w1[i]);
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    acc0[i] = fmaf(e0[i], lo[i] * inv, acc0[i]);
                    acc1[i] = fmaf(e1[i], hi[i] * inv, acc1[i]);
                }
                T* out = static_cast<T*>(p.din[kd]) + tok * p.din_stride[kd] + ho;
                if (s.v0 >= 0) *reinterpret_cast<uint4*>(out + s.v0 * N) = Vec16<T>::narrow(d0);
                if (s.v1 >= 0) *reinterpret_cast<uint4*>(out + s.v1 * N) = Vec16<T>::narrow(d1);
            }
        }
    }
    if (!p.dweight[kd]) return;
    // the lanes of the same slot, in a fixed order: lane groups of the warp by
    // shuffles, then the warps through shared memory
    __shared__ float red[TPB / 32][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i)
        for (int o = lpu; o < 32; o <<= 1) {
            acc0[i] += __shfl_xor_sync(0xffffffffu, acc0[i], o);
            acc1[i] += __shfl_xor_sync(0xffffffffu, acc1[i], o);
        }
    if (lane < lpu) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (s.v0 >= 0) red[warp][s.v0 * N + i] = acc0[i];
            if (s.v1 >= 0) red[warp][s.v1 * N + i] = acc1[i];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.headdim; c += TPB) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < TPB / 32; ++w) v += red[w][c];
        p.partial[kd][static_cast<int64_t>(cta) * p.headdim + c] = v;
    }
}

__global__ void __launch_bounds__(kColSumThreads)
    norm_rope_finish_kernel(NormRopeParams p, int64_t rows_q, int64_t rows_k) {
    grid_dep_wait();
    const int kd = blockIdx.y;
    if (!p.dweight[kd]) return;
    column_sums(p.partial[kd], kd ? rows_k : rows_q, p.headdim,
                [&](int64_t c, float s) { p.dweight[kd][c] = s; });
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

// lanes per unit: the power of two that holds the head's slots
int lanes_per_unit(int n, int headdim, int rot_dim) {
    const int slots = rot_dim / (2 * n) + ((headdim - rot_dim) / n + 1) / 2;
    int lpu = 1;
    while (lpu < slots) lpu *= 2;
    return lpu;
}

// Tokens per CTA: enough for several rounds of units, few enough that the
// grid fills the device and the angles fit 32 KB of shared memory.
int tile_tokens(int64_t tokens, int heads, int lpu, int rot_dim, int64_t ctas) {
    int64_t t = (tokens + ctas - 1) / ctas;
    const int64_t rounds = (static_cast<int64_t>(8) * (TPB / lpu) + heads - 1) / heads;  // 8 rounds
    if (t > rounds) t = rounds;
    if (rot_dim > 0 && t > 32768 / (rot_dim * 4)) t = 32768 / (rot_dim * 4);
    return static_cast<int>(t < 1 ? 1 : t);
}

constexpr int64_t kBwdCtas = 592;  // the backward's persistent CTAs, four per SM

}  // namespace

int64_t norm_rope_bwd_rows() { return kBwdCtas; }

template <typename T> cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
    constexpr int N = Vec16<T>::N;
    const int64_t tokens = p.batch * p.seqlen;
    const int lpu = lanes_per_unit(N, p.headdim, p.rot_dim);
    const int tile = tile_tokens(tokens, p.heads[0] + p.heads[1], lpu, p.rot_dim, 2 * device_sms());
    const size_t smem = static_cast<size_t>(tile) * p.rot_dim * 4;
    norm_rope_kernel<T><<<static_cast<unsigned>((tokens + tile - 1) / tile), TPB, smem, s>>>(p, lpu, tile, tokens);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s) {
    constexpr int N = Vec16<T>::N;
    const int64_t tokens = p.batch * p.seqlen;
    const int lpu = lanes_per_unit(N, p.headdim, p.rot_dim);
    const int H = p.heads[0] + p.heads[1];
    const int tile = tile_tokens(tokens, p.heads[0], lpu, p.rot_dim, 2 * device_sms());
    const int64_t ntiles = (tokens + tile - 1) / tile;
    // the CTAs are shared out between q and k by their heads
    int64_t cq = kBwdCtas * p.heads[0] / H, ck = kBwdCtas - cq;
    if (cq < 1) cq = 1;
    if (cq > ntiles) cq = ntiles;
    if (ck < 1) ck = 1;
    if (ck > ntiles) ck = ntiles;
    if (p.heads[1] == 0) ck = 0;
    const size_t smem = static_cast<size_t>(tile) * p.rot_dim * 4;
    norm_rope_bwd_kernel<T><<<static_cast<unsigned>(cq + ck), TPB, smem, s>>>(p, lpu, tile, tokens,
                                                                            static_cast<int>(cq));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!p.dweight[0] && !p.dweight[1])) return e;
    return launch_kernel(norm_rope_finish_kernel,
                         dim3(static_cast<unsigned>((p.headdim + 31) / 32), ck > 0 ? 2 : 1),
                         dim3(kColSumThreads), 0, s, true, p, cq, ck);
}

template cudaError_t launch_norm_rope<float>(const NormRopeParams&, cudaStream_t);
template cudaError_t launch_norm_rope<__nv_bfloat16>(const NormRopeParams&, cudaStream_t);
template cudaError_t launch_norm_rope_bwd<float>(const NormRopeParams&, cudaStream_t);
template cudaError_t launch_norm_rope_bwd<__nv_bfloat16>(const NormRopeParams&, cudaStream_t);

}  // namespace ssd
