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
//
// Measured (B200, L2 flushed; share of the measured copy bandwidth over the
// call's least bytes).  Forward, bf16: b1 L65536 8 + 8 heads of 128 in packed
// rows 101 us (83 %), b4 L4096 32 + 8 heads of 128 62 us (84 %); fp32: b4 L4096
// 32 + 8 heads of 64, adjacent pairs, 61 us (85 %).  Issue slots are 73 % busy (18
// instructions per element), so instructions and bytes bind about equally.
// Gradient, bf16: b4 L4096 32 + 8 heads of 128 101 us (77 %), heads of 64 59 us
// (66 %); issue 58 %, and without its arithmetic the same loop still takes 99 us:
// the loads in flight of two CTAs per SM bind it.  The forward spills 12 bytes for
// adjacent bf16 pairs at 2, 4 and 8 lanes per unit.  Two units in flight per lane
// (126 registers) measured 115 us, three CTAs per SM (80 registers) spilled, 152.
#include <algorithm>
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

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// (cos, sin) of 2 pi f for a fraction of a turn f in [-1/2, 1/2): the nearest
// quarter turn is taken off and the rest x, |x| <= pi / 4, goes through the two
// Taylor series side by side, sin to x^9 and cos to x^8 (what they leave out is
// below 2^-25).
__device__ __forceinline__ float2 cos_sin_turn(float f) {
    const float q = rintf(4.0f * f);
    const float x = fmaf(q, -0.25f, f) * 6.283185307179586f, x2 = x * x;
    const float2 y = dup(x2);
    // (cos, sin / x)
    float2 v = fma2(make_float2(1.0f / 40320.0f, 1.0f / 362880.0f), y, make_float2(-1.0f / 720.0f, -1.0f / 5040.0f));
    v = fma2(v, y, make_float2(1.0f / 24.0f, 1.0f / 120.0f));
    v = fma2(v, y, make_float2(-0.5f, -1.0f / 6.0f));
    const float c = fmaf(v.x, x2, 1.0f), sn = fmaf(v.y * x2, x, x);
    const int n = static_cast<int>(q);  // quarter turns, -2 .. 2
    const float a = (n & 1) ? sn : c, b = (n & 1) ? c : sn;
    return make_float2(((n + 1) & 2) ? -a : a, (n & 2) ? -b : b);
}

// cos and sin of position * inv_freq for a tile of tokens, in the order the
// lanes read them: a slot's N pairs are N / 2 16-byte chunks (c0, c1, s0, s1),
// chunk k of slot l of token t at ((t * N / 2) + k) * rs + l.  A thread keeps one
// pair j and steps through the tokens.  Its turns per position, inv_freq /
// (2 pi), are held as a 64-bit fraction of a turn (formed in two fp64 parts, so that
// it is right to 2^-63 at any frequency), so the angle is an integer product that
// drops the whole turns by itself: off by less than 2^-25 of a turn at positions up
// to 2^31.
template <int N> struct Angles {
    int t0, tstep, place;  // first token, tokens per step (0: no pair), float offset of the pair in a token's chunks
    int64_t turn;          // the fraction of a turn per position, times 2^64
    __device__ __forceinline__ void init(const NormRopeParams& p) {
        const int half = p.rot_dim / 2, rs = p.rot_dim / (2 * N);
        t0 = tstep = place = 0;
        turn = 0;
        if (half == 0) return;
        tstep = TPB / half;  // (half <= 128)
        t0 = static_cast<int>(threadIdx.x) / half;
        const int j = static_cast<int>(threadIdx.x) - t0 * half;
        if (t0 >= tstep) {
            tstep = 0;
            return;
        }
        // inv_freq / (2 pi) as f + e, 1 / (2 pi) in two parts; whole turns come off f and e
        // exactly (a fraction of 1/2 is cut off at 2^63 - 1)
        constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
        const double v = static_cast<double>(p.inv_freq[j]), f = v * kHi, e = fma(v, kLo, fma(v, kHi, -f));
        turn = static_cast<int64_t>(static_cast<uint64_t>(__double2ll_rn((f - rint(f)) * 18446744073709551616.0)) +
                                    static_cast<uint64_t>(__double2ll_rn((e - rint(e)) * 18446744073709551616.0)));
        int l, w;  // the slot that holds pair j and its place there
        if (!p.adjacent) {
            l = j / N;
            w = j % N;
        } else {  // the first vector's N / 2 pairs, then the second's
            const int q = half / 2, jj = j < q ? j : j - q;
            l = jj / (N / 2);
            w = jj % (N / 2) + (j < q ? 0 : N / 2);
        }
        place = ((w / 2) * rs + l) * 4 + (w & 1);
    }
    __device__ __forceinline__ void fill(float4* cs, const NormRopeParams& p, int64_t tok0, int ntok) const {
        if (tstep == 0) return;
        const uint32_t len = static_cast<uint32_t>(p.seqlen);
        uint32_t own = p.positions ? 0u : static_cast<uint32_t>(tok0 + t0) % len;  // the token's place in its row
        for (int t = t0; t < ntok; t += tstep) {
            const int64_t pos = p.positions ? p.positions[tok0 + t] : static_cast<int64_t>(own);
            own += tstep;
            while (own >= len) own -= len;
            const int64_t part = static_cast<int64_t>(static_cast<uint64_t>(pos) * static_cast<uint64_t>(turn));
            const float f = static_cast<float>(static_cast<int32_t>(part >> 32)) * 2.3283064365386963e-10f;  // 2^-32
            const float2 v = cos_sin_turn(f);
            float* c = reinterpret_cast<float*>(cs) + t * p.rot_dim + place;
            c[0] = v.x;
            c[2] = v.y;
        }
    }
};

// Rotates a slot's N pairs by the angle (BACK: by its negative); lo / hi are its
// two vectors as pairs of elements.
template <int N, bool ADJ, bool BACK>
__device__ __forceinline__ void rotate(float2 (&lo)[N / 2], float2 (&hi)[N / 2], const float4* c4, int rs) {
    const float2 neg = dup(-1.0f);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const float4 v = c4[k * rs];
        const float2 c = make_float2(v.x, v.y), s = make_float2(v.z, v.w);
        if (!ADJ) {
            const float2 a = lo[k], b = hi[k];
            if (!BACK) {
                lo[k] = fma2(mul2(b, s), neg, mul2(a, c));
                hi[k] = fma2(a, s, mul2(b, c));
            } else {
                lo[k] = fma2(b, s, mul2(a, c));
                hi[k] = fma2(mul2(a, s), neg, mul2(b, c));
            }
        } else {  // chunk k: the pairs 2 k and 2 k + 1 of the slot
            float2* q = (k < N / 4) ? lo + 2 * k : hi + 2 * (k - N / 4);
            const float2 x = q[0], y = q[1];
            const float s0 = BACK ? -s.x : s.x, s1 = BACK ? -s.y : s.y;
            q[0] = make_float2(fmaf(x.x, c.x, -x.y * s0), fmaf(x.x, s0, x.y * c.x));
            q[1] = make_float2(fmaf(y.x, c.y, -y.y * s1), fmaf(y.x, s1, y.y * c.y));
        }
    }
}

// The weights of q and k in the order the lanes read them: chunk k (a float4) of
// slot l of kind kd at (kd * N / 2 + k) * LPU + l, the first N / 4 chunks of its
// first vector, then those of its second; 1 without weights or elements.
template <int N, int LPU>
__device__ __forceinline__ void fill_weights(float4* ws, const NormRopeParams& p, int kd0, int kds) {
    for (int e = threadIdx.x; e < kds * (N / 2) * LPU; e += TPB) {
        const int l = e % LPU, k = e / LPU % (N / 2), kd = kd0 + e / LPU / (N / 2);
        const Slot s = slot_of<N>(l, p.headdim, p.rot_dim);
        const int v = k < N / 4 ? s.v0 : s.v1;
        const float* w = p.weight[kd];
        ws[e] = w && v >= 0 ? __ldg(reinterpret_cast<const float4*>(w + v * N) + k % (N / 4))
                            : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    }
}
// pair j of a slot's first (hi = 0) or second vector
template <int N, int LPU>
__device__ __forceinline__ void weight2(const float4* ws, int hi, int k, float2& a, float2& b) {
    const float4 w = ws[(hi * (N / 4) + k) * LPU];
    a = make_float2(w.x, w.y);
    b = make_float2(w.z, w.w);
}

template <typename T> __device__ __forceinline__ void widen2(uint4 raw, float2 (&v)[Vec16<T>::N / 2]) {
    Vec16<T>::widen(raw, reinterpret_cast<float*>(v));
}
template <typename T> __device__ __forceinline__ uint4 narrow2(const float2 (&x)[Vec16<T>::N / 2]) {
    return Vec16<T>::narrow(reinterpret_cast<const float*>(x));
}

// What a lane needs to reach its slot of a head: the byte offset of its first
// vector (in the base pointers), from there to its second, and which it has.
struct Reach {
    int first, delta;
    bool has0, has1;
};
template <int N> __device__ __forceinline__ Reach reach_of(const Slot& s) {
    Reach r;
    r.has0 = s.v0 >= 0;
    r.has1 = s.v1 >= 0;
    r.first = r.has0 ? s.v0 * 16 : 0;
    r.delta = r.has1 ? s.v1 * 16 - r.first : 0;
    return r;
}
// (a vector that is not loaded keeps what the registers held)
__device__ __forceinline__ void load_slot(const char* v, bool live, const Reach& x, uint4& a, uint4& b) {
    if (live && x.has0) a = *reinterpret_cast<const uint4*>(v);
    if (live && x.has1) b = *reinterpret_cast<const uint4*>(v + x.delta);
}
__device__ __forceinline__ void store_slot(char* v, bool live, const Reach& x, uint4 a, uint4 b) {
    if (live && x.has0) *reinterpret_cast<uint4*>(v) = a;
    if (live && x.has1) *reinterpret_cast<uint4*>(v + x.delta) = b;
}

// A lane's place among the units of a tile of tokens: unit u is head u % heads
// of token u / heads, and a lane steps by the CTA's units (dt tokens and dh
// heads) without dividing again.
struct Place {
    int t, h;
    __device__ __forceinline__ void next(int dt, int dh, int heads) {
        t += dt;
        h += dh;
        if (h >= heads) {
            h -= heads;
            ++t;
        }
    }
};
// the byte offset of a place's head from the tile's first token (a token's
// stride fits 32 bits)
__device__ __forceinline__ int64_t head_at(const Place& w, int stride, int head) {
    return static_cast<int64_t>(w.t) * stride + w.h * head;
}

// The forward.  A CTA takes tiles blockIdx.x, + gridDim.x, ... (their angles in
// two buffers by turns: one barrier per tile); a tile's rounds go through the
// heads of q, then those of k.  A lane has its next two units' loads in flight
// while it works on one.
template <typename T, bool ADJ, int LPU>
__global__ void __launch_bounds__(TPB, 3) norm_rope_kernel(NormRopeParams p, int tile, int64_t tokens) {
    constexpr int N = Vec16<T>::N, STEP = TPB / LPU;
    extern __shared__ __align__(16) float4 cs[];
    __shared__ float4 ws[2 * (N / 2) * LPU];
    const int l = threadIdx.x % LPU, u0 = static_cast<int>(threadIdx.x) / LPU;
    const Slot s = slot_of<N>(l, p.headdim, p.rot_dim);
    const int rs = p.rot_dim / (2 * N);
    const float inv_d = 1.0f / static_cast<float>(p.headdim);
    const int nq = p.heads[0], nk = p.heads[1];
    const int dtq = STEP / nq, dhq = STEP - dtq * nq, dtk = nk ? STEP / nk : 0, dhk = STEP - dtk * nk;
    // where the lane's first units lie in a tile
    Place q0, k0;
    q0.t = u0 / nq;
    q0.h = u0 - q0.t * nq;
    k0.t = nk ? u0 / nk : 0;
    k0.h = u0 - k0.t * nk;
    const Reach x = reach_of<N>(s);
    constexpr int E = sizeof(T);
    const int head = p.headdim * E;  // bytes, as the strides
    const int qis = static_cast<int>(p.in_stride[0]) * E, kis = static_cast<int>(p.in_stride[1]) * E;
    const int qos = static_cast<int>(p.out_stride[0]) * E, kos = static_cast<int>(p.out_stride[1]) * E;
    const int64_t ntiles = (tokens + tile - 1) / tile;
    uint4 r[2][2];
    r[0][0] = r[0][1] = r[1][0] = r[1][1] = make_uint4(0, 0, 0, 0);
    fill_weights<N, LPU>(ws, p, 0, 2);
    Angles<N> angles;
    angles.init(p);
    int buf = 0;
    for (int64_t ti = blockIdx.x; ti < ntiles; ti += gridDim.x, buf ^= 1) {
        const int64_t tok0 = ti * tile;
        const int ntok = static_cast<int>(tokens - tok0 < tile ? tokens - tok0 : tile);
        float4* mine = cs + buf * (tile * p.rot_dim / 4);
        const int rq = (ntok * nq + STEP - 1) / STEP, rounds = rq + (ntok * nk + STEP - 1) / STEP;
        const char* const qi = static_cast<const char*>(p.in[0]) + tok0 * qis + x.first;
        const char* const ki = static_cast<const char*>(p.in[1]) + tok0 * kis + x.first;
        char* const qo = static_cast<char*>(p.out[0]) + tok0 * qos + x.first;
        char* const ko = static_cast<char*>(p.out[1]) + tok0 * kos + x.first;
        int fi = 0;  // the round to load next, and its place
        Place at = q0, held[2];
        auto fetch = [&](int b) {
            if (fi == rq) at = k0;
            const bool q = fi < rq, live = fi < rounds && at.t < ntok;
            load_slot(q ? qi + head_at(at, qis, head) : ki + head_at(at, kis, head), live, x, r[b][0], r[b][1]);
            held[b] = at;
            at.next(q ? dtq : dtk, q ? dhq : dhk, q ? nq : nk);
            ++fi;
        };
        fetch(0);
        fetch(1);
        angles.fill(mine, p, tok0, ntok);
        __syncthreads();
        auto work = [&](int i, int b) {
            const Place w = held[b];
            const bool live = w.t < ntok;
            float2 lo[N / 2], hi[N / 2];
            widen2<T>(r[b][0], lo);
            widen2<T>(r[b][1], hi);
            fetch(b);
            float2 ss = dup(0.0f), s2 = ss;
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                ss = fma2(lo[j], lo[j], ss);
                s2 = fma2(hi[j], hi[j], s2);
            }
            float sum = (ss.x + ss.y) + (s2.x + s2.y);
#pragma unroll
            for (int o = LPU / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float2 inv = dup(rsqrtf(fmaf(sum, inv_d, p.eps)));
            const float4* wt = ws + (i < rq ? 0 : (N / 2) * LPU) + l;
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                float2 a, c;
                weight2<N, LPU>(wt, 0, k, a, c);
                lo[2 * k] = mul2(mul2(lo[2 * k], inv), a);
                lo[2 * k + 1] = mul2(mul2(lo[2 * k + 1], inv), c);
                weight2<N, LPU>(wt, 1, k, a, c);
                hi[2 * k] = mul2(mul2(hi[2 * k], inv), a);
                hi[2 * k + 1] = mul2(mul2(hi[2 * k + 1], inv), c);
            }
            if (s.rot) rotate<N, ADJ, false>(lo, hi, mine + (live ? w.t : 0) * (p.rot_dim / 4) + l, rs);
            store_slot(i < rq ? qo + head_at(w, qos, head) : ko + head_at(w, kos, head), live, x, narrow2<T>(lo),
                       narrow2<T>(hi));
        };
        // (a round is the whole CTA's: its shuffles take all lanes)
        for (int i = 0; i < rounds; i += 2) {
            work(i, 0);
            if (i + 1 < rounds) work(i + 1, 1);
        }
    }
}

// The gradient of q (kind 0) or k (kind 1): a CTA takes tiles cta, cta + ctas,
// ... (their angles in two buffers by turns: one barrier per tile) and leaves
// one row of the weight's gradient in partial.  A lane's next unit is on its way
// while it works on one, across tiles too: without that each tile's barrier
// found no load in flight (111 us instead of 107 at b4 L4096 32 + 8 heads of 128
// bf16, 65 instead of 59 at heads of 64).
template <typename T, bool ADJ, int LPU>
__global__ void __launch_bounds__(TPB, 2)
    norm_rope_bwd_kernel(NormRopeParams p, int tile_q, int tile_k, int64_t tokens, int ctas_q) {
    constexpr int N = Vec16<T>::N, STEP = TPB / LPU;
    extern __shared__ __align__(16) float4 cs[];
    __shared__ float4 ws[(N / 2) * LPU];
    const int kd = static_cast<int>(blockIdx.x) < ctas_q ? 0 : 1;
    const int cta = kd ? blockIdx.x - ctas_q : blockIdx.x;
    const int ctas = kd ? gridDim.x - ctas_q : ctas_q, tile = kd ? tile_k : tile_q;
    const int heads = p.heads[kd];
    const int l = threadIdx.x % LPU;
    const Slot s = slot_of<N>(l, p.headdim, p.rot_dim);
    const int rs = p.rot_dim / (2 * N);
    const float inv_d = 1.0f / static_cast<float>(p.headdim);
    const Reach x = reach_of<N>(s);
    const char* const in = static_cast<const char*>(p.in[kd]) + x.first;
    const char* const dout = static_cast<const char*>(p.dout[kd]) + x.first;
    char* const din = static_cast<char*>(p.din[kd]) + x.first;
    // where the lane's first unit lies in a tile
    Place first;
    first.t = static_cast<int>(threadIdx.x) / LPU / heads;
    first.h = static_cast<int>(threadIdx.x) / LPU - first.t * heads;
    const int dt = STEP / heads, dh = STEP - dt * heads;
    constexpr int E = sizeof(T);
    const int head = p.headdim * E;  // bytes, as the strides
    const int is = static_cast<int>(p.in_stride[kd]) * E, es = static_cast<int>(p.dout_stride[kd]) * E;
    const int os = static_cast<int>(p.din_stride[kd]) * E;
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0, q0 = r0, q1 = r0;
    fill_weights<N, LPU>(ws, p, kd, 1);
    float2 acc0[N / 2], acc1[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) acc0[j] = acc1[j] = dup(0.0f);
    Angles<N> angles;
    angles.init(p);
    auto tokens_of = [&](int64_t ti) {
        const int64_t n = tokens - ti * tile;
        return static_cast<int>(n < 0 ? 0 : n < tile ? n : tile);
    };
    auto rounds_of = [&](int ntok) { return (ntok * heads + STEP - 1) / STEP; };
    // the unit to load next, up to a tile ahead
    int64_t fti = cta;
    int fi = 0, fntok = tokens_of(fti);
    const char *vi = in + fti * tile * is, *ei = dout + fti * tile * es;
    Place at = first, held;
    auto fetch = [&]() {
        if (fi == rounds_of(fntok)) {  // (no token past the last tile: nothing is loaded)
            fti += ctas;
            fi = 0;
            fntok = tokens_of(fti);
            vi = in + fti * tile * is;
            ei = dout + fti * tile * es;
            at = first;
        }
        const bool live = at.t < fntok;
        load_slot(vi + head_at(at, is, head), live, x, r0, r1);
        load_slot(ei + head_at(at, es, head), live, x, q0, q1);
        held = at;
        at.next(dt, dh, heads);
        ++fi;
    };
    fetch();
    int buf = 0;
    int64_t tok0 = static_cast<int64_t>(cta) * tile;
    for (int64_t ti = cta; tok0 < tokens; ti += ctas, tok0 = ti * tile, buf ^= 1) {
        const int ntok = tokens_of(ti), rounds = rounds_of(ntok);
        float4* mine = cs + buf * (tile * p.rot_dim / 4);
        char* const vo = din + tok0 * os;
        angles.fill(mine, p, tok0, ntok);
        __syncthreads();
        for (int i = 0; i < rounds; ++i) {
            const Place w = held;
            const bool live = w.t < ntok;
            float2 lo[N / 2], hi[N / 2], e0[N / 2], e1[N / 2];
            widen2<T>(r0, lo);
            widen2<T>(r1, hi);
            widen2<T>(q0, e0);
            widen2<T>(q1, e1);
            fetch();
            if (s.rot) rotate<N, ADJ, true>(e0, e1, mine + (live ? w.t : 0) * (p.rot_dim / 4) + l, rs);
            // e w of both vectors, the sum of squares and of e w v
            float2 ss = dup(0.0f), mm = ss, g0[N / 2], g1[N / 2];
#pragma unroll
            for (int k = 0; k < N / 4; ++k) {
                float2 a, c;
                weight2<N, LPU>(ws + l, 0, k, a, c);
                g0[2 * k] = mul2(e0[2 * k], a);
                g0[2 * k + 1] = mul2(e0[2 * k + 1], c);
                weight2<N, LPU>(ws + l, 1, k, a, c);
                g1[2 * k] = mul2(e1[2 * k], a);
                g1[2 * k + 1] = mul2(e1[2 * k + 1], c);
            }
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                ss = fma2(lo[j], lo[j], fma2(hi[j], hi[j], ss));
                mm = fma2(g0[j], lo[j], fma2(g1[j], hi[j], mm));
            }
            float sum = ss.x + ss.y, m = mm.x + mm.y;
#pragma unroll
            for (int o = LPU / 2; o > 0; o >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                m += __shfl_xor_sync(0xffffffffu, m, o);
            }
            const float s1 = rsqrtf(fmaf(sum, inv_d, p.eps));
            const float2 inv = dup(s1), k = dup(-s1 * s1 * m * inv_d);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float2 n0 = mul2(lo[j], inv), n1 = mul2(hi[j], inv);
                if (live) {  // (a lane without a unit holds an earlier one's values)
                    acc0[j] = fma2(e0[j], n0, acc0[j]);
                    acc1[j] = fma2(e1[j], n1, acc1[j]);
                }
                e0[j] = fma2(n0, k, mul2(g0[j], inv));
                e1[j] = fma2(n1, k, mul2(g1[j], inv));
            }
            store_slot(vo + head_at(w, os, head), live, x, narrow2<T>(e0), narrow2<T>(e1));
        }
    }
    if (!p.dweight[kd]) return;
    // the lanes of the same slot, in a fixed order: lane groups of the warp by
    // shuffles, then the warps through shared memory
    __shared__ float red[TPB / 32][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
#pragma unroll
        for (int o = LPU; o < 32; o <<= 1) {
            acc0[j].x += __shfl_xor_sync(0xffffffffu, acc0[j].x, o);
            acc0[j].y += __shfl_xor_sync(0xffffffffu, acc0[j].y, o);
            acc1[j].x += __shfl_xor_sync(0xffffffffu, acc1[j].x, o);
            acc1[j].y += __shfl_xor_sync(0xffffffffu, acc1[j].y, o);
        }
    if (lane < LPU) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            if (s.v0 >= 0) *reinterpret_cast<float2*>(&red[warp][s.v0 * N + 2 * j]) = acc0[j];
            if (s.v1 >= 0) *reinterpret_cast<float2*>(&red[warp][s.v1 * N + 2 * j]) = acc1[j];
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

constexpr int kSumWarps = 32;  // (up to 296 rows of few columns: 8 warps 7.7 us, 32 6)
__global__ void __launch_bounds__(kSumWarps * 32)
    norm_rope_finish_kernel(NormRopeParams p, int64_t rows_q, int64_t rows_k) {
    grid_dep_wait();
    const int kd = blockIdx.y;
    if (!p.dweight[kd]) return;
    column_sums<kSumWarps>(p.partial[kd], kd ? rows_k : rows_q, p.headdim,
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

// Tokens per tile: about eight rounds of units, evened out so that the CTAs
// (ctas at once) get the same number of tiles, and few enough that two tiles'
// angles fit 64 KB of shared memory.
int tile_tokens(int64_t tokens, int heads, int lpu, int rot_dim, int64_t ctas) {
    int64_t t = (static_cast<int64_t>(8) * (TPB / lpu) + heads - 1) / heads;
    if (rot_dim > 0 && t > 32768 / (rot_dim * 4)) t = 32768 / (rot_dim * 4);
    const int64_t turns = (tokens + ctas * t - 1) / (ctas * t);
    t = (tokens + ctas * turns - 1) / (ctas * turns);
    return static_cast<int>(t < 1 ? 1 : t);
}

// The backward's: up to sixteen rounds of units, shared out evenly over the
// CTAs' turns, with the least turns x (a tile's rounds + its barrier, about one).
// (b4 L4096 32 + 8 heads of 128 bf16: 104 us, with eight rounds 107.)
int bwd_tile_tokens(int64_t tokens, int heads, int lpu, int rot_dim, int64_t ctas) {
    const int64_t step = TPB / lpu;
    int64_t most = 16 * step / heads, best = 1, least = 0;
    if (rot_dim > 0) most = std::min<int64_t>(most, 32768 / (rot_dim * 4));
    most = std::max<int64_t>(most, 1);
    const int64_t turns = (tokens + ctas * most - 1) / (ctas * most);  // at least
    for (int64_t n = turns; n < turns + 16; ++n) {
        const int64_t t = (tokens + ctas * n - 1) / (ctas * n), cost = n * ((t * heads + step - 1) / step + 1);
        if (least == 0 || cost < least) {
            least = cost;
            best = t;
        }
    }
    return static_cast<int>(best);
}

constexpr int64_t kBwdCtas = 296;  // the backward's persistent CTAs, two per SM

}  // namespace

int64_t norm_rope_bwd_rows() { return kBwdCtas; }

namespace {

constexpr int kMaxSmem = 65536;  // two tiles' angles

template <typename T, int LPU> cudaError_t launch_fwd(const NormRopeParams& p, cudaStream_t s) {
    const int64_t tokens = p.batch * p.seqlen, slots = 3 * device_sms();
    const int tile = tile_tokens(tokens, p.heads[0] + p.heads[1], LPU, p.rot_dim, slots);
    const int64_t ntiles = (tokens + tile - 1) / tile, grid = ntiles < slots ? ntiles : slots;
    const auto kern = p.adjacent ? norm_rope_kernel<T, true, LPU> : norm_rope_kernel<T, false, LPU>;
    const cudaError_t e = p.adjacent ? prepare_kernel<norm_rope_kernel<T, true, LPU>>(kMaxSmem, false)
                                     : prepare_kernel<norm_rope_kernel<T, false, LPU>>(kMaxSmem, false);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(grid), TPB, 2 * static_cast<size_t>(tile) * p.rot_dim * 4, s>>>(p, tile, tokens);
    return cudaGetLastError();
}

template <typename T, int LPU> cudaError_t launch_bwd(const NormRopeParams& p, cudaStream_t s) {
    const int64_t tokens = p.batch * p.seqlen;
    const int H = p.heads[0] + p.heads[1];
    // the CTAs are shared out between q and k by their heads
    int64_t cq = kBwdCtas * p.heads[0] / H, ck = kBwdCtas - cq;
    if (cq < 1) cq = 1;
    if (ck < 1) ck = 1;
    const int tile_q = bwd_tile_tokens(tokens, p.heads[0], LPU, p.rot_dim, cq);
    const int tile_k = p.heads[1] ? bwd_tile_tokens(tokens, p.heads[1], LPU, p.rot_dim, ck) : 1;
    cq = std::min(cq, (tokens + tile_q - 1) / tile_q);
    ck = p.heads[1] ? std::min(ck, (tokens + tile_k - 1) / tile_k) : 0;
    const size_t smem = 2 * static_cast<size_t>(std::max(tile_q, tile_k)) * p.rot_dim * 4;
    const auto kern = p.adjacent ? norm_rope_bwd_kernel<T, true, LPU> : norm_rope_bwd_kernel<T, false, LPU>;
    cudaError_t e = p.adjacent ? prepare_kernel<norm_rope_bwd_kernel<T, true, LPU>>(kMaxSmem, false)
                               : prepare_kernel<norm_rope_bwd_kernel<T, false, LPU>>(kMaxSmem, false);
    if (e != cudaSuccess) return e;
    kern<<<static_cast<unsigned>(cq + ck), TPB, smem, s>>>(p, tile_q, tile_k, tokens, static_cast<int>(cq));
    e = cudaGetLastError();
    if (e != cudaSuccess || (!p.dweight[0] && !p.dweight[1])) return e;
    return launch_kernel(norm_rope_finish_kernel,
                         dim3(static_cast<unsigned>((p.headdim + 31) / 32), ck > 0 ? 2 : 1),
                         dim3(kSumWarps * 32), 0, s, true, p, cq, ck);
}

template <typename T, bool BWD> cudaError_t launch(const NormRopeParams& p, cudaStream_t s) {
    switch (lanes_per_unit(Vec16<T>::N, p.headdim, p.rot_dim)) {
        case 1: return BWD ? launch_bwd<T, 1>(p, s) : launch_fwd<T, 1>(p, s);
        case 2: return BWD ? launch_bwd<T, 2>(p, s) : launch_fwd<T, 2>(p, s);
        case 4: return BWD ? launch_bwd<T, 4>(p, s) : launch_fwd<T, 4>(p, s);
        case 8: return BWD ? launch_bwd<T, 8>(p, s) : launch_fwd<T, 8>(p, s);
        case 16: return BWD ? launch_bwd<T, 16>(p, s) : launch_fwd<T, 16>(p, s);
        default: return BWD ? launch_bwd<T, 32>(p, s) : launch_fwd<T, 32>(p, s);
    }
}

}  // namespace

template <typename T> cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t s) {
    return launch<T, false>(p, s);
}
template <typename T> cudaError_t launch_norm_rope_bwd(const NormRopeParams& p, cudaStream_t s) {
    return launch<T, true>(p, s);
}

template cudaError_t launch_norm_rope<float>(const NormRopeParams&, cudaStream_t);
template cudaError_t launch_norm_rope<__nv_bfloat16>(const NormRopeParams&, cudaStream_t);
template cudaError_t launch_norm_rope_bwd<float>(const NormRopeParams&, cudaStream_t);
template cudaError_t launch_norm_rope_bwd<__nv_bfloat16>(const NormRopeParams&, cudaStream_t);

}  // namespace ssd
