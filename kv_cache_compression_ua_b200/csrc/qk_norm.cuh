// qk_norm.cuh -- one head's norm and position rotation, shared by the norm operator and the
// append to the 8-bit cache.
#pragma once

#include "ua_common.cuh"
#include "ua_kernels.h"

namespace ua {

// 8 activations as loaded: one 16-byte vector (bf16) or two (f32).
template <typename T> struct Raw8 {
    static constexpr int NV = sizeof(T) / 2;
    uint4 u[NV];
    __device__ __forceinline__ void ld(const T* p) {
#pragma unroll
        for (int i = 0; i < NV; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NV; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) Vec16<T>::unpack(u[i], x + i * Vec16<T>::N);
    }
    // rounds to the activation type (once)
    __device__ __forceinline__ void put(const float* x) {
        if constexpr (NV == 1) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<uint32_t*>(&h);
            }
            u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                u[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                  __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
        }
    }
    __device__ __forceinline__ void st(T* p) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
    }
};

// cos / sin of pos * f: the angle in turns is formed in double precision and its nearest integer
// removed exactly, so far positions keep the accuracy of the fp32 sine of the remainder.
__device__ __forceinline__ void rope_cs_pi(int pos, double f, float* c, float* s) {
    const double a = (double)pos * (f * 0.15915494309189535);      // 1 / (2 pi)
    sincospif(2.f * (float)(a - rint(a)), s, c);
}

// Rows are spread over a CTA as CH = DH/16 consecutive lanes a head, each lane with elements
// 8c .. 8c+7 and their rotation partners d/2 + 8c ...; every lane of the warp calls.
template <int CH> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = CH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int DH> __device__ __forceinline__ void norm_row(float* x0, float* x1, const float* w0, const float* w1,
                                                           float eps) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
    const float r = rsqrtf(row_sum<DH / 16>(ss) * (1.f / DH) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x0[e] = x0[e] * r * w0[e];
        x1[e] = x1[e] * r * w1[e];
    }
}

__device__ __forceinline__ void rotate_row(float* x0, float* x1, const float* cs, const float* sn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float a = x0[e], b = x1[e];
        x0[e] = a * cs[e] - b * sn[e];
        x1[e] = b * cs[e] + a * sn[e];
    }
}

// Geometry of the norm kernels: 64 rows at a time in 64 * CH threads, as 16 tokens x 4 heads;
// a thread keeps its token and chunk, so its 8 cosines and sines stay in registers while it
// walks the heads four by four.
constexpr int kNormTokens = 16, kNormHeads = 4;

// cos / sin of a tile's tokens into shared memory ([16][DH/2] each), then this thread's eight.
// posf(n): position of flat token n.
template <int DH, typename F>
__device__ __forceinline__ void tile_angles(float* s_cos, float* s_sin, long long n0, long long N, const RopeFreq& rf,
                                            double* s_f, F posf, float* cs, float* sn) {
    constexpr int HALF = DH / 2, NTH = 64 * (DH / 16);
    const int tid = threadIdx.x;
    if (tid < HALF) s_f[tid] = rf.f[tid];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kNormTokens * HALF / NTH; ++i) {
        const int e = i * NTH + tid, tk = e / HALF, m = e % HALF;
        const long long n = n0 + tk;
        rope_cs_pi(n < N ? posf(n) : 0, s_f[m], s_cos + e, s_sin + e);
    }
    __syncthreads();
    const int c = tid % (DH / 16), tk = tid / (DH / 16) / kNormHeads;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = s_cos[tk * HALF + 8 * c + e];
        sn[e] = s_sin[tk * HALF + 8 * c + e];
    }
}

// Forward of tokens n0 .. n0+15: head quads y, y + ny, ... of the queries, then of the keys.
template <typename T, int DH>
__device__ __forceinline__ void norm_rope_tile(const QkNormParams& p, long long n0, int y, int ny, const float* cs,
                                               const float* sn) {
    constexpr int CH = DH / 16, HALF = DH / 2;
    const int tid = threadIdx.x, c = tid % CH, hp = (tid / CH) % kNormHeads;
    const long long n = n0 + tid / CH / kNormHeads;
    const int nq4 = p.q ? (p.H + kNormHeads - 1) / kNormHeads : 0;
    const int nk4 = p.k ? (p.Hkv + kNormHeads - 1) / kNormHeads : 0;
    auto src = [&](int i, bool* ok) -> const T* {
        const bool is_q = i < nq4;
        const int h = (is_q ? i : i - nq4) * kNormHeads + hp;
        *ok = i < nq4 + nk4 && n < p.N && h < (is_q ? p.H : p.Hkv);
        return is_q ? static_cast<const T*>(p.q) + n * p.q_ld + h * DH + 8 * c
                    : static_cast<const T*>(p.k) + n * p.k_ld + h * DH + 8 * c;
    };
    Raw8<T> a, b;
    bool ok;
    const T* s = src(y, &ok);
    a.zero();
    b.zero();
    if (ok) { a.ld(s); b.ld(s + HALF); }
    float w0[8], w1[8];
    const float* have = nullptr;                        // gain the registers hold
    for (int i = y; i < nq4 + nk4; i += ny) {
        Raw8<T> an, bn;                                 // the next quad's loads fly over this one's work
        bool okn;
        const T* sx = src(i + ny, &okn);
        an.zero();
        bn.zero();
        if (okn) { an.ld(sx); bn.ld(sx + HALF); }
        const bool is_q = i < nq4;
        const float* w = is_q ? p.wq : p.wk;
        if (w != nullptr && w != have) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w0[e] = __ldg(w + 8 * c + e);
                w1[e] = __ldg(w + HALF + 8 * c + e);
            }
            have = w;
        }
        float x0[8], x1[8];
        a.get(x0);
        b.get(x1);
        if (w != nullptr) norm_row<DH>(x0, x1, w0, w1, p.eps);
        if (p.rope) rotate_row(x0, x1, cs, sn);
        if (ok) {
            const int h = (is_q ? i : i - nq4) * kNormHeads + hp;
            T* d = is_q ? static_cast<T*>(p.q_out) + (n * p.H + h) * DH + 8 * c
                        : static_cast<T*>(p.k_out) + (n * p.Hkv + h) * DH + 8 * c;
            a.put(x0);
            b.put(x1);
            a.st(d);
            b.st(d + HALF);
        }
        a = an;
        b = bn;
        ok = okn;
    }
}

}  // namespace ua
