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
    // bits of the largest magnitude (non-negative floats order as their bits, NaN last)
    __device__ __forceinline__ uint32_t amax_bits() const {
        if constexpr (NV == 1) {
            const uint32_t m = 0x7fff7fffu;
            const uint32_t a = __vmaxu2(__vmaxu2(u[0].x & m, u[0].y & m), __vmaxu2(u[0].z & m, u[0].w & m));
            return max(a & 0xffff0000u, a << 16);
        } else {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                a = max(max(a, max(u[i].x & 0x7fffffffu, u[i].y & 0x7fffffffu)),
                        max(u[i].z & 0x7fffffffu, u[i].w & 0x7fffffffu));
            return a;
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

// Geometry of the norm kernels: NTH threads take NTH / CH rows at a time, as 4 heads of
// NTH / CH / 4 tokens; a thread keeps its token and chunk, so its 8 cosines and sines stay in
// registers while it walks the heads four by four.
constexpr int kNormHeads = 4;
template <int DH, int NTH> constexpr int norm_tokens() { return NTH / (DH / 16) / kNormHeads; }

// A thread's own queue of 16-byte pieces in shared memory, filled by asynchronous copies several
// steps ahead: loads in flight that cost no registers.  No other thread reads them, so a thread waits
// for its own copies only.  Layout [stage][piece][thread]: neighbouring threads, neighbouring chunks.
template <int NTH, int PIECES, int DEPTH> struct LaneQueue {
    static constexpr int kBytes = NTH * PIECES * DEPTH * 16;
    uint4* base;                                     // this thread's first piece
    __device__ __forceinline__ LaneQueue(void* smem) : base(static_cast<uint4*>(smem) + threadIdx.x) {}
    __device__ __forceinline__ void put(int stage, int piece, const void* src, bool ok) {
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(base + (stage * PIECES + piece) * NTH));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
    }
    __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int PENDING> __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
    }
    __device__ __forceinline__ uint4 get(int stage, int piece) const { return base[(stage * PIECES + piece) * NTH]; }
};

// cos / sin of a tile's tokens into shared memory ([tokens][DH/2] each), then this thread's eight.
// posf(n): position of flat token n.
template <int DH, int NTH, typename F>
__device__ __forceinline__ void tile_angles(float* s_cos, float* s_sin, int n0, int N, const RopeFreq& rf,
                                            double* s_f, F posf, float* cs, float* sn) {
    constexpr int HALF = DH / 2, TOK = norm_tokens<DH, NTH>();
    const int tid = threadIdx.x;
    if (tid < HALF) s_f[tid] = rf.f[tid];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TOK * HALF / NTH; ++i) {
        const int e = i * NTH + tid, tk = e / HALF, m = e % HALF;
        const int n = n0 + tk;
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

// Forward of the tokens n0 ..: head quads y, y + ny, ... of the queries, then of the keys.
// angles(cs, sn) is called once the first loads are on their way.
template <typename T, int DH, int NTH> struct NormTile {
    static constexpr int NV = Raw8<T>::NV, DEPTH = 4;
    using Queue = LaneQueue<NTH, 2 * NV, DEPTH>;
    template <typename A>
    static __device__ __forceinline__ void run(const QkNormParams& p, int n0, int y, int ny, void* smem, A angles) {
        constexpr int CH = DH / 16, HALF = DH / 2;
        const int tid = threadIdx.x, c = tid % CH, hp = (tid / CH) % kNormHeads;
        const int n = n0 + tid / CH / kNormHeads, N = (int)p.N;
        const int nq4 = p.q ? (p.H + kNormHeads - 1) / kNormHeads : 0;
        const int all = nq4 + (p.k ? (p.Hkv + kNormHeads - 1) / kNormHeads : 0);
        Queue queue(smem);
        auto fetch = [&](int i, int stage) {
            if (i < all) {
                const bool is_q = i < nq4;
                const int h = (is_q ? i : i - nq4) * kNormHeads + hp;
                const bool ok = n < N && h < (is_q ? p.H : p.Hkv);
                const T* x = is_q ? static_cast<const T*>(p.q) : static_cast<const T*>(p.k);
                const T* s = ok ? x + (long long)n * (is_q ? p.q_ld : p.k_ld) + h * DH + 8 * c : x;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    queue.put(stage, v, s + v * Vec16<T>::N, ok);
                    queue.put(stage, NV + v, s + HALF + v * Vec16<T>::N, ok);
                }
            }
            queue.commit();
        };
#pragma unroll
        for (int i = 0; i < DEPTH - 1; ++i) fetch(y + i * ny, i);
        float cs[8], sn[8], w0[8], w1[8];
        angles(cs, sn);
        const float* have = nullptr;                    // gain the registers hold
        int stage = 0;
        for (int i = y; i < all; i += ny) {
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
            fetch(i + (DEPTH - 1) * ny, (stage + DEPTH - 1) % DEPTH);
            queue.template wait<DEPTH - 1>();
            Raw8<T> a, b;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                a.u[v] = queue.get(stage, v);
                b.u[v] = queue.get(stage, NV + v);
            }
            stage = (stage + 1) % DEPTH;
            float x0[8], x1[8];
            a.get(x0);
            b.get(x1);
            if (w != nullptr) norm_row<DH>(x0, x1, w0, w1, p.eps);
            if (p.rope) rotate_row(x0, x1, cs, sn);
            const int h = (is_q ? i : i - nq4) * kNormHeads + hp;
            if (n < N && h < (is_q ? p.H : p.Hkv)) {
                T* d = is_q ? static_cast<T*>(p.q_out) + ((long long)n * p.H + h) * DH + 8 * c
                            : static_cast<T*>(p.k_out) + ((long long)n * p.Hkv + h) * DH + 8 * c;
                a.put(x0);
                b.put(x1);
                a.st(d);
                b.st(d + HALF);
            }
        }
        queue.template wait<0>();
    }
};

}  // namespace ua
