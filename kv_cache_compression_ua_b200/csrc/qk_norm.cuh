// qk_norm.cuh -- one head's norm and position rotation, shared by the norm operator and the
// append to the 8-bit cache.
#pragma once

#include "ua_common.cuh"
#include "ua_kernels.h"

namespace ua {

// Two fp32 operations an instruction (sm_100a's packed arithmetic): the norm kernels would otherwise be
// bound by instruction issue before memory.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un2(F2 a, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 neg2(F2 a) { return F2{a.v ^ 0x8000000080000000ull}; }
__device__ __forceinline__ float hsum(F2 a) {
    float x, y;
    un2(a, x, y);
    return x + y;
}
// 8 floats as 4 pairs
__device__ __forceinline__ void pairs(const float* x, F2* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f2(x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ void unpairs(const F2* p, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) un2(p[i], x[2 * i], x[2 * i + 1]);
}

// A head's row is spread over CH = DH/16 consecutive lanes; lane c holds 8 elements of the first half and
// their rotation partners DH/2 further: the 16-byte pieces c (bf16), or c and c + CH (f32) of
// each half, so that neighbouring lanes always touch neighbouring pieces (f32 rows as 8 contiguous
// elements a lane cost half of every 32-byte sector: 1B backward 38 us).
template <typename T, int DH> constexpr int kPieceStep = Vec16<T>::N * (DH / 16);      // elements from a lane's piece to its next
template <typename T> __device__ __forceinline__ int lane_at(int c) { return Vec16<T>::N * c; }   // its first element
template <typename T, int DH> __device__ __forceinline__ int elem_at(int c, int e) {              // its e-th
    return lane_at<T>(c) + e / Vec16<T>::N * kPieceStep<T, DH> + e % Vec16<T>::N;
}

// 8 activations as loaded: one 16-byte vector (bf16) or two (f32).
template <typename T> struct Raw8 {
    static constexpr int NV = sizeof(T) / 2;
    uint4 u[NV];
    __device__ __forceinline__ void get(float* x) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) Vec16<T>::unpack(u[i], x + i * Vec16<T>::N);
    }
    __device__ __forceinline__ void get(F2* p) const {
        float x[8];
        get(x);
        pairs(x, p);
    }
    __device__ __forceinline__ void put(const F2* p) {
        float x[8];
        unpairs(p, x);
        put(x);
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
    // bits of the largest magnitude of this and another's (non-negative floats order as their bits, NaN
    // above all)
    __device__ __forceinline__ uint32_t amax_bits(const Raw8& o) const {
        if constexpr (NV == 1) {
            uint32_t a = amax2(amax2(amax2(u[0].x, u[0].y), amax2(u[0].z, u[0].w)),
                               amax2(amax2(o.u[0].x, o.u[0].y), amax2(o.u[0].z, o.u[0].w)));
            a &= 0x7fff7fffu;
            return max(a & 0xffff0000u, a << 16);
        } else {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                a = max(max(a, max(u[i].x & 0x7fffffffu, u[i].y & 0x7fffffffu)),
                        max(u[i].z & 0x7fffffffu, u[i].w & 0x7fffffffu));
                a = max(max(a, max(o.u[i].x & 0x7fffffffu, o.u[i].y & 0x7fffffffu)),
                        max(o.u[i].z & 0x7fffffffu, o.u[i].w & 0x7fffffffu));
            }
            return a;
        }
    }
    // larger magnitudes of two bf16 pairs, NaN kept; the signs are of no meaning
    static __device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    template <int DH> __device__ __forceinline__ void st(T* p) const {   // p: the lane's first piece
#pragma unroll
        for (int i = 0; i < NV; ++i) *reinterpret_cast<uint4*>(p + i * kPieceStep<T, DH>) = u[i];
    }
};

// A lane's 8 of a half row of floats in shared memory (16-byte aligned)
template <typename T, int DH> __device__ __forceinline__ void pairs_at(const float* x, int c, F2* p) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 a = *reinterpret_cast<const float4*>(x + elem_at<T, DH>(c, 4 * i));
        p[2 * i] = f2(a.x, a.y);
        p[2 * i + 1] = f2(a.z, a.w);
    }
}

// cos / sin of pos * f, given gt = f / (2 pi): the angle in turns is formed in double precision and its
// nearest integer removed exactly, so far positions keep the accuracy of the sine of the remainder.
// fp32 results take sincospi (1 to 2 ulp); bf16 ones the fast unit, whose absolute error on
// [-pi, pi], below 2^-20, is far under their half step of 2^-8 of the pair's size.
template <typename T> __device__ __forceinline__ void rope_cs_turn(int pos, double gt, float* c, float* s) {
    const double a = (double)pos * gt;
    const float r = (float)(a - rint(a));
    if constexpr (sizeof(T) == 4) {
        sincospif(2.f * r, s, c);
    } else {
        __sincosf(6.28318530717958648f * r, s, c);
    }
}

// Sum over a row's lanes; every lane of the warp calls.
template <int CH> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = CH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 / sqrt(mean square + eps) of a head
template <int DH> __device__ __forceinline__ float row_rstd(const F2* x0, const F2* x1, float eps) {
    F2 ss = mul2(x0[0], x0[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) ss = fma2(x0[i], x0[i], ss);
#pragma unroll
    for (int i = 0; i < 4; ++i) ss = fma2(x1[i], x1[i], ss);
    return rsqrtf(row_sum<DH / 16>(hsum(ss)) * (1.f / DH) + eps);
}

template <int DH> __device__ __forceinline__ void norm_row(F2* x0, F2* x1, const F2* w0, const F2* w1, float eps) {
    const float r = row_rstd<DH>(x0, x1, eps);
    const F2 r2 = f2(r, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x0[i] = mul2(mul2(x0[i], r2), w0[i]);
        x1[i] = mul2(mul2(x1[i], r2), w1[i]);
    }
}

// R(pos) x; with -sn for sn and sn for ns (the negated sines), R(-pos) x
__device__ __forceinline__ void rotate_row(F2* x0, F2* x1, const F2* cs, const F2* sn, const F2* ns) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const F2 a = x0[i], b = x1[i];
        x0[i] = fma2(b, ns[i], mul2(a, cs[i]));
        x1[i] = fma2(a, sn[i], mul2(b, cs[i]));
    }
}
__device__ __forceinline__ void negate(const F2* a, F2* b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = neg2(a[i]);
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
    __device__ __forceinline__ void put(int stage, int piece, const void* src) {
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(base + (stage * PIECES + piece) * NTH));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    }
    __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int PENDING> __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
    }
    __device__ __forceinline__ uint4 get(int stage, int piece) const { return base[(stage * PIECES + piece) * NTH]; }
};

// cos / sin of a tile's tokens into shared memory ([tokens][DH/2] each), then this thread's eight.
// posf(n): position of flat token n.
template <typename T, int DH, int NTH, typename F>
__device__ __forceinline__ void tile_angles(float* s_cos, float* s_sin, int n0, int N, const RopeFreq& rf,
                                            double* s_f, F posf, F2* cs, F2* sn) {
    constexpr int HALF = DH / 2, TOK = norm_tokens<DH, NTH>();
    const int tid = threadIdx.x;
    if (tid < HALF) s_f[tid] = rf.f[tid] * 0.15915494309189535;      // 1 / (2 pi)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TOK * HALF / NTH; ++i) {
        const int e = i * NTH + tid, tk = e / HALF, m = e % HALF;
        const int n = n0 + tk;
        rope_cs_turn<T>(n < N ? posf(n) : 0, s_f[m], s_cos + e, s_sin + e);
    }
    __syncthreads();
    const int c = tid % (DH / 16), tk = tid / (DH / 16) / kNormHeads;
    pairs_at<T, DH>(s_cos + tk * HALF, c, cs);
    pairs_at<T, DH>(s_sin + tk * HALF, c, sn);
}
// A thread's own 8 angles at position pos; s_f: f / (2 pi) of the DH/2 pairs.
template <typename T, int DH> __device__ __forceinline__ void lane_angles(int pos, const double* s_f, int c, F2* cs, F2* sn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float ca, sa, cb, sb;
        rope_cs_turn<T>(pos, s_f[elem_at<T, DH>(c, 2 * i)], &ca, &sa);
        rope_cs_turn<T>(pos, s_f[elem_at<T, DH>(c, 2 * i + 1)], &cb, &sb);
        cs[i] = f2(ca, cb);
        sn[i] = f2(sa, sb);
    }
}
// 8 gains of each half
template <typename T, int DH> __device__ __forceinline__ void load_gains(const float* w, int c, F2* w0, F2* w1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float* a = w + elem_at<T, DH>(c, 2 * i);
        w0[i] = f2(__ldg(a), __ldg(a + 1));
        w1[i] = f2(__ldg(a + DH / 2), __ldg(a + DH / 2 + 1));
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
                const T* s = x + (long long)n * (is_q ? p.q_ld : p.k_ld) + h * DH + lane_at<T>(c);
                if (ok) {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        queue.put(stage, v, s + v * kPieceStep<T, DH>);
                        queue.put(stage, NV + v, s + HALF + v * kPieceStep<T, DH>);
                    }
                }
            }
            queue.commit();
        };
#pragma unroll
        for (int i = 0; i < DEPTH - 1; ++i) fetch(y + i * ny, i);
        F2 cs[4], sn[4], w0[4], w1[4];
        angles(cs, sn);
        F2 ns[4];
        negate(sn, ns);
        const float* have = nullptr;                    // gain the registers hold
        int stage = 0;
        for (int i = y; i < all; i += ny) {
            const bool is_q = i < nq4;
            const float* w = is_q ? p.wq : p.wk;
            if (w != nullptr && w != have) {
                load_gains<T, DH>(w, c, w0, w1);
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
            F2 x0[4], x1[4];
            a.get(x0);
            b.get(x1);
            if (w != nullptr) norm_row<DH>(x0, x1, w0, w1, p.eps);
            if (p.rope) rotate_row(x0, x1, cs, sn, ns);
            const int h = (is_q ? i : i - nq4) * kNormHeads + hp;
            if (n < N && h < (is_q ? p.H : p.Hkv)) {
                T* d = is_q ? static_cast<T*>(p.q_out) + ((long long)n * p.H + h) * DH + lane_at<T>(c)
                            : static_cast<T*>(p.k_out) + ((long long)n * p.Hkv + h) * DH + lane_at<T>(c);
                a.put(x0);
                b.put(x1);
                a.template st<DH>(d);
                b.template st<DH>(d + HALF);
            }
        }
        queue.template wait<0>();
    }
};

}  // namespace ua
