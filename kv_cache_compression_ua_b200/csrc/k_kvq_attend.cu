// k_kvq_attend.cu -- attention of a few queries per sequence over the 8-bit cache (formulas and
// layout in include/ua.h).
//
// Bound: HBM, the codes read once: 2 * DH bytes a slot and KV head, 6.5 TB/s / 148 SMs = 23 bytes
// a clock and SM.  The arithmetic has to hide under that, so nothing is converted twice and no
// thread does a dot product on the CUDA cores:
//   * one warp walks blocks of 64 slots with its own asynchronous copies (16 KB of shared memory a
//     warp, no block barrier in the walk);
//   * both products run on the tensor cores with the CODES as the 16-row operand and the (at most 16) query rows
//     as the 8-wide one: S^T = K Q^T and O^T = V^T P^T, so a token with 4 query heads wastes half
//     of a small product and not three quarters of a large one.  (A tcgen05 tile of 128 rows
//     would want the probabilities back through shared memory and TMEM for products of 8
//     columns; mma.sync keeps them in registers, and the products are far from being the bound);
//   * codes become f16 exactly (int8 and e4m3 both are f16 values), two a conversion; the scale of
//     a block multiplies its logits (keys) and its 16 partial sums a thread (values) in fp32;
//   * the contraction may run over the head's elements in any order: a lane takes 16 contiguous bytes of
//     a key as the operand's scattered elements; for the values, four tokens' bytes are
//     transposed in registers.
// Queries enter as f16 scaled by a power of two for each row (bf16 queries exactly; fp32 ones as a high
// and a low part), probabilities as f16 times 2^14 (fp32: high and low part), so that small
// probabilities of long caches keep 2^-38 of the row's maximum; sums and statistics are fp32.
//
// Split: the (sequence, KV head, row tile, block) items of all sequences are laid out flat and cut
// into equal runs, one for each CTA, whatever the lengths; the lengths are read on the device.  A
// unit (sequence, head, row tile) that lies in several CTAs' runs is merged by the last of them
// to arrive, in the order of the runs.
#include <cuda_fp16.h>

#include "tc_common.cuh"
#include "ua_kernels.h"
#include "ua_profile.h"

namespace ua {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 14.f;             // probabilities are held as 2^14 p
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRingBytes = 16384;           // per warp
constexpr int kMinItems = kWarps;           // fewest blocks a CTA is given

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint2 b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four codes of a word -> two f16x2 (bytes 0,1 and 2,3), exactly.  int8: the byte with its sign
// flipped is a mantissa of 1024 + (code + 128).
template <bool E4M3> __device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        w ^= 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));        // 1152
        uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
        __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off), hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
        lo = *reinterpret_cast<uint32_t*>(&ha);
        hi = *reinterpret_cast<uint32_t*>(&hb);
    }
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x0, x1 as a sum of N bf16 pairs (N = 3 holds an fp32 value)
template <int N> __device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t* out) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        out[i] = pack_bf16(x0, x1);
        x0 -= bf16_lo(out[i]);
        x1 -= bf16_hi(out[i]);
    }
}

// Shared-memory placement of a block's codes, in 16-byte chunks, so that the operand reads below
// meet no bank twice: keys are read 16 bytes a lane at tokens t and t + 4, values 8 bytes a lane
// at four neighbouring tokens.
template <int DH> __device__ __forceinline__ int k_place(int tok, int chunk) {
    if constexpr (DH == 64) return (tok >> 1) * 128 + (((tok ^ (tok >> 2)) & 1) << 6) + chunk * 16;
    return tok * 128 + ((chunk ^ (tok & 4)) << 4);
}
template <int DH> __device__ __forceinline__ int v_place(int tok, int chunk) {
    if constexpr (DH == 64) return (tok >> 1) * 128 + ((tok & 1) << 6) + ((chunk ^ (tok & 2)) << 4);
    return tok * 128 + ((chunk ^ ((tok & 3) << 1)) << 4);
}
// Token of operand row m within 16 tokens: the values' operand takes tokens c, c+4, c+8, c+12 as
// rows 2c, 2c+1, 2c+8, 2c+9.
__device__ __forceinline__ int tok_of(int r) { return (r >> 1) + ((r & 1) << 2); }

template <typename T, int DH, int NT, bool E4M3> struct Att {
    static constexpr bool F32 = sizeof(T) == 4;
    static constexpr int R = 8 * NT;                 // query rows of a tile
    static constexpr int QP = F32 ? 2 : 1;           // f16 parts of a query
    static constexpr int PP = F32 ? 2 : 1;           // f16 parts of a probability
    static constexpr int TP = F32 ? 3 : 1;           // bf16 parts of an activation
    static constexpr int TPP = F32 ? 3 : 2;          // bf16 parts of a probability
    static constexpr int NSTG = 128 / DH;            // blocks in a warp's ring
    static constexpr int KB = 64 * DH;               // bytes of a block's keys
    static constexpr int QS = DH + 4;                // row stride of the queries in shared memory
    static constexpr int NM = DH / 16;               // 16-element tiles of the output
    struct Smem {
        alignas(128) unsigned char ring[kWarps][kRingBytes];
        alignas(16) uint16_t q16[QP][R][QS];         // f16, scaled by a power of two a row
        alignas(16) uint16_t qb[TP][R][QS];          // bf16 parts (for the unfinished block)
        float qf[R];                                 // logit scale times the row's power of two
        int lim[R];                                  // last slot the row sees, -1: none
        float m[kWarps][R], l[kWarps][R];
        long long scan[kWarps];
        int found[2];
        int last;
    };
};

// What a warp carries through a unit: O^T (elements 64 * pass + 8r + 2mt + {0, 1} of columns
// 8nt + 2c + {0, 1}, r = lane/4, c = lane%4), the columns' running maximum and this lane's sums.
template <int DH, int NT> struct State {
    float o[DH / 16][NT][4];
    float m[NT][2], l[NT][2];
};

// Online softmax of one block: logits x[mt][nt][e] (rows: tokens tok_of(r) and + 8, columns as in
// State) -> probabilities in place, corr = factor of what was accumulated, any: whether the column sees the block.
template <int DH, int NT>
__device__ __forceinline__ void block_softmax(State<DH, NT>& st, float (&x)[4][NT][4], float (&corr)[NT][2],
                                              bool (&any)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = x[0][nt][e];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) mx = fmaxf(mx, fmaxf(x[mt][nt][e], x[mt][nt][e + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // a NaN logit is no maximum, but it is something seen
            bool seen = mx > -INFINITY;
            bool nan = false;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) nan |= x[mt][nt][e] != x[mt][nt][e] || x[mt][nt][e + 2] != x[mt][nt][e + 2];
            const unsigned who = __ballot_sync(0xffffffffu, nan);
            seen = seen || (who & (0x11111111u << (threadIdx.x & 3))) != 0;
            any[nt][e] = seen;
            const float mn = fmaxf(st.m[nt][e], mx);
            const float ms = mn == -INFINITY ? 0.f : mn;
            corr[nt][e] = ex2((st.m[nt][e] - ms) * kLog2e);
            st.m[nt][e] = mn;
            float sum = 0.f;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float& v = x[mt][nt][e + 2 * k];
                    v = ex2(fmaf(v - ms, kLog2e, kPShift));   // (v - ms first: exact 0 at the lowest float)
                    sum += v;
                }
            st.l[nt][e] = fmaf(st.l[nt][e], corr[nt][e], sum);
        }
}

template <int DH, int NT> __device__ __forceinline__ void init_state(State<DH, NT>& st) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st.m[nt][e] = -INFINITY;
            st.l[nt][e] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < DH / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[i][nt][e] = 0.f;
    }
}

// One unfinished block, its rows in the activation type out of the ring: bf16 products, the
// operands as sums of bf16 parts (bf16 activations are one part, fp32 ones three; pairs of parts
// below 2^-24 of the product are left out).  Read straight into the operands' registers: it is at
// most one block in a unit.
template <typename T, int DH, int NT, bool E4M3>
__device__ __forceinline__ void tail_block(const KvqAttendParams& p, typename Att<T, DH, NT, E4M3>::Smem& sm,
                                        State<DH, NT>& st, int b, int h, int slot0, int n) {
    using A = Att<T, DH, NT, E4M3>;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const size_t ring = ((size_t)b * p.c.Hkv + h) * kKvqRing;
    const T* kr = static_cast<const T*>(p.c.kr) + ring * DH;
    const T* vr = static_cast<const T*>(p.c.vr) + ring * DH;
    const int ring0 = slot0 & (kKvqRing - 1);
    const float* bias = p.bias ? p.bias + ((size_t)b * p.c.Hkv + h) * p.c.cap + slot0 : nullptr;
    float x[4][NT][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][nt][e] = 0.f;
        if (slot0 + 16 * mt < n) {
#pragma unroll 4
            for (int s = 0; s < DH / 16; ++s) {
                const int d0 = (s >> 2) * 64 + 16 * c + 4 * (s & 3);
                uint32_t a[A::TP][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {            // rows r and r + 8: elements d0 .. d0+3
                    const int tok = 16 * mt + tok_of(r) + 8 * k;
                    const bool ok = slot0 + tok < n;
                    const T* src = kr + (size_t)(ring0 + tok) * DH + d0;
                    if constexpr (A::F32) {
                        const float4 f = ok ? *reinterpret_cast<const float4*>(src) : make_float4(0, 0, 0, 0);
                        uint32_t lo[3], hi[3];
                        split_bf16<3>(f.x, f.y, lo);
                        split_bf16<3>(f.z, f.w, hi);
#pragma unroll
                        for (int i = 0; i < A::TP; ++i) { a[i][k] = lo[i]; a[i][2 + k] = hi[i]; }
                    } else {
                        const uint2 u = ok ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
                        a[0][k] = u.x;
                        a[0][2 + k] = u.y;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < A::TP; ++j) {
                        const uint2 q = *reinterpret_cast<const uint2*>(&sm.qb[j][8 * nt + r][d0]);
#pragma unroll
                        for (int i = 0; i + j < A::TP; ++i) mma_bf16(x[mt][nt], a[i], q);
                    }
            }
        }
    }
    bool hidden[4][2];                                   // tokens no row sees: their values may be anything
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int tok = 16 * mt + tok_of(r) + 8 * k, slot = slot0 + tok;
            const float bs = slot >= n ? -INFINITY : bias ? __ldg(bias + tok) : 0.f;
            hidden[mt][k] = bs == -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float& v = x[mt][nt][2 * k + e];
                    v = hidden[mt][k] || slot > sm.lim[8 * nt + 2 * c + e] ? -INFINITY : fmaf(v, p.scale, bs);
                }
        }
    float corr[NT][2];
    bool any[NT][2];
    block_softmax<DH, NT>(st, x, corr, any);
    uint2 pb[A::TPP][4][NT];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t lo[A::TPP], hi[A::TPP];
            split_bf16<A::TPP>(x[mt][nt][0], x[mt][nt][1], lo);
            split_bf16<A::TPP>(x[mt][nt][2], x[mt][nt][3], hi);
#pragma unroll
            for (int i = 0; i < A::TPP; ++i) pb[i][mt][nt] = make_uint2(transpose8x8(lo[i]), transpose8x8(hi[i]));
        }
    // a token's row of the values' operand sits at other lanes than its logit: the bit of token
    // 16 ks + t comes from lane 4 r(t) of the same 16 tokens
    unsigned hid[4][2];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k) hid[ks][k] = __ballot_sync(0xffffffffu, hidden[ks][k]);
#pragma unroll
    for (int pass = 0; pass < DH / 64; ++pass) {
        float acc[4][NT][4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (slot0 + 16 * ks >= n) continue;
            float v[4][8];                               // tokens 4i + c, elements 64 pass + 8r ..
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * i + c;                 // row of the logits' operand: tok_of(row) = t mod 8
                const int row = 2 * (t & 3) + ((t >> 2) & 1);
                const bool ok = ((hid[ks][t >> 3] >> (4 * row)) & 1u) == 0;
                const T* src = vr + (size_t)(ring0 + 16 * ks + t) * DH + 64 * pass + 8 * r;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
                if (ok) {
                    Vec16<T>::ld(src, v[i]);
                    if constexpr (A::F32) Vec16<T>::ld(src + 4, v[i] + 4);
                }
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                uint32_t a[4][A::TP];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    split_bf16<A::TP>(v[0][2 * mt + k], v[1][2 * mt + k], a[k]);
                    split_bf16<A::TP>(v[2][2 * mt + k], v[3][2 * mt + k], a[2 + k]);
                }
#pragma unroll
                for (int i = 0; i < A::TP; ++i) {
                    const uint32_t ai[4] = {a[0][i], a[1][i], a[2][i], a[3][i]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < A::TPP; ++j)
                            if (i + j < 3) mma_bf16(acc[mt][nt], ai, pb[j][ks][nt]);
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st.o[4 * pass + mt][nt][e] =
                        fmaf(st.o[4 * pass + mt][nt][e], corr[nt][e & 1], any[nt][e & 1] ? acc[mt][nt][e] : 0.f);
    }
}

// The warp's walk over blocks first, first + kWarps, ... < last of one unit.
template <typename T, int DH, int NT, bool E4M3>
__device__ __forceinline__ void walk(const KvqAttendParams& p, typename Att<T, DH, NT, E4M3>::Smem& sm,
                                     State<DH, NT>& st, int b, int h, int n, int first, int last) {
    using A = Att<T, DH, NT, E4M3>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int nfull = n / kKvqBlock;
    const long long hrow = (long long)h * p.c.bpp;
    unsigned char* ring = sm.ring[warp];
    const uint32_t ring_s = tc::smem_u32(ring);
    const float* bias0 = p.bias ? p.bias + ((size_t)b * p.c.Hkv + h) * p.c.cap : nullptr;
    // row of block i (or -1: past the run, the unfinished block, or a bad page)
    auto row_of = [&](int blk) -> long long {
        if (blk >= last || blk >= nfull) return -1;
        const long long x = kvq_row(p.c, b, blk);
        return x < 0 ? -1 : x + hrow;
    };
    auto load_k = [&](long long row, int stg) {
        if (row >= 0) {
            const uint8_t* src = p.c.k + row * A::KB;
#pragma unroll
            for (int i = 0; i < A::KB / 512; ++i) {
                const int e = i * 32 + lane, tok = e / (DH / 16), ch = e % (DH / 16);
                cp_async16(ring_s + stg * 2 * A::KB + k_place<DH>(tok, ch), src + e * 16);
            }
        }
        tc::cp_async_commit();
    };
    auto load_v = [&](long long row, int stg) {
        if (row >= 0) {
            const uint8_t* src = p.c.v + row * A::KB;
#pragma unroll
            for (int i = 0; i < A::KB / 512; ++i) {
                const int e = i * 32 + lane, tok = e / (DH / 16), ch = e % (DH / 16);
                cp_async16(ring_s + (stg * 2 + 1) * A::KB + v_place<DH>(tok, ch), src + e * 16);
            }
        }
        tc::cp_async_commit();
    };
    // rows of the blocks in flight, and the scales of the next block, are fetched ahead
    long long rows[A::NSTG + 1];
#pragma unroll
    for (int i = 0; i <= A::NSTG; ++i) rows[i] = row_of(first + i * kWarps);
#pragma unroll
    for (int i = 0; i < A::NSTG; ++i) {
        load_k(rows[i], i);
        load_v(rows[i], i);
    }
    float ks = rows[0] >= 0 ? __ldg(p.c.ks + rows[0]) : 0.f, vs = rows[0] >= 0 ? __ldg(p.c.vs + rows[0]) : 0.f;
    float qf[NT][2];
    int lim[NT][2], lim_min = INT32_MAX;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            qf[nt][e] = sm.qf[8 * nt + 2 * c + e];
            lim[nt][e] = sm.lim[8 * nt + 2 * c + e];
            lim_min = min(lim_min, lim[nt][e]);
        }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    int stg = 0;
#pragma unroll 1
    for (int blk = first; blk < last; blk += kWarps) {
        const long long row = rows[0], next = rows[A::NSTG];
#pragma unroll
        for (int i = 0; i < A::NSTG; ++i) rows[i] = rows[i + 1];
        rows[A::NSTG] = row_of(blk + (A::NSTG + 1) * kWarps);
        const float ksn = rows[0] >= 0 ? __ldg(p.c.ks + rows[0]) : 0.f;
        const float vsn = rows[0] >= 0 ? __ldg(p.c.vs + rows[0]) : 0.f;
        if (row < 0) {                                   // the unfinished block, or one without a page
            if (blk == nfull) tail_block<T, DH, NT, E4M3>(p, sm, st, b, h, blk * kKvqBlock, n);
            load_k(next, stg);
            load_v(next, stg);
        } else {
            const unsigned char* kb = ring + stg * 2 * A::KB;
            const unsigned char* vb = kb + A::KB;
            float bs[4][2];
            if (bias0) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        bs[mt][k] = __ldg(bias0 + blk * kKvqBlock + 16 * mt + tok_of(r) + 8 * k);
            }
            // S^T = K Q^T
            cp_async_wait<2 * A::NSTG - 1>();
            __syncwarp();
            float x[4][NT][4];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[mt][nt][e] = 0.f;
#pragma unroll
            for (int hf = 0; hf < DH / 64; ++hf) {
                uint2 q[A::QP][NT][4];
#pragma unroll
                for (int i = 0; i < A::QP; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            q[i][nt][s] = *reinterpret_cast<const uint2*>(&sm.q16[i][8 * nt + r][64 * hf + 16 * c + 4 * s]);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const int tok = 16 * mt + tok_of(r);
                    const uint4 u0 = *reinterpret_cast<const uint4*>(kb + k_place<DH>(tok, 4 * hf + c));
                    const uint4 u1 = *reinterpret_cast<const uint4*>(kb + k_place<DH>(tok + 8, 4 * hf + c));
                    const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        uint32_t a[4];
                        codes_f16<E4M3>(w0[s], a[0], a[2]);
                        codes_f16<E4M3>(w1[s], a[1], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < A::QP; ++i) mma_f16(x[mt][nt], a, q[i][nt][s]);
                    }
                }
            }
            __syncwarp();
            load_k(next, stg);
            // logits
            const bool masked = blk * kKvqBlock + kKvqBlock - 1 > lim_min;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = qf[nt][e] * ks;
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float& v = x[mt][nt][2 * k + e];
                            v *= f;
                            if (bias0) v = bs[mt][k] == -INFINITY ? -INFINITY : v + bs[mt][k];
                            if (masked && blk * kKvqBlock + 16 * mt + tok_of(r) + 8 * k > lim[nt][e]) v = -INFINITY;
                        }
                }
            float corr[NT][2];
            bool any[NT][2];
            block_softmax<DH, NT>(st, x, corr, any);
            uint2 pb[A::PP][4][NT];
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t lo = pack_f16(x[mt][nt][0], x[mt][nt][1]), hi = pack_f16(x[mt][nt][2], x[mt][nt][3]);
                    pb[0][mt][nt] = make_uint2(transpose8x8(lo), transpose8x8(hi));
                    if constexpr (A::PP == 2) {
                        const float2 l2 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                        const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                        pb[1][mt][nt] = make_uint2(transpose8x8(pack_f16(x[mt][nt][0] - l2.x, x[mt][nt][1] - l2.y)),
                                                   transpose8x8(pack_f16(x[mt][nt][2] - h2.x, x[mt][nt][3] - h2.y)));
                    }
                }
            // O^T += vs * V^T P^T
            cp_async_wait<2 * A::NSTG - 1>();
            __syncwarp();
#pragma unroll
            for (int pass = 0; pass < DH / 64; ++pass) {
                float acc[4][NT][4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) {
                    uint2 w[4];                          // tokens 4i + c, elements 64 pass + 8r ..
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = *reinterpret_cast<const uint2*>(vb + v_place<DH>(16 * kt + 4 * i + c, 4 * pass + (r >> 1)) +
                                                               8 * (r & 1));
#pragma unroll
                    for (int hw = 0; hw < 2; ++hw) {
                        const uint32_t t0 = hw ? w[0].y : w[0].x, t1 = hw ? w[1].y : w[1].x;
                        const uint32_t t2 = hw ? w[2].y : w[2].x, t3 = hw ? w[3].y : w[3].x;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t a[4];
                            const uint32_t sel = k ? 0x7362 : 0x5140;
                            codes_f16<E4M3>(__byte_perm(t0, t1, sel), a[0], a[1]);
                            codes_f16<E4M3>(__byte_perm(t2, t3, sel), a[2], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int i = 0; i < A::PP; ++i) mma_f16(acc[2 * hw + k][nt], a, pb[i][kt][nt]);
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = any[nt][e] ? vs : 0.f;   // (a block no slot of which is seen may have a NaN scale)
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float& o = st.o[4 * pass + mt][nt][2 * k + e];
                                o = fmaf(acc[mt][nt][2 * k + e], f, o * corr[nt][e]);
                            }
                    }
            }
            __syncwarp();
            load_v(next, stg);
        }
        ks = ksn;
        vs = vsn;
        stg = stg + 1 == A::NSTG ? 0 : stg + 1;
    }
    cp_async_wait<0>();
}

template <typename T, int DH, int NT, bool E4M3>
__global__ void __launch_bounds__(kThreads, 3) k_kvq_attend(KvqAttendParams p) {
    using A = Att<T, DH, NT, E4M3>;
    constexpr int R = A::R;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    typename A::Smem& sm = *reinterpret_cast<typename A::Smem*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
    const int Hkv = p.c.Hkv, G = p.G;
    grid_dep_wait();
    // valid queries and slots of sequence b (an out-of-range count: none, with the status raised)
    auto counts = [&](int b, int* nq, int* n) {
        *nq = p.n_q ? p.n_q[b] : p.Tq;
        *n = p.c.n_kept[b];
        if (*nq < 0 || *nq > p.Tq || *n < 0 || *n > p.c.cap) {
            raise_status(UA_ERR_INVALID_ARG);
            *nq = min(max(*nq, 0), p.Tq);
            *n = 0;
        }
    };
    auto tiles_of = [&](int nq) { return (nq * G + R - 1) / R; };
    auto blocks_of = [&](int n) { return max((n + kKvqBlock - 1) / kKvqBlock, 1); };
    auto items_of = [&](int b) -> long long {
        if (b >= p.c.B) return 0;
        int nq, n;
        counts(b, &nq, &n);
        return (long long)Hkv * tiles_of(nq) * blocks_of(n);
    };
    // all items, and this CTA's run [lo, hi) of them
    long long total = 0;
    for (int b = tid; b < p.c.B; b += kThreads) total += items_of(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) sm.scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sm.scan[w];
    const long long ctas = min((long long)gridDim.x, (total + kMinItems - 1) / kMinItems);
    if (blockIdx.x >= ctas) return;
    long long lo = blockIdx.x * total / ctas;
    const long long hi = (blockIdx.x + 1) * total / ctas;
    // the sequence that holds item lo
    int b = 0;
    long long base = 0;
    for (int b0 = 0;; b0 += kThreads) {
        const long long mine = items_of(b0 + tid);
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        __syncthreads();
        if (lane == 31) sm.scan[warp] = inc;
        if (tid == 0) sm.found[0] = -1;
        __syncthreads();
        long long before = base;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) before += sm.scan[w];
        if (lo >= before + inc - mine && lo < before + inc) {
            sm.found[0] = b0 + tid;
            sm.found[1] = (int)(lo - (before + inc - mine));
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) base += sm.scan[w];
        __syncthreads();
        if (sm.found[0] >= 0) break;
    }
    b = sm.found[0];
    int off = sm.found[1];

    while (lo < hi) {
        int nq, n;
        counts(b, &nq, &n);
        const int nt_ = tiles_of(nq), nb = blocks_of(n), units = Hkv * nt_;
        const int u = off / nb, k0 = off - u * nb;
        if (u >= units) {                                // the next sequence with anything to do
            ++b;
            off = 0;
            continue;
        }
        const int h = u / nt_, rt = u - h * nt_;
        const int k1 = (int)min((long long)nb, k0 + (hi - lo));
        const long long g0 = lo - k0;                    // the unit's first item
        const int c_lo = (int)(((g0 + 1) * ctas - 1) / total), c_hi = (int)(((g0 + nb) * ctas - 1) / total);

        // queries of the tile: 8 threads a row
        __syncthreads();
        if (tid < 8 * R) {
            const int row = tid >> 3, part = tid & 7, gr = rt * R + row, i = gr / G, gg = gr - i * G;
            constexpr int E = DH / 8;
            float x[E];
            const bool ok = i < nq;
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.f;
            if (ok) {
                const T* src = static_cast<const T*>(p.q) + (((size_t)b * p.Tq + i) * p.H + h * G + gg) * DH + part * E;
#pragma unroll
                for (int e = 0; e < E; e += Vec16<T>::N) Vec16<T>::ld(src + e, x + e);
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[e]));
            const unsigned mask = __activemask();
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
            // largest element into [2^10, 2^11): f16 then holds 2^-24 of it and more as a normal number
            int ex = amax > 0.f && amax <= 3.4e38f ? 10 - ((int)(__float_as_uint(amax) >> 23) - 127) : 0;
            ex = max(-120, min(120, ex));
            const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const int at = part * E + e;
                const float y0 = x[e] * up, y1 = x[e + 1] * up;
                const uint32_t hq = pack_f16(y0, y1);
                *reinterpret_cast<uint32_t*>(&sm.q16[0][row][at]) = hq;
                if constexpr (A::QP == 2) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hq));
                    *reinterpret_cast<uint32_t*>(&sm.q16[1][row][at]) = pack_f16(y0 - f.x, y1 - f.y);
                }
                uint32_t t[A::TP];
                split_bf16<A::TP>(x[e], x[e + 1], t);
#pragma unroll
                for (int j = 0; j < A::TP; ++j) *reinterpret_cast<uint32_t*>(&sm.qb[j][row][at]) = t[j];
            }
            if (part == 0) {
                sm.qf[row] = p.scale * __uint_as_float((uint32_t)(127 - ex) << 23);
                sm.lim[row] = ok ? min(n - nq + i, n - 1) : INT32_MAX;      // (a row past the last query: anything)
            }
        }
        __syncthreads();
        State<DH, NT> st;
        init_state<DH, NT>(st);
        if (n > 0) walk<T, DH, NT, E4M3>(p, sm, st, b, h, n, k0 + warp, k1);

        // merge the warps: statistics and O through shared memory (the copies' ring is free)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = st.l[nt][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (r == 0) {
                    sm.m[warp][8 * nt + 2 * c + e] = st.m[nt][e];
                    sm.l[warp][8 * nt + 2 * c + e] = l;
                }
            }
        __syncthreads();
        float* buf = reinterpret_cast<float*>(sm.ring[0]) + warp * R * DH;   // [row][element]
        static_assert(kWarps * R * DH * 4 <= kWarps * kRingBytes, "the warps' outputs fit the ring");
#pragma unroll
        for (int i = 0; i < A::NM; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<float2*>(buf + (8 * nt + 2 * c + e) * DH + 64 * (i >> 2) + 8 * r + 2 * (i & 3)) =
                        make_float2(st.o[i][nt][e], st.o[i][nt][e + 2]);
        __syncthreads();
        const float* all = reinterpret_cast<const float*>(sm.ring[0]);
        const int rows = min(R, nq * G - rt * R);
        auto put_out = [&](int row, int d4, float4 o, float M, float L) {
            const int gr = rt * R + row, i = gr / G, head = h * G + gr - i * G;
            const size_t at = (((size_t)b * p.Tq + i) * p.H + head) * DH + d4;
            const float inv = L != 0.f ? 1.f / L : 0.f;
            float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
            if (p.g) {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] *= sigmoid_f(Elem<T>::ld(static_cast<const T*>(p.g) + at + e));
            }
            T* out = static_cast<T*>(p.o) + at;
            if constexpr (A::F32) {
                *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
            } else {
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            }
            if (p.lse && d4 == 0)
                p.lse[((size_t)b * p.H + head) * p.Tq + i] = L != 0.f ? M + (logf(L) - kPShift * 0.6931471805599453f) : -INFINITY;
        };
        const bool whole = c_lo == c_hi;
        const int slot = 2 * blockIdx.x + ((int)blockIdx.x == c_lo ? 1 : 0);
        float* mine = p.part + (size_t)slot * R * (DH + 2);
        for (int e = tid; e < rows * (DH / 4); e += kThreads) {
            const int row = e / (DH / 4), d4 = (e % (DH / 4)) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][row]);
            const float ms = M == -INFINITY ? 0.f : M;
            float4 o = make_float4(0, 0, 0, 0);
            float L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2((sm.m[w][row] - ms) * kLog2e);
                const float4 v = *reinterpret_cast<const float4*>(all + (w * R + row) * DH + d4);
                o.x = fmaf(v.x, f, o.x);
                o.y = fmaf(v.y, f, o.y);
                o.z = fmaf(v.z, f, o.z);
                o.w = fmaf(v.w, f, o.w);
                L = fmaf(sm.l[w][row], f, L);
            }
            if (whole) {
                put_out(row, d4, o, M, L);
            } else {
                *reinterpret_cast<float4*>(mine + 2 * R + row * DH + d4) = o;
                if (d4 == 0) {
                    mine[row] = M;
                    mine[R + row] = L;
                }
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                unsigned* cnt = p.cnt + ((size_t)b * Hkv + h) * p.RT + rt;
                const unsigned at = atomicAdd(cnt, 1u);
                sm.last = at == (unsigned)(c_hi - c_lo);
                if (at > (unsigned)(c_hi - c_lo)) raise_status(UA_ERR_INVALID_ARG);   // not zeroed
                if (sm.last) *cnt = 0;
                __threadfence();
            }
            __syncthreads();
            if (sm.last) {
                // runs c_lo .. c_hi hold the unit's parts: c_lo in its second slot, the others in their first
                const size_t ps = (size_t)R * (DH + 2);
                auto part = [&](int cc) { return p.part + (size_t)(2 * cc + (cc == c_lo ? 1 : 0)) * ps; };
                for (int e = tid; e < rows * (DH / 4); e += kThreads) {
                    const int row = e / (DH / 4), d4 = (e % (DH / 4)) * 4;
                    float M = -INFINITY;
                    for (int cc = c_lo; cc <= c_hi; ++cc) M = fmaxf(M, __ldcg(part(cc) + row));
                    const float ms = M == -INFINITY ? 0.f : M;
                    float4 o = make_float4(0, 0, 0, 0);
                    float L = 0.f;
#pragma unroll 4
                    for (int cc = c_lo; cc <= c_hi; ++cc) {
                        const float* q = part(cc);
                        const float f = ex2((__ldcg(q + row) - ms) * kLog2e);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(q + 2 * R + row * DH + d4));
                        o.x = fmaf(v.x, f, o.x);
                        o.y = fmaf(v.y, f, o.y);
                        o.z = fmaf(v.z, f, o.z);
                        o.w = fmaf(v.w, f, o.w);
                        L = fmaf(__ldcg(q + R + row), f, L);
                    }
                    put_out(row, d4, o, M, L);
                }
            }
        }
        lo += k1 - k0;
        off += k1 - k0;
    }
}

template <typename T, int DH, int NT, bool E4M3> cudaError_t attend(const KvqAttendParams& p, cudaStream_t s) {
    using A = Att<T, DH, NT, E4M3>;
    auto kern = k_kvq_attend<T, DH, NT, E4M3>;
    const int smem = (int)sizeof(typename A::Smem);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // at most the blocks of full caches: the lengths are known on the device only
    const long long most = (long long)p.c.B * p.c.Hkv * p.RT * ((p.c.cap + kKvqBlock - 1) / kKvqBlock);
    const long long want = (most + kMinItems - 1) / kMinItems;
    UA_PROFILE("k_kvq_attend", s);
    return launch_dependent(kern, dim3((unsigned)(want < kKvqAttendCtas ? want : kKvqAttendCtas)), dim3(kThreads),
                            (size_t)smem, s, p);
}

template <typename T, int DH> cudaError_t attend_n(const KvqAttendParams& p, bool e4m3, cudaStream_t s) {
    if (kvq_row_tile(p.Tq * p.G) == 8) return e4m3 ? attend<T, DH, 1, true>(p, s) : attend<T, DH, 1, false>(p, s);
    return e4m3 ? attend<T, DH, 2, true>(p, s) : attend<T, DH, 2, false>(p, s);
}

}  // namespace

cudaError_t launch_kvq_attend(const KvqAttendParams& p, int d, bool bf16, bool e4m3, cudaStream_t s) {
    if (d == 64) return bf16 ? attend_n<__nv_bfloat16, 64>(p, e4m3, s) : attend_n<float, 64>(p, e4m3, s);
    return bf16 ? attend_n<__nv_bfloat16, 128>(p, e4m3, s) : attend_n<float, 128>(p, e4m3, s);
}

}  // namespace ua
