// k_kvq_attend.cu -- attention of a few queries per sequence over the 8-bit cache (formulas and
// layout in include/ua.h).
//
// Bound: HBM, the codes read once: 2 * DH bytes a slot and KV head, 6.5 TB/s / 148 SMs = 23 bytes
// a clock and SM.  The arithmetic has to hide under that, so nothing is converted twice and no
// thread does a dot product on the CUDA cores:
//   * one warp walks blocks of 64 slots with its own asynchronous copies (a block's keys and values,
//     8 or 16 KB of shared memory a warp; no block barrier in the walk); one CTA of 16 (DH = 64), 12
//     (DH = 128) or 8 warps (more than 8 rows) an SM, so that few parts have to be merged;
//   * both products run on the tensor cores with the CODES as the 16-row operand and the (at most 16)
//     query rows as the 8-wide one: S^T = K Q^T and O^T = V^T P^T, so a token with 4 query heads wastes
//     half of a small product and not three quarters of a large one.  (A tcgen05 tile of 128 rows
//     would want the probabilities back through shared memory and TMEM for products of 8 columns;
//     mma.sync keeps them in registers, and the tensor pipe is 20 % busy);
//   * codes become f16 exactly and cheaply: e4m3 by its conversion, int8 as subnormals (codes_f16); the
//     scale of a block multiplies its logits (keys) and its partial sums (values) in fp32;
//   * the contraction may run over the head's elements in any order: a lane takes 16 contiguous bytes of
//     a key as the operand's scattered elements; for the values, tokens' bytes are paired in registers;
//   * a logit is one fused multiply-add and an exp2 from the product where nothing is masked.
// Queries enter as f16 scaled by a power of two for each row (bf16 queries exactly; fp32 ones as a high
// and a low part), probabilities as f16 times 2^14 (fp32: high and low part), so that small
// probabilities of long caches keep 2^-38 of the row's maximum; sums and statistics are fp32.  One f16 part rounds a
// probability by 2^-11 of it at most, an eighth of the half step of 2^-8 by which a bf16 output is rounded anyway
// (outputs are off by 1.7e-3 against 64 bits, as with fp32 probabilities), and a second part would double the second
// product; int8's offset of 128 costs two bits of the fp32 sums, far below that.
//
// Split, by lengths read on the device: few units (sequence, KV head, row tile) get whole CTAs each;
// otherwise the blocks of all units are laid out flat, with kUnitCost more for each unit, and cut into equal runs,
// one a CTA.  A unit in several CTAs is merged by the last of them to arrive, in the order of the blocks:
// the result does not depend on who that is.
//
// Measured (in a captured graph): 32 sequences of about 16k slots, 8 heads of 64, int8 (448 MB): 80 us, 5.6 TB/s (85 % of
// the copy bandwidth; the copies alone 74 us; what is left is the ALU pipe, 2 clocks a warp instruction); one of
// 262144 slots, 8 heads of 128, e4m3 (537 MB): 93 us, 5.8 TB/s (88 %; the copies alone 85 us, SMs of the
// larger clusters finish last); 4 of about 8192 with bias and gate (57 MB): 22 us, of it 7 us before the
// first products and 5 us of merging; one of 333 slots: 6.9 us.
#include <cuda_fp16.h>

#include <algorithm>

#include "tc_common.cuh"
#include "ua_kernels.h"
#include "ua_profile.h"

namespace ua {

namespace {

// Logits are held in units of ln 4, so that the lowest finite bias still fits; the running maximum of a
// column is a whole number of them (at or above its logits), so every rescale is a power of two and
// the shift below is exact.
constexpr float kLog4e = 0.72134752044448170f;
constexpr float kLn4 = 1.3862943611198906f;
constexpr float kPShift = 14.f;             // probabilities are held as 2^14 p
constexpr int kUnitCost = 6;                // what starting and merging a unit costs, in blocks

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// d = a b + c, d += a b
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint2 b, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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

// Four codes of a word -> two f16x2, exactly.  e4m3: codes 0, 1 and 2, 3.  int8: codes 0, 2 and 1, 3, each
// as (code + 128) 2^-24: the byte with its sign bit flipped is the mantissa of a subnormal f16, so no
// arithmetic is needed; the 128 are taken off by what the products' sums start from.
__device__ __forceinline__ uint32_t and_xor(uint32_t w) {       // one instruction, the masks in registers
    uint32_t y, keep = 0x00ff00ffu, flip = 0x00800080u;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(w), "r"(keep), "r"(flip));
    return y;
}
// For fp32 results the sums would lose two bits to the 128 (fp32 drafts: 2e-5 against 5e-7): there the
// byte is the mantissa of 1024 + (code + 128), and 1152 is subtracted at once.
enum Kind { kE4m3, kInt8, kInt8Exact };
template <Kind K> __device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (K == kE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else if constexpr (K == kInt8) {
        lo = and_xor(w);
        hi = and_xor(w >> 8);
    } else {
        w ^= 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));        // 1152
        uint32_t a = __byte_perm(w, 0x64646464u, 0x4240), b = __byte_perm(w, 0x64646464u, 0x4341);
        __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off), hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
        lo = *reinterpret_cast<uint32_t*>(&ha);
        hi = *reinterpret_cast<uint32_t*>(&hb);
    }
}
// Bytes of two tokens' words so that codes_f16 pairs the tokens: elements 0, 1 (k = 0) or 2, 3 (k = 1)
// of both.
template <bool E4M3> __device__ __forceinline__ uint32_t token_pair(uint32_t t0, uint32_t t1, int k) {
    return __byte_perm(t0, t1, E4M3 ? (k ? 0x7362 : 0x5140) : (k ? 0x7632 : 0x5410));
}
constexpr float kI8Unit = 5.9604644775390625e-8f;       // 2^-24
// Place of a query's element among its four neighbours, as codes_f16 orders a key's.
template <bool E4M3> __device__ __forceinline__ constexpr int q_order(int e) {
    return E4M3 ? e : (e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1);
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

// Place of an even element of O's row in shared memory: the rows 2c of a warp's store lie in
// different banks.
__device__ __forceinline__ int o_place(int row, int el) { return el ^ (row & 6); }

template <typename T, int DH, int NT, bool E4M3> struct Att {
    static constexpr bool F32 = sizeof(T) == 4;
    static constexpr Kind KIND = E4M3 ? kE4m3 : F32 ? kInt8Exact : kInt8;
    static constexpr bool OFF = KIND == kInt8;       // codes enter the products with 128 added, times 2^-24
    static constexpr int R = 8 * NT;                 // query rows of a tile
    static constexpr int QP = F32 ? 2 : 1;           // f16 parts of a query
    static constexpr int PP = F32 ? 2 : 1;           // f16 parts of a probability
    static constexpr int TP = F32 ? 3 : 1;           // bf16 parts of an activation
    static constexpr int TPP = F32 ? 3 : 2;          // bf16 parts of a probability
    static constexpr int NSTG = 1;                   // blocks in a warp's ring
    static constexpr int KB = 64 * DH;               // bytes of a block's keys
    static constexpr int QS = DH + 4;                // row stride of the queries in shared memory
    static constexpr int NM = DH / 16;               // 16-element tiles of the output
    // One CTA an SM, of as many warps as its registers allow (128, 168 or 255 a thread): few CTAs make few
    // parts to merge.  The forms of one row tile spill 86 to 202 bytes a thread at that (bf16: 86 and 182 at DH = 64,
    // 182 and 190 at 128), those of two 150 to 278 at DH = 128 (at 64 up to 34, fp32 only).  With 12 (DH = 64) and 8
    // warps the bf16 forms of one tile spill nothing, and four bf16 cases measured faster (1B decode step 80.4 ->
    // 77.9 us, the long sequence 93.1 -> 84.9); fp32 has not been measured so.
    static constexpr int kWarps = NT == 1 ? (DH == 64 ? 16 : 12) : 8, kThreads = 32 * kWarps;
    static constexpr int kBufs = kWarps / 4;         // buffers the warps' O are added up in
    static constexpr int kMinItems = kWarps + kUnitCost;    // fewest items (blocks and unit costs) of a run
    struct Smem {
        alignas(128) unsigned char ring[kWarps][NSTG * 2 * KB];
        alignas(16) float bias[kWarps][NSTG][kKvqBlock];
        alignas(16) uint16_t q16[QP][R][QS];         // f16, scaled by a power of two a row
        alignas(16) uint16_t qb[TP][R][QS];          // bf16 parts (for the unfinished block)
        float qf[R];                                 // logit scale in ln 4 times the row's power of two
        float s0[R];                                 // -128 * sum of the row's f16 values (int8, see codes_f16)
        int lim[R];                                  // last slot the row sees, -1: none
        float m[kWarps][R], l[kWarps][R];
        alignas(16) float o[kBufs][R][DH];           // sums of the warps' O, see o_place
        float2 share[kThreads];
        int scan[2][kWarps];
        int last;
    };
    static_assert(sizeof(Smem) <= 227 * 1024, "one CTA an SM");
};

// What a warp carries through a unit: O^T (elements 64 * pass + 8r + 2mt + {0, 1} of columns
// 8nt + 2c + {0, 1}, r = lane/4, c = lane%4), the columns' running maximum and this lane's sums.
template <int DH, int NT> struct State {
    float o[DH / 16][NT][4];
    float m[NT][2], l[NT][2];
};

// Online softmax of 16 * MT tokens: logits x[mt][nt][e] (rows: tokens tok_of(r) and + 8, columns as
// in State) -> 2^14 p in place, corr = factor of what was accumulated, any: whether the column sees one.
// The sums are left to the caller.
template <int DH, int NT, int MT>
__device__ __forceinline__ void block_softmax(State<DH, NT>& st, float (&x)[MT][NT][4], float (&corr)[NT][2],
                                              bool (&any)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = x[0][nt][e];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(x[mt][nt][e], x[mt][nt][e + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // (a NaN logit is no maximum; it makes the sum NaN, and with it every output of the row)
            any[nt][e] = mx > -INFINITY;
            const float mn = fmaxf(st.m[nt][e], ceilf(mx));
            const float ms = mn == -INFINITY ? 0.f : mn;
            corr[nt][e] = ex2(2.f * (st.m[nt][e] - ms));
            st.m[nt][e] = mn;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float& v = x[mt][nt][e + 2 * k];
                    v = ex2(fmaf(v - ms, 2.f, kPShift));
                }
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

// A warp's 16 tokens of the unfinished block (slots slot0 .. of n), its rows in the activation type
// in the warp's ring (kt, vt: [16][DH]; rows at and behind n are not there): bf16 products, the operands
// as sums of bf16 parts (bf16 activations are one part, fp32 ones three; pairs of parts below 2^-24 of
// the product are left out).
// A row past its own slot has probability 0 there, and 0 times a value that is not finite is NaN: where some row ends
// within these tokens (drafts; lim_min: the least of the rows' last slots), such values are left out of the
// products and added to the rows that see them (as bf16 parts: values above bf16's largest, too).
template <typename T, int DH, int NT, bool E4M3>
__device__ __forceinline__ void tail_part(const KvqAttendParams& p, typename Att<T, DH, NT, E4M3>::Smem& sm,
                                          State<DH, NT>& st, const T* kt, const T* vt, const float* bias, int slot0,
                                          int n, int lim_min) {
    using A = Att<T, DH, NT, E4M3>;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    bool hidden[2];                                      // tokens no row sees: their rows may be anything
    float bs[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int tok = tok_of(r) + 8 * k;
        bs[k] = slot0 + tok >= n ? -INFINITY : bias ? bias[tok] : 0.f;
        hidden[k] = bs[k] == -INFINITY;
    }
    float x[1][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[0][nt][e] = 0.f;
#pragma unroll 4
    for (int s = 0; s < DH / 16; ++s) {
        const int d0 = (s >> 2) * 64 + 16 * c + 4 * (s & 3);
        uint32_t a[A::TP][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {                    // rows r and r + 8: elements d0 .. d0+3
            const T* src = kt + (tok_of(r) + 8 * k) * DH + d0;
            if constexpr (A::F32) {
                const float4 f = *reinterpret_cast<const float4*>(src);
                uint32_t lo[3], hi[3];
                split_bf16<3>(f.x, f.y, lo);
                split_bf16<3>(f.z, f.w, hi);
#pragma unroll
                for (int i = 0; i < A::TP; ++i) { a[i][k] = lo[i]; a[i][2 + k] = hi[i]; }
            } else {
                const uint2 u = *reinterpret_cast<const uint2*>(src);
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
                for (int i = 0; i + j < A::TP; ++i) mma_bf16(x[0][nt], a[i], q);
            }
    }
    // a token's row of the values' operand sits at other lanes than its logit: the bit of token t comes
    // from lane 4 row, tok_of(row) = t mod 8
    const unsigned hid[2] = {__ballot_sync(0xffffffffu, hidden[0]), __ballot_sync(0xffffffffu, hidden[1])};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float& v = x[0][nt][2 * k + e];
                v = hidden[k] || slot0 + tok_of(r) + 8 * k > sm.lim[8 * nt + 2 * c + e]
                        ? -INFINITY
                        : fmaf(v, p.scale * kLog4e, bs[k] * kLog4e);
            }
    float corr[NT][2];
    bool any[NT][2];
    block_softmax<DH, NT, 1>(st, x, corr, any);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) st.l[nt][e] = fmaf(st.l[nt][e], corr[nt][e], x[0][nt][e] + x[0][nt][e + 2]);
    const bool drafts = min(n, slot0 + 16) - 1 > lim_min;
    auto held = [](float v) { return fabsf(v) <= 3.3895314e38f; };      // as sums of bf16 parts
    uint2 pb[A::TPP][NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        uint32_t lo[A::TPP], hi[A::TPP];
        split_bf16<A::TPP>(x[0][nt][0], x[0][nt][1], lo);
        split_bf16<A::TPP>(x[0][nt][2], x[0][nt][3], hi);
#pragma unroll
        for (int i = 0; i < A::TPP; ++i) pb[i][nt] = make_uint2(transpose8x8(lo[i]), transpose8x8(hi[i]));
    }
#pragma unroll
    for (int pass = 0; pass < DH / 64; ++pass) {
        float v[4][8];                                   // tokens 4i + c, elements 64 pass + 8r ..
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * i + c, row = 2 * (t & 3) + ((t >> 2) & 1);
            const T* src = vt + t * DH + 64 * pass + 8 * r;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
            if (((hid[t >> 3] >> (4 * row)) & 1u) == 0) {
                Vec16<T>::ld(src, v[i]);
                if constexpr (A::F32) Vec16<T>::ld(src + 4, v[i] + 4);
            }
        }
        bool left_out = false;
        if (drafts) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!held(v[i][e])) {
                        v[i][e] = 0.f;
                        left_out = true;
                    }
            left_out = __any_sync(0xffffffffu, left_out);
        }
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            uint32_t a[4][A::TP];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                split_bf16<A::TP>(v[0][2 * mt + k], v[1][2 * mt + k], a[k]);
                split_bf16<A::TP>(v[2][2 * mt + k], v[3][2 * mt + k], a[2 + k]);
            }
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
                for (int i = 0; i < A::TP; ++i) {
                    const uint32_t ai[4] = {a[0][i], a[1][i], a[2][i], a[3][i]};
#pragma unroll
                    for (int j = 0; j < A::TPP; ++j)
                        if (i + j < 3) mma_bf16(acc[nt], ai, pb[j][nt]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    st.o[4 * pass + mt][nt][e] =
                        fmaf(st.o[4 * pass + mt][nt][e], corr[nt][e & 1], any[nt][e & 1] ? acc[nt][e] : 0.f);
            }
        }
        if (left_out) {
#pragma unroll 1
            for (int t = 0; t < 16; ++t) {
                if (((t < 8 ? hid[0] : hid[1]) >> (4 * (2 * (t & 3) + ((t >> 2) & 1)))) & 1u) continue;
                float w[8];
                Vec16<T>::ld(vt + t * DH + 64 * pass + 8 * r, w);
                if constexpr (A::F32) Vec16<T>::ld(vt + t * DH + 64 * pass + 8 * r + 4, w + 4);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bool sees = slot0 + t <= sm.lim[8 * nt + 2 * c + (e & 1)];
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
                            if (sees && !held(w[2 * mt + (e >> 1)])) st.o[4 * pass + mt][nt][e] += 2.f * w[2 * mt + (e >> 1)];
                    }
            }
        }
    }
}

// The warp's walk through one unit: the finished blocks first, first + kWarps, ... < last, then its 16
// tokens of the unfinished block if the CTA's run ends with it.  begin() starts the first copies; run()
// needs the queries in shared memory.
template <typename T, int DH, int NT, bool E4M3> struct Walk {
    using A = Att<T, DH, NT, E4M3>;
    static constexpr long long kNone = -1, kTail = -2, kNoPage = -3;
    static constexpr int kWarps = A::kWarps;
    static_assert(A::NSTG == 1, "begin_k, begin_v");
    static_assert(16 * DH * sizeof(T) <= A::KB, "a warp's rows of the unfinished block fit a block's place");
    const KvqAttendParams& p;
    typename A::Smem& sm;
    const int warp, lane, r, c;
    int b, first, steps, full, slot0, n;             // steps: blocks and the 16 tokens; full: blocks
    long long unit, hrow, rows[A::NSTG + 1];         // code rows of the steps in flight and of the one after
    const float* bias0;
    float ks, vs;
    // This lane's places of a block (see k_place, v_place): where its first pieces are copied to, and where
    // it reads from first; further ones lie at constant distances.
    uint32_t ring_s;
    int k_to, v_to, k_from, v_from;

    __device__ __forceinline__ Walk(const KvqAttendParams& p_, typename A::Smem& sm_)
        : p(p_), sm(sm_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31), r(lane >> 2), c(lane & 3) {
        constexpr int PER = DH / 16;                     // 16-byte pieces of a token
        ring_s = tc::smem_u32(sm.ring[warp]);
        k_to = k_place<DH>(lane / PER, lane % PER);
        v_to = v_place<DH>(lane / PER, lane % PER);
        k_from = k_place<DH>(tok_of(r), c);
        v_from = v_place<DH>(c, r >> 1) + 8 * (r & 1);
    }

    __device__ __forceinline__ long long row_of(int i) const {
        if (i >= full) return i < steps ? kTail : kNone;
        const long long x = kvq_row(p.c, b, first + i * kWarps);
        return x < 0 ? kNoPage : x + hrow;
    }
    // step i's keys (and bias) / values into place stg
    __device__ __forceinline__ void load_k(long long row, int i, int stg) {
        const uint32_t dst = ring_s + stg * 2 * A::KB;
        if (row >= 0) {
            const uint8_t* src = p.c.k + row * A::KB + lane * 16;
#pragma unroll
            for (int j = 0; j < A::KB / 512; ++j)        // (at 128 bytes a token, tokens 4 .. 7 of 8 are swapped by 64)
                cp_async16(dst + (DH == 128 && (j & 1) ? k_to ^ 64 : k_to) + j * 512, src + j * 512);
            if (bias0 && lane < 16)
                cp_async16(tc::smem_u32(&sm.bias[warp][stg][4 * lane]), bias0 + (first + i * kWarps) * kKvqBlock + 4 * lane);
        } else if (row == kTail) {
            load_tail(dst, p.c.kr);
            if (bias0 && lane < 4) cp_async16(tc::smem_u32(&sm.bias[warp][stg][4 * lane]), bias0 + slot0 + 4 * lane);
        }
        tc::cp_async_commit();
    }
    __device__ __forceinline__ void load_v(long long row, int stg) {
        const uint32_t dst = ring_s + (stg * 2 + 1) * A::KB;
        if (row >= 0) {
            const uint8_t* src = p.c.v + row * A::KB + lane * 16;
#pragma unroll
            for (int j = 0; j < A::KB / 512; ++j) cp_async16(dst + v_to + j * 512, src + j * 512);
        } else if (row == kTail) {
            load_tail(dst, p.c.vr);
        }
        tc::cp_async_commit();
    }
    __device__ __forceinline__ void load_tail(uint32_t dst, const void* ring) {
        constexpr int PER = DH * (int)sizeof(T) / 16;    // 16-byte pieces of a row
        const T* src = static_cast<const T*>(ring) + (unit * kKvqRing + (slot0 & (kKvqRing - 1))) * DH;
        const int left = (n - slot0) * PER;
#pragma unroll
        for (int j = 0; j < 16 * PER / 32; ++j) {
            const int e = j * 32 + lane;
            if (e < left) cp_async16(dst + e * 16, reinterpret_cast<const uint4*>(src) + e);
        }
    }
    // blocks first_ .. last_ - 1 and, with_tail, the unfinished block of n_ slots
    __device__ __forceinline__ void begin(int b_, int h, int first_, int last_, bool with_tail, int n_) {
        b = b_;
        first = first_;
        n = n_;
        full = max(0, (last_ - first + kWarps - 1) / kWarps);
        slot0 = n / kKvqBlock * kKvqBlock + 16 * (kWarps - 1 - warp);   // (the last warps have fewer blocks)
        steps = full + (with_tail && warp >= kWarps - 4 && slot0 < n ? 1 : 0);
        unit = (long long)b * p.c.Hkv + h;
        hrow = (long long)h * p.c.bpp;
        bias0 = p.bias ? p.bias + unit * p.c.cap : nullptr;
#pragma unroll
        for (int i = 0; i <= A::NSTG; ++i) rows[i] = row_of(i);
    }
    __device__ __forceinline__ void begin_k() { load_k(rows[0], 0, 0); }
    __device__ __forceinline__ void begin_v() {
        load_v(rows[0], 0);
        ks = rows[0] >= 0 ? __ldg(p.c.ks + rows[0]) : 0.f;
        vs = rows[0] >= 0 ? __ldg(p.c.vs + rows[0]) : 0.f;
    }
    __device__ __forceinline__ void run(State<DH, NT>& st) {
        float qf[NT][2], s0[NT][4];                      // s0: what the sums of the products start from
        int lim[NT][2], lim_min = INT32_MAX;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qf[nt][e] = sm.qf[8 * nt + 2 * c + e];
                s0[nt][e] = s0[nt][e + 2] = A::OFF ? sm.s0[8 * nt + 2 * c + e] : 0.f;
                lim[nt][e] = sm.lim[8 * nt + 2 * c + e];
                lim_min = min(lim_min, lim[nt][e]);
            }
        lim_min = __reduce_min_sync(0xffffffffu, lim_min);
        int stg = 0;
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
            const long long row = rows[0], next = rows[A::NSTG];
#pragma unroll
            for (int k = 0; k < A::NSTG; ++k) rows[k] = rows[k + 1];
            rows[A::NSTG] = row_of(i + A::NSTG + 1);
            const float ksn = rows[0] >= 0 ? __ldg(p.c.ks + rows[0]) : 0.f;
            const float vsn = rows[0] >= 0 ? __ldg(p.c.vs + rows[0]) : 0.f;
            if (row >= 0) {
                block(st, i, next, stg, qf, s0, lim, lim_min);
            } else {
                if (row == kTail) {                      // the last step
                    cp_async_wait<0>();
                    __syncwarp();
                    const unsigned char* at = sm.ring[warp] + stg * 2 * A::KB;
                    tail_part<T, DH, NT, E4M3>(p, sm, st, reinterpret_cast<const T*>(at),
                                               reinterpret_cast<const T*>(at + A::KB),
                                               bias0 ? sm.bias[warp][stg] : nullptr, slot0, n, lim_min);
                }
                load_k(next, i + A::NSTG, stg);          // (no page: left out)
                load_v(next, stg);
            }
            ks = ksn;
            vs = vsn;
            stg = stg + 1 == A::NSTG ? 0 : stg + 1;
        }
        cp_async_wait<0>();
        __syncwarp();
    }
    __device__ __forceinline__ void block(State<DH, NT>& st, int i, long long next, int stg, const float (&qf)[NT][2],
                                          const float (&s0)[NT][4], const int (&lim)[NT][2], int lim_min) {
        const int blk = first + i * kWarps;
        const unsigned char* kb = sm.ring[warp] + stg * 2 * A::KB;
        const unsigned char* vb = kb + A::KB;
        // S^T = K Q^T
        cp_async_wait<2 * A::NSTG - 1>();
        __syncwarp();
        float x[4][NT][4];
#pragma unroll
        for (int hf = 0; hf < DH / 64; ++hf) {
            uint2 q[A::QP][NT][4];
#pragma unroll
            for (int j = 0; j < A::QP; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        q[j][nt][s] = *reinterpret_cast<const uint2*>(&sm.q16[j][8 * nt + r][64 * hf + 16 * c + 4 * s]);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const unsigned char* at = kb + (k_from ^ (hf << 6)) + 16 * mt * DH;
                const uint4 u0 = *reinterpret_cast<const uint4*>(at);
                const uint4 u1 = *reinterpret_cast<const uint4*>(at + 8 * DH);
                const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t a[4];
                    codes_f16<A::KIND>(w0[s], a[0], a[2]);
                    codes_f16<A::KIND>(w1[s], a[1], a[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < A::QP; ++j) {
                            if (hf + s + j == 0) mma_f16(x[mt][nt], a, q[j][nt][s], s0[nt]);
                            else mma_f16(x[mt][nt], a, q[j][nt][s]);
                        }
                }
            }
        }
        float bs[4][2];
        if (bias0) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int k = 0; k < 2; ++k) bs[mt][k] = sm.bias[warp][stg][16 * mt + tok_of(r) + 8 * k];
        }
        __syncwarp();
        load_k(next, i + A::NSTG, stg);
        // Probabilities.  Where every slot is seen and nothing is added to the logits, they are one fused
        // multiply-add and an exp2 away from the products: the shift 2 m - 14 is checked to be exact.
        float corr[NT][2], f[NT][2];
        bool any[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) f[nt][e] = A::OFF ? qf[nt][e] * ks * (1.f / kI8Unit) : qf[nt][e] * ks;
        bool plain = bias0 == nullptr && blk * kKvqBlock + kKvqBlock - 1 <= lim_min && p.scale > 0.f;
        if (plain) {
            float mn[NT][2], base[NT][2];
            bool exact = true;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = x[0][nt][e];
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt) mx = fmaxf(mx, fmaxf(x[mt][nt][e], x[mt][nt][e + 2]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    mn[nt][e] = fmaxf(st.m[nt][e], ceilf(mx * f[nt][e]));
                    base[nt][e] = 2.f * mn[nt][e] - kPShift;
                    exact = exact && 2.f * mn[nt][e] - base[nt][e] == kPShift;
                }
            plain = __all_sync(0xffffffffu, exact);
            if (plain) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        any[nt][e] = true;
                        corr[nt][e] = ex2(2.f * (st.m[nt][e] - mn[nt][e]));
                        st.m[nt][e] = mn[nt][e];
                        const float f2 = 2.f * f[nt][e];
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float& v = x[mt][nt][2 * k + e];
                                v = ex2(fmaf(v, f2, -base[nt][e]));
                            }
                    }
            }
        }
        if (!plain) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float& v = x[mt][nt][2 * k + e];
                            v *= f[nt][e];
                            if (bias0) v = bs[mt][k] == -INFINITY ? -INFINITY : fmaf(bs[mt][k], kLog4e, v);
                            if (blk * kKvqBlock + 16 * mt + tok_of(r) + 8 * k > lim[nt][e]) v = -INFINITY;
                        }
            block_softmax<DH, NT, 4>(st, x, corr, any);
        }
        // P^T as the products' operand; int8 also needs the sums of the rounded values, by a product
        // with ones
        uint2 pb[A::PP][4][NT];
        float sum[NT][4];
        const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
        const float none[4] = {0.f, 0.f, 0.f, 0.f};
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
                if constexpr (A::OFF) {                  // (bf16: one part)
                    if (mt == 0) mma_f16(sum[nt], ones, pb[0][mt][nt], none);
                    else mma_f16(sum[nt], ones, pb[0][mt][nt]);
                }
            }
        bool rescale = false;
        float o0[NT][4], fv[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = x[0][nt][e] + x[0][nt][e + 2];
#pragma unroll
                for (int mt = 1; mt < 4; ++mt) l += x[mt][nt][e] + x[mt][nt][e + 2];
                st.l[nt][e] = fmaf(st.l[nt][e], corr[nt][e], l);
                rescale = rescale || corr[nt][e] != 1.f;
                o0[nt][e] = o0[nt][e + 2] = A::OFF ? -128.f * kI8Unit * sum[nt][e] : 0.f;
                // (a block no slot of which is seen may have a NaN scale)
                fv[nt][e] = any[nt][e] ? (A::OFF ? vs * (1.f / kI8Unit) : vs) : 0.f;
            }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
            for (int k = 0; k < A::NM; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) st.o[k][nt][e] *= corr[nt][e & 1];
        }
        // O^T += vs * V^T P^T
        cp_async_wait<2 * A::NSTG - 1>();
        __syncwarp();
#pragma unroll
        for (int pass = 0; pass < DH / 64; ++pass) {
            float acc[4][NT][4];
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                uint2 w[4];                              // tokens 4k + c, elements 64 pass + 8r ..
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = *reinterpret_cast<const uint2*>(vb + (v_from ^ (pass << 6)) + (16 * kt + 4 * k) * DH);
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {
                    const uint32_t t0 = hw ? w[0].y : w[0].x, t1 = hw ? w[1].y : w[1].x;
                    const uint32_t t2 = hw ? w[2].y : w[2].x, t3 = hw ? w[3].y : w[3].x;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t a[4];
                        codes_f16<A::KIND>(token_pair<E4M3>(t0, t1, k), a[0], a[1]);
                        codes_f16<A::KIND>(token_pair<E4M3>(t2, t3, k), a[2], a[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < A::PP; ++j) {
                                if (kt + j == 0) mma_f16(acc[2 * hw + k][nt], a, pb[j][kt][nt], o0[nt]);
                                else mma_f16(acc[2 * hw + k][nt], a, pb[j][kt][nt]);
                            }
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st.o[4 * pass + mt][nt][e] = fmaf(acc[mt][nt][e], fv[nt][e & 1], st.o[4 * pass + mt][nt][e]);
        }
        __syncwarp();
        load_v(next, stg);
    }
};

template <typename T, int DH, int NT, bool E4M3>
__global__ void __launch_bounds__(Att<T, DH, NT, E4M3>::kThreads, 1) k_kvq_attend(KvqAttendParams p) {
    using A = Att<T, DH, NT, E4M3>;
    constexpr int R = A::R, kWarps = A::kWarps, kThreads = A::kThreads;
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
    auto items_of = [&](int b, int* units) {
        *units = 0;
        if (b >= p.c.B) return 0;
        int nq, n;
        counts(b, &nq, &n);
        *units = Hkv * tiles_of(nq);
        return *units * (blocks_of(n) + kUnitCost);
    };
    // All items and units (below 2^31: checked on the host).  Up to 32 sequences: every warp for itself,
    // a sequence a lane.
    const bool few = p.c.B <= 32;
    int total = 0, units = 0, my_nq = 0, my_n = 0;
    for (int b = few ? lane : tid; b < p.c.B; b += few ? 32 : kThreads) {
        counts(b, &my_nq, &my_n);
        const int u = Hkv * tiles_of(my_nq);
        total += u * (blocks_of(my_n) + kUnitCost);
        units += u;
    }
    const int my_units = units, my_blocks = blocks_of(my_n);     // (few: of this lane's sequence)
    total = __reduce_add_sync(0xffffffffu, total);
    units = __reduce_add_sync(0xffffffffu, units);
    if (!few) {
        if (lane == 0) {
            sm.scan[0][warp] = total;
            sm.scan[1][warp] = units;
        }
        __syncthreads();
        total = units = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            total += sm.scan[0][w];
            units += sm.scan[1][w];
        }
    }
    const int cta = blockIdx.x, grid = gridDim.x;
    // Few units: whole CTAs for each, `run` blocks each at most -- a CTA with parts of two units would
    // pay for starting and merging twice (3B decode with bias: 29 us; 22 us so).
    const bool aligned = few && units * 2 <= grid;
    // Otherwise equal runs of items, one a CTA.
    const int ctas = max(min(units, grid), min(grid, (total + A::kMinItems - 1) / A::kMinItems));
    if (!aligned && cta >= ctas) return;
    // floor(a * b / c) for products below 2^53 (the quotient's fraction is at least 1 / c off a whole number)
    auto run_start = [&](int k) { return (int)((double)k * (double)total / (double)ctas); };
    auto run_of = [&](int item) { return (int)((((double)item + 1.0) * ctas - 1.0) / total); };

    // A segment: a run's part in one unit (sequence b, KV head h, row tile rt): blocks k0 .. k1 - 1 of
    // nb (none where the run ends within the unit's cost), `len` items; r_lo .. r_hi: the runs with
    // blocks of the unit.
    struct Segment {
        int b, h, rt, nq, n, nb, k0, k1, r_lo, r_hi, off, len;
    };
    int at = aligned ? 0 : run_start(cta);
    const int hi = aligned ? 0 : run_start(cta + 1);
    // the segment that starts with item `at`, item `off` of sequence b
    auto segment = [&](int b, int off) {
        Segment s;
        int pos;
        for (;; ++b, off = 0) {
            counts(b, &s.nq, &s.n);
            s.nb = blocks_of(s.n);
            const int tiles = tiles_of(s.nq), u = off / (s.nb + kUnitCost);
            if (u < Hkv * tiles) {                       // (else: the next sequence with anything to do)
                s.h = u / tiles;
                s.rt = u - s.h * tiles;
                pos = off - u * (s.nb + kUnitCost);
                break;
            }
        }
        s.b = b;
        s.off = off;
        s.len = min(s.nb + kUnitCost - pos, hi - at);
        s.k0 = max(pos - kUnitCost, 0);
        s.k1 = pos + s.len - kUnitCost;
        s.r_lo = run_of(at - pos + kUnitCost);
        s.r_hi = run_of(at - pos + kUnitCost + s.nb - 1);
        return s;
    };
    // the sequence that holds item `at`, 32 sequences at a time
    auto find = [&]() {
        for (int seq = 0, first = 0;; seq += 32) {
            int u, inc = items_of(seq + lane, &u);
            const int mine = inc;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, at < first + inc);
            if (past) {
                const int l = __ffs(past) - 1;
                return segment(seq + l, at - first - __shfl_sync(0xffffffffu, inc - mine, l));
            }
            first += __shfl_sync(0xffffffffu, inc, 31);
        }
    };
    // Whole CTAs for each unit: the least of 32 ascending numbers of blocks a CTA (by a sixteenth
    // of the even share) with which the units need no more CTAs than there are; this CTA's part.
    auto own_part = [&](bool* have) {
        const int blocks = __reduce_add_sync(0xffffffffu, my_units * my_blocks);
        const int even = max((blocks + grid - 1) / grid, kWarps), mine = even + even * lane / 16 + lane;
        int need = 0;
        for (int b = 0; b < p.c.B; ++b) {
            const int nb = __shfl_sync(0xffffffffu, my_blocks, b);
            need += __shfl_sync(0xffffffffu, my_units, b) * ((nb + mine - 1) / mine);
        }
        const unsigned fits = __ballot_sync(0xffffffffu, need <= grid);
        const int run = __shfl_sync(0xffffffffu, mine, __ffs(fits) - 1);
        const int parts = (my_blocks + run - 1) / run;   // CTAs a unit, of this lane's sequence
        int inc = my_units * parts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, cta < inc);
        Segment s = {};
        *have = past != 0;
        if (!past) return s;
        const int l = __ffs(past) - 1, k = __shfl_sync(0xffffffffu, parts, l);
        const int off = cta - __shfl_sync(0xffffffffu, inc - my_units * parts, l), u = off / k, part = off - u * k;
        s.b = l;
        s.nq = __shfl_sync(0xffffffffu, my_nq, l);
        s.n = __shfl_sync(0xffffffffu, my_n, l);
        s.nb = blocks_of(s.n);
        const int tiles = tiles_of(s.nq);
        s.h = tiles == 1 ? u : u / tiles;
        s.rt = u - s.h * tiles;
        s.k0 = (int)((unsigned)part * (unsigned)s.nb / (unsigned)k);         // (at most 148 * 2^24)
        s.k1 = (int)((unsigned)(part + 1) * (unsigned)s.nb / (unsigned)k);
        s.r_lo = cta - part;
        s.r_hi = s.r_lo + k - 1;
        s.off = s.len = 0;
        return s;
    };
    Walk<T, DH, NT, E4M3> walk(p, sm);
    // Queries of a tile: 8 threads a row, fetched before the segment's copies are started.
    constexpr int E = DH / 8, QV = E / Vec16<T>::N;
    uint4 qraw[QV];
    auto start = [&](const Segment& s) {
        const int gr = s.rt * R + (tid >> 3), i = gr / G, gg = gr - i * G;
#pragma unroll
        for (int v = 0; v < QV; ++v) qraw[v] = make_uint4(0, 0, 0, 0);
        if (tid < 8 * R && i < s.nq) {
            const T* src = static_cast<const T*>(p.q) + (((size_t)s.b * p.Tq + i) * p.H + s.h * G + gg) * DH + (tid & 7) * E;
#pragma unroll
            for (int v = 0; v < QV; ++v)
                asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(qraw[v].x), "=r"(qraw[v].y), "=r"(qraw[v].z), "=r"(qraw[v].w)
                             : "l"(reinterpret_cast<const uint4*>(src) + v));
        }
        const int nfull = s.n / kKvqBlock;
        walk.begin(s.b, s.h, s.k0 + warp, min(s.k1, nfull), s.k1 == s.nb, s.n);
    };
    bool have = true;
    Segment cur = aligned ? own_part(&have) : find();
    if (!have) return;
    start(cur);
    bool ahead = false;                                  // the segment's keys are on their way
    for (;;) {
        const int h = cur.h, rt = cur.rt, nq = cur.nq, n = cur.n, b = cur.b, r_lo = cur.r_lo, r_hi = cur.r_hi;
        if (tid < 8 * R) {
            const int row = tid >> 3, part = tid & 7, gr = rt * R + row, i = gr / G;
            float x[E];
#pragma unroll
            for (int v = 0; v < QV; ++v) Vec16<T>::unpack(qraw[v], x + v * Vec16<T>::N);
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
                uint32_t t[A::TP];
                split_bf16<A::TP>(x[e], x[e + 1], t);
#pragma unroll
                for (int j = 0; j < A::TP; ++j) *reinterpret_cast<uint32_t*>(&sm.qb[j][row][part * E + e]) = t[j];
            }
            float qsum = 0.f;
#pragma unroll
            for (int e = 0; e < E; e += 4)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {         // places k, k + 1 of four
                    const float y0 = x[e + q_order<E4M3>(k)] * up, y1 = x[e + q_order<E4M3>(k + 1)] * up;
                    const uint32_t hq = pack_f16(y0, y1);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hq));
                    *reinterpret_cast<uint32_t*>(&sm.q16[0][row][part * E + e + k]) = hq;
                    qsum += f.x + f.y;
                    if constexpr (A::QP == 2) {
                        const uint32_t lq = pack_f16(y0 - f.x, y1 - f.y);
                        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&lq));
                        *reinterpret_cast<uint32_t*>(&sm.q16[1][row][part * E + e + k]) = lq;
                        qsum += g.x + g.y;
                    }
                }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) qsum += __shfl_xor_sync(mask, qsum, o);
            if (part == 0) {
                sm.qf[row] = p.scale * kLog4e * __uint_as_float((uint32_t)(127 - ex) << 23);
                sm.s0[row] = -128.f * kI8Unit * qsum;
                sm.lim[row] = i < nq ? min(n - nq + i, n - 1) : INT32_MAX;  // (a row past the last query: anything)
            }
        }
        __syncthreads();
        // (An SM takes in 25 bytes a clock and a copy waits for room to be issued: with all copies before
        // the barrier the first warp's keys lay there for 5000 clocks until the last warp's were issued.)
        if (!ahead) walk.begin_k();
        walk.begin_v();
        State<DH, NT> st;
        init_state<DH, NT>(st);
        walk.run(st);
        // the next segment's copies run while this one is merged
        at += cur.len;
        bool more = at < hi;
        if (more) {
            cur = segment(b, cur.off + cur.len);
            more = cur.k1 > cur.k0;
            if (more) {
                start(cur);
                walk.begin_k();
            }
            ahead = more;
        }

        // merge the warps: statistics, then O, one warp after the other
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
        {
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float M = sm.m[0][8 * nt + 2 * c + e];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm.m[w][8 * nt + 2 * c + e]);
                    f[nt][e] = ex2(2.f * (st.m[nt][e] - (M == -INFINITY ? 0.f : M)));
                }
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {                // buffer j adds up warps j, j + kBufs, ..
                if (warp / A::kBufs == w) {
#pragma unroll
                    for (int i = 0; i < A::NM; ++i)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float2* to = reinterpret_cast<float2*>(
                                    &sm.o[warp % A::kBufs][8 * nt + 2 * c + e][o_place(2 * c, 64 * (i >> 2) + 8 * r + 2 * (i & 3))]);
                                float2 v = make_float2(st.o[i][nt][e] * f[nt][e], st.o[i][nt][e + 2] * f[nt][e]);
                                if (w > 0) {
                                    const float2 u = *to;
                                    v.x += u.x;
                                    v.y += u.y;
                                }
                                *to = v;
                            }
                }
                __syncthreads();
            }
        }
        const int rows = min(R, nq * G - rt * R);
        // four elements of a row: where they lie, their gates (fetched ahead of the merge), their output
        auto place = [&](int row, int d4, int* head, int* i) {
            const int gr = rt * R + row;
            *i = gr / G;
            *head = h * G + gr - *i * G;
            return (((size_t)b * p.Tq + *i) * p.H + *head) * DH + d4;
        };
        auto gates = [&](int row, int d4) {
            float4 f = make_float4(0, 0, 0, 0);
            if (p.g) {
                int head, i;
                const T* src = static_cast<const T*>(p.g) + place(row, d4, &head, &i);
                if constexpr (A::F32) {
                    f = *reinterpret_cast<const float4*>(src);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(src);
                    f = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
                }
            }
            return f;
        };
        auto put_out = [&](int row, int d4, float4 o, float M, float L, float4 gt) {
            int head, i;
            const size_t at = place(row, d4, &head, &i);
            const float inv = L != 0.f ? 1.f / L : 0.f;
            float y[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
            if (p.g) {
                y[0] *= sigmoid_f(gt.x);
                y[1] *= sigmoid_f(gt.y);
                y[2] *= sigmoid_f(gt.z);
                y[3] *= sigmoid_f(gt.w);
            }
            T* out = static_cast<T*>(p.o) + at;
            if constexpr (A::F32) {
                *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
            } else {
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
            }
            if (p.lse && d4 == 0)
                p.lse[((size_t)b * p.H + head) * p.Tq + i] = L != 0.f ? M * kLn4 + (logf(L) - kPShift * 0.6931471805599453f) : -INFINITY;
        };
        const bool whole = r_lo == r_hi;
        const int slot = 2 * cta + (cta == r_lo ? 1 : 0);
        float* to = p.part + (size_t)slot * R * (DH + 2);
        for (int e = tid; e < rows * (DH / 4); e += kThreads) {
            const int row = e / (DH / 4), d4 = (e % (DH / 4)) * 4;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][row]);
            const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) L = fmaf(sm.l[w][row], ex2(2.f * (sm.m[w][row] - ms)), L);
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < A::kBufs; ++j) {
                const float2 o0 = *reinterpret_cast<const float2*>(&sm.o[j][row][o_place(row, d4)]);
                const float2 o1 = *reinterpret_cast<const float2*>(&sm.o[j][row][o_place(row, d4 + 2)]);
                o.x += o0.x;
                o.y += o0.y;
                o.z += o1.x;
                o.w += o1.y;
            }
            if (whole) {
                put_out(row, d4, o, M, L, gates(row, d4));
            } else {
                __stcg(reinterpret_cast<float4*>(to + 2 * R + row * DH + d4), o);
                if (d4 == 0) {
                    __stcg(to + row, M);
                    __stcg(to + R + row, L);
                }
            }
        }
        __syncthreads();                                 // (sm.m, sm.l and sm.o are free again, the part is written)
        if (!whole) {
            if (tid == 0) {
                unsigned* cnt = p.cnt + ((size_t)b * Hkv + h) * p.RT + rt;
                __threadfence();
                const unsigned at_ = atomicAdd(cnt, 1u);
                sm.last = at_ == (unsigned)(r_hi - r_lo);
                if (at_ > (unsigned)(r_hi - r_lo)) raise_status(UA_ERR_INVALID_ARG);  // not zeroed
                if (sm.last) {
                    *cnt = 0;
                    __threadfence();
                }
            }
            __syncthreads();
            if (sm.last) {
                // Runs r_lo .. r_hi hold the unit's parts: r_lo in its second slot, the others in their
                // first.  A thread sums four elements of a row over its share of the parts with a running
                // maximum (one round of loads), and the shares are joined in order.
                const size_t ps = (size_t)R * (DH + 2);
                const int parts = r_hi - r_lo + 1;
                auto part = [&](int i) { return p.part + (size_t)(2 * (r_lo + i) + (i == 0 ? 1 : 0)) * ps; };
                const int cols = rows * (DH / 4), groups = max(1, min(kThreads / cols, parts));
                float4* share_o = reinterpret_cast<float4*>(&sm.o[0][0][0]);
                float2* share_ml = sm.share;
                static_assert(sizeof(sm.o) >= kThreads * 16, "a share for each thread");
                for (int e0 = 0; e0 < cols; e0 += kThreads) {
                    const int grp = groups > 1 ? tid / cols : 0, e = e0 + tid - grp * cols;
                    const int row = e / (DH / 4), d4 = (e % (DH / 4)) * 4;
                    const bool on = e < cols && grp < groups;
                    const float4 gt = on && grp == 0 ? gates(row, d4) : make_float4(0, 0, 0, 0);
                    float M = -INFINITY, L = 0.f;
                    float4 o = make_float4(0, 0, 0, 0);
                    auto join = [&](float m, float l, float4 v) {
                        const float mn = fmaxf(M, m), ms = mn == -INFINITY ? 0.f : mn;
                        const float f = ex2(2.f * (M - ms)), g = ex2(2.f * (m - ms));
                        M = mn;
                        L = fmaf(L, f, l * g);
                        o.x = fmaf(o.x, f, v.x * g);
                        o.y = fmaf(o.y, f, v.y * g);
                        o.z = fmaf(o.z, f, v.z * g);
                        o.w = fmaf(o.w, f, v.w * g);
                    };
                    if (on) {
                        for (int i = grp; i < parts; i += 4 * groups) {
                            float m[4], l[4];
                            float4 v[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const bool in = i + k * groups < parts;
                                const float* q = part(in ? i + k * groups : i);
                                m[k] = in ? __ldcg(q + row) : -INFINITY;
                                l[k] = in ? __ldcg(q + R + row) : 0.f;
                                v[k] = in ? __ldcg(reinterpret_cast<const float4*>(q + 2 * R + row * DH + d4))
                                          : make_float4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) join(m[k], l[k], v[k]);
                        }
                    }
                    if (groups > 1) {
                        if (on) {
                            share_o[tid] = o;
                            share_ml[tid] = make_float2(M, L);
                        }
                        __syncthreads();
                        for (int g = 1; on && grp == 0 && g < groups; ++g) {
                            const float2 ml = share_ml[g * cols + tid];
                            join(ml.x, ml.y, share_o[g * cols + tid]);
                        }
                    }
                    if (on && grp == 0) put_out(row, d4, o, M, L, gt);
                }
            }
        }
        if (!more) break;
        __syncthreads();
    }
}

template <typename T, int DH, int NT, bool E4M3> cudaError_t attend(const KvqAttendParams& p, cudaStream_t s) {
    using A = Att<T, DH, NT, E4M3>;
    auto kern = k_kvq_attend<T, DH, NT, E4M3>;
    const int smem = (int)sizeof(typename A::Smem), kThreads = A::kThreads;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // at most the blocks of full caches: the lengths are known on the device only
    const long long most = (long long)p.c.B * p.c.Hkv * p.RT * ((p.c.cap + kKvqBlock - 1) / kKvqBlock);
    const long long want = std::max(most * (1 + kUnitCost) / A::kMinItems, (long long)p.c.B * p.c.Hkv * p.RT) + 1;
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
