// k_kvq_append.cu -- append of keys and values to the 8-bit cache: per-head norm and position
// rotation of the keys on the way, the ring of recent rows, and the encoding of every block of 64
// slots that the call fills; a step's queries are normalised and rotated by further CTAs of the
// same launch, a prompt's by k_qk_norm_fwd beside it (formulas and layout in include/ua.h).
//
// Bound: HBM for prompts (each key and value read once in the activation type, written once in
// 8 bits), launch latency for single tokens.  One CTA owns a block of 64 slots of hpc KV heads:
// CH = DH/16 lanes a row, every element of the block in registers between the one read and the
// write of its code, so the block's largest magnitude costs one reduction and no second read.  A
// token's gain and rotation are one set of coefficients for all hpc heads; the next head's rows are
// copied meanwhile (a thread's own queue).  32 x 4096 tokens, 8 heads of 64, bf16 to e4m3: 83 us,
// 4.9 TB/s; issue slots bind (its share of a prompt with 32 query heads: 28 of 68 us for 8 x 4096 tokens).  8 x 4096
// tokens with queries to int8: 73 us; fp32 to e4m3 122, to int8 134.  The step of 32 tokens: 4.5 us.
// At DH = 64 three CTAs an SM leave 80 registers a thread: fp32 to int8 spills 180 bytes, to e4m3 28, bf16 to int8 48.
#include "qk_norm.cuh"
#include "ua_profile.h"

namespace ua {

namespace {

struct SeqState {
    int start, n_new;       // n_new = 0: nothing to append (or a refused sequence)
    int refused;            // status to raise, 0: none
};

// What sequence b appends.  Refused: n_new or start out of range, earlier rows of the start's
// block not in the ring, capacity.  A call that ends with `end` slots keeps the rows of blocks end/64 - 1 and
// end/64 (at a border the latter has none yet).  ring_state says which blocks' rows are there: those from
// ring_state/64 - 1 on.
__device__ __forceinline__ SeqState seq_state(const KvqAppendParams& p, int b) {
    SeqState s;
    const int n0 = p.c.n_kept[b];
    s.start = p.start ? p.start[b] : n0;
    s.n_new = p.n_new ? p.n_new[b] : p.n.T;
    s.refused = 0;
    if (n0 < 0 || n0 > p.c.cap || s.n_new < 0 || s.n_new > p.n.T || s.start < 0 || s.start > n0)
        s.refused = UA_ERR_INVALID_ARG;
    else if (s.start % kKvqBlock != 0 &&
             (p.c.ring_state[b] < s.start || s.start / kKvqBlock < p.c.ring_state[b] / kKvqBlock - 1))
        s.refused = UA_ERR_INVALID_ARG;
    else if (s.n_new > p.c.cap - s.start)
        s.refused = UA_ERR_CAPACITY;
    if (s.refused) {
        s.n_new = 0;
        s.start = 0;
    }
    return s;
}

// Scale of a block from the bits of its largest magnitude, and the factor of its encoding.  int8:
// amax / 127 and 127 / amax.  e4m3: the format floats, so a power of two loses nothing against
// amax / 448 and makes the scaling exact: 2^(E - 8), or 2^(E - 7) where amax > 448 * 2^(E - 8) (448 = 1.75 * 2^8), E
// the exponent of amax; the factor is its reciprocal.  Factor 0 (all codes 0): a block of zeros (below 2^-100: scale 0) or with
// a value that is not finite (scale NaN).
template <bool E4M3> __device__ __forceinline__ float block_scale(uint32_t amax_bits, float* factor) {
    *factor = 0.f;
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    if (amax_bits < 0x0d800000u) return 0.f;
    if constexpr (E4M3) {
        const uint32_t e = (amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        *factor = __uint_as_float((254 - e) << 23);
        return __uint_as_float(e << 23);
    } else {
        const float amax = __uint_as_float(amax_bits);
        *factor = 127.f / amax;
        return amax / 127.f;
    }
}

// 8 codes of a row's chunk
template <typename T, bool E4M3> __device__ __forceinline__ uint2 encode8(const Raw8<T>& raw, float factor) {
    if (factor == 0.f) return make_uint2(0, 0);
    F2 y[4];
    float x[8];
    raw.get(y);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], f2(factor, factor));
    unpairs(y, x);
    uint32_t w[2];
    if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
                "mov.b32 %0, {l, h};\n\t}"
                : "=r"(w[i])
                : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]));
    } else {
        // |x * factor| <= 127 (1 + 2^-23): rounds to 127 at most.  1.5 * 2^23 more leaves the rounded
        // (to even) number in the low byte.
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += 12582912.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = __byte_perm(__byte_perm(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), 0x0040),
                               __byte_perm(__float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]), 0x0040), 0x5410);
    }
    return make_uint2(w[0], w[1]);
}

// ... to where the chunk's pieces lie
template <typename T, int DH> __device__ __forceinline__ void put_codes(uint8_t* d, uint2 w) {
    if constexpr (Raw8<T>::NV == 1) {
        *reinterpret_cast<uint2*>(d) = w;
    } else {
        *reinterpret_cast<uint32_t*>(d) = w.x;
        *reinterpret_cast<uint32_t*>(d + kPieceStep<T, DH>) = w.y;
    }
}

// grid: B * (Hkv / hpc) * nb block CTAs, then q_tiles * q_split query CTAs; 4 * DH threads
template <typename T> struct KvQueue {
    static constexpr int NV = Raw8<T>::NV, DEPTH = 2;
    template <int NTH> using Queue = LaneQueue<NTH, 4 * NV, DEPTH>;
};

template <typename T, int DH, bool E4M3>
__global__ void __launch_bounds__(4 * DH, DH == 64 ? 3 : 1) k_kvq_append(KvqAppendParams p) {
    constexpr int CH = DH / 16, HALF = DH / 2, NTH = 4 * DH, NW = NTH / 32, TOK = norm_tokens<DH, NTH>();
    constexpr int NV = KvQueue<T>::NV, DEPTH = KvQueue<T>::DEPTH;
    extern __shared__ __align__(16) unsigned char s_queue[];
    __shared__ __align__(16) float s_cos[TOK * HALF], s_sin[TOK * HALF];
    __shared__ double s_f[HALF];
    __shared__ __align__(16) uint32_t s_max[2][2][NW];   // the warps' largest magnitudes, keys and values
    __shared__ int s_last;
    grid_dep_wait();
    grid_dep_release();
    const int tid = threadIdx.x, T_ = p.n.T, Hkv = p.c.Hkv;
    const int groups = Hkv / p.hpc, kv_ctas = p.c.B * groups * p.nb;
    // Every CTA arrives once it has read the slot counts; the last to arrive sets them, at its end.
    auto arrive = [&]() {
        if (tid == 0) {
            __threadfence();
            const int at = atomicAdd(p.c.ring_state + p.c.B, 1);
            if (at >= (int)gridDim.x) raise_status(UA_ERR_INVALID_ARG);     // the counter did not start at 0
            s_last = at == (int)gridDim.x - 1;
        }
    };
    if ((int)blockIdx.x >= kv_ctas) {                    // queries
        const int i = blockIdx.x - kv_ctas, n0 = i / p.q_split * TOK;
        QkNormParams q = p.n;
        q.k = nullptr;
        NormTile<T, DH, NTH>::run(q, n0, i % p.q_split, p.q_split, s_queue, [&](F2* cs, F2* sn) {
            auto posf = [&](int n) {
                if (p.n.pos) return p.n.pos[n];
                const int b = n / T_;
                return (p.start ? p.start[b] : p.c.n_kept[b]) + n - b * T_;
            };
            if (p.n.rope) tile_angles<T, DH, NTH>(s_cos, s_sin, n0, (int)p.n.N, p.n.rf, s_f, posf, cs, sn);
            arrive();                                    // (behind the angles' barrier)
        });
    } else {
        const int j = blockIdx.x % p.nb, gi = (blockIdx.x / p.nb) % groups, b = blockIdx.x / p.nb / groups;
        const int row = tid / CH, c = tid % CH;
        const SeqState s = seq_state(p, b);
        if (s.refused && j == 0 && gi == 0 && tid == 0) raise_status(s.refused);
        if (tid < HALF) s_f[tid] = p.n.rf.f[tid] * 0.15915494309189535;      // 1 / (2 pi)
        const int end = s.start + s.n_new, j0 = s.start / kKvqBlock, jl = end / kKvqBlock;   // jl: unfinished block
        const int mine = j0 + j;
        // this row's position (a single token's may be the slot count: read before anyone changes it)
        const int t_mine = mine * kKvqBlock + row - s.start;
        const int pos_mine = p.n.rope && p.n.pos && t_mine >= 0 && t_mine < s.n_new ? p.n.pos[b * T_ + t_mine] : 0;
        __syncthreads();
        arrive();
        if (s.n_new > 0 && mine * kKvqBlock < end) {
            // Ring rows are kept for blocks jl - 1 and jl.  The first block may still need earlier
            // rows out of the ring, from the places that the kept block of the same parity takes:
            // that block's rows are then written by the first block's CTA, after it has read them.
            const bool old_rows = s.start % kKvqBlock != 0 && (j0 + 1) * kKvqBlock <= end;
            auto shares_first = [&](int blk) { return old_rows && blk > j0 && ((blk - j0) & 1) == 0; };
            const bool kept_here = mine >= jl - 1 && !shares_first(mine);
            const int kept_too = j == 0 ? (shares_first(jl) ? jl : shares_first(jl - 1) ? jl - 1 : -1) : -1;
            typename KvQueue<T>::template Queue<NTH> queue(s_queue);
            int buf = 0;
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                const int blk = pass == 0 ? mine : kept_too;
                if (blk < 0) continue;
                const bool keep = pass == 1 || kept_here;
                const bool full = pass == 0 && (blk + 1) * kKvqBlock <= end;
                const int slot = blk * kKvqBlock + row, t = slot - s.start;
                const bool is_new = t >= 0 && slot < end, old = full && t < 0;
                const int n = b * T_ + t;
                // this thread's chunk in the ring, of head h: ring + h * kKvqRing * DH
                const size_t ring = (((size_t)b * Hkv + gi * p.hpc) * kKvqRing + (slot & (kKvqRing - 1))) * DH + lane_at<T>(c);
                T* kr = static_cast<T*>(p.c.kr) + ring;
                T* vr = static_cast<T*>(p.c.vr) + ring;
                const T* ksrc = old ? kr : static_cast<const T*>(p.n.k);
                const T* vsrc = old ? vr : static_cast<const T*>(p.v);
                if (is_new) {
                    ksrc += (long long)n * p.n.k_ld + gi * p.hpc * DH + lane_at<T>(c);
                    vsrc += (long long)n * p.v_ld + gi * p.hpc * DH + lane_at<T>(c);
                }
                const int hstep = old ? kKvqRing * DH : DH;
                auto fetch = [&](int hh, int stage) {
                    if (hh < p.hpc) {
                        if (is_new || old) {
                            const T* k = ksrc + hh * hstep;
                            const T* v = vsrc + hh * hstep;
#pragma unroll
                            for (int i = 0; i < NV; ++i) {
                                queue.put(stage, i, k + i * kPieceStep<T, DH>);
                                queue.put(stage, NV + i, k + HALF + i * kPieceStep<T, DH>);
                                queue.put(stage, 2 * NV + i, v + i * kPieceStep<T, DH>);
                                queue.put(stage, 3 * NV + i, v + HALF + i * kPieceStep<T, DH>);
                            }
                        }
                    }
                    queue.commit();
                };
#pragma unroll
                for (int i = 0; i < DEPTH - 1; ++i) fetch(i, i);
                const long long crow = full ? kvq_row(p.c, b, blk) : -1;
                // The gain and the rotation of a token's pairs together, the same for every head:
                // (a0, a1) -> r (a0 w0 cos - a1 w1 sin, a1 w1 cos + a0 w0 sin), r the head's own.
                F2 c00[4], c01[4], c11[4], c10[4];
                if (is_new && p.n.rope) {
                    F2 cs[4], sn[4];
                    lane_angles<T, DH>(!p.n.pos ? slot : pass == 0 ? pos_mine : p.n.pos[n], s_f, c, cs, sn);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        c00[i] = c11[i] = cs[i];
                        c01[i] = neg2(sn[i]);
                        c10[i] = sn[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        c00[i] = c11[i] = f2(1.f, 1.f);
                        c01[i] = c10[i] = f2(0.f, 0.f);
                    }
                }
                if (p.n.wk != nullptr) {
                    F2 w0[4], w1[4];
                    load_gains<T, DH>(p.n.wk, c, w0, w1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        c00[i] = mul2(c00[i], w0[i]);
                        c10[i] = mul2(c10[i], w0[i]);
                        c01[i] = mul2(c01[i], w1[i]);
                        c11[i] = mul2(c11[i], w1[i]);
                    }
                }
                const bool changed = p.n.wk != nullptr || p.n.rope;
                int stage = 0;
#pragma unroll 1
                for (int hh = 0; hh < p.hpc; ++hh) {
                    fetch(hh + DEPTH - 1, (stage + DEPTH - 1) % DEPTH);
                    queue.template wait<DEPTH - 1>();
                    Raw8<T> ka, kb, va, vb;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        ka.u[i] = queue.get(stage, i);
                        kb.u[i] = queue.get(stage, NV + i);
                    }
                    if (changed) {
                        F2 x0[4], x1[4];
                        ka.get(x0);
                        kb.get(x1);
                        F2 r2 = f2(1.f, 1.f);
                        if (p.n.wk != nullptr) {
                            const float r = row_rstd<DH>(x0, x1, p.n.eps);
                            r2 = f2(r, r);
                        }
                        if (is_new) {                    // rounded to the activation type: codes are formed
#pragma unroll                                           // from what the ring would hold
                            for (int i = 0; i < 4; ++i) {
                                const F2 a = mul2(x0[i], r2), b2 = mul2(x1[i], r2);
                                x0[i] = fma2(b2, c01[i], mul2(a, c00[i]));
                                x1[i] = fma2(a, c10[i], mul2(b2, c11[i]));
                            }
                            ka.put(x0);
                            kb.put(x1);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        va.u[i] = queue.get(stage, 2 * NV + i);
                        vb.u[i] = queue.get(stage, 3 * NV + i);
                    }
                    stage = (stage + 1) % DEPTH;
                    if (full) {
                        uint32_t mk = __reduce_max_sync(0xffffffffu, ka.amax_bits(kb));
                        uint32_t mv = __reduce_max_sync(0xffffffffu, va.amax_bits(vb));
                        if ((tid & 31) == 0) {
                            s_max[buf][0][tid >> 5] = mk;
                            s_max[buf][1][tid >> 5] = mv;
                        }
                        __syncthreads();                 // (also: this head's earlier rows have been read from the ring)
#pragma unroll
                        for (int i = 0; i < NW; i += 4) {
                            const uint4 a = *reinterpret_cast<const uint4*>(&s_max[buf][0][i]);
                            const uint4 b4 = *reinterpret_cast<const uint4*>(&s_max[buf][1][i]);
                            mk = max(max(mk, max(a.x, a.y)), max(a.z, a.w));
                            mv = max(max(mv, max(b4.x, b4.y)), max(b4.z, b4.w));
                        }
                        buf ^= 1;
                        if (crow >= 0) {
                            const long long r = crow + (long long)(gi * p.hpc + hh) * p.c.bpp;
                            float fk, fv;
                            const float sk = block_scale<E4M3>(mk, &fk), sv = block_scale<E4M3>(mv, &fv);
                            uint8_t* dk = p.c.k + r * (kKvqBlock * DH) + row * DH + lane_at<T>(c);
                            uint8_t* dv = p.c.v + r * (kKvqBlock * DH) + row * DH + lane_at<T>(c);
                            put_codes<T, DH>(dk, encode8<T, E4M3>(ka, fk));
                            put_codes<T, DH>(dk + HALF, encode8<T, E4M3>(kb, fk));
                            put_codes<T, DH>(dv, encode8<T, E4M3>(va, fv));
                            put_codes<T, DH>(dv + HALF, encode8<T, E4M3>(vb, fv));
                            if (tid == 0) {
                                p.c.ks[r] = sk;
                                p.c.vs[r] = sv;
                            }
                        }
                    }
                    if (is_new && keep) {
                        T* kd = kr + (size_t)hh * kKvqRing * DH;
                        T* vd = vr + (size_t)hh * kKvqRing * DH;
                        ka.template st<DH>(kd); kb.template st<DH>(kd + HALF);
                        va.template st<DH>(vd); vb.template st<DH>(vd + HALF);
                    }
                }
                queue.template wait<0>();
                __syncthreads();                         // every earlier row of every head has been read
            }
        }
    }
    __syncthreads();
    if (s_last) {
        for (int b = tid; b < p.c.B; b += blockDim.x) {
            const SeqState s = seq_state(p, b);
            if (s.refused) continue;
            const int end = s.start + s.n_new;
            p.c.n_kept[b] = end;
            // from a start on, the rows of its block are the newest whatever was there before (a start inside
            // the block found its earlier rows there); the block before keeps what was known of it (nothing, where
            // the count was set by hand to a border: ring_state below the start)
            const int border = (s.start / kKvqBlock + 1) * kKvqBlock, was = p.c.ring_state[b];
            p.c.ring_state[b] = max(end, was < s.start ? border : min(was, border));
        }
        if (tid == 0) p.c.ring_state[p.c.B] = 0;
    }
}

template <typename T, int DH, bool E4M3> cudaError_t append(const KvqAppendParams& p, cudaStream_t s) {
    const int ctas = p.c.B * (p.c.Hkv / p.hpc) * p.nb + p.q_tiles * p.q_split;
    constexpr int q_smem = NormTile<T, DH, 4 * DH>::Queue::kBytes, kv_smem = KvQueue<T>::template Queue<4 * DH>::kBytes;
    constexpr int smem = q_smem > kv_smem ? q_smem : kv_smem;
    cudaError_t e = cudaFuncSetAttribute(k_kvq_append<T, DH, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    UA_PROFILE("k_kvq_append", s);
    return launch_dependent(k_kvq_append<T, DH, E4M3>, dim3(ctas), dim3(4 * DH), smem, s, p);
}

template <typename T> cudaError_t append_t(const KvqAppendParams& p, int d, bool e4m3, cudaStream_t s) {
    if (d == 64) return e4m3 ? append<T, 64, true>(p, s) : append<T, 64, false>(p, s);
    return e4m3 ? append<T, 128, true>(p, s) : append<T, 128, false>(p, s);
}

}  // namespace

cudaError_t launch_kvq_append(const KvqAppendParams& p, int d, bool bf16, bool e4m3, cudaStream_t s) {
    return bf16 ? append_t<__nv_bfloat16>(p, d, e4m3, s) : append_t<float>(p, d, e4m3, s);
}

}  // namespace ua
