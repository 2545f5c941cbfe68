// k_qk_norm.cu -- RMS norm of every query and key head with a learned gain, and the position
// rotation, in one pass; and its backward (formulas in include/ua.h).
//
// Bound: HBM.  The forward reads and writes every activation once (4 bytes an element in bf16), the
// backward reads x and dy and writes dx (6 bytes).  What it took to get near:
//   * loads in flight that cost no registers: a thread's own queue of asynchronous copies, three (two)
//     steps ahead.  3B shape (4 x 8192 tokens, 24 + 8 heads of 128, bf16): forward 161 -> 90 us;
//   * few instructions an element, for at 6.5 TB/s an SM has some 280 issue slots a warp for 3 KB: packed
//     fp32 arithmetic, a token's angles once for all its heads (90 -> 83 us; copy bandwidth: 82);
//   * the backward's angles a thread's own, without barriers, from positions fetched a tile ahead: 169 ->
//     139 us (123), 88 % of the copy bandwidth; what is left is issue slots (60 % busy at 16 warps an SM,
//     128 registers a thread; with the rotation 24 (bf16) or 32 bytes of them spill).
#include "qk_norm.cuh"
#include "ua_profile.h"

namespace ua {

constexpr int kNth = 256;               // threads of a CTA

// grid (token tiles, head splits).  p.beside: it runs beside the append of the same call, whose results
// it does not need: that kernel releases it once everything before the call is done.
template <typename T, int DH>
__global__ void __launch_bounds__(kNth, 3) k_qk_norm_fwd(QkNormParams p) {
    constexpr int HALF = DH / 2, TOK = norm_tokens<DH, kNth>();
    extern __shared__ __align__(16) unsigned char s_queue[];
    __shared__ __align__(16) float s_cos[TOK * HALF], s_sin[TOK * HALF];
    __shared__ double s_f[HALF];
    if (!p.beside) grid_dep_wait();
    const int n0 = blockIdx.x * TOK;
    NormTile<T, DH, kNth>::run(p, n0, blockIdx.y, gridDim.y, s_queue, [&](F2* cs, F2* sn) {
        auto posf = [&](int n) {
            if (p.pos) return p.pos[n];
            const int b = (unsigned)n / (unsigned)p.T;
            return n - b * p.T + (p.start ? p.start[b] : 0);
        };
        if (p.rope) tile_angles<T, DH, kNth>(s_cos, s_sin, n0, (int)p.N, p.rf, s_f, posf, cs, sn);
    });
    if (p.beside) grid_dep_wait();                      // whoever waits for this kernel waits for that one
}

// Backward.  The first ctas_q CTAs take the queries, the others the keys (in proportion to their
// heads), each an equal run of (token tile, four heads) items; the loads of the next items are always on their way (a thread's own queue in shared memory).  It keeps the gain
// gradient of its lanes' elements in registers (fp32: no chain is longer than a lane's own terms; off by 2.4e-7 of
// the largest for 270000 tokens of 128 heads), sums it over its rows in shared memory at the
// end and writes one partial row; k_qk_norm_dw adds the CTAs' rows in a fixed order.
template <typename T> struct BwdQueue {
    static constexpr int NV = Raw8<T>::NV, DEPTH = 3;
    using Queue = LaneQueue<kNth, 4 * NV, DEPTH>;
};

template <typename T, int DH, bool ROPE, bool NORM>
__device__ __forceinline__ void bwd_run(const QkNormParams& p, bool is_q, int cta, int ctas, unsigned char* s_queue,
                                        const double* s_f) {
    constexpr int CH = DH / 16, HALF = DH / 2, TOK = norm_tokens<DH, kNth>(), ROWS = kNth / CH;
    constexpr int NV = BwdQueue<T>::NV, DEPTH = BwdQueue<T>::DEPTH;
    const int tid = threadIdx.x, c = tid % CH, hp = (tid / CH) % kNormHeads, row = tid / CH, N = (int)p.N;
    const T* dy = static_cast<const T*>(is_q ? p.dq_out : p.dk_out);
    const int nh = is_q ? p.H : p.Hkv, quads = (nh + kNormHeads - 1) / kNormHeads;
    const long long ld = is_q ? p.q_ld : p.k_ld;
    // an equal run of (token tile, head quad) items
    const int tiles = (N + TOK - 1) / TOK;
    const int lo = (int)((long long)tiles * quads * cta / ctas);
    const int count = (int)((long long)tiles * quads * (cta + 1) / ctas) - lo;
    typename BwdQueue<T>::Queue queue(s_queue);
    // the next item to fetch: its place in dy (and dx) and in x
    int left = count, fi = lo % quads, fn = lo / quads * TOK + row / kNormHeads, fstage = 0;
    const T* fg = dy + ((long long)fn * nh + fi * kNormHeads + hp) * DH + lane_at<T>(c);
    const T* fx = static_cast<const T*>(is_q ? p.q : p.k) + fn * ld + (fi * kNormHeads + hp) * DH + lane_at<T>(c);
    const long long g_jump = ((long long)TOK * nh - (quads - 1) * kNormHeads) * DH;   // from a tile's last quad to the
    const long long x_jump = TOK * ld - (long long)(quads - 1) * kNormHeads * DH;     // next tile's first
    auto fetch = [&]() {
        if (left > 0) {
            --left;
            if (fn < N && fi * kNormHeads + hp < nh) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    queue.put(fstage, v, fg + v * kPieceStep<T, DH>);
                    queue.put(fstage, NV + v, fg + HALF + v * kPieceStep<T, DH>);
                    if (NORM) {
                        queue.put(fstage, 2 * NV + v, fx + v * kPieceStep<T, DH>);
                        queue.put(fstage, 3 * NV + v, fx + HALF + v * kPieceStep<T, DH>);
                    }
                }
            }
            if (++fi == quads) {
                fi = 0;
                fn += TOK;
                fg += g_jump;
                fx += x_jump;
            } else {
                fg += kNormHeads * DH;
                fx += kNormHeads * DH;
            }
        }
        queue.commit();
        fstage = fstage + 1 == DEPTH ? 0 : fstage + 1;
    };
    int i = fi, n = fn, stage = 0;
    T* out = static_cast<T*>(is_q ? p.dq : p.dk) + (fg - dy);
#pragma unroll
    for (int j = 0; j < DEPTH - 1; ++j) fetch();
    F2 w0[4], w1[4], dw[8], cs[4], sn[4], ns[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = f2(0.f, 0.f);
    if (NORM) load_gains<T, DH>(is_q ? p.wq : p.wk, c, w0, w1);
    const float eps = p.eps;
    auto pos_of = [&](int m) { return m >= N ? 0 : p.pos ? __ldg(p.pos + m) : (int)((unsigned)m % (unsigned)p.T); };
    int pos = ROPE ? pos_of(n) : 0;
    bool new_tile = true;
#pragma unroll 1
    for (int item = 0; item < count; ++item) {
        if (ROPE && new_tile) {                         // (its position was fetched with the tile before)
            lane_angles<T, DH>(pos, s_f, c, cs, sn);
            negate(sn, ns);
            pos = pos_of(n + TOK);
        }
        const bool ok = n < N && i * kNormHeads + hp < nh;
        fetch();
        queue.template wait<DEPTH - 1>();
        Raw8<T> ga, gb;
        F2 g0[4], g1[4];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            ga.u[v] = queue.get(stage, v);
            gb.u[v] = queue.get(stage, NV + v);
        }
        ga.get(g0);
        gb.get(g1);
        if (ROPE) rotate_row(g0, g1, cs, ns, sn);       // R(-pos) dy
        if (NORM) {
            Raw8<T> xa, xb;
            F2 x0[4], x1[4], n0[4], n1[4];              // n: g (.) w
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                xa.u[v] = queue.get(stage, 2 * NV + v);
                xb.u[v] = queue.get(stage, 3 * NV + v);
            }
            xa.get(x0);
            xb.get(x1);
            F2 ss = f2(0.f, 0.f), dot = ss;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                n0[j] = mul2(g0[j], w0[j]);
                n1[j] = mul2(g1[j], w1[j]);
                ss = fma2(x0[j], x0[j], fma2(x1[j], x1[j], ss));
                dot = fma2(n0[j], x0[j], fma2(n1[j], x1[j], dot));
            }
            const float r = rsqrtf(row_sum<CH>(hsum(ss)) * (1.f / DH) + eps);
            const float rm = r * row_sum<CH>(hsum(dot)) * r * (1.f / DH);    // r * mean(n (.) xh)
            if (ok) {                                   // (a row past the end holds anything)
                const F2 r2 = f2(r, r), m2 = f2(-rm, -rm);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const F2 h0 = mul2(x0[j], r2), h1 = mul2(x1[j], r2);
                    dw[j] = fma2(g0[j], h0, dw[j]);
                    dw[4 + j] = fma2(g1[j], h1, dw[4 + j]);
                    g0[j] = fma2(h0, m2, mul2(n0[j], r2));
                    g1[j] = fma2(h1, m2, mul2(n1[j], r2));
                }
            }
        }
        stage = stage + 1 == DEPTH ? 0 : stage + 1;
        if (ok) {
            ga.put(g0);
            gb.put(g1);
            ga.template st<DH>(out);
            gb.template st<DH>(out + HALF);
        }
        new_tile = ++i == quads;
        if (new_tile) {
            i = 0;
            n += TOK;
            out += g_jump;
        } else {
            out += kNormHeads * DH;
        }
    }
    queue.template wait<0>();
    if (!NORM) return;
    __syncthreads();                                    // the queue becomes the rows' sums [row][element]
    float* s_sum = reinterpret_cast<float*>(s_queue);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float* mine = s_sum + row * DH + elem_at<T, DH>(c, 2 * j);
        un2(dw[j], mine[0], mine[1]);
        un2(dw[4 + j], mine[HALF], mine[HALF + 1]);
    }
    __syncthreads();
    if (tid < DH) {
        float s = 0.f;
        for (int r = 0; r < ROWS; ++r) s += s_sum[r * DH + tid];
        p.part[(size_t)blockIdx.x * DH + tid] = s;
    }
}

template <typename T, int DH, bool ROPE>
__global__ void __launch_bounds__(kNth, 2) k_qk_norm_bwd(const __grid_constant__ QkNormParams p, int ctas_q) {
    extern __shared__ __align__(16) unsigned char s_queue[];
    __shared__ double s_f[DH / 2];
    static_assert(BwdQueue<T>::Queue::kBytes >= kNth / (DH / 16) * DH * 4, "the rows' sums fit the queue");
    grid_dep_wait();
    grid_dep_release();                                 // (k_qk_norm_dw may be made ready)
    if (ROPE) {
        if (threadIdx.x < DH / 2) s_f[threadIdx.x] = p.rf.f[threadIdx.x] * 0.15915494309189535;  // 1 / (2 pi)
        __syncthreads();
    }
    const bool is_q = (int)blockIdx.x < ctas_q;
    const int cta = is_q ? blockIdx.x : blockIdx.x - ctas_q, ctas = is_q ? ctas_q : gridDim.x - ctas_q;
    if ((is_q ? p.wq : p.wk) != nullptr) bwd_run<T, DH, ROPE, true>(p, is_q, cta, ctas, s_queue, s_f);
    else bwd_run<T, DH, ROPE, false>(p, is_q, cta, ctas, s_queue, s_f);
}

// Sum of the CTAs' partial gain gradients: grid (d/32, 2), block (32, 32); rows [0, ctas_q) are the
// queries', the others the keys'
__global__ void __launch_bounds__(1024) k_qk_norm_dw(const float* part, int ctas_q, int ctas, int d, float* dwq,
                                                     float* dwk) {
    __shared__ float s_sum[32][33];
    grid_dep_wait();
    float* out = blockIdx.y ? dwk : dwq;
    if (out == nullptr) return;
    // every load at once, then a column a warp: a chain of 10 + 5 sums (serial loops: 0.5 us more)
    const int e = blockIdx.x * 32 + threadIdx.x, lo = (blockIdx.y ? ctas_q : 0) + threadIdx.y, hi = blockIdx.y ? ctas : ctas_q;
    constexpr int K = (kQkNormBwdCtas + 2 + 31) / 32;
    float v[K], s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lo + 32 * k < hi ? part[(size_t)(lo + 32 * k) * d + e] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) s += v[k];
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = row_sum<32>(s_sum[threadIdx.x][threadIdx.y]);
    if (threadIdx.x == 0) out[blockIdx.x * 32 + threadIdx.y] = s;
}

namespace {

int head_quads(const QkNormParams& p) {
    return (p.q ? (p.H + kNormHeads - 1) / kNormHeads : 0) + (p.k ? (p.Hkv + kNormHeads - 1) / kNormHeads : 0);
}

template <typename T, int DH> cudaError_t fwd(const QkNormParams& p, cudaStream_t s) {
    constexpr int TOK = norm_tokens<DH, kNth>(), smem = NormTile<T, DH, kNth>::Queue::kBytes;
    const long long tiles = (p.N + TOK - 1) / TOK;
    // few tokens: the heads are split over CTAs too, while all of them fit the SMs' three places (2 x 777
    // tokens, 32 + 8 heads of 64: 6.6 us with a CTA an SM, 4.6 with three; in two rounds, 5.6)
    const int quads = head_quads(p), places = 3 * 148;
    const int split = (int)(tiles >= places ? 1 : (quads < places / tiles ? quads : places / tiles));
    cudaError_t e = cudaFuncSetAttribute(k_qk_norm_fwd<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    UA_PROFILE("k_qk_norm_fwd", s);
    return launch_dependent(k_qk_norm_fwd<T, DH>, dim3((unsigned)tiles, split < 1 ? 1 : split), dim3(kNth), smem, s, p);
}

template <typename T, int DH> cudaError_t bwd(const QkNormParams& p, cudaStream_t s) {
    constexpr int TOK = norm_tokens<DH, kNth>(), smem = BwdQueue<T>::Queue::kBytes;
    const long long tiles = (p.N + TOK - 1) / TOK;
    // two resident CTAs for each SM, shared between queries and keys in proportion to their heads
    const int nq = p.q ? p.H : 0, nk = p.k ? p.Hkv : 0;
    auto most = [&](int heads) {
        const long long n = heads ? (kQkNormBwdCtas * (long long)heads + (nq + nk) / 2) / (nq + nk) : 0;
        const long long items = tiles * ((heads + kNormHeads - 1) / kNormHeads);
        return (int)(heads == 0 ? 0 : n < 1 ? 1 : n < items ? n : items);
    };
    const int ctas_q = most(nq), ctas = ctas_q + most(nk);
    auto kern = p.rope ? k_qk_norm_bwd<T, DH, true> : k_qk_norm_bwd<T, DH, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    {
        UA_PROFILE("k_qk_norm_bwd", s);
        e = launch_dependent(kern, dim3(ctas), dim3(kNth), smem, s, p, ctas_q);
        if (e != cudaSuccess) return e;
    }
    float* dwq = p.q && p.wq ? p.dwq : nullptr;
    float* dwk = p.k && p.wk ? p.dwk : nullptr;
    if (dwq == nullptr && dwk == nullptr) return cudaSuccess;
    UA_PROFILE("k_qk_norm_dw", s);
    return launch_dependent(k_qk_norm_dw, dim3(DH / 32, 2), dim3(32, 32), 0, s, (const float*)p.part, ctas_q, ctas, DH,
                            dwq, dwk);
}

}  // namespace

cudaError_t launch_qk_norm_fwd(const QkNormParams& p, int d, bool bf16, cudaStream_t s) {
    if (d == 64) return bf16 ? fwd<__nv_bfloat16, 64>(p, s) : fwd<float, 64>(p, s);
    return bf16 ? fwd<__nv_bfloat16, 128>(p, s) : fwd<float, 128>(p, s);
}

cudaError_t launch_qk_norm_bwd(const QkNormParams& p, int d, bool bf16, cudaStream_t s) {
    if (d == 64) return bf16 ? bwd<__nv_bfloat16, 64>(p, s) : bwd<float, 64>(p, s);
    return bf16 ? bwd<__nv_bfloat16, 128>(p, s) : bwd<float, 128>(p, s);
}

}  // namespace ua
