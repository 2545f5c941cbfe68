// k_qk_norm.cu -- RMS norm of every query and key head with a learned gain, and the position
// rotation, in one pass; and its backward (formulas in include/ua.h).
//
// Bound: HBM.  The forward reads and writes every activation once (4 bytes an element in bf16),
// the backward reads x and dy and writes dx (6 bytes); the angles (double precision, one set for
// each token, shared by its heads through shared memory) and the arithmetic hide under the
// loads, which are issued one head quad ahead.
#include "qk_norm.cuh"
#include "ua_profile.h"

namespace ua {

constexpr int kNth = 256;               // threads of a CTA

// grid (token tiles, head splits)
template <typename T, int DH>
__global__ void __launch_bounds__(kNth, 3) k_qk_norm_fwd(QkNormParams p) {
    constexpr int HALF = DH / 2, TOK = norm_tokens<DH, kNth>();
    extern __shared__ __align__(16) unsigned char s_queue[];
    __shared__ float s_cos[TOK * HALF], s_sin[TOK * HALF];
    __shared__ double s_f[HALF];
    grid_dep_wait();
    const int n0 = blockIdx.x * TOK;
    NormTile<T, DH, kNth>::run(p, n0, blockIdx.y, gridDim.y, s_queue, [&](float* cs, float* sn) {
        if (p.rope)
            tile_angles<DH, kNth>(s_cos, s_sin, n0, (int)p.N, p.rf, s_f,
                                  [&](int n) { return p.pos ? p.pos[n] : (int)((unsigned)n % (unsigned)p.T); }, cs, sn);
    });
}

// Backward.  The first ctas_q CTAs take the queries, the others the keys (in proportion to their
// heads).  A persistent CTA walks token tiles; the loads of the next head quads, the next tile's
// among them, are always on their way (a thread's own queue in shared memory).  It keeps the gain
// gradient of its lanes' elements in registers (fp32), sums it over its rows in shared memory at the
// end and writes one partial row; k_qk_norm_dw adds the CTAs' rows in a fixed order.
template <typename T> struct BwdQueue {
    static constexpr int NV = Raw8<T>::NV, DEPTH = 3;
    using Queue = LaneQueue<kNth, 4 * NV, DEPTH>;
};

template <typename T, int DH>
__global__ void __launch_bounds__(kNth, 2) k_qk_norm_bwd(QkNormParams p, int ctas_q) {
    constexpr int CH = DH / 16, HALF = DH / 2, TOK = norm_tokens<DH, kNth>(), ROWS = kNth / CH;
    constexpr int NV = BwdQueue<T>::NV, DEPTH = BwdQueue<T>::DEPTH;
    extern __shared__ __align__(16) unsigned char s_queue[];
    __shared__ float s_cos[TOK * HALF], s_sin[TOK * HALF];
    __shared__ double s_f[HALF];
    static_assert(BwdQueue<T>::Queue::kBytes >= ROWS * DH * 4, "the rows' sums fit the queue");
    grid_dep_wait();
    const int tid = threadIdx.x, c = tid % CH, hp = (tid / CH) % kNormHeads, row = tid / CH, N = (int)p.N;
    const bool is_q = (int)blockIdx.x < ctas_q;
    const int first = is_q ? blockIdx.x : blockIdx.x - ctas_q, step = is_q ? ctas_q : gridDim.x - ctas_q;
    const T* x = static_cast<const T*>(is_q ? p.q : p.k);
    const T* dy = static_cast<const T*>(is_q ? p.dq_out : p.dk_out);
    T* dx = static_cast<T*>(is_q ? p.dq : p.dk);
    const float* w = is_q ? p.wq : p.wk;
    const int nh = is_q ? p.H : p.Hkv, quads = (nh + kNormHeads - 1) / kNormHeads;
    const long long ld = is_q ? p.q_ld : p.k_ld;
    const int tiles = (N + TOK - 1) / TOK;
    typename BwdQueue<T>::Queue queue(s_queue);
    int ft = first, fi = 0, fstage = 0;              // the next (tile, quad) to fetch
    auto fetch = [&]() {
        if (ft < tiles) {
            const int n = ft * TOK + row / kNormHeads, h = fi * kNormHeads + hp;
            const bool ok = n < N && h < nh;
            const T* g = ok ? dy + ((long long)n * nh + h) * DH + 8 * c : dy;
            const T* s = ok ? x + n * ld + h * DH + 8 * c : x;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                queue.put(fstage, v, g + v * Vec16<T>::N, ok);
                queue.put(fstage, NV + v, g + HALF + v * Vec16<T>::N, ok);
                if (w != nullptr) {
                    queue.put(fstage, 2 * NV + v, s + v * Vec16<T>::N, ok);
                    queue.put(fstage, 3 * NV + v, s + HALF + v * Vec16<T>::N, ok);
                }
            }
            if (++fi == quads) {
                fi = 0;
                ft += step;
            }
        }
        queue.commit();
        fstage = (fstage + 1) % DEPTH;
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) fetch();
    float w0[8], w1[8], dw[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[e] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w0[e] = w ? __ldg(w + 8 * c + e) : 1.f;
        w1[e] = w ? __ldg(w + HALF + 8 * c + e) : 1.f;
    }
    int stage = 0;
    for (int tile = first; tile < tiles; tile += step) {
        const int n0 = tile * TOK, n = n0 + row / kNormHeads;
        float cs[8], sn[8];
        if (p.rope) {
            __syncthreads();                            // the last tile's angles have been read
            tile_angles<DH, kNth>(s_cos, s_sin, n0, N, p.rf, s_f,
                                  [&](int m) { return p.pos ? p.pos[m] : (int)((unsigned)m % (unsigned)p.T); }, cs, sn);
        }
        for (int i = 0; i < quads; ++i) {
            const int h = i * kNormHeads + hp;
            const bool ok = n < N && h < nh;
            fetch();
            queue.template wait<DEPTH - 1>();
            Raw8<T> ga, gb;
            float g0[8], g1[8];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                ga.u[v] = queue.get(stage, v);
                gb.u[v] = queue.get(stage, NV + v);
            }
            ga.get(g0);
            gb.get(g1);
            if (p.rope) {                               // R(-pos) dy
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = g0[e], v = g1[e];
                    g0[e] = u * cs[e] + v * sn[e];
                    g1[e] = v * cs[e] - u * sn[e];
                }
            }
            if (w != nullptr) {
                Raw8<T> xa, xb;
                float x0[8], x1[8], ss = 0.f, dot = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    xa.u[v] = queue.get(stage, 2 * NV + v);
                    xb.u[v] = queue.get(stage, 3 * NV + v);
                }
                xa.get(x0);
                xb.get(x1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
                    dot = fmaf(g0[e] * w0[e], x0[e], fmaf(g1[e] * w1[e], x1[e], dot));
                }
                const float r = rsqrtf(row_sum<CH>(ss) * (1.f / DH) + p.eps);
                const float rm = r * row_sum<CH>(dot) * r * (1.f / DH);      // r * mean(n' (.) xh)
                if (ok) {                               // (a row past the end would add 0 * rsqrt(eps))
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float h0 = x0[e] * r, h1 = x1[e] * r;
                        dw[e] = fmaf(g0[e], h0, dw[e]);
                        dw[8 + e] = fmaf(g1[e], h1, dw[8 + e]);
                        g0[e] = fmaf(r, g0[e] * w0[e], -h0 * rm);
                        g1[e] = fmaf(r, g1[e] * w1[e], -h1 * rm);
                    }
                }
            }
            stage = (stage + 1) % DEPTH;
            if (ok) {
                T* d = dx + ((long long)n * nh + h) * DH + 8 * c;
                ga.put(g0);
                gb.put(g1);
                ga.st(d);
                gb.st(d + HALF);
            }
        }
    }
    queue.template wait<0>();
    if (w == nullptr) return;
    __syncthreads();                                    // the queue becomes the rows' sums [row][element]
    float* s_sum = reinterpret_cast<float*>(s_queue);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        s_sum[row * DH + 8 * c + e] = dw[e];
        s_sum[row * DH + HALF + 8 * c + e] = dw[8 + e];
    }
    __syncthreads();
    if (tid < DH) {
        float s = 0.f;
        for (int r = 0; r < ROWS; ++r) s += s_sum[r * DH + tid];
        p.part[(size_t)blockIdx.x * DH + tid] = s;
    }
}

// Sum of the CTAs' partial gain gradients: grid (d/32, 2), block (32, 32); rows [0, ctas_q) are the
// queries', the others the keys'
__global__ void __launch_bounds__(1024) k_qk_norm_dw(const float* part, int ctas_q, int ctas, int d, float* dwq,
                                                     float* dwk) {
    __shared__ float s_sum[32][33];
    grid_dep_wait();
    float* out = blockIdx.y ? dwk : dwq;
    if (out == nullptr) return;
    const int e = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    for (int r = (blockIdx.y ? ctas_q : 0) + threadIdx.y; r < (blockIdx.y ? ctas : ctas_q); r += 32)
        s += part[(size_t)r * d + e];
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
        for (int r = 1; r < 32; ++r) s += s_sum[r][threadIdx.x];
        out[e] = s;
    }
}

namespace {

int head_quads(const QkNormParams& p) {
    return (p.q ? (p.H + kNormHeads - 1) / kNormHeads : 0) + (p.k ? (p.Hkv + kNormHeads - 1) / kNormHeads : 0);
}

template <typename T, int DH> cudaError_t fwd(const QkNormParams& p, cudaStream_t s) {
    constexpr int TOK = norm_tokens<DH, kNth>(), smem = NormTile<T, DH, kNth>::Queue::kBytes;
    const long long tiles = (p.N + TOK - 1) / TOK;
    // few tokens: the heads are split over CTAs too, until there is about one for each SM
    const int quads = head_quads(p);
    const int split = (int)(tiles >= 148 ? 1 : (quads < 148 / tiles ? quads : 148 / tiles));
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
        return (int)(heads == 0 ? 0 : n < 1 ? 1 : n < tiles ? n : tiles);
    };
    const int ctas_q = most(nq), ctas = ctas_q + most(nk);
    cudaError_t e = cudaFuncSetAttribute(k_qk_norm_bwd<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    {
        UA_PROFILE("k_qk_norm_bwd", s);
        e = launch_dependent(k_qk_norm_bwd<T, DH>, dim3(ctas), dim3(kNth), smem, s, p, ctas_q);
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
