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

// grid (token tiles of 16, head splits), 64 * DH/16 threads
template <typename T, int DH>
__global__ void __launch_bounds__(4 * DH) k_qk_norm_fwd(QkNormParams p) {
    constexpr int HALF = DH / 2;
    __shared__ float s_cos[kNormTokens * HALF], s_sin[kNormTokens * HALF];
    __shared__ double s_f[HALF];
    grid_dep_wait();
    const long long n0 = (long long)blockIdx.x * kNormTokens;
    float cs[8], sn[8];
    if (p.rope)
        tile_angles<DH>(s_cos, s_sin, n0, p.N, p.rf, s_f,
                        [&](long long n) { return p.pos ? p.pos[n] : (int)(n % p.T); }, cs, sn);
    norm_rope_tile<T, DH>(p, n0, blockIdx.y, gridDim.y, cs, sn);
}

// Backward.  A persistent CTA walks token tiles and keeps the gain gradients of its lanes'
// elements in registers (fp32, one set for queries and one for keys), sums them over its rows in
// shared memory at the end and writes one partial row; k_qk_norm_dw adds the CTAs' rows in a
// fixed order.
template <typename T, int DH>
__global__ void __launch_bounds__(4 * DH) k_qk_norm_bwd(QkNormParams p) {
    constexpr int CH = DH / 16, HALF = DH / 2, NTH = 64 * CH, ROWS = 64;
    __shared__ float s_buf[ROWS * DH / 2];              // angles of a tile, later half of the row sums
    __shared__ double s_f[HALF];
    static_assert(2 * kNormTokens * HALF <= ROWS * DH / 2, "angles fit the buffer");
    float* s_cos = s_buf;
    float* s_sin = s_buf + kNormTokens * HALF;
    grid_dep_wait();
    const int tid = threadIdx.x, c = tid % CH, hp = (tid / CH) % kNormHeads, row = tid / CH;
    float dw[2][16];
#pragma unroll
    for (int e = 0; e < 16; ++e) dw[0][e] = dw[1][e] = 0.f;
    const long long tiles = (p.N + kNormTokens - 1) / kNormTokens;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long long n0 = tile * kNormTokens, n = n0 + row / kNormHeads;
        float cs[8], sn[8];
        if (p.rope) {
            __syncthreads();                            // the last tile's angles have been read
            tile_angles<DH>(s_cos, s_sin, n0, p.N, p.rf, s_f,
                            [&](long long m) { return p.pos ? p.pos[m] : (int)(m % p.T); }, cs, sn);
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {          // queries, then keys
            const T* x = static_cast<const T*>(side ? p.k : p.q);
            if (x == nullptr) continue;
            const T* dy = static_cast<const T*>(side ? p.dk_out : p.dq_out);
            T* dx = static_cast<T*>(side ? p.dk : p.dq);
            const float* w = side ? p.wk : p.wq;
            const int nh = side ? p.Hkv : p.H;
            const long long ld = side ? p.k_ld : p.q_ld;
            float w0[8], w1[8];
            if (w != nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w0[e] = __ldg(w + 8 * c + e);
                    w1[e] = __ldg(w + HALF + 8 * c + e);
                }
            }
            for (int h = hp; h - hp < nh; h += kNormHeads) {
                const bool ok = n < p.N && h < nh;
                const long long at = (n * nh + h) * DH + 8 * c;
                Raw8<T> xa, xb, ga, gb;
                xa.zero(); xb.zero(); ga.zero(); gb.zero();
                if (ok) {
                    const T* s = x + n * ld + (long long)h * DH + 8 * c;
                    ga.ld(dy + at);
                    gb.ld(dy + at + HALF);
                    if (w != nullptr) { xa.ld(s); xb.ld(s + HALF); }
                }
                float g0[8], g1[8];
                ga.get(g0);
                gb.get(g1);
                if (p.rope) {                           // R(-pos) dy
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float u = g0[e], v = g1[e];
                        g0[e] = u * cs[e] + v * sn[e];
                        g1[e] = v * cs[e] - u * sn[e];
                    }
                }
                if (w != nullptr) {
                    float x0[8], x1[8], ss = 0.f, dot = 0.f;
                    xa.get(x0);
                    xb.get(x1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
                        dot = fmaf(g0[e] * w0[e], x0[e], fmaf(g1[e] * w1[e], x1[e], dot));
                    }
                    const float r = rsqrtf(row_sum<CH>(ss) * (1.f / DH) + p.eps);
                    const float mean = row_sum<CH>(dot) * r * (1.f / DH);   // mean(n' (.) xh)
                    if (ok) {                           // (a row past the end would add 0 * rsqrt(eps))
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float h0 = x0[e] * r, h1 = x1[e] * r;
                            dw[side][e] = fmaf(g0[e], h0, dw[side][e]);
                            dw[side][8 + e] = fmaf(g1[e], h1, dw[side][8 + e]);
                            g0[e] = r * (g0[e] * w0[e] - h0 * mean);
                            g1[e] = r * (g1[e] * w1[e] - h1 * mean);
                        }
                    }
                }
                if (ok) {
                    ga.put(g0);
                    gb.put(g1);
                    ga.st(dx + at);
                    gb.st(dx + at + HALF);
                }
            }
        }
    }
    // rows' sums: one half of the elements at a time through the buffer
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        if ((side ? p.wk : p.wq) == nullptr) continue;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) s_buf[row * HALF + 8 * c + e] = dw[side][8 * hf + e];
            __syncthreads();
            if (tid < HALF) {
                float s = 0.f;
                for (int r = 0; r < ROWS; ++r) s += s_buf[r * HALF + tid];
                p.part[((size_t)blockIdx.x * 2 + side) * DH + hf * HALF + tid] = s;
            }
        }
    }
    static_assert(NTH >= HALF, "one thread per element of a half");
}

// Sum of the CTAs' partial gain gradients: grid (d/32, 2), block (32, 16)
__global__ void __launch_bounds__(512) k_qk_norm_dw(const float* part, int rows, int d, float* dwq, float* dwk) {
    __shared__ float s_sum[16][33];
    grid_dep_wait();
    float* out = blockIdx.y ? dwk : dwq;
    if (out == nullptr) return;
    const int e = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    for (int r = threadIdx.y; r < rows; r += 16) s += part[((size_t)r * 2 + blockIdx.y) * d + e];
    s_sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0) {
        for (int r = 1; r < 16; ++r) s += s_sum[r][threadIdx.x];
        out[e] = s;
    }
}

namespace {

int head_quads(const QkNormParams& p) {
    return (p.q ? (p.H + kNormHeads - 1) / kNormHeads : 0) + (p.k ? (p.Hkv + kNormHeads - 1) / kNormHeads : 0);
}

template <typename T, int DH> cudaError_t fwd(const QkNormParams& p, cudaStream_t s) {
    const long long tiles = (p.N + kNormTokens - 1) / kNormTokens;
    // few tokens: the heads are split over CTAs too, until there is about one for each SM
    const int quads = head_quads(p);
    const int split = (int)(tiles >= 148 ? 1 : (quads < 148 / tiles ? quads : 148 / tiles));
    UA_PROFILE("k_qk_norm_fwd", s);
    return launch_dependent(k_qk_norm_fwd<T, DH>, dim3((unsigned)tiles, split < 1 ? 1 : split), dim3(4 * DH), 0, s, p);
}

template <typename T, int DH> cudaError_t bwd(const QkNormParams& p, cudaStream_t s) {
    const long long tiles = (p.N + kNormTokens - 1) / kNormTokens;
    const int ctas = (int)(tiles < kQkNormBwdCtas ? tiles : kQkNormBwdCtas);
    {
        UA_PROFILE("k_qk_norm_bwd", s);
        cudaError_t e = launch_dependent(k_qk_norm_bwd<T, DH>, dim3(ctas), dim3(4 * DH), 0, s, p);
        if (e != cudaSuccess) return e;
    }
    float* dwq = p.q && p.wq ? p.dwq : nullptr;
    float* dwk = p.k && p.wk ? p.dwk : nullptr;
    if (dwq == nullptr && dwk == nullptr) return cudaSuccess;
    UA_PROFILE("k_qk_norm_dw", s);
    return launch_dependent(k_qk_norm_dw, dim3(DH / 32, 2), dim3(32, 16), 0, s, (const float*)p.part, ctas, DH, dwq,
                            dwk);
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
