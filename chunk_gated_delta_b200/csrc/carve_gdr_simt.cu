// Scalar-gated delta rule on the CUDA cores, fp32 throughout (include/carve_mixers.h): the path
// of fp32 tensors, and the step by which single tokens are decoded.
//
// Chunks of C = 32 tokens with start state S0 and G_t = sum of log a over the chunk up to t:
//   M[t,s] = w_t e^{G_t - G_s} k_t.k_s (s < t),  Tm = (I + M)^-1,  A[t,s] = e^{G_t - G_s} q_t.k_s (s <= t)
//   R = V - e^G K S0^T,  U = Tm (w R),  O = e^G Q S0^T + A U,  S1 = e^{G_C} S0 + (e^{G_C - G} U)^T K
// Every decay factor is applied as e^{difference <= 0}, so nothing overflows at any decay.
// Tm and A need no state: they are formed for all chunks at once (prep), then one CTA per
// (sequence, head, 32 value rows) carries its rows of the state through the chunks (sweep).
// The backward is the adjoint: a reverse sweep carries dS (it needs only Tm, A, K, Q, dO), and
// the gradients of q, k and the gates, which need S0, dS1 and U, are formed for all chunks at
// once from what the two sweeps stored:
//   dU = A^T dO + e^{G_C - G} K dS1^T,  dY = Tm^T dU,  dV = w dY,
//   dS0 = e^{G_C} dS1 + (e^G dO)^T Q - (w e^G dY)^T K
// Rows past a sequence's end are inert: q = k = v = dO = 0, log a = 0, w = 0.
#include "carve_mixers.cuh"

namespace carve {

__device__ int g_gdr_bad_seqlens;   // set when a packed sequence's offsets are out of range

int gdr_take_bad_seqlens() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gdr_bad_seqlens, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_gdr_bad_seqlens, &z, sizeof(int));
    }
    return v;
}

namespace {

constexpr int C = 32;          // tokens of a chunk
constexpr int NT = 256;        // threads of a CTA, as 16 x 16
constexpr int LC = C + 1;      // row stride of [C][C] and [C][32] tiles

// per-tile operands (floats): Tm [C][C], A [C][C], G [C], w [C]
constexpr int kPrep = 2 * C * C + 2 * C;

// acc[i][j] += sum_x fa(ty + 16 i, x) fb(tx + 16 j, x): a 32 x (16 NJ) product over X terms
template <int NJ, int X, class FA, class FB>
__device__ __forceinline__ void mm(float (&acc)[2][NJ], FA fa, FB fb) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll 4
    for (int x = 0; x < X; ++x) {
        const float a0 = fa(ty, x), a1 = fa(ty + 16, x);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float b = fb(tx + 16 * j, x);
            acc[0][j] = fmaf(a0, b, acc[0][j]);
            acc[1][j] = fmaf(a1, b, acc[1][j]);
        }
    }
}
// f(row, column, acc) over the same product's elements
template <int NJ, class F>
__device__ __forceinline__ void each(float (&acc)[2][NJ], F f) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) f(ty + 16 * i, tx + 16 * j, acc[i][j]);
}
template <int NJ>
__device__ __forceinline__ void zero(float (&acc)[2][NJ]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[0][j] = acc[1][j] = 0.f;
}

// rows t < n of W columns (col0 ..) of a token tensor [rows, H, width], rows beyond as zero
template <class IO>
__device__ __forceinline__ void load_tile(float *dst, int ld, const void *src, long long row0, int n, int H, int h,
                                          int width, int col0, int W) {
    const IO *s = static_cast<const IO *>(src);
    for (int i = threadIdx.x; i < C * W; i += NT) {
        const int t = i / W, x = i - t * W;
        dst[t * ld + x] = t < n ? ld_io(s + ((size_t)(row0 + t) * H + h) * width + col0 + x) : 0.f;
    }
}
__device__ __forceinline__ void load_f32(float *dst, int ld, const float *src, int rows, int W) {
    for (int i = threadIdx.x; i < rows * W; i += NT) dst[(i / W) * ld + i % W] = src[i];
}

// prep: Tm, A, G, w of one tile and value head
template <int K, class IO>
__global__ void __launch_bounds__(NT) gdr_simt_prep(GdrArgs a) {
    __shared__ float k[C][K + 1], q[C][K + 1], M[C][LC], X[C][LC], G[C], w[C];
    const int tile = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, tid = threadIdx.x;
    int n, c, len;
    long long row0;
    if (!a.seq.find(tile, C, n, c, row0, len)) return;
    row0 += (long long)c * C;
    const int m = min(C, len - c * C), hk = h / (a.Hv / a.Hk);
    load_tile<IO>(&k[0][0], K + 1, a.k, row0, m, a.Hk, hk, K, 0, K);
    load_tile<IO>(&q[0][0], K + 1, a.q, row0, m, a.Hk, hk, K, 0, K);
    if (tid < C) {
        float la = 0.f, ww = 0.f;
        if (tid < m) {
            const size_t at = (size_t)(row0 + tid) * a.Hv + h;
            const float x = ld_io(static_cast<const IO *>(a.g_logit) + at) + (a.tau ? a.tau[h] : 0.f);
            la = -decay_amp(a.A_dec, h) * softplus_f(x);
            ww = sigmoid_f(ld_io(static_cast<const IO *>(a.w_logit) + at));
        }
#pragma unroll
        for (int off = 1; off < C; off <<= 1) {
            const float up = __shfl_up_sync(0xffffffffu, la, off);
            if (tid >= off) la += up;
        }
        G[tid] = la;
        w[tid] = ww;
    }
    __syncthreads();
    float *out = reinterpret_cast<float *>(a.prep) + ((size_t)tile * a.Hv + h) * kPrep;
    float acc[2][2];
    zero(acc);
    mm<2, K>(acc, [&](int t, int x) { return k[t][x]; }, [&](int s, int x) { return k[s][x]; });
    each(acc, [&](int t, int s, float x) { M[t][s] = s < t ? w[t] * expf(G[t] - G[s]) * x : 0.f; });
    zero(acc);
    mm<2, K>(acc, [&](int t, int x) { return q[t][x]; }, [&](int s, int x) { return k[s][x]; });
    each(acc, [&](int t, int s, float x) { out[C * C + t * C + s] = s <= t ? expf(G[t] - G[s]) * x : 0.f; });
    __syncthreads();
    if (tid < C) {   // column tid of Tm by forward substitution
        for (int t = 0; t < C; ++t) {
            float x = t == tid ? 1.f : 0.f;
            for (int s = 0; s < t; ++s) x -= M[t][s] * X[s][tid];
            X[t][tid] = x;
        }
        out[2 * C * C + tid] = G[tid];
        out[2 * C * C + C + tid] = w[tid];
    }
    __syncthreads();
    each(acc, [&](int t, int s, float) { out[t * C + s] = X[t][s]; });
}

template <int K>
struct SweepSmem {
    float k[C][K + 1], q[C][K + 1], S[32][K + 1], Tm[C][LC], A[C][LC], v[C][LC], y[C][LC], u[C][LC], G[C], w[C];
};

// tiles of the sweeps: K, Q, Tm, A, G, w of (tile, h)
template <int K, class IO>
__device__ __forceinline__ void load_common(SweepSmem<K> &sm, const GdrArgs &a, long long tile, long long row, int m,
                                            int h) {
    const int hk = h / (a.Hv / a.Hk);
    load_tile<IO>(&sm.k[0][0], K + 1, a.k, row, m, a.Hk, hk, K, 0, K);
    load_tile<IO>(&sm.q[0][0], K + 1, a.q, row, m, a.Hk, hk, K, 0, K);
    const float *p = reinterpret_cast<const float *>(a.prep) + ((size_t)tile * a.Hv + h) * kPrep;
    load_f32(&sm.Tm[0][0], LC, p, C, C);
    load_f32(&sm.A[0][0], LC, p + C * C, C, C);
    if (threadIdx.x < C) {
        sm.G[threadIdx.x] = p[2 * C * C + threadIdx.x];
        sm.w[threadIdx.x] = p[2 * C * C + C + threadIdx.x];
    }
}

// forward sweep of 32 value rows of one (sequence, head); saved: per tile S0 [V][K] and U [C][V]
template <int K, int V, class IO>
__global__ void __launch_bounds__(NT) gdr_simt_sweep(GdrArgs a, bool save) {
    extern __shared__ __align__(16) unsigned char raw[];
    SweepSmem<K> &sm = *reinterpret_cast<SweepSmem<K> *>(raw);
    constexpr int NK = K / 16;
    const int v0 = (blockIdx.x % (V / 32)) * 32, unit = blockIdx.x / (V / 32), h = unit % a.Hv, n = unit / a.Hv;
    long long row0;
    int len;
    a.seq.rows(n, row0, len, threadIdx.x == 0 ? &g_gdr_bad_seqlens : nullptr);
    const size_t st = ((size_t)unit * V + v0) * K;
    for (int i = threadIdx.x; i < 32 * K; i += NT) sm.S[i / K][i % K] = a.S0 ? a.S0[st + i] : 0.f;
    const long long t0 = a.seq.tile0(n, C);
    for (int c = 0; c * C < len; ++c) {
        const int m = min(C, len - c * C);
        const long long tile = t0 + c, row = row0 + (long long)c * C;
        __syncthreads();
        load_common<K, IO>(sm, a, tile, row, m, h);
        load_tile<IO>(&sm.v[0][0], LC, a.v, row, m, a.Hv, h, V, v0, 32);
        __syncthreads();
        if (save) {
            float *s0 = reinterpret_cast<float *>(a.saved) + ((size_t)tile * a.Hv + h) * ((size_t)V * K + C * V);
            for (int i = threadIdx.x; i < 32 * K; i += NT) s0[(size_t)v0 * K + i] = sm.S[i / K][i % K];
        }
        float acc[2][2];
        zero(acc);
        mm<2, K>(acc, [&](int t, int x) { return sm.k[t][x]; }, [&](int v, int x) { return sm.S[v][x]; });
        each(acc, [&](int t, int v, float x) { sm.y[t][v] = sm.w[t] * (sm.v[t][v] - expf(sm.G[t]) * x); });
        __syncthreads();
        zero(acc);
        mm<2, C>(acc, [&](int t, int s) { return sm.Tm[t][s]; }, [&](int v, int s) { return sm.y[s][v]; });
        each(acc, [&](int t, int v, float x) { sm.u[t][v] = x; });
        __syncthreads();
        if (save) {
            float *u = reinterpret_cast<float *>(a.saved) + ((size_t)tile * a.Hv + h) * ((size_t)V * K + C * V) + (size_t)V * K;
            each(acc, [&](int t, int v, float x) { u[t * V + v0 + v] = x; });
        }
        zero(acc);
        mm<2, K>(acc, [&](int t, int x) { return sm.q[t][x]; }, [&](int v, int x) { return sm.S[v][x]; });
        each(acc, [&](int t, int, float &x) { x *= expf(sm.G[t]); });
        mm<2, C>(acc, [&](int t, int s) { return sm.A[t][s]; }, [&](int v, int s) { return sm.u[s][v]; });
        each(acc, [&](int t, int v, float x) {
            if (t < m) st_io(static_cast<IO *>(a.o) + ((size_t)(row + t) * a.Hv + h) * V + v0 + v, x);
        });
        __syncthreads();
        const float gl = sm.G[C - 1];
        float s1[2][NK];
        each(s1, [&](int v, int x, float &s) { s = expf(gl) * sm.S[v][x]; });
        mm<NK, C>(s1, [&](int v, int t) { return sm.u[t][v] * expf(gl - sm.G[t]); }, [&](int x, int t) { return sm.k[t][x]; });
        each(s1, [&](int v, int x, float s) { sm.S[v][x] = s; });
    }
    __syncthreads();
    if (a.S_final)
        for (int i = threadIdx.x; i < 32 * K; i += NT) a.S_final[st + i] = sm.S[i / K][i % K];
}

// reverse sweep of 32 value rows; ws: per tile dS1 [V][K] and dY [C][V]
template <int K, int V, class IO>
__global__ void __launch_bounds__(NT) gdr_simt_bsweep(GdrArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    SweepSmem<K> &sm = *reinterpret_cast<SweepSmem<K> *>(raw);
    constexpr int NK = K / 16;
    const int v0 = (blockIdx.x % (V / 32)) * 32, unit = blockIdx.x / (V / 32), h = unit % a.Hv, n = unit / a.Hv;
    long long row0;
    int len;
    a.seq.rows(n, row0, len, threadIdx.x == 0 ? &g_gdr_bad_seqlens : nullptr);
    const size_t st = ((size_t)unit * V + v0) * K;
    for (int i = threadIdx.x; i < 32 * K; i += NT) sm.S[i / K][i % K] = a.dS_final ? a.dS_final[st + i] : 0.f;
    const long long t0 = a.seq.tile0(n, C);
    for (int c = (len + C - 1) / C - 1; c >= 0; --c) {
        const int m = min(C, len - c * C);
        const long long tile = t0 + c, row = row0 + (long long)c * C;
        __syncthreads();
        load_common<K, IO>(sm, a, tile, row, m, h);
        load_tile<IO>(&sm.v[0][0], LC, a.dO, row, m, a.Hv, h, V, v0, 32);   // sm.v = dO
        __syncthreads();
        float *out = reinterpret_cast<float *>(a.ws) + ((size_t)tile * a.Hv + h) * ((size_t)V * K + C * V);
        for (int i = threadIdx.x; i < 32 * K; i += NT) out[(size_t)v0 * K + i] = sm.S[i / K][i % K];
        const float gl = sm.G[C - 1];
        float acc[2][2];
        zero(acc);
        mm<2, K>(acc, [&](int t, int x) { return sm.k[t][x]; }, [&](int v, int x) { return sm.S[v][x]; });
        each(acc, [&](int t, int, float &x) { x *= expf(gl - sm.G[t]); });
        mm<2, C>(acc, [&](int t, int s) { return sm.A[s][t]; }, [&](int v, int s) { return sm.v[s][v]; });
        each(acc, [&](int t, int v, float x) { sm.u[t][v] = x; });   // dU
        __syncthreads();
        zero(acc);
        mm<2, C>(acc, [&](int t, int s) { return sm.Tm[s][t]; }, [&](int v, int s) { return sm.u[s][v]; });
        each(acc, [&](int t, int v, float x) {
            out[(size_t)V * K + t * V + v0 + v] = x;
            sm.y[t][v] = sm.w[t] * x;   // dV
            if (t < m) st_io(static_cast<IO *>(a.dv) + ((size_t)(row + t) * a.Hv + h) * V + v0 + v, sm.w[t] * x);
        });
        __syncthreads();
        float s0[2][NK];
        each(s0, [&](int v, int x, float &s) { s = expf(gl) * sm.S[v][x]; });
        mm<NK, C>(s0, [&](int v, int t) { return sm.v[t][v] * expf(sm.G[t]); }, [&](int x, int t) { return sm.q[t][x]; });
        mm<NK, C>(s0, [&](int v, int t) { return -sm.y[t][v] * expf(sm.G[t]); }, [&](int x, int t) { return sm.k[t][x]; });
        each(s0, [&](int v, int x, float s) { sm.S[v][x] = s; });
    }
    __syncthreads();
    if (a.dS0)
        for (int i = threadIdx.x; i < 32 * K; i += NT) a.dS0[st + i] = sm.S[i / K][i % K];
}

template <int K, int V>
struct GradSmem {
    float k[C][K + 1], q[C][K + 1], S[V][K], dO[C][V + 1], dY[C][V + 1], U[C][V + 1], v[C][V + 1];
    float P1[C][LC], P2[C][LC], kk[C][LC], row[4][C], G[C], w[C], red[NT / 32];
};

// sum over the 16 lanes that share a row of the 16 x 16 thread grid
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// gradients of q, k (summed over the value heads of a key head, in order) and of the gates
template <int K, int V, class IO>
__global__ void __launch_bounds__(NT) gdr_simt_grad(GdrArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<K, V> &sm = *reinterpret_cast<GradSmem<K, V> *>(raw);
    constexpr int NK = K / 16;
    const int tile = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk, share = a.Hv / a.Hk, tid = threadIdx.x;
    int n, c, len;
    long long row;
    if (!a.seq.find(tile, C, n, c, row, len)) {
        if (a.dA_dec || a.dtau) {   // unused numbers count as zero in the fixed-order sums
            float *p = reinterpret_cast<float *>(a.ws) + (size_t)a.seq.n_tiles(C) * a.Hv * ((size_t)V * K + C * V);
            for (int i = tid; i < 2 * share; i += NT) p[((size_t)tile * a.Hv + hk * share) * 2 + i] = 0.f;
        }
        return;
    }
    row += (long long)c * C;
    const int m = min(C, len - c * C);
    load_tile<IO>(&sm.k[0][0], K + 1, a.k, row, m, a.Hk, hk, K, 0, K);
    load_tile<IO>(&sm.q[0][0], K + 1, a.q, row, m, a.Hk, hk, K, 0, K);
    float dq[2][NK], dk[2][NK];
    zero(dq);
    zero(dk);
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        const size_t slot = (size_t)tile * a.Hv + h, per = (size_t)V * K + C * V;
        const float *fwd = reinterpret_cast<const float *>(a.saved) + slot * per;
        const float *bwd = reinterpret_cast<const float *>(a.ws) + slot * per;
        const float *prep = reinterpret_cast<const float *>(a.prep) + slot * kPrep;
        __syncthreads();
        load_tile<IO>(&sm.dO[0][0], V + 1, a.dO, row, m, a.Hv, h, V, 0, V);
        load_tile<IO>(&sm.v[0][0], V + 1, a.v, row, m, a.Hv, h, V, 0, V);
        load_f32(&sm.dY[0][0], V + 1, bwd + (size_t)V * K, C, V);
        load_f32(&sm.U[0][0], V + 1, fwd + (size_t)V * K, C, V);
        load_f32(&sm.S[0][0], K, fwd, V, K);
        if (tid < C) {
            sm.G[tid] = prep[2 * C * C + tid];
            sm.w[tid] = prep[2 * C * C + C + tid];
        }
        __syncthreads();
        const float gl = sm.G[C - 1];
        float acc[2][2], x1[2][NK];
        // per-row partial sums of this thread's two rows: gate gradients
        float dG[2] = {0.f, 0.f}, dw[2] = {0.f, 0.f}, kb[2] = {0.f, 0.f}, lastp = 0.f;
        // the products with the chunk's start state
        zero(x1);
        mm<NK, V>(x1, [&](int t, int v) { return sm.dO[t][v]; }, [&](int x, int v) { return sm.S[v][x]; });
        each(x1, [&](int t, int x, float &y) { y *= expf(sm.G[t]); });
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int t = tid / 16 + 16 * i, x = tid % 16 + 16 * j;
                dq[i][j] += x1[i][j];
                dG[i] += sm.q[t][x] * x1[i][j];
            }
        zero(x1);
        mm<NK, V>(x1, [&](int t, int v) { return sm.dY[t][v]; }, [&](int x, int v) { return sm.S[v][x]; });
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int t = tid / 16 + 16 * i, x = tid % 16 + 16 * j;
                const float y = expf(sm.G[t]) * x1[i][j];
                dk[i][j] -= sm.w[t] * y;
                dw[i] -= sm.k[t][x] * y;
                dG[i] -= sm.w[t] * sm.k[t][x] * y;
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            for (int v = tid % 16; v < V; v += 16) dw[i] += sm.dY[tid / 16 + 16 * i][v] * sm.v[tid / 16 + 16 * i][v];
        // <S0, dS1>, then dS1 in place of S0
        for (int i = tid; i < V * K; i += NT) lastp += sm.S[i / K][i % K] * bwd[i];
        lastp *= expf(gl);
        __syncthreads();
        load_f32(&sm.S[0][0], K, bwd, V, K);
        __syncthreads();
        zero(x1);
        mm<NK, V>(x1, [&](int t, int v) { return sm.U[t][v]; }, [&](int x, int v) { return sm.S[v][x]; });
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int t = tid / 16 + 16 * i, x = tid % 16 + 16 * j;
                const float y = expf(gl - sm.G[t]) * x1[i][j];
                dk[i][j] += y;
                kb[i] += sm.k[t][x] * y;
            }
        // the products within the chunk
        zero(acc);
        mm<2, K>(acc, [&](int t, int x) { return sm.k[t][x]; }, [&](int s, int x) { return sm.k[s][x]; });
        each(acc, [&](int t, int s, float x) { sm.kk[t][s] = x; });
        float kq[2][2];
        zero(kq);
        mm<2, K>(kq, [&](int t, int x) { return sm.q[t][x]; }, [&](int s, int x) { return sm.k[s][x]; });
        zero(acc);
        mm<2, V>(acc, [&](int t, int v) { return sm.dO[t][v]; }, [&](int s, int v) { return sm.U[s][v]; });
        float pr[2][2];   // contributions of the pairs (t, s < t), whose factor is e^{G_t - G_s}
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = tid / 16 + 16 * i, s = tid % 16 + 16 * j;
                const float p = s <= t ? acc[i][j] * expf(sm.G[t] - sm.G[s]) : 0.f;
                sm.P1[t][s] = p;
                pr[i][j] = s < t ? p * kq[i][j] : 0.f;
            }
        zero(acc);
        mm<2, V>(acc, [&](int t, int v) { return sm.dY[t][v]; }, [&](int s, int v) { return sm.U[s][v]; });
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = tid / 16 + 16 * i, s = tid % 16 + 16 * j;
                const float p = s < t ? -acc[i][j] * expf(sm.G[t] - sm.G[s]) : 0.f;
                dw[i] += p * sm.kk[t][s];
                sm.P2[t][s] = sm.w[t] * p;
                pr[i][j] += sm.w[t] * p * sm.kk[t][s];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) sm.kk[tid / 16 + 16 * i][tid % 16 + 16 * j] = pr[i][j];
        mm<NK, C>(dq, [&](int t, int s) { return sm.P1[t][s]; }, [&](int x, int s) { return sm.k[s][x]; });
        mm<NK, C>(dk, [&](int t, int s) { return sm.P2[t][s] + sm.P2[s][t]; }, [&](int x, int s) { return sm.k[s][x]; });
        mm<NK, C>(dk, [&](int t, int s) { return sm.P1[s][t]; }, [&](int x, int s) { return sm.q[s][x]; });
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float g = sum16(dG[i]), ww = sum16(dw[i]), b = sum16(kb[i]);
            if (tid % 16 == 0) {
                sm.row[0][tid / 16 + 16 * i] = g;
                sm.row[1][tid / 16 + 16 * i] = ww;
                sm.row[2][tid / 16 + 16 * i] = b;
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) lastp += __shfl_xor_sync(0xffffffffu, lastp, off);
        if (tid % 32 == 0) sm.red[tid / 32] = lastp;
        __syncthreads();
        if (tid < C) {
            // Gradient of log a_t: the sum over every path that crosses the decay of token t, each
            // term as it is (rows minus columns of a cumulative sum would cancel): queries and
            // keys r >= t that read the start state, keys s < t that reach the end, S0 itself,
            // and pairs r >= t > s.
            float run = 0.f;   // row tid of the pairs: sums over s < t
            for (int t = 0; t < C; ++t) {
                const float p = sm.kk[tid][t];
                sm.kk[tid][t] = run;
                run += p;
            }
            __syncwarp();
            float g = sm.row[0][tid], b = sm.row[2][tid];
#pragma unroll
            for (int off = 1; off < C; off <<= 1) {
                const float dn = __shfl_down_sync(0xffffffffu, g, off), up = __shfl_up_sync(0xffffffffu, b, off);
                if (tid + off < C) g += dn;
                if (tid >= off) b += up;
            }
            b = __shfl_up_sync(0xffffffffu, b, 1);
            if (tid > 0) g += b;
            for (int i = 0; i < NT / 32; ++i) g += sm.red[i];
            for (int r = tid; r < C; ++r) g += sm.kk[r][tid];
            float dlog = 0.f, damp = 0.f;
            if (tid < m) {
                const size_t at = (size_t)(row + tid) * a.Hv + h;
                const float x = ld_io(static_cast<const IO *>(a.g_logit) + at) + (a.tau ? a.tau[h] : 0.f);
                const float amp = decay_amp(a.A_dec, h), w = sm.w[tid];
                dlog = -amp * sigmoid_f(x) * g;
                damp = -amp * softplus_f(x) * g;
                st_io(static_cast<IO *>(a.dg_logit) + at, dlog);
                st_io(static_cast<IO *>(a.dw_logit) + at, sm.row[1][tid] * w * (1.f - w));
            }
            if (a.dA_dec || a.dtau) {
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1) {
                    dlog += __shfl_xor_sync(0xffffffffu, dlog, off);
                    damp += __shfl_xor_sync(0xffffffffu, damp, off);
                }
                if (tid == 0) {
                    float *p = reinterpret_cast<float *>(a.ws) + (size_t)a.seq.n_tiles(C) * a.Hv * per + slot * 2;
                    p[0] = damp;
                    p[1] = dlog;
                }
            }
        }
    }
    each(dq, [&](int t, int x, float y) {
        if (t < m) st_io(static_cast<IO *>(a.dq) + ((size_t)(row + t) * a.Hk + hk) * K + x, y);
    });
    each(dk, [&](int t, int x, float y) {
        if (t < m) st_io(static_cast<IO *>(a.dk) + ((size_t)(row + t) * a.Hk + hk) * K + x, y);
    });
}

}  // namespace

// dA_dec, dtau of head blockIdx.x: the tiles' partial sums [tiles][Hv][2], in a fixed order
__global__ void __launch_bounds__(256) gdr_reduce_decay(const float *p, long long tiles, int Hv, float *dA_dec,
                                                        float *dtau) {
    __shared__ float red[2][256];
    float x = 0.f, y = 0.f;
    for (long long t = threadIdx.x; t < tiles; t += 256) {
        x += p[(t * Hv + blockIdx.x) * 2];
        y += p[(t * Hv + blockIdx.x) * 2 + 1];
    }
    red[0][threadIdx.x] = x;
    red[1][threadIdx.x] = y;
    for (int off = 128; off >= 1; off >>= 1) {
        __syncthreads();
        if (threadIdx.x < off) {
            red[0][threadIdx.x] += red[0][threadIdx.x + off];
            red[1][threadIdx.x] += red[1][threadIdx.x + off];
        }
    }
    if (threadIdx.x == 0) {
        if (dA_dec) dA_dec[blockIdx.x] = red[0][0];
        if (dtau) dtau[blockIdx.x] = red[1][0];
    }
}

void launch_gdr_reduce_decay(const float *p, long long tiles, int Hv, float *dA_dec, float *dtau, cudaStream_t st) {
    gdr_reduce_decay<<<Hv, 256, 0, st>>>(p, tiles, Hv, dA_dec, dtau);
}

GdrSizes gdr_simt_sizes(const Seqs &s, int Hv, int K, int V) {
    const size_t slots = (size_t)s.n_tiles(C) * Hv, per = sizeof(float) * ((size_t)V * K + C * V);
    return {sizeof(float) * slots * kPrep, slots * per, slots * (per + 2 * sizeof(float))};
}

namespace {

template <int K, int V, class IO>
cudaError_t fwd_t(const GdrArgs &a, bool save, cudaStream_t st) {
    const long long tiles = a.seq.n_tiles(C);
    if (tiles) gdr_simt_prep<K, IO><<<(unsigned)(tiles * a.Hv), NT, 0, st>>>(a);
    auto kern = gdr_simt_sweep<K, V, IO>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), sizeof(SweepSmem<K>));
    if (e != cudaSuccess) return e;
    kern<<<a.seq.N * a.Hv * (V / 32), NT, sizeof(SweepSmem<K>), st>>>(a, save);
    return cudaGetLastError();
}

template <int K, int V, class IO>
cudaError_t bwd_t(const GdrArgs &a, cudaStream_t st) {
    auto sweep = gdr_simt_bsweep<K, V, IO>;
    auto grad = gdr_simt_grad<K, V, IO>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(sweep), sizeof(SweepSmem<K>));
    if (e == cudaSuccess) e = set_smem_once(reinterpret_cast<const void *>(grad), sizeof(GradSmem<K, V>));
    if (e != cudaSuccess) return e;
    const long long tiles = a.seq.n_tiles(C);
    sweep<<<a.seq.N * a.Hv * (V / 32), NT, sizeof(SweepSmem<K>), st>>>(a);
    if (tiles) grad<<<(unsigned)(tiles * a.Hk), NT, sizeof(GradSmem<K, V>), st>>>(a);
    if (a.dA_dec || a.dtau)
        launch_gdr_reduce_decay(reinterpret_cast<const float *>(a.ws) + (size_t)tiles * a.Hv * ((size_t)V * K + C * V), tiles, a.Hv,
                                a.dA_dec, a.dtau, st);
    return cudaGetLastError();
}

template <class F>
cudaError_t by_shape(int K, int V, F f) {
    if (K == 64) return V == 64 ? f.template operator()<64, 64>() : f.template operator()<64, 128>();
    return V == 64 ? f.template operator()<128, 64>() : f.template operator()<128, 128>();
}

struct Fwd {
    const GdrArgs &a;
    bool save;
    cudaStream_t st;
    template <int K, int V>
    cudaError_t operator()() const {
        return fwd_t<K, V, float>(a, save, st);
    }
};
struct Bwd {
    const GdrArgs &a;
    cudaStream_t st;
    template <int K, int V>
    cudaError_t operator()() const {
        return bwd_t<K, V, float>(a, st);
    }
};

// One token: 32 value rows of one (batch element, head) per CTA of 128 threads; the 8 lanes of an
// octet share a row pair (rows r, r + 16) and hold float4 columns seg, seg + 8, ...  The state is
// read once and written once from registers.
template <int K, int V, class IO>
__global__ void __launch_bounds__(128) gdr_step_kernel(GdrArgs a) {
    constexpr int CP = K / 32;
    const int v0 = (blockIdx.x % (V / 32)) * 32, unit = blockIdx.x / (V / 32), h = unit % a.Hv, b = unit / a.Hv;
    const int hk = h / (a.Hv / a.Hk), seg = threadIdx.x % 8, r = threadIdx.x / 8;
    float4 *S = reinterpret_cast<float4 *>(a.S_final) + ((size_t)unit * V + v0 + r) * (K / 4) + seg;
    float4 s[2][CP];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < CP; ++j) s[i][j] = __ldcs(S + i * 16 * (K / 4) + 8 * j);
    const float x = ld_io(static_cast<const IO *>(a.g_logit) + unit) + (a.tau ? a.tau[h] : 0.f);
    const float al = expf(-decay_amp(a.A_dec, h) * softplus_f(x));
    const float w = sigmoid_f(ld_io(static_cast<const IO *>(a.w_logit) + unit));
    const IO *kp = static_cast<const IO *>(a.k) + ((size_t)b * a.Hk + hk) * K, *qp = static_cast<const IO *>(a.q) + ((size_t)b * a.Hk + hk) * K;
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = ld_io(static_cast<const IO *>(a.v) + (size_t)unit * V + v0 + r + 16 * i);
    float4 k[CP], q[CP];
#pragma unroll
    for (int j = 0; j < CP; ++j) {
        const int c = 4 * (seg + 8 * j);
        k[j] = make_float4(ld_io(kp + c), ld_io(kp + c + 1), ld_io(kp + c + 2), ld_io(kp + c + 3));
        q[j] = make_float4(ld_io(qp + c), ld_io(qp + c + 1), ld_io(qp + c + 2), ld_io(qp + c + 3));
    }
    float ks[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            s[i][j].x *= al;
            s[i][j].y *= al;
            s[i][j].z *= al;
            s[i][j].w *= al;
            ks[i] += s[i][j].x * k[j].x + s[i][j].y * k[j].y + s[i][j].z * k[j].z + s[i][j].w * k[j].w;
        }
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) ks[i] += __shfl_xor_sync(0xffffffffu, ks[i], off);
    float o[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float u = w * (v[i] - ks[i]);
#pragma unroll
        for (int j = 0; j < CP; ++j) {
            float4 y = s[i][j];
            y.x += u * k[j].x;
            y.y += u * k[j].y;
            y.z += u * k[j].z;
            y.w += u * k[j].w;
            __stcs(S + i * 16 * (K / 4) + 8 * j, y);
            o[i] += y.x * q[j].x + y.y * q[j].y + y.z * q[j].z + y.w * q[j].w;
        }
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], off);
    if (seg == 0) {
        st_io(static_cast<IO *>(a.o) + (size_t)unit * V + v0 + r, o[0]);
        st_io(static_cast<IO *>(a.o) + (size_t)unit * V + v0 + r + 16, o[1]);
    }
}

struct Step {
    const GdrArgs &a;
    bool bf16;
    cudaStream_t st;
    template <int K, int V>
    cudaError_t operator()() const {
        const unsigned grid = (unsigned)((long long)a.seq.N * a.Hv * (V / 32));
        if (bf16)
            gdr_step_kernel<K, V, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
        else
            gdr_step_kernel<K, V, float><<<grid, 128, 0, st>>>(a);
        return cudaGetLastError();
    }
};

}  // namespace

cudaError_t launch_gdr_fwd_simt(int K, int V, const GdrArgs &a, bool save, cudaStream_t st) {
    return by_shape(K, V, Fwd{a, save, st});
}
cudaError_t launch_gdr_bwd_simt(int K, int V, const GdrArgs &a, cudaStream_t st) {
    return by_shape(K, V, Bwd{a, st});
}
cudaError_t launch_gdr_step(int K, int V, bool bf16, const GdrArgs &a, cudaStream_t st) {
    return by_shape(K, V, Step{a, bf16, st});
}

}  // namespace carve
