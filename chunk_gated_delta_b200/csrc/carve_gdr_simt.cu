// Scalar-gated delta rule on the CUDA cores, fp32 throughout (include/carve_mixers.h): the path
// of fp32 tensors, and the step by which single tokens are decoded.
//
// Chunks of C = 32 tokens with start state S0 and G_t = sum of log a over the chunk up to t:
//   M[t,s] = w_t e^{G_t - G_s} k_t.k_s (s < t),  Tm = (I + M)^-1,  A[t,s] = e^{G_t - G_s} q_t.k_s (s <= t)
//   R = V - e^G K S0^T,  U = Tm (w R),  O = e^G Q S0^T + A U,  S1 = e^{G_C} S0 + (e^{G_C - G} U)^T K
// Every decay factor is applied as e^{difference <= 0}, so nothing overflows at any decay.
// Tm and A need no state: they are formed for all chunks at once (prep), then one CTA per
// (sequence, head, 16 value rows) carries its rows of the state through the chunks (sweep).
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

// per-tile operands (floats): Tm [C][C], A [C][C], G [C], w [C], L [C] (G's low part)
constexpr int kPrep = 2 * C * C + 3 * C;

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) { return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c)))); }
// acc[i][j] += <row ty + 16 i of a, row tx + 16 j of b> over X terms (rows 16-byte aligned)
template <int X>
__device__ __forceinline__ void mm_rows(float (&acc)[2][2], const float *a, int lda, const float *b, int ldb) {
    a += threadIdx.x / 16 * lda;
    b += threadIdx.x % 16 * ldb;
#pragma unroll 4
    for (int x = 0; x < X; x += 4) {
        const float4 a0 = *reinterpret_cast<const float4 *>(a + x), a1 = *reinterpret_cast<const float4 *>(a + 16 * lda + x);
        const float4 b0 = *reinterpret_cast<const float4 *>(b + x), b1 = *reinterpret_cast<const float4 *>(b + 16 * ldb + x);
        acc[0][0] = dot4(a0, b0, acc[0][0]);
        acc[0][1] = dot4(a0, b1, acc[0][1]);
        acc[1][0] = dot4(a1, b0, acc[1][0]);
        acc[1][1] = dot4(a1, b1, acc[1][1]);
    }
}

// f(row, column, acc) over such a product's elements
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

__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {   // zeros where !there
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;\n" ::: "memory"); }

// rows t < n of a token tensor [rows, H, width] to rows of stride ld, rows behind as zero; X x Y floats to rows of
// stride ld: copies of NT threads, waited for by the caller
__device__ __forceinline__ void copy_tile(float *dst, int ld, const void *src, long long row0, int n, int H, int h, int width) {
    const float *s = static_cast<const float *>(src);
    for (int i = threadIdx.x; i < C * width / 4; i += NT) {
        const int t = i / (width / 4), x = i % (width / 4) * 4;
        copy16(dst + t * ld + x, s + ((size_t)(row0 + (t < n ? t : 0)) * H + h) * width + x, t < n);
    }
}
__device__ __forceinline__ void copy_f32(float *dst, int ld, const float *src, int rows, int W) {
    for (int i = threadIdx.x; i < rows * W / 4; i += NT) copy16(dst + i / (W / 4) * ld + i % (W / 4) * 4, src + 4 * i, true);
}

// prep: Tm, A, G, w of one tile and value head
template <int K>
__global__ void __launch_bounds__(NT) gdr_simt_prep(GdrArgs a) {
    __shared__ __align__(16) float k[C][K + 4], q[C][K + 4];
    __shared__ float M[C][LC], X[C][LC], G[C], L[C], w[C];
    const int tile = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, tid = threadIdx.x;
    int n, c, len;
    long long row0;
    if (!a.seq.find(tile, C, n, c, row0, len)) return;
    row0 += (long long)c * C;
    const int m = min(C, len - c * C), hk = h / (a.Hv / a.Hk);
    copy_tile(&k[0][0], K + 4, a.k, row0, m, a.Hk, hk, K);
    copy_tile(&q[0][0], K + 4, a.q, row0, m, a.Hk, hk, K);
    copies_commit();
    if (tid < C) {
        float la = 0.f, ww = 0.f;
        if (tid < m) {
            const size_t at = (size_t)(row0 + tid) * a.Hv + h;
            const float x = static_cast<const float *>(a.g_logit)[at] + (a.tau ? a.tau[h] : 0.f);
            la = least_log(-decay_amp(a.A_dec, h) * softplus_f(x));
            ww = sigmoid_f(static_cast<const float *>(a.w_logit)[at]);
        }
        float lo = 0.f;
        sum2_scan(la, lo, tid);
        G[tid] = la;
        L[tid] = lo;
        w[tid] = ww;
    }
    copies_wait();
    __syncthreads();
    float *out = reinterpret_cast<float *>(a.prep) + ((size_t)tile * a.Hv + h) * kPrep;
    float acc[2][2];
    zero(acc);
    mm_rows<K>(acc, &k[0][0], K + 4, &k[0][0], K + 4);
    each(acc, [&](int t, int s, float x) { M[t][s] = s < t ? w[t] * expf(sum2_diff(G[t], L[t], G[s], L[s])) * x : 0.f; });
    zero(acc);
    mm_rows<K>(acc, &q[0][0], K + 4, &k[0][0], K + 4);
    each(acc, [&](int t, int s, float x) { out[C * C + t * C + s] = s <= t ? expf(sum2_diff(G[t], L[t], G[s], L[s])) * x : 0.f; });
    __syncthreads();
    if (tid < C) {   // column tid of Tm by forward substitution, the column in registers
        float x[C];
#pragma unroll
        for (int t = 0; t < C; ++t) {
            float y[4] = {t == tid ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < t; ++s) y[s % 4] = fmaf(-M[t][s], x[s], y[s % 4]);
            x[t] = (y[0] + y[1]) + (y[2] + y[3]);
            X[t][tid] = x[t];
        }
        out[2 * C * C + tid] = G[tid];
        out[2 * C * C + C + tid] = w[tid];
        out[2 * C * C + 2 * C + tid] = L[tid];
    }
    __syncthreads();
    each(acc, [&](int t, int s, float) { out[t * C + s] = X[t][s]; });
}

// The sweeps: VR value rows of one (sequence, head) a CTA of 128 threads, so that small calls fill more of
// the GPU; thread = four tokens t4 .. t4 + 3 and one value row, contractions in 16-byte steps.  The
// next chunk's tiles are copied (cp.async) while this one is computed: of a chunk's 9 us in the form
// that loaded them in turn, most was the wait for them.
constexpr int VR = 16, ST = 128, LT = C + 4;

template <int K>
struct SweepStage {
    float k[C][K + 4], q[C][K + 4], Tm[C][LT], A[C][LT], v[C][VR + 4], G[C], w[C], L[C];
};
template <int K>
struct SweepSmem {
    SweepStage<K> st[2];
    float S[VR][K + 4], y[VR][LT], u[VR][LT], ue[VR][LT], x[C][VR + 4];
};

// tiles of a chunk: K, Q, Tm, A, G, w, L of (tile, h), and VR columns from v0 of `v` (values or dO); rows behind m: zero
template <int K>
__device__ __forceinline__ void copy_stage(SweepStage<K> &st, const GdrArgs &a, const void *v, int V, int v0, long long tile, long long row,
                                           int m, int h) {
    const int hk = h / (a.Hv / a.Hk);
    const float *k = static_cast<const float *>(a.k), *q = static_cast<const float *>(a.q), *vv = static_cast<const float *>(v);
    for (int i = threadIdx.x; i < C * K / 4; i += ST) {
        const int t = i / (K / 4), x = i % (K / 4) * 4;
        const size_t at = ((size_t)(row + (t < m ? t : 0)) * a.Hk + hk) * K + x;
        copy16(&st.k[t][x], k + at, t < m);
        copy16(&st.q[t][x], q + at, t < m);
    }
    const float *p = reinterpret_cast<const float *>(a.prep) + ((size_t)tile * a.Hv + h) * kPrep;
    for (int i = threadIdx.x; i < C * C / 4; i += ST) {
        copy16(&st.Tm[i / (C / 4)][i % (C / 4) * 4], p + 4 * i, true);
        copy16(&st.A[i / (C / 4)][i % (C / 4) * 4], p + C * C + 4 * i, true);
    }
    for (int i = threadIdx.x; i < C * VR / 4; i += ST) {
        const int t = i / (VR / 4), x = i % (VR / 4) * 4;
        copy16(&st.v[t][x], vv + ((size_t)(row + (t < m ? t : 0)) * a.Hv + h) * V + v0 + x, t < m);
    }
    if (threadIdx.x < C / 4) {
        copy16(st.G + 4 * threadIdx.x, p + 2 * C * C + 4 * threadIdx.x, true);
        copy16(st.w + 4 * threadIdx.x, p + 2 * C * C + C + 4 * threadIdx.x, true);
        copy16(st.L + 4 * threadIdx.x, p + 2 * C * C + 2 * C + 4 * threadIdx.x, true);
    }
    copies_commit();
}

// acc[i] += <rows[t4 + i], col> over X terms, rows at stride ld
template <int X>
__device__ __forceinline__ void rows4(float (&acc)[4], const float *rows, int ld, const float *col) {
#pragma unroll 4
    for (int x = 0; x < X; x += 4) {
        const float4 b = *reinterpret_cast<const float4 *>(col + x);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = dot4(*reinterpret_cast<const float4 *>(rows + i * ld + x), b, acc[i]);
    }
}
// acc[i] += sum_s m[s][t4 + i] x[s][v]: m at stride LT from column t4, x at stride VR + 4 from column v
__device__ __forceinline__ void columns4(float (&acc)[4], const float *m, const float *x) {
#pragma unroll 8
    for (int s = 0; s < C; ++s) {
        const float4 a = *reinterpret_cast<const float4 *>(m + s * LT);
        const float b = x[s * (VR + 4)];
        acc[0] = fmaf(a.x, b, acc[0]);
        acc[1] = fmaf(a.y, b, acc[1]);
        acc[2] = fmaf(a.z, b, acc[2]);
        acc[3] = fmaf(a.w, b, acc[3]);
    }
}
// S rows r, r + 8 (columns 4 x + 64 j of this thread) += sum_t f[row][t] m[t][column]
template <int K>
__device__ __forceinline__ void outer(float4 (&acc)[2][K / 64], const float (*f)[LT], int r, const float *m) {
#pragma unroll 2
    for (int t = 0; t < C; t += 4) {
        const float4 a0 = *reinterpret_cast<const float4 *>(&f[r][t]), a1 = *reinterpret_cast<const float4 *>(&f[r + 8][t]);
        const float x0[4] = {a0.x, a0.y, a0.z, a0.w}, x1[4] = {a1.x, a1.y, a1.z, a1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < K / 64; ++j) {
                const float4 b = *reinterpret_cast<const float4 *>(m + (t + e) * (K + 4) + 64 * j);
                float4 &c0 = acc[0][j], &c1 = acc[1][j];
                c0 = make_float4(fmaf(x0[e], b.x, c0.x), fmaf(x0[e], b.y, c0.y), fmaf(x0[e], b.z, c0.z), fmaf(x0[e], b.w, c0.w));
                c1 = make_float4(fmaf(x1[e], b.x, c1.x), fmaf(x1[e], b.y, c1.y), fmaf(x1[e], b.z, c1.z), fmaf(x1[e], b.w, c1.w));
            }
    }
}
template <int K>
__device__ __forceinline__ void scaled_state(float4 (&acc)[2][K / 64], const float (*S)[K + 4], int r, int x, float f) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < K / 64; ++j) {
            const float4 s = *reinterpret_cast<const float4 *>(&S[r + 8 * i][x + 64 * j]);
            acc[i][j] = make_float4(f * s.x, f * s.y, f * s.z, f * s.w);
        }
}
template <int K>
__device__ __forceinline__ void state_back(float (*S)[K + 4], const float4 (&acc)[2][K / 64], int r, int x) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < K / 64; ++j) *reinterpret_cast<float4 *>(&S[r + 8 * i][x + 64 * j]) = acc[i][j];
}

// forward sweep of VR value rows of one (sequence, head); saved: per tile S0 [V][K] and U [C][V]
template <int K, int V>
__global__ void __launch_bounds__(ST) gdr_simt_sweep(GdrArgs a, bool save) {
    extern __shared__ __align__(16) unsigned char raw[];
    SweepSmem<K> &sm = *reinterpret_cast<SweepSmem<K> *>(raw);
    const int v0 = (blockIdx.x % (V / VR)) * VR, unit = blockIdx.x / (V / VR), h = unit % a.Hv, n = unit / a.Hv;
    const int t4 = threadIdx.x / 16 * 4, v = threadIdx.x % 16;      // tokens and value row of the products
    const int sr = threadIdx.x / 16, sx = threadIdx.x % 16 * 4;     // rows and columns of the state
    long long row0;
    int len;
    a.seq.rows(n, row0, len, threadIdx.x == 0 ? &g_gdr_bad_seqlens : nullptr);
    const size_t st = ((size_t)unit * V + v0) * K;
    for (int i = threadIdx.x; i < VR * K; i += ST) sm.S[i / K][i % K] = a.S0 ? a.S0[st + i] : 0.f;
    const long long t0 = a.seq.tile0(n, C);
    const int chunks = (len + C - 1) / C;
    if (chunks) copy_stage<K>(sm.st[0], a, a.v, V, v0, t0, row0, min(C, len), h);
    for (int c = 0; c < chunks; ++c) {
        const int m = min(C, len - c * C);
        const long long tile = t0 + c, row = row0 + (long long)c * C;
        const SweepStage<K> &s = sm.st[c & 1];
        copies_wait();
        __syncthreads();   // the stage is there, the other one and S, u are free
        if (c + 1 < chunks) copy_stage<K>(sm.st[(c + 1) & 1], a, a.v, V, v0, tile + 1, row + C, min(C, len - (c + 1) * C), h);
        float *keep = save ? reinterpret_cast<float *>(a.saved) + ((size_t)tile * a.Hv + h) * ((size_t)V * K + C * V) : nullptr;
        if (save)
            for (int i = threadIdx.x; i < VR * K; i += ST) keep[(size_t)v0 * K + i] = sm.S[i / K][i % K];
        float g[4] = {}, o[4] = {};
        rows4<K>(g, s.k[t4], K + 4, sm.S[v]);
        rows4<K>(o, s.q[t4], K + 4, sm.S[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float eG = expf(s.G[t4 + i]);
            o[i] *= eG;
            sm.y[v][t4 + i] = s.w[t4 + i] * (s.v[t4 + i][v] - eG * g[i]);
        }
        __syncthreads();
        const float gl = s.G[C - 1], ll = s.L[C - 1];
        float u[4] = {};
        rows4<C>(u, s.Tm[t4], LT, sm.y[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sm.u[v][t4 + i] = u[i];
            sm.ue[v][t4 + i] = u[i] * expf(sum2_diff(gl, ll, s.G[t4 + i], s.L[t4 + i]));
            if (save) keep[(size_t)V * K + (t4 + i) * V + v0 + v] = u[i];
        }
        __syncthreads();
        rows4<C>(o, s.A[t4], LT, sm.u[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t4 + i < m) static_cast<float *>(a.o)[((size_t)(row + t4 + i) * a.Hv + h) * V + v0 + v] = o[i];
        float4 acc[2][K / 64];
        scaled_state<K>(acc, sm.S, sr, sx, expf(gl));
        outer<K>(acc, sm.ue, sr, &s.k[0][sx]);
        state_back<K>(sm.S, acc, sr, sx);
    }
    __syncthreads();
    if (a.S_final)
        for (int i = threadIdx.x; i < VR * K; i += ST) a.S_final[st + i] = sm.S[i / K][i % K];
}

// reverse sweep of VR value rows; ws: per tile dS1 [V][K] and dY [C][V]
template <int K, int V>
__global__ void __launch_bounds__(ST) gdr_simt_bsweep(GdrArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    SweepSmem<K> &sm = *reinterpret_cast<SweepSmem<K> *>(raw);
    const int v0 = (blockIdx.x % (V / VR)) * VR, unit = blockIdx.x / (V / VR), h = unit % a.Hv, n = unit / a.Hv;
    const int t4 = threadIdx.x / 16 * 4, v = threadIdx.x % 16, sr = threadIdx.x / 16, sx = threadIdx.x % 16 * 4;
    long long row0;
    int len;
    a.seq.rows(n, row0, len, threadIdx.x == 0 ? &g_gdr_bad_seqlens : nullptr);
    const size_t st = ((size_t)unit * V + v0) * K;
    for (int i = threadIdx.x; i < VR * K; i += ST) sm.S[i / K][i % K] = a.dS_final ? a.dS_final[st + i] : 0.f;
    const long long t0 = a.seq.tile0(n, C);
    const int chunks = (len + C - 1) / C;
    auto fetch = [&](int c) {   // sm.st[].v = dO
        copy_stage<K>(sm.st[c & 1], a, a.dO, V, v0, t0 + c, row0 + (long long)c * C, min(C, len - c * C), h);
    };
    if (chunks) fetch(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
        const int m = min(C, len - c * C);
        const long long tile = t0 + c, row = row0 + (long long)c * C;
        const SweepStage<K> &s = sm.st[c & 1];
        copies_wait();
        __syncthreads();
        if (c > 0) fetch(c - 1);
        float *out = reinterpret_cast<float *>(a.ws) + ((size_t)tile * a.Hv + h) * ((size_t)V * K + C * V);
        for (int i = threadIdx.x; i < VR * K; i += ST) out[(size_t)v0 * K + i] = sm.S[i / K][i % K];
        const float gl = s.G[C - 1], ll = s.L[C - 1];
        float d[4] = {};
        rows4<K>(d, s.k[t4], K + 4, sm.S[v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] *= expf(sum2_diff(gl, ll, s.G[t4 + i], s.L[t4 + i]));
            sm.u[v][t4 + i] = s.v[t4 + i][v] * expf(s.G[t4 + i]);   // e^G dO
        }
        columns4(d, &s.A[0][t4], &s.v[0][v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sm.x[t4 + i][v] = d[i];   // dU
        __syncthreads();
        float y[4] = {};
        columns4(y, &s.Tm[0][t4], &sm.x[0][v]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float dv = s.w[t4 + i] * y[i];
            out[(size_t)V * K + (t4 + i) * V + v0 + v] = y[i];
            sm.y[v][t4 + i] = -dv * expf(s.G[t4 + i]);
            if (t4 + i < m) static_cast<float *>(a.dv)[((size_t)(row + t4 + i) * a.Hv + h) * V + v0 + v] = dv;
        }
        __syncthreads();
        float4 acc[2][K / 64];
        scaled_state<K>(acc, sm.S, sr, sx, expf(gl));
        outer<K>(acc, sm.u, sr, &s.q[0][sx]);
        outer<K>(acc, sm.y, sr, &s.k[0][sx]);
        state_back<K>(sm.S, acc, sr, sx);
    }
    __syncthreads();
    if (a.dS0)
        for (int i = threadIdx.x; i < VR * K; i += ST) a.dS0[st + i] = sm.S[i / K][i % K];
}

template <int K, int V>
struct GradSmem {
    float k[C][K + 4], q[C][K + 4], S[V][K], dO[C][V + 4], dY[C][V + 4], U[C][V + 4], v[C][V + 4];
    float P1[C][LC], P2[C][LC], kk[C][LC], row[4][C], G[C], L[C], w[C], red[NT / 32];
};

// column j of a thread's K / 16: groups of four
__device__ __forceinline__ int col4(int j) { return 4 * (threadIdx.x % 16) + 64 * (j / 4) + j % 4; }
// acc[i][j] += sum_x f(ty + 16 i, x) m[x][col4(j)] over X rows of m (stride ld)
template <int NJ, int X, class F>
__device__ __forceinline__ void mm_wide(float (&acc)[2][NJ], F f, const float *m, int ld) {
    const int ty = threadIdx.x / 16;
    const float *b = m + 4 * (threadIdx.x % 16);
#pragma unroll 4
    for (int x = 0; x < X; ++x) {
        const float a0 = f(ty, x), a1 = f(ty + 16, x);
#pragma unroll
        for (int j = 0; j < NJ; j += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(b + x * ld + 16 * j);
            const float yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[0][j + e] = fmaf(a0, yy[e], acc[0][j + e]);
                acc[1][j + e] = fmaf(a1, yy[e], acc[1][j + e]);
            }
        }
    }
}
// sum over the 16 lanes that share a row of the 16 x 16 thread grid
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// gradients of q, k (summed over the value heads of a key head, in order) and of the gates
template <int K, int V>
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
    copy_tile(&sm.k[0][0], K + 4, a.k, row, m, a.Hk, hk, K);
    copy_tile(&sm.q[0][0], K + 4, a.q, row, m, a.Hk, hk, K);
    float dq[2][NK], dk[2][NK];
    zero(dq);
    zero(dk);
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        const size_t slot = (size_t)tile * a.Hv + h, per = (size_t)V * K + C * V;
        const float *fwd = reinterpret_cast<const float *>(a.saved) + slot * per;
        const float *bwd = reinterpret_cast<const float *>(a.ws) + slot * per;
        const float *prep = reinterpret_cast<const float *>(a.prep) + slot * kPrep;
        __syncthreads();
        copy_tile(&sm.dO[0][0], V + 4, a.dO, row, m, a.Hv, h, V);
        copy_tile(&sm.v[0][0], V + 4, a.v, row, m, a.Hv, h, V);
        copy_f32(&sm.dY[0][0], V + 4, bwd + (size_t)V * K, C, V);
        copy_f32(&sm.U[0][0], V + 4, fwd + (size_t)V * K, C, V);
        copy_f32(&sm.S[0][0], K, fwd, V, K);
        copies_commit();
        if (tid < C) {
            sm.G[tid] = prep[2 * C * C + tid];
            sm.w[tid] = prep[2 * C * C + C + tid];
            sm.L[tid] = prep[2 * C * C + 2 * C + tid];
        }
        copies_wait();
        __syncthreads();
        const float gl = sm.G[C - 1], ll = sm.L[C - 1];
        float acc[2][2], x1[2][NK];
        // per-row partial sums of this thread's two rows: gate gradients
        float dG[2] = {0.f, 0.f}, dw[2] = {0.f, 0.f}, kb[2] = {0.f, 0.f}, lastp = 0.f;
        // the products with the chunk's start state
        zero(x1);
        mm_wide<NK, V>(x1, [&](int t, int v) { return sm.dO[t][v]; }, &sm.S[0][0], K);
        each(x1, [&](int t, int, float &y) { y *= expf(sm.G[t]); });
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int t = tid / 16 + 16 * i, x = col4(j);
                dq[i][j] += x1[i][j];
                dG[i] += sm.q[t][x] * x1[i][j];
            }
        zero(x1);
        mm_wide<NK, V>(x1, [&](int t, int v) { return sm.dY[t][v]; }, &sm.S[0][0], K);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int t = tid / 16 + 16 * i, x = col4(j);
                const float y = expf(sm.G[t]) * x1[i][j];
                dk[i][j] -= sm.w[t] * y;
                dw[i] -= sm.k[t][x] * y;
                dG[i] -= sm.w[t] * sm.k[t][x] * y;
            }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            for (int v = tid % 16; v < V; v += 16) dw[i] += sm.dY[tid / 16 + 16 * i][v] * sm.v[tid / 16 + 16 * i][v];
        // <S0, dS1>, then dS1 in place of S0
        #pragma unroll 4
        for (int i = tid; i < V * K / 4; i += NT)
            lastp = dot4(reinterpret_cast<const float4 *>(&sm.S[0][0])[i], reinterpret_cast<const float4 *>(bwd)[i], lastp);
        lastp *= expf(gl);
        __syncthreads();
        copy_f32(&sm.S[0][0], K, bwd, V, K);
        copies_commit();
        copies_wait();
        __syncthreads();
        zero(x1);
        mm_wide<NK, V>(x1, [&](int t, int v) { return sm.U[t][v]; }, &sm.S[0][0], K);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int t = tid / 16 + 16 * i, x = col4(j);
                const float y = expf(sum2_diff(gl, ll, sm.G[t], sm.L[t])) * x1[i][j];
                dk[i][j] += y;
                kb[i] += sm.k[t][x] * y;
            }
        // the products within the chunk
        zero(acc);
        mm_rows<K>(acc, &sm.k[0][0], K + 4, &sm.k[0][0], K + 4);
        each(acc, [&](int t, int s, float x) { sm.kk[t][s] = x; });
        float kq[2][2];
        zero(kq);
        mm_rows<K>(kq, &sm.q[0][0], K + 4, &sm.k[0][0], K + 4);
        zero(acc);
        mm_rows<V>(acc, &sm.dO[0][0], V + 4, &sm.U[0][0], V + 4);
        float pr[2][2];   // contributions of the pairs (t, s < t), whose factor is e^{G_t - G_s}
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = tid / 16 + 16 * i, s = tid % 16 + 16 * j;
                const float p = s <= t ? acc[i][j] * expf(sum2_diff(sm.G[t], sm.L[t], sm.G[s], sm.L[s])) : 0.f;
                sm.P1[t][s] = p;
                pr[i][j] = s < t ? p * kq[i][j] : 0.f;
            }
        zero(acc);
        mm_rows<V>(acc, &sm.dY[0][0], V + 4, &sm.U[0][0], V + 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = tid / 16 + 16 * i, s = tid % 16 + 16 * j;
                const float p = s < t ? -acc[i][j] * expf(sum2_diff(sm.G[t], sm.L[t], sm.G[s], sm.L[s])) : 0.f;
                dw[i] += p * sm.kk[t][s];
                sm.P2[t][s] = sm.w[t] * p;
                pr[i][j] += sm.w[t] * p * sm.kk[t][s];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) sm.kk[tid / 16 + 16 * i][tid % 16 + 16 * j] = pr[i][j];
        mm_wide<NK, C>(dq, [&](int t, int s) { return sm.P1[t][s]; }, &sm.k[0][0], K + 4);
        mm_wide<NK, C>(dk, [&](int t, int s) { return sm.P2[t][s] + sm.P2[s][t]; }, &sm.k[0][0], K + 4);
        mm_wide<NK, C>(dk, [&](int t, int s) { return sm.P1[s][t]; }, &sm.q[0][0], K + 4);
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
                const float x = static_cast<const float *>(a.g_logit)[at] + (a.tau ? a.tau[h] : 0.f);
                const float amp = decay_amp(a.A_dec, h), w = sm.w[tid];
                dlog = -amp * sigmoid_f(x) * g;
                damp = softplus_f(x) * (-amp * g);   // of a reset g is 0, and amp softplus may be beyond fp32
                static_cast<float *>(a.dg_logit)[at] = dlog;
                static_cast<float *>(a.dw_logit)[at] = sm.row[1][tid] * w * (1.f - w);
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
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int t = tid / 16 + 16 * i;
            const size_t at = ((size_t)(row + t) * a.Hk + hk) * K + col4(j);
            if (t < m) {
                static_cast<float *>(a.dq)[at] = dq[i][j];
                static_cast<float *>(a.dk)[at] = dk[i][j];
            }
        }
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

template <int K, int V>
cudaError_t fwd_t(const GdrArgs &a, bool save, cudaStream_t st) {
    const long long tiles = a.seq.n_tiles(C);
    if (tiles) gdr_simt_prep<K><<<(unsigned)(tiles * a.Hv), NT, 0, st>>>(a);
    auto kern = gdr_simt_sweep<K, V>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), sizeof(SweepSmem<K>));
    if (e != cudaSuccess) return e;
    kern<<<a.seq.N * a.Hv * (V / VR), ST, sizeof(SweepSmem<K>), st>>>(a, save);
    return cudaGetLastError();
}

template <int K, int V>
cudaError_t bwd_t(const GdrArgs &a, cudaStream_t st) {
    auto sweep = gdr_simt_bsweep<K, V>;
    auto grad = gdr_simt_grad<K, V>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(sweep), sizeof(SweepSmem<K>));
    if (e == cudaSuccess) e = set_smem_once(reinterpret_cast<const void *>(grad), sizeof(GradSmem<K, V>));
    if (e != cudaSuccess) return e;
    const long long tiles = a.seq.n_tiles(C);
    sweep<<<a.seq.N * a.Hv * (V / VR), ST, sizeof(SweepSmem<K>), st>>>(a);
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
        return fwd_t<K, V>(a, save, st);
    }
};
struct Bwd {
    const GdrArgs &a;
    cudaStream_t st;
    template <int K, int V>
    cudaError_t operator()() const {
        return bwd_t<K, V>(a, st);
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
