// Sliding-window attention with sink tokens on the CUDA cores, fp32 throughout
// (include/carve_mixers.h): the path of fp32 tensors.
//
// Forward: one CTA per (16 queries, head) walks the key tiles that its queries see (the window's,
// and before them the ones that hold sinks) with the running maximum m and sum l of the softmax:
//   m' = max(m, s), l' = e^{m - m'} l + sum e^{s - m'}, o' = e^{m - m'} o + sum e^{s - m'} v
// Backward, from lse = m + log l and delta_i = sum_c dO_ic o_ic:
//   p_ij = e^{s_ij - lse_i},  ds_ij = p_ij (dO_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dO_i
// in two passes, by queries for dq and by keys for dk, dv (over the query heads of a key head in
// order), so that no sum goes through atomics.
#include "carve_mixers.cuh"

namespace carve {

__device__ int g_swa_bad_seqlens;   // set when a packed sequence's offsets are out of range

int swa_take_bad_seqlens() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_swa_bad_seqlens, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_swa_bad_seqlens, &z, sizeof(int));
    }
    return v;
}

namespace {

constexpr int BR = 16;    // rows of a CTA: queries (forward, dq) or keys (dk, dv)
constexpr int BC = 32;    // rows of a tile of the other side
constexpr int NT = 256;   // threads, as 16 x 16: row ty, columns tx, tx + 16 of the scores, channels 4 tx + 64 j

template <int D>
struct Smem {
    float r1[BR][D + 4], r2[BR][D + 4], c1[2][BC][D + 4], c2[2][BC][D + 4], lse[2][BC], delta[2][BC], p[BR][BC + 4], ds[BR][BC + 4];
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) {   // zeros where !there
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
// N rows of a token tensor from row0 on, those from `n` on as zeros
template <int D, int N>
__device__ __forceinline__ void copy_rows(float (*dst)[D + 4], const void *src, long long row0, int n, int H, int h) {
    for (int i = threadIdx.x; i < N * D / 4; i += NT) {
        const int t = i / (D / 4), x = i % (D / 4) * 4;
        copy16(&dst[t][x], static_cast<const float *>(src) + ((size_t)(row0 + (t < n ? t : 0)) * H + h) * D + x, t < n);
    }
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) { return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c)))); }
// s[j] = <r[ty], c[tx + 16 j]>
template <int D>
__device__ __forceinline__ void scores(float (&s)[2], const float (*r)[D + 4], const float (*c)[D + 4]) {
    const float *a = r[threadIdx.x / 16], *b0 = c[threadIdx.x % 16], *b1 = c[threadIdx.x % 16 + 16];
    s[0] = s[1] = 0.f;
#pragma unroll 8
    for (int x = 0; x < D; x += 4) {
        const float4 y = *reinterpret_cast<const float4 *>(a + x);
        s[0] = dot4(y, *reinterpret_cast<const float4 *>(b0 + x), s[0]);
        s[1] = dot4(y, *reinterpret_cast<const float4 *>(b1 + x), s[1]);
    }
}
// acc[j] += sum_c p[ty][c] m[c][4 tx + 64 j ..]
template <int D>
__device__ __forceinline__ void gather(float4 (&acc)[D / 64], const float (*p)[BC + 4], const float (*m)[D + 4]) {
    const float *f = p[threadIdx.x / 16];
    const int x = 4 * (threadIdx.x % 16);
#pragma unroll 2
    for (int c = 0; c < BC; c += 4) {
        const float4 y = *reinterpret_cast<const float4 *>(f + c);
        const float w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const float4 b = *reinterpret_cast<const float4 *>(&m[c + e][x + 64 * j]);
                acc[j] = make_float4(fmaf(w[e], b.x, acc[j].x), fmaf(w[e], b.y, acc[j].y), fmaf(w[e], b.z, acc[j].z), fmaf(w[e], b.w, acc[j].w));
            }
    }
}
template <int D>
__device__ __forceinline__ void store_rows(void *dst, const float4 (&acc)[D / 64], long long row0, int n, int H, int h) {
    const int ty = threadIdx.x / 16, x = 4 * (threadIdx.x % 16);
    if (ty < n)
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            *reinterpret_cast<float4 *>(static_cast<float *>(dst) + ((size_t)(row0 + ty) * H + h) * D + x + 64 * j) = acc[j];
}

__global__ void __launch_bounds__(NT) swa_check(Seqs s) { check_seqs(s, &g_swa_bad_seqlens); }

enum Mode { FWD, DQ, DKV };

// One CTA: BR rows of one (sequence, head), resident, and the tiles of the other side that they see (DKV:
// of every query head of the key head in turn), the next tile's copies in flight while one is computed.
//          r1   r2   c1   c2
//   FWD    q         k    v
//   DQ     q    dO   k    v
//   DKV    k    v    q    dO
template <int D, Mode MODE>
__global__ void __launch_bounds__(NT) swa_simt(SwaArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int heads = MODE == DKV ? a.Hkv : a.Hq, share = a.Hq / a.Hkv;
    const int tile = blockIdx.x / heads, h = blockIdx.x % heads, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (MODE != DQ && blockIdx.x == 0) check_seqs(a.seq, &g_swa_bad_seqlens);
    int n, c, len;
    long long row0;
    if (!a.seq.find(tile, BR, n, c, row0, len)) return;
    const int r0 = c * BR, r1 = min(r0 + BR, len), row = r0 + ty;
    KeyTiles kt;
    int per = 0, first = 0, count;   // DKV: tiles of a query head, from `first` on
    if (MODE == DKV) {
        first = r0 / BC;
        per = last_query(r0, r1, len, a.window, a.sinks) / BC - first + 1;
        count = per * share;
    } else {
        kt = KeyTiles(r0, r1, BC, a.window, a.sinks);
        count = kt.count();
    }
    auto fetch = [&](int b) {
        const int s = b & 1, c0 = (MODE == DKV ? first + b % per : kt.tile(b)) * BC, there = min(BC, len - c0);
        const int hc = MODE == DKV ? h * share + b / per : h / share, Hc = MODE == DKV ? a.Hq : a.Hkv;
        copy_rows<D, BC>(sm.c1[s], MODE == DKV ? a.q : a.k, row0 + c0, there, Hc, hc);
        copy_rows<D, BC>(sm.c2[s], MODE == DKV ? a.dO : a.v, row0 + c0, there, Hc, hc);
        if (MODE == DKV && threadIdx.x < BC) {
            const size_t at = (size_t)(row0 + c0 + threadIdx.x) * a.Hq + hc;
            sm.lse[s][threadIdx.x] = (int)threadIdx.x < there ? a.lse[at] : 0.f;
            sm.delta[s][threadIdx.x] = (int)threadIdx.x < there ? a.delta[at] : 0.f;
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    copy_rows<D, BR>(sm.r1, MODE == DKV ? a.k : a.q, row0 + r0, r1 - r0, heads, h);
    if (MODE != FWD) copy_rows<D, BR>(sm.r2, MODE == DKV ? a.v : a.dO, row0 + r0, r1 - r0, heads, h);
    fetch(0);
    float lse = 0.f, delta = 0.f, m = -INFINITY, l = 0.f;
    if (MODE == DQ && row < r1) {
        lse = a.lse[(size_t)(row0 + row) * a.Hq + h];
        delta = a.delta[(size_t)(row0 + row) * a.Hq + h];
    }
    float4 acc[D / 64], acc2[D / 64];
#pragma unroll
    for (int j = 0; j < D / 64; ++j) acc[j] = acc2[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = 0; b < count; ++b) {
        const int s = b & 1, c0 = (MODE == DKV ? first + b % per : kt.tile(b)) * BC;
        asm volatile("cp.async.wait_group 0;\n" ::: "memory");
        __syncthreads();   // the tile is there; the other stage, p and ds are free
        if (b + 1 < count) fetch(b + 1);
        float x[2], dp[2];
        scores<D>(x, sm.r1, sm.c1[s]);
        if (MODE != FWD) scores<D>(dp, sm.r2, sm.c2[s]);
        bool seen[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = c0 + tx + 16 * j;
            seen[j] = MODE == DKV ? col < len && swa_sees(col, row, a.window, a.sinks) : swa_sees(row, col, a.window, a.sinks);
        }
        if (MODE == FWD) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x[j] = seen[j] ? x[j] * a.scale : -INFINITY;
                mx = fmaxf(mx, x[j]);
            }
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float m1 = fmaxf(m, mx), base = m1 == -INFINITY ? 0.f : m1, f = expf(m - base);
            m = m1;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p = expf(x[j] - base);
                sm.p[ty][tx + 16 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l = l * f + sum;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) acc[j] = make_float4(f * acc[j].x, f * acc[j].y, f * acc[j].z, f * acc[j].w);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int y = tx + 16 * j;
                const float p = seen[j] ? expf(x[j] * a.scale - (MODE == DKV ? sm.lse[s][y] : lse)) : 0.f;
                sm.ds[ty][y] = seen[j] ? p * (dp[j] - (MODE == DKV ? sm.delta[s][y] : delta)) * a.scale : 0.f;
                if (MODE == DKV) sm.p[ty][y] = p;
            }
        }
        __syncwarp();   // a warp's two rows of p and ds are its own
        if (MODE == FWD) gather<D>(acc, sm.p, sm.c2[s]);
        if (MODE != FWD) gather<D>(acc, sm.ds, sm.c1[s]);
        if (MODE == DKV) gather<D>(acc2, sm.p, sm.c2[s]);
        __syncwarp();
    }
    if (MODE == FWD) {
        const float inv = 1.f / l;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] = make_float4(inv * acc[j].x, inv * acc[j].y, inv * acc[j].z, inv * acc[j].w);
        if (a.lse && tx == 0 && row < r1) a.lse[(size_t)(row0 + row) * a.Hq + h] = m + logf(l);
    }
    store_rows<D>(MODE == FWD ? a.o : MODE == DQ ? a.dq : a.dk, acc, row0 + r0, r1 - r0, heads, h);
    if (MODE == DKV) store_rows<D>(a.dv, acc2, row0 + r0, r1 - r0, heads, h);
}

// delta[row, h] = sum_c dO o: 8 lanes per (row, head)
template <int D>
__global__ void __launch_bounds__(256) swa_delta(SwaArgs a, long long heads) {
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x / 8;
    const int seg = threadIdx.x % 8;
    float x = 0.f;
    if (i < heads) {
        const float *o = static_cast<const float *>(a.o) + i * D, *g = static_cast<const float *>(a.dO) + i * D;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x += o[seg * (D / 8) + c] * g[seg * (D / 8) + c];
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if (seg == 0 && i < heads) a.delta[i] = x;
}

template <int D, Mode MODE>
cudaError_t launch(const SwaArgs &a, cudaStream_t st) {
    auto kern = swa_simt<D, MODE>;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), sizeof(Smem<D>));
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(a.seq.n_tiles(BR) * (MODE == DKV ? a.Hkv : a.Hq)), NT, sizeof(Smem<D>), st>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t bwd_t(const SwaArgs &a, cudaStream_t st) {
    const long long heads = (a.seq.cu ? a.seq.total : (long long)a.seq.N * a.seq.T) * a.Hq;
    swa_delta<D><<<(unsigned)((heads + 31) / 32), 256, 0, st>>>(a, heads);
    const cudaError_t e = launch<D, DKV>(a, st);
    return e == cudaSuccess ? launch<D, DQ>(a, st) : e;
}

}  // namespace

cudaError_t launch_swa_check(const Seqs &s, cudaStream_t st) {
    swa_check<<<1, NT, 0, st>>>(s);
    return cudaGetLastError();
}
cudaError_t launch_swa_fwd_simt(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? launch<64, FWD>(a, st) : launch<128, FWD>(a, st);
}
cudaError_t launch_swa_bwd_simt(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? bwd_t<64>(a, st) : bwd_t<128>(a, st);
}

}  // namespace carve
