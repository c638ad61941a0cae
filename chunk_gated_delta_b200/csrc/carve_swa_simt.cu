// Sliding-window attention with sink tokens on the CUDA cores, fp32 throughout
// (include/carve_mixers.h): the path of fp32 tensors.
//
// Forward: one CTA per (32 queries, head) walks the key tiles that its queries see (the window's,
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

constexpr int BT = 32;    // queries and keys of a tile
constexpr int NT = 256;   // threads, as 16 x 16: rows ty, ty + 16 and columns tx + 16 j

template <int D>
struct Smem {
    float q[BT][D + 1], k[BT][D + 1], v[BT][D + 1], dO[BT][D + 1], p[BT][BT + 1], ds[BT][BT + 1], lse[BT], delta[BT];
};

template <class IO, int D>
__device__ __forceinline__ void load(float (*dst)[D + 1], const void *src, long long row0, int n, int H, int h) {
    const IO *s = static_cast<const IO *>(src);
    for (int i = threadIdx.x; i < BT * D; i += NT) {
        const int t = i / D, x = i % D;
        dst[t][x] = t < n ? ld_io(s + ((size_t)(row0 + t) * H + h) * D + x) : 0.f;
    }
}
template <class IO, int D>
__device__ __forceinline__ void store(void *dst, const float (&acc)[2][D / 16], long long row0, int n, int H, int h) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            if (ty + 16 * i < n)
                st_io(static_cast<IO *>(dst) + ((size_t)(row0 + ty + 16 * i) * H + h) * D + tx + 16 * j, acc[i][j]);
}

// acc[i][j] += sum_x fa(ty + 16 i, x) fb(tx + 16 j, x)
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

template <int D, class IO>
__global__ void __launch_bounds__(NT) swa_simt_fwd(SwaArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int tile = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hkv);
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    if (blockIdx.x == 0) check_seqs(a.seq, &g_swa_bad_seqlens);
    int n, c, len;
    long long row0;
    if (!a.seq.find(tile, BT, n, c, row0, len)) return;
    const int i0 = c * BT, i1 = min(i0 + BT, len);
    load<IO, D>(sm.q, a.q, row0 + i0, i1 - i0, a.Hq, h);
    float o[2][D / 16], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[0][j] = o[1][j] = 0.f;
    const KeyTiles kt(i0, i1, BT, a.window, a.sinks);
    for (int x = 0; x < kt.count(); ++x) {
        const int j0 = kt.tile(x) * BT, nk = min(BT, len - j0);
        __syncthreads();
        load<IO, D>(sm.k, a.k, row0 + j0, nk, a.Hkv, hk);
        load<IO, D>(sm.v, a.v, row0 + j0, nk, a.Hkv, hk);
        __syncthreads();
        float s[2][2] = {};
        mm<2, D>(s, [&](int i, int y) { return sm.q[i][y]; }, [&](int j, int y) { return sm.k[j][y]; });
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[i][j] = swa_sees(i0 + ty + 16 * i, j0 + tx + 16 * j, a.window, a.sinks) ? s[i][j] * a.scale : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float m1 = fmaxf(m[i], mx), base = m1 == -INFINITY ? 0.f : m1, f = expf(m[i] - base);
            m[i] = m1;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p = expf(s[i][j] - base);
                sm.p[ty + 16 * i][tx + 16 * j] = p;
                sum += p;
            }
#pragma unroll
            for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[i][j] *= f;
        }
        __syncthreads();
        mm<D / 16, BT>(o, [&](int i, int j) { return sm.p[i][j]; }, [&](int y, int j) { return sm.v[j][y]; });
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float inv = 1.f / l[i];
#pragma unroll
        for (int j = 0; j < D / 16; ++j) o[i][j] *= inv;
        if (a.lse && tx == 0 && i0 + ty + 16 * i < i1)
            a.lse[(size_t)(row0 + i0 + ty + 16 * i) * a.Hq + h] = m[i] + logf(l[i]);
    }
    store<IO, D>(a.o, o, row0 + i0, i1 - i0, a.Hq, h);
}

// p and ds of the tile (queries in q, dO, lse, delta; keys in k, v) into sm.p, sm.ds
template <int D>
__device__ __forceinline__ void p_ds(Smem<D> &sm, const SwaArgs &a, int i0, int i1, int j0) {
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float s[2][2] = {}, dp[2][2] = {};
    mm<2, D>(s, [&](int i, int y) { return sm.q[i][y]; }, [&](int j, int y) { return sm.k[j][y]; });
    mm<2, D>(dp, [&](int i, int y) { return sm.dO[i][y]; }, [&](int j, int y) { return sm.v[j][y]; });
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = ty + 16 * i, x = tx + 16 * j;
            const bool seen = i0 + r < i1 && swa_sees(i0 + r, j0 + x, a.window, a.sinks);
            const float p = seen ? expf(s[i][j] * a.scale - sm.lse[r]) : 0.f;
            sm.p[r][x] = p;
            sm.ds[r][x] = seen ? p * (dp[i][j] - sm.delta[r]) * a.scale : 0.f;
        }
}

template <int D, class IO>
__device__ __forceinline__ void load_queries(Smem<D> &sm, const SwaArgs &a, long long row, int n, int h) {
    load<IO, D>(sm.q, a.q, row, n, a.Hq, h);
    load<IO, D>(sm.dO, a.dO, row, n, a.Hq, h);
    if (threadIdx.x < BT) {
        const bool there = (int)threadIdx.x < n;
        sm.lse[threadIdx.x] = there ? a.lse[(size_t)(row + threadIdx.x) * a.Hq + h] : 0.f;
        sm.delta[threadIdx.x] = there ? a.delta[(size_t)(row + threadIdx.x) * a.Hq + h] : 0.f;
    }
}

template <int D, class IO>
__global__ void __launch_bounds__(NT) swa_simt_dq(SwaArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int tile = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hkv);
    int n, c, len;
    long long row0;
    if (!a.seq.find(tile, BT, n, c, row0, len)) return;
    const int i0 = c * BT, i1 = min(i0 + BT, len);
    load_queries<D, IO>(sm, a, row0 + i0, i1 - i0, h);
    float dq[2][D / 16] = {};
    const KeyTiles kt(i0, i1, BT, a.window, a.sinks);
    for (int x = 0; x < kt.count(); ++x) {
        const int j0 = kt.tile(x) * BT, nk = min(BT, len - j0);
        __syncthreads();
        load<IO, D>(sm.k, a.k, row0 + j0, nk, a.Hkv, hk);
        load<IO, D>(sm.v, a.v, row0 + j0, nk, a.Hkv, hk);
        __syncthreads();
        p_ds<D>(sm, a, i0, i1, j0);
        __syncthreads();
        mm<D / 16, BT>(dq, [&](int i, int j) { return sm.ds[i][j]; }, [&](int y, int j) { return sm.k[j][y]; });
    }
    store<IO, D>(a.dq, dq, row0 + i0, i1 - i0, a.Hq, h);
}

template <int D, class IO>
__global__ void __launch_bounds__(NT) swa_simt_dkv(SwaArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(raw);
    const int tile = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv, share = a.Hq / a.Hkv;
    if (blockIdx.x == 0) check_seqs(a.seq, &g_swa_bad_seqlens);
    int n, c, len;
    long long row0;
    if (!a.seq.find(tile, BT, n, c, row0, len)) return;
    const int j0 = c * BT, j1 = min(j0 + BT, len), last = last_query(j0, j1, len, a.window, a.sinks);
    load<IO, D>(sm.k, a.k, row0 + j0, j1 - j0, a.Hkv, hk);
    load<IO, D>(sm.v, a.v, row0 + j0, j1 - j0, a.Hkv, hk);
    float dk[2][D / 16] = {}, dv[2][D / 16] = {};
    for (int h = hk * share; h < (hk + 1) * share; ++h)
        for (int i0 = j0; i0 <= last; i0 += BT) {
            const int i1 = min(i0 + BT, len);
            __syncthreads();
            load_queries<D, IO>(sm, a, row0 + i0, i1 - i0, h);
            __syncthreads();
            p_ds<D>(sm, a, i0, i1, j0);
            __syncthreads();
            mm<D / 16, BT>(dv, [&](int j, int i) { return sm.p[i][j]; }, [&](int y, int i) { return sm.dO[i][y]; });
            mm<D / 16, BT>(dk, [&](int j, int i) { return sm.ds[i][j]; }, [&](int y, int i) { return sm.q[i][y]; });
        }
    store<IO, D>(a.dk, dk, row0 + j0, j1 - j0, a.Hkv, hk);
    store<IO, D>(a.dv, dv, row0 + j0, j1 - j0, a.Hkv, hk);
}

// delta[row, h] = sum_c dO o: 8 lanes per (row, head)
template <int D, class IO>
__global__ void __launch_bounds__(256) swa_delta(SwaArgs a, long long heads) {
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x / 8;
    const int seg = threadIdx.x % 8;
    float x = 0.f;
    if (i < heads) {
        const IO *o = static_cast<const IO *>(a.o) + i * D, *g = static_cast<const IO *>(a.dO) + i * D;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) x += ld_io(o + seg * (D / 8) + c) * ld_io(g + seg * (D / 8) + c);
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if (seg == 0 && i < heads) a.delta[i] = x;
}

template <int D, class IO>
cudaError_t fwd_t(const SwaArgs &a, cudaStream_t st) {
    auto kern = swa_simt_fwd<D, IO>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), sizeof(Smem<D>));
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(a.seq.n_tiles(BT) * a.Hq), NT, sizeof(Smem<D>), st>>>(a);
    return cudaGetLastError();
}

template <int D, class IO>
cudaError_t bwd_t(const SwaArgs &a, cudaStream_t st) {
    auto dq = swa_simt_dq<D, IO>;
    auto dkv = swa_simt_dkv<D, IO>;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(dq), sizeof(Smem<D>));
    if (e == cudaSuccess) e = set_smem_once(reinterpret_cast<const void *>(dkv), sizeof(Smem<D>));
    if (e != cudaSuccess) return e;
    const long long heads = (a.seq.cu ? a.seq.total : (long long)a.seq.N * a.seq.T) * a.Hq;
    swa_delta<D, IO><<<(unsigned)((heads + 31) / 32), 256, 0, st>>>(a, heads);
    dkv<<<(unsigned)(a.seq.n_tiles(BT) * a.Hkv), NT, sizeof(Smem<D>), st>>>(a);
    dq<<<(unsigned)(a.seq.n_tiles(BT) * a.Hq), NT, sizeof(Smem<D>), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swa_fwd_simt(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? fwd_t<64, float>(a, st) : fwd_t<128, float>(a, st);
}
cudaError_t launch_swa_bwd_simt(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? bwd_t<64, float>(a, st) : bwd_t<128, float>(a, st);
}

}  // namespace carve
