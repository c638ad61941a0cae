// Shared pieces of the mixers declared in include/carve_mixers.h: argument structs, sequence
// tables and launch declarations (product code; independent of the oracle).
#pragma once
#include "carve_device.cuh"

namespace carve {

// The sequences of a call: B batch elements of T tokens each, or (cu) N sequences packed in
// `total` rows.
struct Seqs {
    const int *cu;
    long long total;
    int N, T;

    // rows [row0, row0 + len) of sequence n; a packed sequence that leaves [0, total] is empty
    // and *bad (when given) records it
    __device__ __forceinline__ void rows(int n, long long &row0, int &len, int *bad = nullptr, int mark = 1) const {
        if (!cu) {
            row0 = (long long)n * T;
            len = T;
            return;
        }
        const int c0 = cu[n], c1 = cu[n + 1];
        row0 = c0;
        len = c1 - c0;
        if (c0 < 0 || c1 < c0 || (long long)c1 > total) {
            row0 = 0;
            len = 0;
            if (bad) atomicOr(bad, mark);
        }
    }

    // Tiles of C tokens, each sequence starting its own: sequence n's tiles are numbered from
    // tile0(n, C).  Packed, cu[n] / C + n leaves every sequence at least ceil(len / C) numbers and
    // needs no table of lengths on the host; the numbers between two sequences' tiles stay unused.
    __host__ __device__ __forceinline__ long long n_tiles(int C) const {
        return cu ? total / C + N : (long long)N * ((T + C - 1) / C);
    }
    __device__ __forceinline__ long long tile0(int n, int C) const {
        return cu ? cu[n] / C + n : (long long)n * ((T + C - 1) / C);
    }
    // the sequence n and the tile c within it that number `tile` stands for; false where it is
    // unused.  Packed, the last n with tile0(n) <= tile is found by bisection (tile0 grows with n).
    __device__ __forceinline__ bool find(int tile, int C, int &n, int &c, long long &row0, int &len) const {
        if (!cu) {
            const int per = (T + C - 1) / C;
            n = tile / per;
            c = tile - n * per;
        } else {
            int lo = 0, hi = N - 1;
#pragma unroll 1
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] / C + mid <= tile)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            n = lo;
            c = tile - (cu[n] / C + n);
        }
        rows(n, row0, len);
        return c >= 0 && (long long)c * C < len;
    }
};

// Threads of one CTA together: records packed sequences whose offsets are out of range.
__device__ __forceinline__ void check_seqs(const Seqs &s, int *bad, int mark = 1) {
    if (!s.cu) return;
    long long r;
    int len;
    for (int n = threadIdx.x; n < s.N; n += blockDim.x) s.rows(n, r, len, bad, mark);
}
// A kernel's status word for carve_check: bits of what happened.
constexpr int kTimedOut = 1;     // a bounded wait gave up (never expected)
constexpr int kBadOffsets = 2;   // a packed sequence's offsets are out of range

// Running sums of log decays as hi + lo.  A decay between two tokens is the difference of two such sums, and
// behind a token that resets the state (log a of -1e3, say) an fp32 sum of the whole chunk has lost the low
// bits of the mild steps: the factors were off by 6e-5 there, 1e-3 at -1e4.  lo holds what the roundings of hi
// drop (exactly, addition by addition), so a difference is good to 2^-40 of the largest step.
__device__ __forceinline__ void sum2_add(float &hi, float &lo, float h, float l) {
    const float s = hi + h, y = s - hi;
    lo += l + ((hi - (s - y)) + (h - y));
    hi = s;
}
// inclusive over the lanes of a warp
__device__ __forceinline__ void sum2_scan(float &hi, float &lo, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float h = __shfl_up_sync(0xffffffffu, hi, off), l = __shfl_up_sync(0xffffffffu, lo, off);
        if (lane >= off) sum2_add(hi, lo, h, l);
    }
}
__device__ __forceinline__ float sum2_diff(float hi, float lo, float hi0, float lo0) { return (hi - hi0) + (lo - lo0); }
// log a, not below -1e4 (in either base: a decay of zero in fp32 long before), so that sums and their
// differences are finite; a NaN stays one
__device__ __forceinline__ float least_log(float la) { return la < -1e4f ? -1e4f : la; }

struct GdrArgs {
    Seqs seq;
    int Hk, Hv;
    const void *q, *k, *v, *g_logit, *w_logit;
    const float *A_dec, *tau, *S0;
    void *o;
    float *S_final;
    // backward
    const void *dO;
    const float *dS_final;
    void *dq, *dk, *dv, *dg_logit, *dw_logit;
    float *dA_dec, *dtau, *dS0;
    char *prep, *saved, *ws;   // per-tile operands; what the forward saves beside them; backward scratch
};

struct SwaArgs {
    Seqs seq;
    int Hq, Hkv, d, window, sinks;
    float scale;
    const void *q, *k, *v;
    void *o;
    float *lse;
    // backward
    const void *dO;
    void *dq, *dk, *dv;
    float *delta;              // rowsum(dO * o), [rows, Hq] (tensor-core path: see there)
    float *partial;            // dk, dv of the parts of the keys' pass [2][parts][rows, Hkv, d], when there are parts
    int parts;
    // cache
    void *k_cache, *v_cache;
    const long long *pos;
};

// The window: key j of a sequence is seen by query i.
__device__ __forceinline__ bool swa_sees(int i, int j, int window, int sinks) {
    return j <= i && (i - j < window || j < sinks);
}

// Key tiles of BN that queries [i0, i1) of a sequence see, in order: `near` tiles from tile `lo` that
// the window reaches, and before them the `far` first tiles that hold sinks only.
struct KeyTiles {
    int far, lo, near;
    KeyTiles() = default;
    __device__ __forceinline__ KeyTiles(int i0, int i1, int BN, int window, int sinks) {
        lo = i0 - window + 1 > 0 ? (i0 - window + 1) / BN : 0;
        near = (i1 - 1) / BN - lo + 1;
        const int s = sinks < i1 ? sinks : i1;
        far = (s + BN - 1) / BN;
        far = far < lo ? far : lo;
    }
    __device__ __forceinline__ int count() const { return far + near; }
    __device__ __forceinline__ int tile(int x) const { return x < far ? x : lo + x - far; }
};

// Last query of a sequence of `len` tokens that sees a key of [j0, j1).
__device__ __forceinline__ int last_query(int j0, int j1, int len, int window, int sinks) {
    if (j0 < sinks) return len - 1;
    const long long i = (long long)j1 - 1 + window - 1;
    return i < len - 1 ? (int)i : len - 1;
}

// Polls of a bounded barrier wait of the tensor-core kernels here (each poll may suspend the thread
// for a while: of the order of a second, far beyond any copy or product that completes).
constexpr uint32_t kSwaWait = 1u << 22;
constexpr uint32_t kIdleWait = 1u << 17;   // of polls that suspend for up to 20 us

// sizes of the delta rule's buffers for one path, in bytes
struct GdrSizes {
    size_t prep, saved, bwd;
};
GdrSizes gdr_simt_sizes(const Seqs &s, int Hv, int K, int V);
cudaError_t launch_gdr_fwd_simt(int K, int V, const GdrArgs &a, bool save, cudaStream_t st);
cudaError_t launch_gdr_bwd_simt(int K, int V, const GdrArgs &a, cudaStream_t st);
// dA_dec, dtau [Hv] from the tiles' partial sums [tiles][Hv][2], in a fixed order
void launch_gdr_reduce_decay(const float *p, long long tiles, int Hv, float *dA_dec, float *dtau, cudaStream_t st);
GdrSizes gdr_tc_sizes(const Seqs &s, int Hv, int K, int V);
cudaError_t launch_gdr_fwd_tc(int K, int V, const GdrArgs &a, bool save, cudaStream_t st);
cudaError_t launch_gdr_bwd_tc(int K, int V, const GdrArgs &a, cudaStream_t st);
cudaError_t launch_gdr_step(int K, int V, bool bf16, const GdrArgs &a, cudaStream_t st);
cudaError_t launch_swa_fwd_simt(const SwaArgs &a, cudaStream_t st);
cudaError_t launch_swa_bwd_simt(const SwaArgs &a, cudaStream_t st);
cudaError_t launch_swa_fwd_tc(const SwaArgs &a, cudaStream_t st);
cudaError_t launch_swa_bwd_tc(const SwaArgs &a, cudaStream_t st);
int swa_bwd_parts(const SwaArgs &a);
int swa_fwd_take_status();
int swa_bwd_take_status();
int swa_fill_take_bad_seqlens();
cudaError_t launch_swa_check(const Seqs &s, cudaStream_t st);   // the offsets alone (no rows)
cudaError_t launch_swa_fill(bool bf16, const SwaArgs &a, cudaStream_t st);
cudaError_t launch_swa_step(bool bf16, const SwaArgs &a, cudaStream_t st);
int gdr_tc_fwd_take_timeout();
int gdr_tc_bwd_take_timeout();
int gdr_take_bad_seqlens();
int gdr_tc_fwd_take_bad_seqlens();
int gdr_tc_bwd_take_bad_seqlens();
int swa_take_bad_seqlens();
// kTimedOut, kBadOffsets of all kernels of a mixer since the last call (0 when none ran)
int gdr_take_status();
int swa_take_status();

}  // namespace carve
