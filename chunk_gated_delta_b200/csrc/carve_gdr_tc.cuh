// Scalar-gated delta rule on the tensor core (bf16 tensors): the chunked form and the layouts that
// its kernels share.
//
// Chunks of kC = 64 tokens, start state S0, G_t = sum of log a over the chunk up to t, D[t,s] =
// e^{G_t - G_s} (only s <= t, so never above 1):
//   M[t,s] = w_t D[t,s] k_t.k_s (s < t),  Tm = (I + M)^-1,  A[t,s] = D[t,s] q_t.k_s (s <= t)
//   R = V - e^G K S0^T,  U = Tm (w R),  O = e^G Q S0^T + A U,  S1 = e^{G_C} S0 + (e^{G_C - G} U)^T K
// The decay is one scalar a token, so it never touches a matrix operand: K, Q, V, dO enter the
// products as the bf16 values that they are, and the factors act on fp32 accumulators.  Operands that
// are results (S, w R, e^{G_C - G} U, Tm) are split into two bf16 terms, hi + lo (16 bits
// together), where they carry the state; so the state that a prompt leaves is good to a few 1e-6.
//
// Tiles are in the tensor core's operand layout (carve_umma.cuh): blocks of rows x 64 channels, 128
// bytes a row, 16-byte chunk c of row r at c ^ (r % 8).
#pragma once
#include "carve_mixers.cuh"
#include "carve_umma.cuh"

namespace carve {

constexpr int kC = 64;
constexpr uint32_t kTile64 = kC * 128;   // bytes of a 64-row block

// Per (tile, value head), written by the preparation: Tm hi, Tm lo, A (each [64][64]), then vectors.
struct GdrPrep {
    __nv_bfloat16 t_hi[kC * 64], t_lo[kC * 64], A[kC * 64];
    float eG[kC], eK[kC], w[kC], G[kC];   // e^{G_t}, e^{G_C - G_t}, w_t, G_t
};
static_assert(sizeof(GdrPrep) == 25600, "slots are copied in bulk");

// Per (tile, value head): the state [V][K] and a token tile [64][V], bf16 operand layout.
template <int K, int V>
struct GdrKeep {
    __nv_bfloat16 S[V * K], x[kC * V];
};

// element offset of (row r, column c) in a tile of `rows` rows
__device__ __forceinline__ int op_off(int r, int c, int rows) { return umma_off(r, c, rows); }

__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

// zero rows `first` .. 63 of a [64][64 x halves] tile whose halves are `stride` bytes apart (one warp)
__device__ __forceinline__ void zero_rows(void *tile, int first, int halves, uint32_t stride, int lane) {
    for (int y = 0; y < halves; ++y)
        for (int i = first * 8 + lane; i < kC * 8; i += 32)
            reinterpret_cast<uint4 *>(static_cast<char *>(tile) + y * stride)[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Column of 16 tokens (slice kk of 4) of a split [lane][64 tokens] operand in tensor memory: each half
// of 32 tokens keeps its hi terms (16 columns) and then its lo terms, over the 32 columns of the
// accumulator it comes from, so a thread overwrites only what it has read itself.
__device__ __forceinline__ uint32_t half_col(int kk) { return 32 * (kk / 2) + 8 * (kk % 2); }

constexpr uint32_t kUmmaAmn = 1u << 15;   // instruction descriptor: A is MN-contiguous

}  // namespace carve
