// Scalar-gated delta rule on the tensor core (bf16 tensors): the chunked form and the layouts that
// its kernels share.
//
// Chunks of kC = 64 tokens, start state S0, G_t = sum of log a over the chunk up to t, D[t,s] =
// e^{G_t - G_s} (only s <= t, so never above 1):
//   M[t,s] = w_t D[t,s] k_t.k_s (s < t),  Tm = (I + M)^-1,  A[t,s] = D[t,s] q_t.k_s (s <= t)
//   R = V - e^G K S0^T,  U = Tm (w R),  O = e^G Q S0^T + A U,  S1 = e^{G_C} S0 + (e^{G_C - G} U)^T K
// G is a sum in two floats (carve_mixers.cuh); its low part enters D as a factor of the row and one of the column.
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
    float eG[kC], eK[kC], w[kC], G[kC];   // e^{G_t}, e^{G_C - G_t}, w_t, G_t log2 e
    float eB[kC], rL[kC];                 // e^{G_r - G_t}, r the last of t's 16 tokens; e^{-G_t's low part}
    float pad[128];
};
static_assert(sizeof(GdrPrep) == 26624, "slots are copied in bulk, tiles on 1024-byte boundaries");
constexpr uint32_t kVecBytes = 6 * kC * 4;   // eG .. rL

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

// The sweeps' register warps: four a lane quarter, each with a quarter of the columns (state) or 16
// of the chunk's tokens.  Half as many threads with twice the columns spilled (6.8 us a chunk), and with shared
// memory taken by the tiles a spill goes to L2.  At d = 128 the sweeps still spill a little, 54 to 70 bytes a thread
// forward, 120 backward.
constexpr int kRegWarps = 16, kSweepThreads = (kRegWarps + 4) * 32;
// Registers: 640 threads start with 96 (61440 in all); the register warps take 112 and the others go
// down to 32 (512 x 112 + 128 x 32 = 61440), or 104 and 64.
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }

// A split [lane][64 tokens] operand in tensor memory lies over the accumulator it comes from: 16
// tokens' hi terms in 8 columns, then their lo terms, so that a warp overwrites only what it has read
// itself.
__device__ __forceinline__ uint32_t split_col(int kk, int lo) { return 16 * kk + 8 * lo; }

// A register warp's 32 value rows x 16 tokens of an accumulator as fragments: x[y][4 j + 2 i + e] is row
// 16 y + 8 i + lane / 4, token 8 j + 2 (lane % 4) + e.  In this layout a token tile's rows [token][channel]
// are read and written by ldmatrix / stmatrix.trans (two each) and a factor of the tokens is two
// 8-byte loads; with a lane a row they took 16 two-byte accesses and 16 loads.
struct Frag {
    float x[2][8];
    __device__ __forceinline__ void load(uint32_t taddr) {   // followed by ready()
        tmem_ld_frag2(taddr, reinterpret_cast<uint32_t *>(x[0]));
        tmem_ld_frag2(taddr + (16u << 16), reinterpret_cast<uint32_t *>(x[1]));
    }
    __device__ __forceinline__ void ready() { tmem_tie16(reinterpret_cast<uint32_t *>(x[0])); }
};
// the thread's four of 16 factors
struct Factor {
    float f[4];
    __device__ __forceinline__ Factor(const float *p, int lane) {
        const float2 a = *reinterpret_cast<const float2 *>(p + 2 * (lane % 4)), b = *reinterpret_cast<const float2 *>(p + 8 + 2 * (lane % 4));
        f[0] = a.x;
        f[1] = a.y;
        f[2] = b.x;
        f[3] = b.y;
    }
    __device__ __forceinline__ float operator[](int i) const { return f[2 * (i / 4) + i % 2]; }   // of x[.][i]
};
// fragments as a split operand over the accumulator at taddr
__device__ __forceinline__ void put_split(uint32_t taddr, const Frag &a) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        uint32_t p[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_pair(a.x[y][2 * i], a.x[y][2 * i + 1], p[i], p[4 + i]);
        tmem_st_frag4(taddr + ((16u * y) << 16), p);
    }
}
// the address of this lane's row of the four 8 x 8 matrices (tokens c16 .. + 15, channels r0 .. + 15) of a
// [64][channels] tile in operand layout
__device__ __forceinline__ uint32_t tile_row(const __nv_bfloat16 *tile, int c16, int r0, int lane) {
    return smem_u32(tile + op_off(c16 + (lane / 16) * 8 + lane % 8, r0 + ((lane / 8) & 1) * 8, kC));
}
__device__ __forceinline__ void load_tokens(uint32_t (&v)[2][4], const __nv_bfloat16 *tile, int c16, int r0, int lane) {
    ldsm_x4_t(v[0], tile_row(tile, c16, r0, lane));
    ldsm_x4_t(v[1], tile_row(tile, c16, r0 + 16, lane));
}
__device__ __forceinline__ float bf16_of(const uint32_t (&v)[4], int i) {   // x[.][i]'s counterpart
    return __uint_as_float(i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
}
__device__ __forceinline__ void store_tokens(__nv_bfloat16 *tile, int c16, int r0, int lane, const Frag &a) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
        stsm_x4_t(tile_row(tile, c16, r0 + 16 * y, lane), pack_bf16(a.x[y][0], a.x[y][1]), pack_bf16(a.x[y][2], a.x[y][3]),
                  pack_bf16(a.x[y][4], a.x[y][5]), pack_bf16(a.x[y][6], a.x[y][7]));
}
// a [64][V] tile in operand layout to rows row .. of head h (one warp, its own bulk group): by TMA, or, when only m
// rows are the sequence's, row by row
template <int V>
__device__ __forceinline__ void store_tile(const CUtensorMap *map, void *dst, const __nv_bfloat16 *tile, long long row, int m, int H,
                                           int h, int lane) {
    if (m >= kC) {
        if (elect_one()) {
            for (int x = 0; x < V / 64; ++x) tma_store_3d(map, tile + x * kC * 64, 64 * x, h, (int)row);
            bulk_commit();
            bulk_wait_read<0>();
        }
    } else {
        for (int i = lane; i < m * (V / 8); i += 32) {
            const int t = i / (V / 8), x = i % (V / 8) * 8;
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(dst) + ((size_t)(row + t) * H + h) * V + x) =
                *reinterpret_cast<const uint4 *>(tile + op_off(t, x, kC));
        }
    }
    __syncwarp();
}
// A row's part of the state, COLS columns from x0: operands hi, lo and the accumulator times gl; the hi
// terms stay in hi[] when the state is kept
template <int COLS>
__device__ __forceinline__ void put_state(uint32_t acc, uint32_t hi_at, uint32_t lo_at, const float *S, float gl, uint32_t *hi) {
#pragma unroll
    for (int b = 0; b < COLS; b += 16) {
        uint32_t lo[8], sc[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) split_pair(S[b + 2 * i], S[b + 2 * i + 1], hi[b / 2 + i], lo[i]);
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[i] = __float_as_uint(S[b + i] * gl);
        tmem_st8(hi_at + b / 2, hi + b / 2);
        tmem_st8(lo_at + b / 2, lo);
        tmem_st16(acc + b, sc);
    }
    tmem_wait_st();
    tc_fence_before_sync();
}
template <int COLS>
__device__ __forceinline__ void get_state(uint32_t acc, float *S) {
    uint32_t *x = reinterpret_cast<uint32_t *>(S);
#pragma unroll
    for (int b = 0; b < COLS; b += 16) tmem_ld16(acc + b, x + b);
    tmem_wait_ld();
#pragma unroll
    for (int b = 0; b < COLS; b += 16) tmem_tie16(x + b);
}
template <int COLS>
__device__ __forceinline__ void load_row(float *S, const float *src) {
#pragma unroll
    for (int x = 0; x < COLS; x += 4) {
        const float4 y = src ? *reinterpret_cast<const float4 *>(src + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        S[x] = y.x;
        S[x + 1] = y.y;
        S[x + 2] = y.z;
        S[x + 3] = y.w;
    }
}
template <int COLS>
__device__ __forceinline__ void store_row(float *dst, const float *S) {
#pragma unroll
    for (int x = 0; x < COLS; x += 4) *reinterpret_cast<float4 *>(dst + x) = make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]);
}

// A kernel that reads what the one before it in the stream writes may start beside that one's last CTAs
// (launch_after) and sets itself up; what it reads of it comes after wait_for_last().  Its own
// outputs touch nothing that the last kernel reads.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// `early` false: an ordinary launch, after everything before it (where that is not a kernel of the same call)
template <class... P, class... A>
cudaError_t launch_after(bool early, void (*kern)(P...), unsigned grid, unsigned block, int smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

constexpr uint32_t kUmmaAmn = 1u << 15;   // instruction descriptor: A is MN-contiguous

}  // namespace carve
