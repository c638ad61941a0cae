// Scalar-gated delta rule, forward, on the 5th-generation tensor core (carve_gdr_tc.cuh).
//
// gdr_tc_prep: one CTA per (tile, key head) forms [Q; K] K^T with one M = 128 product and, for each
// value head of the key head, the decayed A and M, Tm by blocked inversion (fp32 substitution on the
// diagonal, three tf32 products off it), and the gate vectors.  It needs no state, so all tiles run
// at once; instruction issue and latency bound it (8 sequences of 4096 tokens, 16 heads, d = 128: 111
// us, 4.5 TB/s; four CTAs an SM and gates after the product 123, with the inverse in plain fp32 and an
// exponential a pair 204).
//
// gdr_tc_sweep: one CTA per (sequence, value head) carries the state through the chunks.  The state is
// a tensor-memory accumulator with the value channels as its 128 lanes, so every product of the
// recurrence has A in tensor memory (what the last step produced) and B in shared memory (K, Q, Tm or
// A as copied), and a thread owns a quarter of a state row:
//   G = S K^T (hi, lo), Q S^T       -> R = w (v - e^G G), split
//   U = R Tm^T (three terms)        -> e^{G_C - G} U, split; U
//   S += (e^{G_C - G} U) K (hi, lo)  -> S split for the next chunk, S scaled by its e^{G_C}
//   O = e^G Q S^T + U A^T (S, U hi, lo), two accumulators, off the chain
// The chain of one chunk is three products and three register passes; what bounds the sweep is
// their latency (B H units on 148 SMs, one chain each): 2.9 us a chunk, of which the products
// take 1.2.  With the states kept (the sizes above: 230 us, 1.15 GB) HBM is as near, 5.0 TB/s.
// Chunks of 64: the products of 128 tokens need 576 columns of tensor memory, and an inverse of four
// times the work.
// Warps 0-15 register passes, 16 copies in (TMA and bulk, two stages), 17 products, 18 and 19 copies out.  What
// is not on the chain (outputs of the chunk before, copies of S and U) is done while a product runs.
#include "carve_gdr_tc.cuh"

namespace carve {

__device__ int g_gdr_timeout;   // set when a bounded wait gives up (never expected)
__device__ int g_gdr_tc_bad_seqlens;

int gdr_tc_fwd_take_timeout() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gdr_timeout, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_gdr_timeout, &z, sizeof(int));
    }
    return v;
}
int gdr_tc_fwd_take_bad_seqlens() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gdr_tc_bad_seqlens, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_gdr_tc_bad_seqlens, &z, sizeof(int));
    }
    return v;
}

namespace {

constexpr int LM = 68;   // row stride of the fp32 64 x 64 matrices

template <int K>
struct PrepSmem {
    union {
        __nv_bfloat16 qk[K / 64][128 * 64];   // [Q; K], rows 0-63 and 64-127
        struct {
            union {
                float M[kC][LM];
                __nv_bfloat16 t[2][kC * 64];   // Tm hi, lo on their way out
            };
            float X[kC][LM];
        };
    };
    __nv_bfloat16 A[kC * 64];
    float eG[kC], eK[kC], w[kC], G[kC], eB[kC], rL[kC], half[2];
    uint64_t full, done;
    uint32_t tmem;
};

// acc (16 x 16, m16n8 fragments) = A B over KD terms of fp32 matrices in shared memory (row stride LM), by
// one warp: each factor in two tf32 terms, three products, about 2^-21 relative
template <int KD>
__device__ __forceinline__ void mm16(float (&acc)[2][4], const float *A, const float *B, int lane) {
    const int g = lane / 4, c = lane % 4;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    auto mma = [](float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
        asm volatile(
            "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    };
    auto split = [](float x, uint32_t &hi, uint32_t &lo) {
        hi = __float_as_uint(x) & 0xffffe000u;
        lo = __float_as_uint(x - __uint_as_float(hi));
    };
#pragma unroll
    for (int k = 0; k < KD; k += 8) {
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split(A[(g + 8 * (i % 2)) * LM + k + c + 4 * (i / 2)], ah[i], al[i]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) split(B[(k + c + 4 * i) * LM + 8 * n + g], bh[i], bl[i]);
            mma(acc[n], al, bh);
            mma(acc[n], ah, bl);
            mma(acc[n], ah, bh);
        }
    }
}
// C (16 x 16 at row stride LM) = f acc
__device__ __forceinline__ void put16(float *C, const float (&acc)[2][4], float f, int lane) {
    const int g = lane / 4, c = 2 * (lane % 4);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2 *>(C + (g + 8 * i) * LM + 8 * n + c) = make_float2(f * acc[n][2 * i], f * acc[n][2 * i + 1]);
}

// The lower blocks of X = (I + M)^-1 for a strictly lower-triangular M (64 x 64; its blocks of 16 above the
// diagonal are not read); M is overwritten.  16 x 16 diagonal blocks by substitution in fp32, then
// off-diagonal blocks by T21 = -T22 (M21 T11), first of size 16 (a warp each), then of size 32.  128 threads.
__device__ __forceinline__ void invert64(float (*M)[LM], float (*X)[LM]) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid < kC) {   // column c of a block
        const int o = tid / 16 * 16, c = tid % 16;
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float y = t == c ? 1.f : 0.f;
#pragma unroll
            for (int s = 0; s < t; s += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(&M[o + t][o + s]);
                const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (s + e < t) y = fmaf(-mm[e], x[s + e], y);
            }
            x[t] = y;
            X[o + t][o + c] = y;
        }
    }
    __syncthreads();
    float acc[2][4];
    if (warp < 2) {
        const int o = 32 * warp;
        mm16<16>(acc, &M[o + 16][o], &X[o][o], lane);
        __syncwarp();
        put16(&M[o + 16][o], acc, 1.f, lane);
        __syncwarp();
        mm16<16>(acc, &X[o + 16][o + 16], &M[o + 16][o], lane);
        put16(&X[o + 16][o], acc, -1.f, lane);
    }
    __syncthreads();
    const int r = warp / 2 * 16, c = warp % 2 * 16;
    mm16<32>(acc, &M[32 + r][0], &X[0][c], lane);
    __syncthreads();
    put16(&M[32 + r][c], acc, 1.f, lane);
    __syncthreads();
    mm16<32>(acc, &X[32 + r][32], &M[32][c], lane);
    put16(&X[32 + r][c], acc, -1.f, lane);
    __syncthreads();
}

template <int K>
__global__ void __launch_bounds__(128) gdr_tc_prep(GdrArgs a, const __grid_constant__ CUtensorMap mq,
                                                   const __grid_constant__ CUtensorMap mk) {
    // Without room for alignment five CTAs share an SM (four with it); no static shared memory stands before this
    extern __shared__ __align__(1024) unsigned char raw[];
    PrepSmem<K> &sm = *reinterpret_cast<PrepSmem<K> *>(raw);
    if (smem_u32(raw) & 1023u) {
        if (threadIdx.x == 0) atomicOr(&g_gdr_timeout, 1);
        return;
    }
    const int tile = blockIdx.x / a.Hk, hk = blockIdx.x % a.Hk, share = a.Hv / a.Hk;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    int n, c, len;
    long long row;
    if (!a.seq.find(tile, kC, n, c, row, len)) return;
    row += (long long)c * kC;
    const int m = min(kC, len - c * kC);
    if (tid == 0) {
        mbar_init(&sm.full, 1);
        mbar_init(&sm.done, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(&sm.tmem, 64);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;
    let_next_start();   // not before the allocation: a sweep's CTA takes all tensor memory of its SM and waits for this kernel
    bool ok = true;
    if (warp == 3) {
        if (elect_one()) {
            mbar_expect_tx(&sm.full, 128 * K * 2);
            for (int x = 0; x < K / 64; ++x) {
                tma_load_3d(sm.qk[x], &mq, 64 * x, hk, (int)row, &sm.full);
                tma_load_3d(sm.qk[x] + kC * 64, &mk, 64 * x, hk, (int)row, &sm.full);
            }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&sm.full, 0, kSwaWait));
        if (ok && elect_one()) {
#pragma unroll
            for (int kk = 0; kk < K / 16; ++kk)
                umma_bf16(tm, umma_desc(smem_u32(sm.qk[kk / 4]) + 32 * (kk % 4)),
                          umma_desc(smem_u32(sm.qk[kk / 4]) + kTile64 + 32 * (kk % 4)), umma_idesc_bf16(128, 64), kk > 0);
            umma_commit(&sm.done);
        }
        __syncwarp();
    }
    // gates of a head and the running sums of log a, by warps 0 and 1; rows behind the end: log a = 0, w = 0
    auto gates = [&](int h) {
        if (tid >= kC) return;
        float la = 0.f, lo = 0.f, w = 0.f;
        if (tid < m) {
            const size_t at = (size_t)(row + tid) * a.Hv + h;
            const float x = ld_io(static_cast<const __nv_bfloat16 *>(a.g_logit) + at) + (a.tau ? a.tau[h] : 0.f);
            la = least_log(-1.4426950408889634f * decay_amp(a.A_dec, h) * softplus_f(x));
            w = sigmoid_f(ld_io(static_cast<const __nv_bfloat16 *>(a.w_logit) + at));
        }
        sum2_scan(la, lo, lane);
        if (tid == 31) {
            sm.half[0] = la;
            sm.half[1] = lo;
        }
        asm volatile("bar.sync 1, 64;\n" ::: "memory");
        if (warp == 1) sum2_add(la, lo, sm.half[0], sm.half[1]);
        sm.G[tid] = la;
        sm.rL[tid] = exp2f(-lo);
        sm.w[tid] = w;
        asm volatile("bar.sync 1, 64;\n" ::: "memory");
        sm.eG[tid] = exp2f(la);
        sm.eK[tid] = exp2f(sm.G[kC - 1] - la) * (sm.rL[tid] / sm.rL[kC - 1]);
        sm.eB[tid] = exp2f(sm.G[tid | 15] - la) * (sm.rL[tid] / sm.rL[tid | 15]);
    };
    gates(hk * share);   // the first head's while the tiles and their product are under way
    ok = ok && mbar_wait(&sm.done, 0, kSwaWait);
    if (__syncthreads_or(!ok)) {   // give up together, with the copy landed and the product finished
        if (tid == 0) {
            atomicOr(&g_gdr_timeout, 1);
            mbar_wait(&sm.full, 0, kSwaWait);
        }
        __syncthreads();
        if (warp == 0) tmem_dealloc(tm, 64);
        return;
    }
    tc_fence_after_sync();
    // row tid of [Q; K] K^T: q_t.k_s for tid = t < 64, k_t.k_s for tid = 64 + t; A in the lower half of
    // sm.A, M (w D k.k below the diagonal) in sm.M; blocks of 16 above the diagonal stay zero
    const int t = tid % kC;
    const bool key = tid >= kC, here = t < m;
    for (int i = tid; i < kC * 8; i += 128) reinterpret_cast<uint4 *>(sm.A)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < kC * LM / 4; i += 128) reinterpret_cast<float4 *>(sm.X)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
        if (h > hk * share) {
            if (tid == 0) bulk_wait_read<0>();   // the last head's copies out have left the buffers
            __syncthreads();
            gates(h);
            __syncthreads();
        }
        const float Gt = sm.G[t], f0 = (key ? sm.w[t] : 1.f) / sm.rL[t];   // D[t,s] = 2^{G_t - G_s} rL_s / rL_t
#pragma unroll 1
        for (int s0 = 0; s0 <= (t | 31); s0 += 16) {
            uint32_t g[16];
            tmem_ld16(tm + ((uint32_t)warp << 21) + s0, g);
            tmem_wait_ld();
            tmem_tie16(g);
            float y[16];
            if (s0 + 15 < (t & 32)) {   // all below the diagonal: one factor a row, one a column
                const float f = f0 * ex2(Gt - sm.G[s0 + 15]) * sm.rL[s0 + 15];
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = here ? f * sm.eB[s0 + e] * __uint_as_float(g[e]) : 0.f;
            } else {
                const int lim = here ? t + !key - s0 : 0;   // s < t, and s = t for queries
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = e < lim ? f0 * ex2(Gt - sm.G[s0 + e]) * sm.rL[s0 + e] * __uint_as_float(g[e]) : 0.f;
            }
            if (!key) {
#pragma unroll
                for (int e = 0; e < 16; e += 8)
                    *reinterpret_cast<uint4 *>(sm.A + op_off(t, s0 + e, kC)) =
                        make_uint4(pack_bf16(y[e], y[e + 1]), pack_bf16(y[e + 2], y[e + 3]), pack_bf16(y[e + 4], y[e + 5]), pack_bf16(y[e + 6], y[e + 7]));
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4 *>(&sm.M[t][s0 + e]) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
        }
        __syncthreads();
        invert64(sm.M, sm.X);
        {   // Tm into two bf16 terms
            const int r = tid / 2, c0 = tid % 2 * 32;
#pragma unroll
            for (int x = c0; x < c0 + 32; x += 8) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split_pair(sm.X[r][x + 2 * e], sm.X[r][x + 2 * e + 1], hi[e], lo[e]);
                *reinterpret_cast<uint4 *>(sm.t[0] + op_off(r, x, kC)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(sm.t[1] + op_off(r, x, kC)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            GdrPrep *out = reinterpret_cast<GdrPrep *>(a.prep) + (size_t)tile * a.Hv + h;
            bulk_s2g(out->t_hi, sm.t, sizeof(sm.t));
            bulk_s2g(out->A, sm.A, sizeof(sm.A));
            bulk_s2g(out->eG, sm.eG, kVecBytes);
            bulk_commit();
        }
    }
    if (tid == 0) bulk_wait_read<0>();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, 64);
}

template <int K, int V, bool SAVE>
struct SweepSmem {
    __nv_bfloat16 k[2][K / 64][kC * 64], q[2][K / 64][kC * 64];
    GdrPrep p[2];
    __nv_bfloat16 v[2][V / 64][kC * 64];
    __nv_bfloat16 S[SAVE ? V * K : 512], u[SAVE ? kC * V : 512], o[kC * V];   // on their way out
    float eG[2][kC];   // kept for the outputs beyond the stage
    uint64_t full[2], free[2], sready, gfull, rready, ufull, uready, sfull, ofull, oread, ofree;
    uint64_t Sout, Sfree, uout, ufree, oout, drain;
    uint32_t tmem;
};

template <int K, int V, bool SAVE>
__global__ void __launch_bounds__(kSweepThreads, 1)
    gdr_tc_sweep(GdrArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    extern __shared__ __align__(1024) unsigned char raw[];
    typedef SweepSmem<K, V, SAVE> Smem;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    constexpr int KH = K / 64, KQ = K / 4;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int h = blockIdx.x % a.Hv, n = blockIdx.x / a.Hv, hk = h / (a.Hv / a.Hk);
    long long row0;
    int len;
    a.seq.rows(n, row0, len, threadIdx.x == 0 ? &g_gdr_tc_bad_seqlens : nullptr);
    const long long t0 = a.seq.tile0(n, kC);
    const int chunks = (len + kC - 1) / kC;
    if (threadIdx.x == 0) {
        for (uint64_t *b : {&sm.full[0], &sm.full[1], &sm.free[0], &sm.free[1], &sm.gfull, &sm.ufull, &sm.sfull,
                            &sm.ofull, &sm.Sfree, &sm.ufree, &sm.ofree, &sm.drain})
            mbar_init(b, 1);
        for (uint64_t *b : {&sm.sready, &sm.rready, &sm.uready, &sm.oread, &sm.Sout, &sm.uout, &sm.oout}) mbar_init(b, kRegWarps);
        fence_mbar_init();
    }
    if (warp == kRegWarps + 1) tmem_alloc(&sm.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;
    // tensor memory: S 0-127, S hi 128, S lo 192, G (then R hi, lo, then U hi, lo) 256, U (then
    // e^{G_C - G} U hi, lo) 320, Q S^T 384, U A^T 448
    constexpr uint32_t cHi = 128, cLo = 192, cG = 256, cU = 320, cQ = 384, cA = 448;
    bool ok = true;
    auto wait = [&](uint64_t &bar, int phase) {   // by a whole warp
        return mbar_wait_warp(&bar, phase & 1, kIdleWait);
    };

    if (warp >= kRegWarps) regs_down<64>();
    if (warp == kRegWarps) {
        wait_for_last();   // the preparation
        int c = 0;
        for (; c < chunks; ++c) {
            const int s = c & 1;
            if (c >= 2) ok = wait(sm.free[s], c / 2 - 1);
            if (!ok) break;
            if (elect_one()) {
                const int row = (int)(row0 + (long long)c * kC);
                mbar_expect_tx(&sm.full[s], 2 * kC * K * 2 + kC * V * 2 + sizeof(GdrPrep));
                for (int x = 0; x < KH; ++x) tma_load_3d(sm.k[s][x], &mk, 64 * x, hk, row, &sm.full[s]);
                bulk_g2s(&sm.p[s], reinterpret_cast<const GdrPrep *>(a.prep) + (size_t)(t0 + c) * a.Hv + h, sizeof(GdrPrep),
                         &sm.full[s]);
                for (int x = 0; x < V / 64; ++x) tma_load_3d(sm.v[s][x], &mv, 64 * x, h, row, &sm.full[s]);
                for (int x = 0; x < KH; ++x) tma_load_3d(sm.q[s][x], &mq, 64 * x, hk, row, &sm.full[s]);
            }
        }
        if (!ok)
            for (int i = max(0, c - 2); i < c; ++i) wait(sm.full[i & 1], i / 2);
    } else if (warp == kRegWarps + 1) {
        constexpr uint32_t iN64 = umma_idesc_bf16(128, 64), iS = umma_idesc_bf16(128, K) | kUmmaBmn;
        const uint64_t dk0 = umma_desc(smem_u32(sm.k)), dq0 = umma_desc(smem_u32(sm.q)), dt0 = umma_desc(smem_u32(sm.p)),
                       ds0 = umma_desc_mn(smem_u32(sm.k), kTile64);
        for (int c = 0; c < chunks; ++c) {
            const int s = c & 1;
            const uint64_t dk = desc_at(dk0, s * KH * kTile64), dq = desc_at(dq0, s * KH * kTile64),
                           dt = desc_at(dt0, s * sizeof(GdrPrep)), ds = desc_at(ds0, s * KH * kTile64);
            if (!(ok = wait(sm.full[s], c / 2))) break;
            if (len - c * kC < kC) {   // key rows behind the end meet U = 0 in the state update
                zero_rows(sm.k[s], len - c * kC, KH, kTile64, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (!(ok = wait(sm.sready, c))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < K / 16; ++kk)
                        umma_bf16_ta(tm + cG, tm + (lo ? cLo : cHi) + 8 * kk, desc_at(dk, kTile64 * (kk / 4) + 32 * (kk % 4)),
                                     iN64, lo > 0 || kk > 0);
                umma_commit(&sm.gfull);
            }
            __syncwarp();
            if (!(ok = wait(sm.rready, c))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int x = 0; x < 3; ++x)   // R hi Tm hi, R lo Tm hi, R hi Tm lo
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tm + cU, tm + cG + split_col(kk, x == 1), desc_at(dt, (x == 2 ? kTile64 : 0) + 32 * kk), iN64,
                                     x > 0 || kk > 0);
                umma_commit(&sm.ufull);
            }
            __syncwarp();
            // in the shadow of the pass over U
            if (c > 0 && !(ok = wait(sm.oread, c - 1))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < K / 16; ++kk)
                        umma_bf16_ta(tm + cQ, tm + (lo ? cLo : cHi) + 8 * kk, desc_at(dq, kTile64 * (kk / 4) + 32 * (kk % 4)),
                                     iN64, lo > 0 || kk > 0);
            }
            __syncwarp();
            if (!(ok = wait(sm.uready, c))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tm, tm + cU + split_col(kk, lo), desc_at(ds, 2048 * kk), iS, 1);
                umma_commit(&sm.sfull);
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) 
                        umma_bf16_ta(tm + cA, tm + cG + split_col(kk, lo), desc_at(dt, 2 * kTile64 + 32 * kk), iN64, lo > 0 || kk > 0);
                umma_commit(&sm.ofull);
                umma_commit(&sm.free[s]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(&sm.drain);   // products in flight finish before the tensor memory is freed
        __syncwarp();
        wait(sm.drain, 0);
    } else if (warp == kRegWarps + 2) {
        typedef GdrKeep<K, V> Keep;
        Keep *keep = SAVE ? reinterpret_cast<Keep *>(a.saved) + (size_t)t0 * a.Hv + h : nullptr;
        for (int c = 0; SAVE && c < chunks; ++c) {
            if (!(ok = wait(sm.Sout, c))) break;
            if (elect_one()) {
                bulk_s2g(keep[(size_t)c * a.Hv].S, sm.S, sizeof(sm.S));
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&sm.Sfree);
            }
            __syncwarp();
            if (!(ok = wait(sm.uout, c))) break;
            if (elect_one()) {
                bulk_s2g(keep[(size_t)c * a.Hv].x, sm.u, sizeof(sm.u));
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&sm.ufree);
            }
            __syncwarp();
        }
        bulk_wait<0>();
    } else if (warp == kRegWarps + 3) {
        for (int c = 0; c < chunks; ++c) {
            if (!(ok = wait(sm.oout, c))) break;
            store_tile<V>(&mo, a.o, sm.o, row0 + (long long)c * kC, len - c * kC, a.Hv, h, lane);
            if (elect_one()) mbar_arrive(&sm.ofree);
            __syncwarp();
        }
        bulk_wait<0>();
    } else if (warp < kRegWarps) {
        regs_up<104>();
        const int part = warp / 4, quarter = warp % 4, r = quarter * 32 + lane;
        const uint32_t tl = tm + ((uint32_t)quarter << 21);
        const int x0 = part * KQ, c16 = part * 16;   // this warp's columns of S, its tokens
        const bool live = quarter * 32 < V;          // value rows (others carry zeros)
        const size_t st = (((size_t)n * a.Hv + h) * V + (live ? r : 0)) * K + x0;
        float S[KQ];
        load_row<KQ>(S, live && a.S0 ? a.S0 + st : nullptr);
        Frag y;
        for (int c = 0; c <= chunks; ++c) {
            const GdrPrep &p = sm.p[c & 1];
            uint32_t hi[KQ / 2];
            if (c < chunks) {
                if (!(ok = wait(sm.full[c & 1], c / 2))) break;
                put_state<KQ>(tl + x0, tl + cHi + x0 / 2, tl + cLo + x0 / 2, S, p.eG[kC - 1], hi);
                mbar_arrive_warp(&sm.sready);
            }
            if (c > 0) {   // outputs of the chunk before, while the product runs
                const Factor eG(sm.eG[(c - 1) & 1] + c16, lane);
                if (!(ok = wait(sm.ofull, c - 1))) break;
                tc_fence_after_sync();
                Frag z;
                y.load(tl + cQ + c16);
                z.load(tl + cA + c16);
                tmem_wait_ld();
                y.ready();
                z.ready();
                tc_fence_before_sync();
                mbar_arrive_warp(&sm.oread);
#pragma unroll
                for (int e = 0; e < 16; ++e) y.x[e / 8][e % 8] = fmaf(eG[e % 8], y.x[e / 8][e % 8], z.x[e / 8][e % 8]);
                if (c > 1 && !(ok = wait(sm.ofree, c - 2))) break;
                if (live) store_tokens(sm.o, c16, quarter * 32, lane, y);
                fence_proxy_async_smem();
                mbar_arrive_warp(&sm.oout);
            }
            if (c == chunks) break;
            const int m = min(kC, len - c * kC);
            if (quarter == 0 && lane < 16) sm.eG[c & 1][c16 + lane] = p.eG[c16 + lane];
            // R = w (v - e^G G)
            {
                uint32_t v[2][4] = {};
                if (live) load_tokens(v, sm.v[c & 1][0], c16, quarter * 32, lane);
                const Factor eG(p.eG + c16, lane), w(p.w + c16, lane);
                if (!(ok = wait(sm.gfull, c))) break;
                tc_fence_after_sync();
                y.load(tl + cG + c16);
                tmem_wait_ld();
                y.ready();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float &x = y.x[e / 8][e % 8];
                    x = w[e % 8] * fmaf(-eG[e % 8], x, bf16_of(v[e / 8], e % 8));
                }
                if (m < kC)   // value rows behind the end may hold anything
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c16 + 8 * (e % 8 / 4) + 2 * (lane % 4) + e % 2 >= m) y.x[e / 8][e % 8] = 0.f;
            }
            put_split(tl + cG + c16, y);
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive_warp(&sm.rready);
            if (SAVE) {
                if (c > 0 && !(ok = wait(sm.Sfree, c - 1))) break;
                if (live)
#pragma unroll
                    for (int i = 0; i < KQ / 2; i += 4)
                        *reinterpret_cast<uint4 *>(sm.S + op_off(r, x0 + 2 * i, V)) = make_uint4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
                fence_proxy_async_smem();
                mbar_arrive_warp(&sm.Sout);
            }
            // U
            const Factor eK(p.eK + c16, lane);
            if (!(ok = wait(sm.ufull, c))) break;
            tc_fence_after_sync();
            y.load(tl + cU + c16);
            tmem_wait_ld();
            y.ready();
            {
                Frag z;
#pragma unroll
                for (int e = 0; e < 16; ++e) z.x[e / 8][e % 8] = eK[e % 8] * y.x[e / 8][e % 8];
                put_split(tl + cU + c16, z);
            }
            put_split(tl + cG + c16, y);
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive_warp(&sm.uready);
            if (SAVE) {
                if (c > 0 && !(ok = wait(sm.ufree, c - 1))) break;
                if (live) store_tokens(sm.u, c16, quarter * 32, lane, y);
                fence_proxy_async_smem();
                mbar_arrive_warp(&sm.uout);
            }
            // the state after the chunk
            if (!(ok = wait(sm.sfull, c))) break;
            tc_fence_after_sync();
            get_state<KQ>(tl + x0, S);
        }
        if (ok && a.S_final && live) store_row<KQ>(a.S_final + st, S);
    }
    if (!ok && lane == 0) atomicOr(&g_gdr_timeout, 1);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kRegWarps + 1) tmem_dealloc(tm, 512);
}

template <int K, int V, bool SAVE>
cudaError_t sweep_t(const GdrArgs &a, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const CUtensorMap &mo,
                    bool prepared, cudaStream_t st) {
    auto kern = gdr_tc_sweep<K, V, SAVE>;
    const int bytes = (int)sizeof(SweepSmem<K, V, SAVE>) + 1024;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), bytes);
    if (e != cudaSuccess) return e;
    // beside the preparation, an ordinary launch, so that the states and offsets are there; without one, after all
    return launch_after(prepared, kern, (unsigned)(a.seq.N * a.Hv), kSweepThreads, bytes, st, a, mq, mk, mv, mo);
}

template <int K, int V>
cudaError_t fwd_t(const GdrArgs &a, bool save, cudaStream_t st) {
    const long long rows = a.seq.cu ? a.seq.total : (long long)a.seq.N * a.seq.T;
    CUtensorMap mq{}, mk{}, mv{}, mo{};
    if (rows > 0) {   // without rows no tile is copied; the sweep hands the states on
        cudaError_t e = make_operand_tile_map(&mq, a.q, K, a.Hk, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mk, a.k, K, a.Hk, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mv, a.v, V, a.Hv, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mo, a.o, V, a.Hv, rows, kC);
        auto prep = gdr_tc_prep<K>;
        const int bytes = (int)sizeof(PrepSmem<K>);
        if (e == cudaSuccess) e = set_smem_once(reinterpret_cast<const void *>(prep), bytes);
        if (e != cudaSuccess) return e;
        prep<<<(unsigned)(a.seq.n_tiles(kC) * a.Hk), 128, bytes, st>>>(a, mq, mk);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return save ? sweep_t<K, V, true>(a, mq, mk, mv, mo, rows > 0, st) : sweep_t<K, V, false>(a, mq, mk, mv, mo, rows > 0, st);
}

}  // namespace

GdrSizes gdr_tc_sizes(const Seqs &s, int Hv, int K, int V) {
    const size_t slots = (size_t)s.n_tiles(kC) * Hv, keep = 2 * ((size_t)V * K + kC * V);
    return {slots * sizeof(GdrPrep), slots * keep, slots * (keep + 2 * sizeof(float))};
}

cudaError_t launch_gdr_fwd_tc(int K, int V, const GdrArgs &a, bool save, cudaStream_t st) {
    if (K == 64) return V == 64 ? fwd_t<64, 64>(a, save, st) : fwd_t<64, 128>(a, save, st);
    return V == 64 ? fwd_t<128, 64>(a, save, st) : fwd_t<128, 128>(a, save, st);
}

}  // namespace carve
