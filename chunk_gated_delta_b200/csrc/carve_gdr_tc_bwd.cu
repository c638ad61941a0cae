// Scalar-gated delta rule, backward, on the 5th-generation tensor core (carve_gdr_tc.cuh).
//
// gdr_tc_bsweep: one CTA per (sequence, value head) carries dS backwards through the chunks, the
// mirror of the forward's sweep (value channels = lanes of the accumulator, A in tensor memory, a
// thread owns a quarter of a state row; only dO^T A takes its A from shared memory, read transposed):
//   X = dS1 K^T (hi, lo), dO^T A    -> dU = dO^T A + e^{G_C - G} X, split
//   dY = dU Tm (three terms)         -> -w e^G dY, split; dV = w dY; dY
//   dS0 = e^{G_C} dS1 + (e^G dO)^T Q - (w e^G dY)^T K   (hi, lo) -> split for the next chunk
// It leaves dS1 and dY of every chunk in bf16.  Bound as the forward's sweep, by the chain and by what it
// leaves: 8 sequences of 4096 tokens, 16 heads, d = 128 take 214 us.
//
// gdr_tc_grad: with S0, U (forward) and dS1, dY known, the gradients of q, k and the gates have no
// order: persistent CTAs take (tile, key head), all value heads of the key head in turn.  Tokens are the
// lanes, queries in 0-63 and keys in 64-127, so that one product serves both:
//   [dO; dY] U^T  -> P1 = D (dO U^T), P2 = -w D (dY U^T) below the diagonal, bf16
//   [dO; dY] S0   -> dq += e^G x, dk -= w e^G x;   [.; U] dS1 -> dk += e^{G_C - G} x
//   [P1; P2] K + [0; P1^T] Q + [0; P2^T] K  accumulated over the value heads
// P1^T and P2^T are the same tile read along its other index; the zero block beside it fills the
// lanes that have no part.  It reads two states, U, dY, dO, q and k a chunk: 1.5 GB of the sizes above
// in 320 us, 4.6 TB/s; beside HBM it is bound by instruction issue (20 thousand warp instructions a
// tile and head, a quarter of them waits and arrivals).  A pass that would fuse it with the sweep
// saves 0.9 GB but needs 448 more columns of tensor memory than there are.
#include "carve_gdr_tc.cuh"

namespace carve {

__device__ int g_gdr_bwd_timeout;   // set when a bounded wait gives up (never expected)
__device__ int g_gdr_tc_bwd_bad_seqlens;

int gdr_tc_bwd_take_timeout() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gdr_bwd_timeout, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_gdr_bwd_timeout, &z, sizeof(int));
    }
    return v;
}
int gdr_tc_bwd_take_bad_seqlens() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_gdr_tc_bwd_bad_seqlens, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_gdr_tc_bwd_bad_seqlens, &z, sizeof(int));
    }
    return v;
}

namespace {

template <int K, int V>
struct BsweepSmem {
    __nv_bfloat16 k[2][K / 64][kC * 64], q[2][K / 64][kC * 64], dO[2][2][kC * 64];   // dO's second half zero at V = 64
    GdrPrep p[2];
    __nv_bfloat16 S[V * K], y[kC * V], dv[kC * V];   // on their way out
    uint64_t full[2], free[2], sready, gfull, uready, yfull, yready, sfull, Sout, Sfree, yout, yfree, drain;
    uint32_t tmem;
};

template <int K, int V>
__global__ void __launch_bounds__(kSweepThreads, 1)
    gdr_tc_bsweep(GdrArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap md, const __grid_constant__ CUtensorMap mdv) {
    let_next_start();
    extern __shared__ __align__(16) unsigned char raw[];
    typedef BsweepSmem<K, V> Smem;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    constexpr int KH = K / 64, VH = V / 64, KQ = K / 4;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int h = blockIdx.x % a.Hv, n = blockIdx.x / a.Hv, hk = h / (a.Hv / a.Hk);
    long long row0;
    int len;
    a.seq.rows(n, row0, len, threadIdx.x == 0 ? &g_gdr_tc_bwd_bad_seqlens : nullptr);
    const long long t0 = a.seq.tile0(n, kC);
    const int chunks = (len + kC - 1) / kC;
    if (threadIdx.x == 0) {
        for (uint64_t *b : {&sm.full[0], &sm.full[1], &sm.free[0], &sm.free[1], &sm.gfull, &sm.yfull, &sm.sfull, &sm.Sfree,
                            &sm.drain})
            mbar_init(b, 1);
        mbar_init(&sm.yfree, 2);
        for (uint64_t *b : {&sm.sready, &sm.uready, &sm.yready, &sm.Sout, &sm.yout}) mbar_init(b, kRegWarps);
        fence_mbar_init();
    }
    if (VH == 1) {
        for (int i = threadIdx.x; i < 2 * kC * 8; i += blockDim.x)
            reinterpret_cast<uint4 *>(sm.dO[i / (kC * 8)][1])[i % (kC * 8)] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (warp == kRegWarps + 1) tmem_alloc(&sm.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;
    // tensor memory: dS 0-127, dS hi 128, lo 192, X (then dU hi, lo) 256, dO^T A 320, dY (then
    // -w e^G dY hi, lo) 384, e^G dO hi, lo 448
    constexpr uint32_t cHi = 128, cLo = 192, cX = 256, cP = 320, cY = 384, cD = 448;
    bool ok = true;
    auto wait = [&](uint64_t &bar, int phase) {   // by a whole warp
        return mbar_wait_warp(&bar, phase & 1, kIdleWait);
    };

    if (warp >= kRegWarps) regs_down<64>();
    if (warp == kRegWarps) {
        int i = 0;
        for (; i < chunks; ++i) {
            const int s = i & 1, c = chunks - 1 - i;
            if (i >= 2) ok = wait(sm.free[s], i / 2 - 1);
            if (!ok) break;
            if (elect_one()) {
                const int row = (int)(row0 + (long long)c * kC);
                mbar_expect_tx(&sm.full[s], 2 * kC * K * 2 + kC * V * 2 + sizeof(GdrPrep));
                for (int x = 0; x < VH; ++x) tma_load_3d(sm.dO[s][x], &md, 64 * x, h, row, &sm.full[s]);
                bulk_g2s(&sm.p[s], reinterpret_cast<const GdrPrep *>(a.prep) + (size_t)(t0 + c) * a.Hv + h, sizeof(GdrPrep),
                         &sm.full[s]);
                for (int x = 0; x < KH; ++x) tma_load_3d(sm.k[s][x], &mk, 64 * x, hk, row, &sm.full[s]);
                for (int x = 0; x < KH; ++x) tma_load_3d(sm.q[s][x], &mq, 64 * x, hk, row, &sm.full[s]);
            }
        }
        if (!ok)
            for (int j = max(0, i - 2); j < i; ++j) wait(sm.full[j & 1], j / 2);
    } else if (warp == kRegWarps + 1) {
        constexpr uint32_t iN64 = umma_idesc_bf16(128, 64), iS = umma_idesc_bf16(128, K) | kUmmaBmn;
        const uint64_t dk0 = umma_desc(smem_u32(sm.k)), dkt0 = umma_desc_mn(smem_u32(sm.k), kTile64),
                       dqt0 = umma_desc_mn(smem_u32(sm.q), kTile64), dt0 = umma_desc_mn(smem_u32(sm.p), kTile64),
                       do0 = umma_desc_mn(smem_u32(sm.dO), kTile64);
        for (int i = 0; i < chunks; ++i) {
            const int s = i & 1, c = chunks - 1 - i;
            const uint64_t dk = desc_at(dk0, s * KH * kTile64), dkt = desc_at(dkt0, s * KH * kTile64),
                           dqt = desc_at(dqt0, s * KH * kTile64), dt = desc_at(dt0, s * sizeof(GdrPrep)),
                           dd = desc_at(do0, s * 2 * kTile64);
            if (!(ok = wait(sm.full[s], i / 2))) break;
            if (len - c * kC < kC) {   // rows behind the end meet zero factors, so they have to be finite
                zero_rows(sm.k[s], len - c * kC, KH, kTile64, lane);
                zero_rows(sm.q[s], len - c * kC, KH, kTile64, lane);
                zero_rows(sm.dO[s], len - c * kC, VH, kTile64, lane);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_bf16(tm + cP, desc_at(dd, 2048 * kk), desc_at(dt, 2 * kTile64 + 2048 * kk), iN64 | kUmmaAmn | kUmmaBmn, kk > 0);
            }
            __syncwarp();
            if (!(ok = wait(sm.sready, i))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < K / 16; ++kk)
                        umma_bf16_ta(tm + cX, tm + (lo ? cLo : cHi) + 8 * kk, desc_at(dk, kTile64 * (kk / 4) + 32 * (kk % 4)),
                                     iN64, lo > 0 || kk > 0);
                umma_commit(&sm.gfull);
            }
            __syncwarp();
            if (!(ok = wait(sm.uready, i))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int x = 0; x < 3; ++x)   // dU hi Tm hi, dU lo Tm hi, dU hi Tm lo
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tm + cY, tm + cX + split_col(kk, x == 1),
                                     desc_at(dt, (x == 2 ? kTile64 : 0) + 2048 * kk), iN64 | kUmmaBmn, x > 0 || kk > 0);
                umma_commit(&sm.yfull);
                // in the shadow of the pass over dY
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tm, tm + cD + split_col(kk, lo), desc_at(dqt, 2048 * kk),
                                     iS, 1);
            }
            __syncwarp();
            if (!(ok = wait(sm.yready, i))) break;
            tc_fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ta(tm, tm + cY + split_col(kk, lo), desc_at(dkt, 2048 * kk),
                                     iS, 1);
                umma_commit(&sm.sfull);
                umma_commit(&sm.free[s]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(&sm.drain);   // products in flight finish before the tensor memory is freed
        __syncwarp();
        wait(sm.drain, 0);
    } else if (warp == kRegWarps + 2) {
        typedef GdrKeep<K, V> Keep;
        Keep *keep = reinterpret_cast<Keep *>(a.ws) + (size_t)t0 * a.Hv + h;
        for (int i = 0; i < chunks; ++i) {
            const int c = chunks - 1 - i;
            if (!(ok = wait(sm.Sout, i))) break;
            if (elect_one()) {
                bulk_s2g(keep[(size_t)c * a.Hv].S, sm.S, sizeof(sm.S));
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&sm.Sfree);
            }
            __syncwarp();
            if (!(ok = wait(sm.yout, i))) break;
            if (elect_one()) {
                bulk_s2g(keep[(size_t)c * a.Hv].x, sm.y, sizeof(sm.y));
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&sm.yfree);
            }
            __syncwarp();
        }
        bulk_wait<0>();
    } else if (warp == kRegWarps + 3) {
        for (int i = 0; i < chunks; ++i) {
            const int c = chunks - 1 - i;
            if (!(ok = wait(sm.yout, i))) break;
            store_tile<V>(&mdv, a.dv, sm.dv, row0 + (long long)c * kC, len - c * kC, a.Hv, h, lane);
            if (elect_one()) mbar_arrive(&sm.yfree);
            __syncwarp();
        }
        bulk_wait<0>();
    } else if (warp < kRegWarps) {
        regs_up<104>();
        const int part = warp / 4, quarter = warp % 4, r = quarter * 32 + lane;
        const uint32_t tl = tm + ((uint32_t)quarter << 21);
        const int x0 = part * KQ, c16 = part * 16;   // this warp's columns of dS, its tokens
        const bool live = quarter * 32 < V;          // value rows (others carry zeros)
        const size_t st = (((size_t)n * a.Hv + h) * V + (live ? r : 0)) * K + x0;
        float S[KQ];
        load_row<KQ>(S, live && a.dS_final ? a.dS_final + st : nullptr);
        Frag y;
        for (int i = 0; i < chunks; ++i) {
            const int s = i & 1, c = chunks - 1 - i, m = min(kC, len - c * kC);
            const GdrPrep &p = sm.p[s];
            uint32_t hi[KQ / 2];
            // dS1 as operands, the accumulator scaled by e^{G_C}
            if (!(ok = wait(sm.full[s], i / 2))) break;
            put_state<KQ>(tl + x0, tl + cHi + x0 / 2, tl + cLo + x0 / 2, S, p.eG[kC - 1], hi);
            mbar_arrive_warp(&sm.sready);
            if (i > 0 && !(ok = wait(sm.Sfree, i - 1))) break;
            if (live)
#pragma unroll
                for (int e = 0; e < KQ / 2; e += 4)
                    *reinterpret_cast<uint4 *>(sm.S + op_off(r, x0 + 2 * e, V)) = make_uint4(hi[e], hi[e + 1], hi[e + 2], hi[e + 3]);
            fence_proxy_async_smem();
            mbar_arrive_warp(&sm.Sout);
            const Factor eG(p.eG + c16, lane), w(p.w + c16, lane);
            {   // e^G dO, transposed
                uint32_t d[2][4] = {};
                if (live) load_tokens(d, sm.dO[s][0], c16, quarter * 32, lane);
#pragma unroll
                for (int e = 0; e < 16; ++e) y.x[e / 8][e % 8] = eG[e % 8] * bf16_of(d[e / 8], e % 8);
                if (m < kC)   // rows behind the end may hold anything
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c16 + 8 * (e % 8 / 4) + 2 * (lane % 4) + e % 2 >= m) y.x[e / 8][e % 8] = 0.f;
                put_split(tl + cD + c16, y);
            }
            // dU
            {
                Frag pa;
                const Factor eK(p.eK + c16, lane);
                if (!(ok = wait(sm.gfull, i))) break;
                tc_fence_after_sync();
                y.load(tl + cX + c16);
                pa.load(tl + cP + c16);
                tmem_wait_ld();
                y.ready();
                pa.ready();
#pragma unroll
                for (int e = 0; e < 16; ++e) y.x[e / 8][e % 8] = fmaf(eK[e % 8], y.x[e / 8][e % 8], pa.x[e / 8][e % 8]);
            }
            put_split(tl + cX + c16, y);
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive_warp(&sm.uready);
            // dY
            if (!(ok = wait(sm.yfull, i))) break;
            tc_fence_after_sync();
            y.load(tl + cY + c16);
            tmem_wait_ld();
            y.ready();
            Frag z;
#pragma unroll
            for (int e = 0; e < 16; ++e) z.x[e / 8][e % 8] = -eG[e % 8] * (w[e % 8] * y.x[e / 8][e % 8]);
            put_split(tl + cY + c16, z);
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive_warp(&sm.yready);
            if (i > 0 && !(ok = wait(sm.yfree, i - 1))) break;
            if (live) {
                store_tokens(sm.y, c16, quarter * 32, lane, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y.x[e / 8][e % 8] *= w[e % 8];
                store_tokens(sm.dv, c16, quarter * 32, lane, y);
            }
            fence_proxy_async_smem();
            mbar_arrive_warp(&sm.yout);
            // dS0
            if (!(ok = wait(sm.sfull, i))) break;
            tc_fence_after_sync();
            get_state<KQ>(tl + x0, S);
        }
        if (ok && a.dS0 && live) store_row<KQ>(a.dS0 + st, S);
    }
    if (!ok && lane == 0) atomicOr(&g_gdr_bwd_timeout, 1);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kRegWarps + 1) tmem_dealloc(tm, 512);
}

template <int K, int V>
struct GradSmem {
    __nv_bfloat16 d[V / 64][192 * 64];         // dO, dY, U
    __nv_bfloat16 S0[V * K], S1[V * K];        // S0, dS1
    __nv_bfloat16 qk[2][K / 64][128 * 64];     // [stage]: Q, K, then dq, dk on their way out
    __nv_bfloat16 P[192 * 64];                 // zeros, P1, P2
    float vec[2][6][kC];                       // [stage]: e^G, e^{G_C - G}, w, G, e^{G_r - G}, e^{-low part of G}
    float dg[4][128], dw[kC], kb[4][kC], tot[3][128], col[4][kC], last[8];   // partial sums of a head
    uint64_t vfull[2], vfree[2], qkfull[2], qkfree[2], dfull, dfree, s0full, s0free, s1full, s1free, Dfull, Dfree, xfull,
        xfree, yfull, yfree, pready, pfull, afree, gready, gfree, oready[2], drain;   // oready: [stage]
    uint32_t tmem;
};

// <rows v0 .. v0 + 15 of S0, the same of S1> of [V][K] tiles in operand layout, by this warp: the diagonal of
// S0 S1^T from m16n8k16 products (the sum of 64 products a lane took four times as many instructions)
template <int K, int V>
__device__ __forceinline__ float inner16(const __nv_bfloat16 *S0, const __nv_bfloat16 *S1, int v0, int lane) {
    float d[2][4] = {};
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t a[4], b[4];
        load_a_um(a, S0, V, v0, k, lane);
        ldsm_x4(b, smem_u32(S1 + umma_off(v0 + (lane & 7) + ((lane >> 4) << 3), k + ((lane >> 3) & 1) * 8, V)));
        mma_bf16(d[0], a, b[0], b[1]);
        mma_bf16(d[1], a, b[2], b[3]);
    }
    const int g = lane / 4;   // this thread's rows g, g + 8 meet their columns in lane 4 g + g / 2
    float x = lane % 4 == g / 2 ? (g & 1 ? d[0][1] + d[1][3] : d[0][0] + d[1][2]) : 0.f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// lane l returns the sum over the warp's lanes of their x[l % 16]
__device__ __forceinline__ float column_sum(float (&x)[16], int lane) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], 16);
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float keep = up ? x[i + w] : x[i], give = up ? x[i] : x[i + w];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    return x[0];
}

// acc += f times COLS columns x of an accumulator; returns <x, row r of [Q; K]>; `read` follows the last load
template <int COLS, class F>
__device__ __forceinline__ float product_row(uint32_t taddr, float f, const __nv_bfloat16 *qk, int r, int x0, float *acc, F read) {
    float d = 0.f;
#pragma unroll
    for (int b = 0; b < COLS; b += 16) {
        uint32_t x[16];
        tmem_ld16(taddr + b, x);
        tmem_wait_ld();
        tmem_tie16(x);
        if (b + 16 == COLS) read();
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            const uint4 y = *reinterpret_cast<const uint4 *>(qk + op_off(r, x0 + b + i, 128));
            const uint32_t yy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = __uint_as_float(x[i + e]);
                d = fmaf(z, __uint_as_float(e % 2 ? yy[e / 2] & 0xffff0000u : yy[e / 2] << 16), d);
                acc[b + i + e] = fmaf(f, z, acc[b + i + e]);
            }
        }
    }
    return d;
}

template <int K, int V>
__global__ void __launch_bounds__(kSweepThreads, 1)
    gdr_tc_grad(GdrArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap md, const __grid_constant__ CUtensorMap mdq,
                const __grid_constant__ CUtensorMap mdk) {
    extern __shared__ __align__(16) unsigned char raw[];
    typedef GradSmem<K, V> Smem;
    typedef GdrKeep<K, V> Keep;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    constexpr int KH = K / 64, VH = V / 64, KQ = K / 4;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, share = a.Hv / a.Hk;
    if (threadIdx.x == 0) {
        for (uint64_t *b : {&sm.vfull[0], &sm.vfull[1], &sm.qkfull[0], &sm.qkfull[1], &sm.qkfree[0], &sm.qkfree[1], &sm.dfull,
                            &sm.dfree, &sm.s0full, &sm.s1full, &sm.Dfull, &sm.xfull, &sm.yfull, &sm.pfull, &sm.gfree, &sm.drain})
            mbar_init(b, 1);
        for (uint64_t *b : {&sm.vfree[0], &sm.vfree[1], &sm.Dfree, &sm.xfree, &sm.pready, &sm.afree, &sm.gready, &sm.oready[0], &sm.oready[1]})
            mbar_init(b, kRegWarps);
        for (uint64_t *b : {&sm.s0free, &sm.s1free}) mbar_init(b, kRegWarps / 2 + 1);   // readers and the products
        mbar_init(&sm.yfree, kRegWarps / 2);
        fence_mbar_init();
    }
    // the zero block, and what stays zero: blocks of 16 above the diagonal
    for (int i = threadIdx.x; i < (int)sizeof(sm.P) / 16; i += blockDim.x) reinterpret_cast<uint4 *>(sm.P)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < 4 * kC; i += blockDim.x) sm.col[i / kC][i % kC] = 0.f;
    for (int i = threadIdx.x; i < 3 * 128; i += blockDim.x) sm.tot[i / 128][i % 128] = 0.f;
    for (int i = threadIdx.x; i < 8; i += blockDim.x) sm.last[i] = 0.f;
    fence_proxy_async_smem();
    if (warp == kRegWarps + 1) tmem_alloc(&sm.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;
    constexpr uint32_t cX = 0, cY = 128, cA = 256, cD = 384, cKK = 448;
    bool ok = true;
    auto wait = [&](uint64_t &bar, int phase) {   // by a whole warp
        return mbar_wait_warp(&bar, phase & 1, kIdleWait);
    };
    const int items = (int)a.seq.n_tiles(kC) * a.Hk;   // below 2^28
    int it = 0, j = 0;   // items and heads so far (those of used tiles)

    // The sweep, by every warp: a long sequence may keep it busy for seconds after this CTA has started, beyond
    // what the waits below allow for
    wait_for_last();
    if (warp >= kRegWarps) regs_down<64>();
    if (warp == kRegWarps) {
#pragma unroll 1
        for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
            const int tile = w / a.Hk, hk = w - tile * a.Hk;
            int n, c, len;
            long long row;
            if (!a.seq.find(tile, kC, n, c, row, len)) continue;
            row += (long long)c * kC;
#pragma unroll 1
            for (int g = 0; g < share && ok; ++g, ++j) {
                const int s = j & 1, h = hk * share + g;
                const size_t slot = (size_t)tile * a.Hv + h;
                const Keep *fwd = reinterpret_cast<const Keep *>(a.saved) + slot, *bwd = reinterpret_cast<const Keep *>(a.ws) + slot;
                if (j >= 2 && !(ok = wait(sm.vfree[s], j / 2 - 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&sm.vfull[s], kVecBytes);
                    bulk_g2s(sm.vec[s], reinterpret_cast<const GdrPrep *>(a.prep)[slot].eG, kVecBytes, &sm.vfull[s]);
                }
                __syncwarp();
                if (g == 0) {
                    const int b = it & 1;
                    if (it >= 2 && !(ok = wait(sm.qkfree[b], it / 2 - 1))) break;
                    if (elect_one()) {
                        mbar_expect_tx(&sm.qkfull[b], 2 * kC * K * 2);
                        for (int x = 0; x < KH; ++x) {
                            tma_load_3d(sm.qk[b][x], &mq, 64 * x, hk, (int)row, &sm.qkfull[b]);
                            tma_load_3d(sm.qk[b][x] + kC * 64, &mk, 64 * x, hk, (int)row, &sm.qkfull[b]);
                        }
                    }
                    __syncwarp();
                }
                if (j > 0 && !(ok = wait(sm.dfree, j - 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&sm.dfull, 3 * kC * V * 2);
                    for (int x = 0; x < VH; ++x) {
                        tma_load_3d(sm.d[x], &md, 64 * x, h, (int)row, &sm.dfull);
                        bulk_g2s(sm.d[x] + kC * 64, bwd->x + x * kC * 64, kTile64, &sm.dfull);
                        bulk_g2s(sm.d[x] + 2 * kC * 64, fwd->x + x * kC * 64, kTile64, &sm.dfull);
                    }
                }
                __syncwarp();
                if (j > 0 && !(ok = wait(sm.s0free, j - 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&sm.s0full, sizeof(sm.S0));
                    bulk_g2s(sm.S0, fwd->S, sizeof(sm.S0), &sm.s0full);
                }
                __syncwarp();
                if (j > 0 && !(ok = wait(sm.s1free, j - 1))) break;
                if (elect_one()) {
                    mbar_expect_tx(&sm.s1full, sizeof(sm.S1));
                    bulk_g2s(sm.S1, bwd->S, sizeof(sm.S1), &sm.s1full);
                }
                __syncwarp();
            }
            ++it;
        }
        // every copy has landed before the memory is given back (those not issued wait in vain, with a limit)
        if (!ok) {
            for (int i = max(0, j - 1); i <= j; ++i) wait(sm.vfull[i & 1], i / 2);
            for (int i = max(0, it - 1); i <= it; ++i) wait(sm.qkfull[i & 1], i / 2);
            wait(sm.dfull, j);
            wait(sm.s0full, j);
            wait(sm.s1full, j);
        }
    } else if (warp == kRegWarps + 1) {
        constexpr uint32_t iN64 = umma_idesc_bf16(128, 64), iK = umma_idesc_bf16(128, K) | kUmmaBmn;
        const uint32_t P = smem_u32(sm.P);
        const uint64_t dd = umma_desc(smem_u32(sm.d)), dS0 = umma_desc_mn(smem_u32(sm.S0), V * 128), dS1 = umma_desc_mn(smem_u32(sm.S1), V * 128);
        const uint64_t dP = umma_desc(P + kTile64), dP1 = umma_desc_mn(P, kTile64), dP2 = umma_desc_mn(P, 2 * kTile64);
#pragma unroll 1
        for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
            const int tile = w / a.Hk;
            int n, c, len;
            long long row;
            if (!a.seq.find(tile, kC, n, c, row, len)) continue;
            const uint64_t dqk = umma_desc(smem_u32(sm.qk[it & 1])), dqkt = umma_desc_mn(smem_u32(sm.qk[it & 1]), 2 * kTile64);
#pragma unroll 1
            for (int g = 0; g < share && ok; ++g, ++j) {
                if (g == 0) {
                    if (!(ok = wait(sm.qkfull[it & 1], it / 2))) break;
                    if (len - c * kC < kC) {   // rows behind the end meet zero factors, so they have to be finite
                        zero_rows(sm.qk[it & 1][0], len - c * kC, KH, 2 * kTile64, lane);
                        zero_rows(sm.qk[it & 1][0] + kC * 64, len - c * kC, KH, 2 * kTile64, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (j > 0 && !(ok = wait(sm.Dfree, j - 1))) break;
                tc_fence_after_sync();
                if (g == 0 && elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < K / 16; ++kk) {
                        const uint32_t x = 2 * kTile64 * (kk / 4) + 32 * (kk % 4);
                        umma_bf16(tm + cKK, desc_at(dqk, x), desc_at(dqk, x + kTile64), iN64, kk > 0);
                    }
                }
                __syncwarp();
                if (!(ok = wait(sm.dfull, j))) break;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < V / 16; ++kk) {
                        const uint32_t x = 3 * kTile64 * (kk / 4) + 32 * (kk % 4);
                        umma_bf16(tm + cD, desc_at(dd, x), desc_at(dd, x + 2 * kTile64), iN64, kk > 0);
                    }
                    umma_commit(&sm.Dfull);
                }
                __syncwarp();
                if (!(ok = wait(sm.s0full, j))) break;
                if (j > 0 && !(ok = wait(sm.xfree, j - 1))) break;
                tc_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < V / 16; ++kk)
                        umma_bf16(tm + cX, desc_at(dd, 3 * kTile64 * (kk / 4) + 32 * (kk % 4)), desc_at(dS0, 2048 * kk), iK, kk > 0);
                    umma_commit(&sm.xfull);
                    umma_commit(&sm.s0free);
                }
                __syncwarp();
                if (!(ok = wait(sm.s1full, j))) break;
                if (j > 0 && !(ok = wait(sm.yfree, j - 1))) break;
                tc_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < V / 16; ++kk)   // [dY; U] dS1, of which the lanes of U count
                        umma_bf16(tm + cY, desc_at(dd, kTile64 + 3 * kTile64 * (kk / 4) + 32 * (kk % 4)), desc_at(dS1, 2048 * kk), iK,
                                  kk > 0);
                    umma_commit(&sm.yfull);
                umma_commit(&sm.s1free);
                    umma_commit(&sm.dfree);
                }
                __syncwarp();
                if (!(ok = wait(sm.pready, j))) break;
                if (g == 0 && it > 0 && !(ok = wait(sm.afree, it - 1))) break;
                tc_fence_after_sync();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // [P1; P2] K
                        umma_bf16(tm + cA, desc_at(dP, 32 * kk), desc_at(dqkt, kTile64 + 2048 * kk), iK, g > 0 || kk > 0);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // [0; P1^T] Q
                        umma_bf16(tm + cA, desc_at(dP1, 2048 * kk), desc_at(dqkt, 2048 * kk), iK | kUmmaAmn, 1);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // [0; P2^T] K
                        umma_bf16(tm + cA, desc_at(dP2, 2048 * kk), desc_at(dqkt, kTile64 + 2048 * kk), iK | kUmmaAmn, 1);
                    umma_commit(&sm.pfull);
                }
                __syncwarp();
            }
            ++it;
        }
        if (elect_one()) umma_commit(&sm.drain);
        __syncwarp();
        wait(sm.drain, 0);
    } else if (warp == kRegWarps + 2) {
        // gate gradients from the partial sums: lane = tokens lane and lane + 32.  The gradient of log a_t
        // is the sum over every path that crosses the decay of token t, each term as it is (rows minus
        // columns of a cumulative sum would cancel): queries and keys r >= t that read the start state,
        // keys s < t that reach the end, S0 itself, and pairs r >= t > s.
        float *part = a.dA_dec || a.dtau ? reinterpret_cast<float *>(a.ws + (size_t)a.seq.n_tiles(kC) * a.Hv * sizeof(Keep)) : nullptr;
#pragma unroll 1
        for (int wk = blockIdx.x; wk < items && ok; wk += gridDim.x) {
            const int tile = wk / a.Hk, hk = wk - tile * a.Hk;
            int n, c, len;
            long long row;
            if (!a.seq.find(tile, kC, n, c, row, len)) {
                if (part)   // unused numbers count as zero in the fixed-order sums
                    for (int i = lane; i < 2 * share; i += 32) part[((size_t)tile * a.Hv + hk * share) * 2 + i] = 0.f;
                continue;
            }
            row += (long long)c * kC;
            const int m = min(kC, len - c * kC);
#pragma unroll 1
            for (int g = 0; g < share && ok; ++g, ++j) {
                const int h = hk * share + g;
                const float amp = decay_amp(a.A_dec, h), bias = a.tau ? a.tau[h] : 0.f;
                if (!(ok = wait(sm.gready, j))) break;
                // row sums; sums of key rows; dY.U = w dL/dw (from (I + M) U = w R: dL/dw = dY.(R - M U / w) = dY.U / w);
                // columns of the pairs; row totals of the pairs of tokens 0-15, 16-31, 32-47
                float G[2], B[2], dw[2], C[2], T[3][2], last = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = lane + 32 * e;
                    G[e] = B[e] = C[e] = 0.f;
                    dw[e] = sm.dw[t];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        G[e] += sm.dg[p][t] + sm.dg[p][t + 64];
                        B[e] += sm.kb[p][t];
                        C[e] += sm.col[p][t];
                    }
#pragma unroll
                    for (int p = 0; p < 3; ++p) T[p][e] = sm.tot[p][t] + sm.tot[p][t + 64];
                }
#pragma unroll
                for (int p = 0; p < 8; ++p) last += sm.last[p];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.gfree);
                // suffix sums of G and the T, exclusive prefix of B
#pragma unroll 1
                for (int off = 1; off < 32; off <<= 1) {
                    const bool down = lane + off < 32;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float g1 = __shfl_down_sync(0xffffffffu, G[e], off), b1 = __shfl_up_sync(0xffffffffu, B[e], off);
                        G[e] += down ? g1 : 0.f;
                        B[e] += lane >= off ? b1 : 0.f;
#pragma unroll
                        for (int p = 0; p < 3; ++p) {
                            const float t1 = __shfl_down_sync(0xffffffffu, T[p][e], off);
                            T[p][e] += down ? t1 : 0.f;
                        }
                    }
                }
                G[0] += __shfl_sync(0xffffffffu, G[1], 0);
                const float t0 = __shfl_sync(0xffffffffu, T[0][1], 0), all0 = __shfl_sync(0xffffffffu, B[0], 31);
                float b0 = __shfl_up_sync(0xffffffffu, B[0], 1), b1 = __shfl_up_sync(0xffffffffu, B[1], 1);
                b0 = lane ? b0 : 0.f;
                b1 = (lane ? b1 : 0.f) + all0;
                const float gr0 = G[0] + b0 + last + C[0] + (lane >= 16 ? T[0][0] + t0 : 0.f);
                const float gr1 = G[1] + b1 + last + C[1] + T[0][1] + T[1][1] + (lane >= 16 ? T[2][1] : 0.f);
                float dlog = 0.f, damp = 0.f;
#pragma unroll 1
                for (int t = lane; t < m; t += 32) {
                    const size_t at = (size_t)(row + t) * a.Hv + h;
                    const float x = ld_io(static_cast<const __nv_bfloat16 *>(a.g_logit) + at) + bias;
                    const float w = sigmoid_f(ld_io(static_cast<const __nv_bfloat16 *>(a.w_logit) + at));
                    const float gr = -amp * (t < 32 ? gr0 : gr1), dl = sigmoid_f(x) * gr;
                    dlog += dl;
                    damp += softplus_f(x) * gr;
                    st_io(static_cast<__nv_bfloat16 *>(a.dg_logit) + at, dl);
                    st_io(static_cast<__nv_bfloat16 *>(a.dw_logit) + at, (t < 32 ? dw[0] : dw[1]) * (1.f - w));
                }
                __syncwarp();
                if (part) {
#pragma unroll
                    for (int off = 16; off >= 1; off >>= 1) {
                        dlog += __shfl_xor_sync(0xffffffffu, dlog, off);
                        damp += __shfl_xor_sync(0xffffffffu, damp, off);
                    }
                    if (elect_one()) {
                        part[((size_t)tile * a.Hv + h) * 2] = damp;
                        part[((size_t)tile * a.Hv + h) * 2 + 1] = dlog;
                    }
                }
            }
        }
    } else if (warp == kRegWarps + 3) {
#pragma unroll 1
        for (int w = blockIdx.x; w < items && ok; w += gridDim.x) {
            const int tile = w / a.Hk, hk = w - tile * a.Hk;
            int n, c, len;
            long long row;
            if (!a.seq.find(tile, kC, n, c, row, len)) continue;
            row += (long long)c * kC;
            // one barrier a stage: the register warps may finish the next item before this warp has seen this one, and
            // the one after it only when this stage was given back
            if (!(ok = wait(sm.oready[it & 1], it / 2))) break;
            if (elect_one()) {
                if (len - c * kC >= kC)
                    for (int x = 0; x < KH; ++x) {
                        tma_store_3d(&mdq, sm.qk[it & 1][x], 64 * x, hk, (int)row);
                        tma_store_3d(&mdk, sm.qk[it & 1][x] + kC * 64, 64 * x, hk, (int)row);
                    }
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&sm.qkfree[it & 1]);
            }
            __syncwarp();
            ++it;
        }
        bulk_wait<0>();
    } else if (warp < kRegWarps) {
        regs_up<104>();
        const int part = warp / 4, quarter = warp % 4, r = quarter * 32 + lane, t = r % kC;
        const bool key = r >= kC;   // lane of a key (the same for a whole warp)
        const uint32_t tl = tm + ((uint32_t)quarter << 21);
        const int x0 = part * KQ, s0 = part * 16;
        // this warp's 32 tokens x 16 pairs: above the diagonal, across it, below it
        const int pairs = s0 > (t | 31) ? 0 : s0 + 15 < (t & 32) ? 2 : 1;
        float acc[KQ];
#pragma unroll 1
        for (int wk = blockIdx.x; wk < items && ok; wk += gridDim.x) {
            const int tile = wk / a.Hk, hk = wk - tile * a.Hk;
            int n, c, len;
            long long row;
            if (!a.seq.find(tile, kC, n, c, row, len)) continue;
            row += (long long)c * kC;
            const int m = min(kC, len - c * kC);
            const bool here = t < m;
            const int lim = here ? t + !key - s0 : 0;   // pairs of this token among its 16: s < t, and s = t for queries
            __nv_bfloat16 *qk = sm.qk[it & 1][0];
#pragma unroll
            for (int x = 0; x < KQ; ++x) acc[x] = 0.f;
#pragma unroll 1
            for (int g = 0; g < share && ok; ++g, ++j) {
                const int s = j & 1;
                if (!(ok = wait(sm.vfull[s], j / 2))) break;
                const float *eG = sm.vec[s][0], *eK = sm.vec[s][1], *G = sm.vec[s][3] + s0, *rL = sm.vec[s][5] + s0;
                const float Gt = sm.vec[s][3][t], sign = (key ? -sm.vec[s][2][t] : 1.f) * __frcp_rn(sm.vec[s][5][t]);
                // pairs of the chunk: y = D (dO U^T) or -w D (dY U^T), times k.k or q.k
                if (!(ok = wait(sm.Dfull, j))) break;
                tc_fence_after_sync();
                if (pairs) {
                    uint32_t D[16], kk[16];
                    tmem_ld16(tl + cD + s0, D);
                    tmem_ld16(tl + cKK + s0, kk);
                    tmem_wait_ld();
                    tmem_tie16(D);
                    tmem_tie16(kk);
                    tc_fence_before_sync();
                    mbar_arrive_warp(&sm.Dfree);
                    float pr[16], own = 0.f, run = 0.f;
                    if (pairs == 2) {   // all of them below the diagonal: one factor a row, one a column
                        const float f = here ? sign * ex2(Gt - G[15]) * rL[15] : 0.f;
                        const float *eB = sm.vec[s][4] + s0;
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 b = *reinterpret_cast<const float4 *>(eB + e);
                            const float c[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float y = here ? f * c[i] * __uint_as_float(D[e + i]) : 0.f;
                                pr[e + i] = y * __uint_as_float(kk[e + i]);
                                D[e + i] = __float_as_uint(y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = __uint_as_float(D[e]);
                            own = t - s0 == e ? x : own;
                            const float y = e < lim ? sign * ex2(Gt - G[e]) * rL[e] * x : 0.f;
                            pr[e] = y * __uint_as_float(kk[e]);
                            D[e] = __float_as_uint(y);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) kk[e] = pack_bf16(__uint_as_float(D[2 * e]), __uint_as_float(D[2 * e + 1]));
                    if (j > 0 && !(ok = wait(sm.pfull, j - 1))) break;
#pragma unroll
                    for (int e = 0; e < 8; e += 4)
                        *reinterpret_cast<uint4 *>(sm.P + kC * 64 + op_off(r, s0 + 2 * e, 128)) = make_uint4(kk[e], kk[e + 1], kk[e + 2], kk[e + 3]);
                    fence_proxy_async_smem();
                    mbar_arrive_warp(&sm.pready);
                    // sums over s before u, for u up to t (what a query's own pair adds is behind its last u)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float y = pr[e];
                        pr[e] = pairs == 2 || s0 + e <= t ? run : 0.f;
                        run += y;
                    }
                    const float cs = column_sum(pr, lane);
                    if (j > 0 && !(ok = wait(sm.gfree, j - 1))) break;
                    if (lane < 16) sm.col[quarter][s0 + lane] = cs;
                    if (part < 3) sm.tot[part][r] = run;
                    if (key && t / 16 == part) sm.dw[t] = own;
                } else {
                    mbar_arrive_warp(&sm.Dfree);
                    mbar_arrive_warp(&sm.pready);
                    if (j > 0 && !(ok = wait(sm.gfree, j - 1))) break;
                }
                if (key) {   // end state
                    if (!(ok = wait(sm.yfull, j))) break;
                    tc_fence_after_sync();
                    const float f = eK[t];
                    const float d = product_row<KQ>(tl + cY + x0, f, qk, r, x0, acc, [&] {
                        tc_fence_before_sync();
                        mbar_arrive_warp(&sm.yfree);
                    });
                    sm.kb[part][t] = here ? f * d : 0.f;
                } else {   // <S0, dS1>: both are laid out alike
                    if (!(ok = wait(sm.s0full, j))) break;
                    if (!(ok = wait(sm.s1full, j))) break;
                    const int v0 = (part * 2 + quarter) * 16;
                    float y = 0.f;
                    if (v0 < V) y = inner16<K, V>(sm.S0, sm.S1, v0, lane);
                    mbar_arrive_warp(&sm.s0free);
                    mbar_arrive_warp(&sm.s1free);
                    if (lane == 0 && v0 < V) sm.last[part * 2 + quarter] = y * eG[kC - 1];
                }
                // start state
                if (!(ok = wait(sm.xfull, j))) break;
                tc_fence_after_sync();
                const float f = sign * eG[t];
                const float d = product_row<KQ>(tl + cX + x0, f, qk, r, x0, acc, [&] {
                    tc_fence_before_sync();
                    mbar_arrive_warp(&sm.xfree);
                });
                sm.dg[part][r] = here ? f * d : 0.f;
                mbar_arrive_warp(&sm.gready);
                mbar_arrive_warp(&sm.vfree[s]);
            }
            if (!ok) break;
            if (!(ok = wait(sm.pfull, j - 1))) break;
            tc_fence_after_sync();
            // dq, dk in the place of this thread's part of q, k (rows of a last tile straight to memory: those
            // behind the end are others')
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(key ? a.dk : a.dq) +
                                                   ((size_t)(row + t) * a.Hk + hk) * K + x0);
#pragma unroll
            for (int b = 0; b < KQ; b += 16) {
                uint32_t x[16], o[8];
                tmem_ld16(tl + cA + x0 + b, x);
                tmem_wait_ld();
                tmem_tie16(x);
                if (b + 16 == KQ) {
                    tc_fence_before_sync();
                    mbar_arrive_warp(&sm.afree);
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    o[e / 2] = pack_bf16(acc[b + e] + __uint_as_float(x[e]), acc[b + e + 1] + __uint_as_float(x[e + 1]));
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const uint4 y = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    if (m == kC)
                        *reinterpret_cast<uint4 *>(qk + op_off(r, x0 + b + 2 * e, 128)) = y;
                    else if (here)
                        out[(b + 2 * e) / 8] = y;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive_warp(&sm.oready[it & 1]);
            ++it;
        }
    }
    if (!ok && lane == 0) atomicOr(&g_gdr_bwd_timeout, 1);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kRegWarps + 1) tmem_dealloc(tm, 512);
}

template <int K, int V>
cudaError_t bwd_t(const GdrArgs &a, cudaStream_t st) {
    const long long rows = a.seq.cu ? a.seq.total : (long long)a.seq.N * a.seq.T;
    CUtensorMap mq{}, mk{}, md{}, mdq{}, mdk{}, mdv{};
    auto sweep = gdr_tc_bsweep<K, V>;
    auto grad = gdr_tc_grad<K, V>;
    const int sb = (int)sizeof(BsweepSmem<K, V>) + 1024, gb = (int)sizeof(GradSmem<K, V>) + 1024;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(sweep), sb);
    if (e == cudaSuccess) e = set_smem_once(reinterpret_cast<const void *>(grad), gb);
    if (rows > 0) {   // without rows no tile is copied; the sweep hands the states on
        if (e == cudaSuccess) e = make_operand_tile_map(&mq, a.q, K, a.Hk, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mk, a.k, K, a.Hk, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&md, a.dO, V, a.Hv, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mdv, a.dv, V, a.Hv, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mdq, a.dq, K, a.Hk, rows, kC);
        if (e == cudaSuccess) e = make_operand_tile_map(&mdk, a.dk, K, a.Hk, rows, kC);
    }
    if (e != cudaSuccess) return e;
    sweep<<<a.seq.N * a.Hv, kSweepThreads, sb, st>>>(a, mq, mk, md, mdv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long tiles = a.seq.n_tiles(kC), items = tiles * a.Hk;
    if (items) e = launch_after(true, grad, (unsigned)(items < sm_count() ? items : sm_count()), kSweepThreads, gb, st, a, mq, mk, md, mdq, mdk);
    if (e != cudaSuccess) return e;
    if (a.dA_dec || a.dtau)
        launch_gdr_reduce_decay(reinterpret_cast<const float *>(a.ws + (size_t)tiles * a.Hv * sizeof(GdrKeep<K, V>)), tiles, a.Hv,
                                a.dA_dec, a.dtau, st);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_bwd_tc(int K, int V, const GdrArgs &a, cudaStream_t st) {
    if (K == 64) return V == 64 ? bwd_t<64, 64>(a, st) : bwd_t<64, 128>(a, st);
    return V == 64 ? bwd_t<128, 64>(a, st) : bwd_t<128, 128>(a, st);
}

}  // namespace carve
