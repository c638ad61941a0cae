// Sliding-window attention with sink tokens, forward, on the 5th-generation tensor core (bf16;
// include/carve_mixers.h).
//
// A CTA holds two query tiles of 128 rows that read the same keys: two query heads of one key
// head when the heads pair up (the keys of one 128-row window), else 256 rows of one head.  For
// each 128-key block that a tile sees:
//   S = Q K^T                    tcgen05.mma, accumulator in tensor memory (128 columns)
//   P = 2^{S scale log2 e - m}   two threads a row, 64 scores each in registers; they exchange
//                                their maxima through shared memory; P goes back as bf16 over S
//   O += P V                     A = P from tensor memory, O stays in tensor memory
// The two tiles alternate, so the tensor core works on one while the other's rows are in
// softmax.  m is the maximum that was current when O was last rescaled: O is rescaled (a round
// trip through registers) only when some row's maximum has grown by more than 2^8 since, which
// keeps P below 2^8 and sums in fp32 exact to rounding; the last division removes the reference.
// Roles: warps 0-7 and 8-15 softmax of tile 0 and 1 (the second four of each take columns 64 ..
// 127: four warps a scheduler hide each other's latency, one half as many took 1.7 times as
// long), warp 16 copies (TMA, ring of four 128-row key or value tiles), warp 17 issues the products.
//
// Blocks that a tile does not see are skipped; only blocks that a window edge or the diagonal
// crosses are masked, by selection.  Value rows behind the sequence's end are zeroed in shared
// memory, so nothing that belongs to another sequence meets a product with P = 0.
#include "carve_mixers.cuh"
#include "carve_umma.cuh"

namespace carve {

__device__ int g_swa_timeout;   // set when a bounded wait gives up (never expected)

int swa_fwd_take_timeout() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_swa_timeout, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_swa_timeout, &z, sizeof(int));
    }
    return v;
}

namespace {

constexpr int BM = 128, BN = 128, kStages = 4, kThreadsTc = 576;
constexpr float kLazy = 8.f;   // growth of a row's maximum, in powers of two, that O may lag behind

template <int D>
struct FwdSmem {
    __nv_bfloat16 q[2][D / 64][BM * 64];
    __nv_bfloat16 kv[kStages][D / 64][BN * 64];
    float part[2][2][BM];   // a row's maximum, at the end its sum, by tile and column half
    uint64_t qfull, kvfull[kStages], kvfree[kStages], sfull[2], pfull[2], ofull[2], xbar[2][4];
    uint32_t tmem;
};

// The two query tiles of a CTA and the key blocks that they see.
struct Work {
    long long row0;
    int len, i0[2], i1[2], h[2], hk;
    KeyTiles kt;
    __device__ __forceinline__ bool sees(const SwaArgs &a, int t, int j0) const {
        return i0[t] < i1[t] && j0 < i1[t] && (j0 < a.sinks || (long long)j0 + BN - 1 + a.window > i0[t]);
    }
};

template <int D>
__global__ void __launch_bounds__(kThreadsTc, 1)
    swa_tc_fwd(SwaArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, int paired) {
    extern __shared__ __align__(16) unsigned char raw[];
    FwdSmem<D> &sm = *reinterpret_cast<FwdSmem<D> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int KH = D / 64;
    constexpr uint32_t kTile = BN * D * 2;   // bytes of one operand tile

    // ---- which work
    int n, c, len;
    long long row0;
    const int units = paired ? a.Hq / 2 : a.Hq, u = blockIdx.x % units, rows = paired ? BM : 2 * BM;
    if (!a.seq.find(blockIdx.x / units, rows, n, c, row0, len)) return;
    const int q0 = c * rows, h0 = paired ? 2 * u : u;
    const Work w{row0, len, {q0, paired ? q0 : q0 + BM},
                 {min(q0 + BM, len), paired ? min(q0 + BM, len) : min(q0 + 2 * BM, len)},
                 {h0, paired ? h0 + 1 : h0}, h0 / (a.Hq / a.Hkv), KeyTiles(q0, min(q0 + rows, len), BN, a.window, a.sinks)};
    const int blocks = w.kt.count();

    if (threadIdx.x == 0) {
        mbar_init(&sm.qfull, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.kvfull[i], 1);
            mbar_init(&sm.kvfree[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.sfull[t], 1);
            mbar_init(&sm.pfull[t], 256);
            for (int i = 0; i < 4; ++i) mbar_init(&sm.xbar[t][i], 2);
            mbar_init(&sm.ofull[t], 1);
        }
        fence_mbar_init();
    }
    if (warp == 17) tmem_alloc(&sm.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;   // S of tile t at column 128 t, O at 256 + 128 t
    bool ok = true;
    auto wait = [&](uint64_t &bar, int phase) {   // by a whole warp
        return mbar_wait_warp(&bar, phase & 1, kIdleWait);
    };

    if (warp == 16) {
        if (elect_one()) {
            mbar_expect_tx(&sm.qfull, 2 * BM * D * 2);
            for (int t = 0; t < 2; ++t)
                for (int x = 0; x < KH; ++x)
                    tma_load_3d(sm.q[t][x], &mq, 64 * x, w.h[t], (int)(w.row0 + w.i0[t]), &sm.qfull);
            int filled = 0;
            for (int b = 0; b < blocks && ok; ++b) {
                const int row = (int)w.row0 + w.kt.tile(b) * BN;
                for (int kv = 0; kv < 2 && ok; ++kv, ++filled) {
                    const int s = filled % kStages;
                    if (filled >= kStages) ok = mbar_wait(&sm.kvfree[s], (filled / kStages - 1) & 1, kSwaWait);
                    if (!ok) break;
                    mbar_expect_tx(&sm.kvfull[s], kTile);
                    for (int x = 0; x < KH; ++x) tma_load_3d(sm.kv[s][x], kv ? &mv : &mk, 64 * x, w.hk, row, &sm.kvfull[s]);
                }
            }
            if (!ok) {   // the copies in flight land before the CTA leaves
                mbar_wait(&sm.qfull, 0, kSwaWait);
                for (int i = max(0, filled - kStages); i < filled; ++i)
                    mbar_wait(&sm.kvfull[i % kStages], (i / kStages) & 1, kSwaWait);
            }
        }
    } else if (warp == 17) {
        constexpr uint32_t iS = umma_idesc_bf16(BM, BN), iO = umma_idesc_bf16(BM, D) | kUmmaBmn;
        int ns[2] = {0, 0}, np[2] = {0, 0};   // products S and P V issued, per tile
        const uint64_t dq = umma_desc(smem_u32(sm.q)), dk = umma_desc(smem_u32(sm.kv)), dv = umma_desc_mn(smem_u32(sm.kv), BN * 128);
        auto issue_s = [&](int t, int slot) {
            if (elect_one()) {
                const uint64_t q = desc_at(dq, t * sizeof(sm.q[0])), k = desc_at(dk, slot * sizeof(sm.kv[0]));
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16(tm + 128 * t, desc_at(q, BM * 128 * (kk / 4) + 32 * (kk % 4)), desc_at(k, BN * 128 * (kk / 4) + 32 * (kk % 4)),
                              iS, kk > 0);
                umma_commit(&sm.sfull[t]);
            }
            __syncwarp();
            ++ns[t];
        };
        ok = wait(sm.qfull, 0) && wait(sm.kvfull[0], 0);
        tc_fence_after_sync();
        if (ok) {
            for (int t = 0; t < 2; ++t)
                if (w.sees(a, t, w.kt.tile(0) * BN)) issue_s(t, 0);
            if (elect_one()) umma_commit(&sm.kvfree[0]);
        }
        for (int b = 0; b < blocks && ok; ++b) {
            const int vs = (2 * b + 1) % kStages, ks = (2 * b + 2) % kStages;
            const int j0 = w.kt.tile(b) * BN, j1 = b + 1 < blocks ? w.kt.tile(b + 1) * BN : 0;
            ok = wait(sm.kvfull[vs], (2 * b + 1) / kStages);
            if (ok && w.len - j0 < BN) {   // value rows behind the end: zero
                const int first = w.len - j0;
                for (int x = 0; x < KH; ++x)
                    for (int i = first * 8 + lane; i < BN * 8; i += 32)
                        reinterpret_cast<uint4 *>(sm.kv[vs][x])[i] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (ok && b + 1 < blocks) ok = wait(sm.kvfull[ks], (2 * b + 2) / kStages);
            for (int t = 0; t < 2 && ok; ++t) {
                if (w.sees(a, t, j0)) {
                    ok = wait(sm.pfull[t], np[t]);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t v = desc_at(dv, vs * sizeof(sm.kv[0]));
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            umma_bf16_ta(tm + 256 + 128 * t, tm + 128 * t + 8 * kk + (kk < 4 ? 0 : 32),
                                         desc_at(v, 2048 * kk), iO, kk > 0 || np[t] > 0);
                        umma_commit(&sm.ofull[t]);
                    }
                    __syncwarp();
                    ++np[t];
                }
                if (b + 1 < blocks && w.sees(a, t, j1)) issue_s(t, ks);
            }
            if (elect_one()) {
                umma_commit(&sm.kvfree[vs]);
                if (b + 1 < blocks) umma_commit(&sm.kvfree[ks]);
            }
        }
        // products in flight finish before the tensor memory is freed: the softmax warps wait for
        // the last of each tile, and on the way out after a timeout this warp does
        if (!ok)
            for (int t = 0; t < 2; ++t) {
                if (ns[t]) wait(sm.sfull[t], ns[t] - 1);
                if (np[t]) wait(sm.ofull[t], np[t] - 1);
            }
    } else {
        const int t = warp / 8, half = (warp / 4) % 2, quarter = warp % 4, r = quarter * 32 + lane, i = w.i0[t] + r;
        const uint32_t lanes = (uint32_t)quarter << 21;   // lane quarter in bits 16+
        // this thread's 64 scores (and over the first 32 of them its 64 values of P), its half of O
        const uint32_t tS = tm + 128 * t + 64 * half + lanes, tO = tm + 256 + 128 * t + (D / 2) * half + lanes;
        const bool plain = a.scale > 0.f;   // else the scores are scaled first (its sign, or zero)
        const float sc = (plain ? a.scale : 1.f) * 1.4426950408889634f;
        float m = -INFINITY, l = 0.f;   // reference maximum (of unscaled scores) and this half's sum
        int nb = 0, nx = 0;
        auto other = [&](float x) {     // exchange with the thread of the row's other half
            sm.part[t][half][r] = x;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.xbar[t][quarter]);
            ok = wait(sm.xbar[t][quarter], nx++);
            return sm.part[t][1 - half][r];
        };
        for (int b = 0; b < blocks && ok; ++b) {
            const int j0 = w.kt.tile(b) * BN;
            if (!w.sees(a, t, j0)) continue;
            ok = wait(sm.sfull[t], nb);
            if (!ok) break;
            tc_fence_after_sync();
            uint32_t s[64];
            tmem_ld32(tS, s);
            tmem_ld32(tS + 32, s + 32);
            tmem_wait_ld();
            tmem_tie(s);
            tmem_tie(s + 32);
            if (!plain) {
#pragma unroll
                for (int x = 0; x < 64; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * a.scale);
            }
            // masked only where the diagonal or the window's far edge crosses the block
            if (!(j0 + BN - 1 <= w.i0[t] && (w.i0[t] + BM - 1 - j0 < a.window || j0 + BN <= a.sinks))) {
                const int c0 = j0 + 64 * half, hi = i - c0;                      // seen: columns 0 .. hi that are
                const int lo = (int)max((long long)i - a.window + 1 - c0, 0LL);  // from lo on, or before sk
                const int sk = a.sinks - c0;
#pragma unroll
                for (int y = 0; y < 64; y += 32) {
                    const int top = hi - y, from = lo - y, before = sk - y;
                    const uint32_t past = top >= 31 ? 0xffffffffu : top < 0 ? 0u : (2u << top) - 1u;
                    const uint32_t near = from <= 0 ? 0xffffffffu : from > 31 ? 0u : 0xffffffffu << from;
                    const uint32_t sink = before >= 32 ? 0xffffffffu : before <= 0 ? 0u : (1u << before) - 1u;
                    const uint32_t seen = past & (near | sink);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!((seen >> x) & 1u)) s[y + x] = 0xff800000u;   // -inf
                }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 64; ++x) mx[x & 3] = fmaxf(mx[x & 3], __uint_as_float(s[x]));
            float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            mb = fmaxf(mb, other(mb));
            if (!ok) break;
            const bool grown = (mb - m) * sc > kLazy;   // of this row alone: a row's result depends on no other
            if (__any_sync(0xffffffffu, grown)) {       // rare after the first block
                const float m1 = grown ? mb : m, f = grown ? ex2((m - m1) * sc) : 1.f;
                if (nb > 0) {
                    ok = wait(sm.ofull[t], nb - 1);
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int x = 0; x < D / 2; x += 16) {
                        uint32_t o[16];
                        tmem_ld16(tO + x, o);
                        tmem_wait_ld();
                        tmem_tie16(o);
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                        tmem_st16(tO + x, o);
                    }
                }
                l *= f;
                m = m1;
            }
            const float base = m == -INFINITY ? 0.f : m * sc;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
                const float p0 = ex2(fmaf(__uint_as_float(s[x]), sc, -base)), p1 = ex2(fmaf(__uint_as_float(s[x + 1]), sc, -base));
                sum[x & 2] += p0;
                sum[(x & 2) + 1] += p1;
                s[x / 2] = pack_bf16(p0, p1);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st32(tS, s);
            tmem_wait_st();
            tc_fence_before_sync();
            mbar_arrive(&sm.pfull[t]);
            ++nb;
        }
        if (ok && nb > 0) {
            l += other(l);
            ok = ok && wait(sm.ofull[t], nb - 1);
            tc_fence_after_sync();
            const float inv = 1.f / l;
            const size_t at = (size_t)(w.row0 + i) * a.Hq + w.h[t];
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.o) + at * D + (D / 2) * half;
#pragma unroll
            for (int x = 0; x < D / 2; x += 32) {
                uint32_t o[32];
                tmem_ld32(tO + x, o);
                tmem_wait_ld();
                tmem_tie(o);
                if (ok && i < w.i1[t]) {
#pragma unroll
                    for (int y = 0; y < 32; y += 8) {
                        uint4 v;
                        v.x = pack_bf16(__uint_as_float(o[y]) * inv, __uint_as_float(o[y + 1]) * inv);
                        v.y = pack_bf16(__uint_as_float(o[y + 2]) * inv, __uint_as_float(o[y + 3]) * inv);
                        v.z = pack_bf16(__uint_as_float(o[y + 4]) * inv, __uint_as_float(o[y + 5]) * inv);
                        v.w = pack_bf16(__uint_as_float(o[y + 6]) * inv, __uint_as_float(o[y + 7]) * inv);
                        *reinterpret_cast<uint4 *>(out + x + y) = v;
                    }
                }
            }
            if (ok && a.lse && half == 0 && i < w.i1[t]) a.lse[at] = (m * sc + log2f(l)) * 0.6931471805599453f;
        }
    }
    if (!ok && lane == 0) atomicOr(&g_swa_timeout, 1);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 17) tmem_dealloc(tm, 512);
}

template <int D>
cudaError_t fwd_t(const SwaArgs &a, cudaStream_t st) {
    auto kern = swa_tc_fwd<D>;
    const int bytes = (int)sizeof(FwdSmem<D>) + 1024;
    cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), bytes);
    const long long rows = a.seq.cu ? a.seq.total : (long long)a.seq.N * a.seq.T;
    CUtensorMap mq, mk, mv;
    if (e == cudaSuccess) e = make_operand_tile_map(&mq, a.q, D, a.Hq, rows, BM);
    if (e == cudaSuccess) e = make_operand_tile_map(&mk, a.k, D, a.Hkv, rows, BN);
    if (e == cudaSuccess) e = make_operand_tile_map(&mv, a.v, D, a.Hkv, rows, BN);
    if (e != cudaSuccess) return e;
    const int paired = (a.Hq / a.Hkv) % 2 == 0;
    const long long grid = paired ? a.seq.n_tiles(BM) * (a.Hq / 2) : a.seq.n_tiles(2 * BM) * a.Hq;
    kern<<<(unsigned)grid, kThreadsTc, bytes, st>>>(a, mq, mk, mv, paired);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swa_fwd_tc(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? fwd_t<64>(a, st) : fwd_t<128>(a, st);
}

}  // namespace carve
