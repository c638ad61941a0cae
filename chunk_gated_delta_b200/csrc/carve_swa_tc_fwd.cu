// Sliding-window attention with sink tokens, forward, on the 5th-generation tensor core (bf16;
// include/carve_mixers.h).
//
// A CTA holds two query tiles of 128 rows that read the same keys: two query heads of one key
// head when the heads pair up (the keys of one 128-row window), else 256 rows of one head.  For
// each 64-key block that a tile sees:
//   S = Q K^T                    tcgen05.mma, accumulator in tensor memory (64 columns, two buffers)
//   P = 2^{S scale log2 e - m}   two threads a row, 32 scores each in registers; they exchange
//                                their maxima through shared memory; P goes back as bf16 over S
//   O += P V                     A = P from tensor memory, O stays in tensor memory
// The next block's S is there while this one is in softmax.  (With 128-key blocks tensor memory has room
// for one S a tile: softmax, P V and the next S of a tile then wait for one another, 3850 cycles for 128
// keys of both tiles where their products take 2048.)  m is the maximum that was current when O was last
// rescaled: O is rescaled (a round trip through registers) only when some row's maximum has grown
// by more than 2^8 since, which keeps P below 2^8 and sums in fp32 exact to rounding; the last
// division removes the reference.
// Roles: warps 0-7 and 8-15 softmax of tile 0 and 1 (the second four of each take the upper half of the
// columns), warp 16 copies (TMA, ring of five 64-row key or value tiles, queries of the next unit),
// warps 17 and 18 issue the products of a tile each.  Persistent: a unit's copies and first products run
// beside the last one's outputs (the two took a fifth of a CTA's time at W = 1024, a quarter at 512).
// Softmax bounds it: 2000 cycles for 64 keys of both tiles, of which the exponentials need 1024 and the
// products 1280.  8 sequences of 4096 tokens, 16 query and 4 key heads, d = 128, W = 1024: 310 us, 780
// TFLOP/s of products; 4 of 2048, W = 512: 68 us.
//
// Blocks that a tile does not see are skipped; only blocks that a window edge or the diagonal
// crosses are masked, by selection.  Value rows behind the sequence's end are zeroed in shared
// memory, so nothing that belongs to another sequence meets a product with P = 0.
#include "carve_mixers.cuh"
#include "carve_umma.cuh"

namespace carve {

__device__ int g_swa_fwd_status;   // kTimedOut, kBadOffsets

int swa_fwd_take_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_swa_fwd_status, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_swa_fwd_status, &z, sizeof(int));
    }
    return v;
}

namespace {

// rows `first` .. 63 of a block of 64 rows x 64 KH channels in operand layout become zero (one warp)
__device__ __forceinline__ void zero_block_rows(void *tile, int first, int halves, int lane) {
    for (int y = 0; y < halves; ++y)
        for (int i = max(first, 0) * 8 + lane; i < 64 * 8; i += 32)
            reinterpret_cast<uint4 *>(tile)[y * 64 * 8 + i] = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int BM = 128, BN = 64, kStages = 5, kThreadsTc = 608;
constexpr float kLazy = 8.f;   // growth of a row's maximum, in powers of two, that O may lag behind

template <int D>
struct FwdSmem {
    __nv_bfloat16 q[2][2][D / 64][BM * 64];   // [unit's parity][tile], then the tile's outputs
    __nv_bfloat16 kv[kStages][D / 64][BN * 64];
    float part[2][2][2][BM];   // a row's maximum, at the end its sum, by turn, tile and column half
    uint64_t qfull[2], qfree[2], kvfull[kStages], kvfree[kStages], ofree[2];
    uint64_t sfull[2][2], pfull[2][2], ofull[2][2];   // [tile][parity of its block]: two blocks may be under way
    uint32_t tmem;
};

// A unit: two query tiles and the key blocks that they see.
struct Work {
    long long row0;
    int len, i0[2], i1[2], h[2], hk, blocks;
    KeyTiles kt;
    __device__ __forceinline__ bool set(const SwaArgs &a, int unit, int paired) {
        const int per = paired ? a.Hq / 2 : a.Hq, rows = paired ? BM : 2 * BM, tile = unit / per, u = unit - tile * per;
        int n, c;
        if (!a.seq.find(tile, rows, n, c, row0, len)) return false;
        i0[0] = c * rows;
        i0[1] = paired ? i0[0] : i0[0] + BM;
        i1[0] = min(i0[0] + BM, len);
        i1[1] = min(i0[1] + BM, len);
        h[0] = paired ? 2 * u : u;
        h[1] = paired ? h[0] + 1 : u;
        hk = h[0] / (a.Hq / a.Hkv);
        kt = KeyTiles(i0[0], min(i0[0] + rows, len), BN, a.window, a.sinks);
        blocks = kt.count();
        return true;
    }
    __device__ __forceinline__ bool sees(const SwaArgs &a, int t, int j0) const {
        return i0[t] < i1[t] && j0 < i1[t] && (j0 < a.sinks || (long long)j0 + BN - 1 + a.window > i0[t]);
    }
};

template <int D>
__global__ void __launch_bounds__(kThreadsTc, 1)
    swa_tc_fwd(SwaArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, int paired, int items) {
    extern __shared__ __align__(16) unsigned char raw[];
    FwdSmem<D> &sm = *reinterpret_cast<FwdSmem<D> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int KH = D / 64;
    constexpr uint32_t kTile = BN * D * 2;   // bytes of one operand tile

    // The copying lane initialises the barriers and sends for the first unit's tiles before the CTA meets:
    // their way here and the allocation of tensor memory take 1 us each.
    Work w;
    bool ok = true;
    const bool copier = warp == 16 && elect_one();
    int filled = 0, nu = 0;   // ring tiles copied; units so far
    auto fill = [&](const CUtensorMap *map, int b) {
        const int s = filled % kStages;
        if (filled >= kStages) ok = mbar_wait(&sm.kvfree[s], (filled / kStages - 1) & 1, kSwaWait);
        if (!ok) return;
        mbar_expect_tx(&sm.kvfull[s], kTile);
        for (int x = 0; x < KH; ++x) tma_load_3d(sm.kv[s][x], map, 64 * x, w.hk, (int)w.row0 + w.kt.tile(b) * BN, &sm.kvfull[s]);
        ++filled;
    };
    auto begin = [&] {   // a unit's queries, and its first keys; in the order in which they are used: K0, K1, V0, K2, V1, ...
        const int x2 = nu & 1;
        if (nu >= 2) ok = mbar_wait(&sm.qfree[x2], (nu / 2 - 1) & 1, kSwaWait);
        if (!ok) return;
        mbar_expect_tx(&sm.qfull[x2], 2 * BM * D * 2);
        for (int t = 0; t < 2; ++t)
            for (int x = 0; x < KH; ++x)
                tma_load_3d(sm.q[x2][t][x], &mq, 64 * x, w.h[t], (int)(w.row0 + w.i0[t]), &sm.qfull[x2]);
        ++nu;
        fill(&mk, 0);
        if (w.blocks > 1 && ok) fill(&mk, 1);
    };
    int first = blockIdx.x;   // the copying lane's first unit
    if (copier) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.kvfull[i], 1);
            mbar_init(&sm.kvfree[i], 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.qfull[t], 1);
            mbar_init(&sm.qfree[t], 2);
            mbar_init(&sm.ofree[t], 8);
            mbar_init(&sm.sfull[t][0], 1);
            mbar_init(&sm.sfull[t][1], 1);
            mbar_init(&sm.pfull[t][0], 8);
            mbar_init(&sm.pfull[t][1], 8);
            mbar_init(&sm.ofull[t][0], 1);
            mbar_init(&sm.ofull[t][1], 1);
        }
        fence_mbar_init();
        while (first < items && !w.set(a, first, paired)) first += gridDim.x;
        if (first < items) begin();
    }
    if (warp == 17) tmem_alloc(&sm.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;   // S of tile t at column 128 t, two buffers of 64, O at 256 + 128 t
    auto wait = [&](uint64_t &bar, int phase) {   // by a whole warp
        return mbar_wait_warp(&bar, phase & 1, kIdleWait);
    };

    if (warp == 16) {
        if (copier) {
            for (int u = first; u < items && ok; u += gridDim.x) {
                if (u != first) {
                    if (!w.set(a, u, paired)) continue;
                    begin();
                }
                for (int b = 0; b < w.blocks && ok; ++b) {
                    fill(&mv, b);
                    if (b + 2 < w.blocks && ok) fill(&mk, b + 2);
                }
            }
            if (!ok) {   // the copies in flight land before the CTA leaves
                for (int i = max(0, nu - 2); i < nu; ++i) mbar_wait(&sm.qfull[i & 1], (i / 2) & 1, kSwaWait);
                for (int i = max(0, filled - kStages); i < filled; ++i)
                    mbar_wait(&sm.kvfull[i % kStages], (i / kStages) & 1, kSwaWait);
            }
        }
    } else if (warp >= 17) {
        // a warp for each tile: what one does between its products runs beside the other's
        constexpr uint32_t iS = umma_idesc_bf16(BM, BN), iO = umma_idesc_bf16(BM, D) | kUmmaBmn;
        const int t = warp - 17;
        const uint32_t tS = tm + 128 * t, tO = tm + 256 + 128 * t;
        const uint64_t dq0 = umma_desc(smem_u32(sm.q[0][t])), dk0 = umma_desc(smem_u32(sm.kv)), dv0 = umma_desc_mn(smem_u32(sm.kv), BN * 128);
        int ns = 0, np = 0, no = 0;     // products S and P V issued, units with outputs
        uint64_t dq = dq0;
        int slot = 0, turn = 0;         // the ring, in the order of its copies
        auto next = [&] {
            if (elect_one()) umma_commit(&sm.kvfree[slot]);
            __syncwarp();
            slot = (slot + 1) % kStages;
            turn += slot == 0;
        };
        auto issue_s = [&](bool sees) {   // S of a key block
            ok = wait(sm.kvfull[slot], turn);
            if (!ok) return;
            if (sees) {
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t k = desc_at(dk0, slot * sizeof(sm.kv[0]));
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_bf16(tS + 64 * (ns & 1), desc_at(dq, BM * 128 * (kk / 4) + 32 * (kk % 4)),
                                  desc_at(k, BN * 128 * (kk / 4) + 32 * (kk % 4)), iS, kk > 0);
                    umma_commit(&sm.sfull[t][ns & 1]);
                }
                __syncwarp();
                ++ns;
            }
            next();
        };
        auto sees = [&](int b) { return b < w.blocks && w.sees(a, t, w.kt.tile(b) * BN); };
        for (int u = blockIdx.x; u < items && ok; u += gridDim.x) {
            if (!w.set(a, u, paired)) continue;
            bool s0 = sees(0), s1 = sees(1), some = false;   // of blocks b and b + 1; any P V yet
            dq = desc_at(dq0, (nu & 1) * (uint32_t)sizeof(sm.q[0]));
            ok = wait(sm.qfull[nu & 1], nu / 2);
            // a tile without rows: nothing else of it waits for the queries, and they may be copied over only once
            // this warp has seen them
            if (ok && w.i0[t] >= w.i1[t]) {
                if (elect_one()) mbar_arrive(&sm.qfree[nu & 1]);
                __syncwarp();
            }
            ++nu;
            if (ok) issue_s(s0);
            if (ok && w.blocks > 1) issue_s(s1);
            for (int b = 0; b < w.blocks && ok; ++b) {
                const bool s2 = sees(b + 2);
                ok = wait(sm.kvfull[slot], turn);
                if (!ok) break;
                if (s0) {
                    const int there = w.len - w.kt.tile(b) * BN;
                    if (there < BN) {   // value rows behind the end: zero (by both warps, each before its product)
                        zero_block_rows(sm.kv[slot][0], there, KH, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (!some && no > 0) ok = wait(sm.ofree[t], no - 1);   // the last unit's outputs are read
                    ok = ok && wait(sm.pfull[t][np & 1], np / 2);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t v = desc_at(dv0, slot * sizeof(sm.kv[0]));
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            umma_bf16_ta(tO, tS + 64 * (np & 1) + 8 * kk + (kk < 2 ? 0 : 16), desc_at(v, 2048 * kk), iO, kk > 0 || some);
                        umma_commit(&sm.ofull[t][np & 1]);
                    }
                    __syncwarp();
                    ++np;
                    some = true;
                }
                next();
                // the buffer of block b, whose P has been issued for, takes block b + 2
                if (b + 2 < w.blocks) issue_s(s2);
                s0 = s1;
                s1 = s2;
            }
            no += some;
        }
        // products in flight finish before the tensor memory is freed: the softmax warps wait for
        // the last P V, and on the way out after a timeout this warp does
        if (!ok) {
            for (int i = max(0, ns - 2); i < ns; ++i) wait(sm.sfull[t][i & 1], i / 2);
            for (int i = max(0, np - 2); i < np; ++i) wait(sm.ofull[t][i & 1], i / 2);
        }
    } else {
        const int t = warp / 8, half = (warp / 4) % 2, quarter = warp % 4, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;   // lane quarter in bits 16+
        // this thread's 32 scores (and over the first 16 of them its 32 values of P), its half of O
        const uint32_t tS0 = tm + 128 * t + 32 * half + lanes, tO = tm + 256 + 128 * t + (D / 2) * half + lanes;
        const bool plain = a.scale > 0.f;   // else the scores are scaled first (its sign, or zero)
        const float sc = (plain ? a.scale : 1.f) * 1.4426950408889634f;
        int nb = 0;   // blocks so far
        // exchange with the thread of the row's other half: a barrier of the two warps that both reach once a
        // block whatever else fails (after a wait that ran out the loop goes on without waiting)
        int nx = 0;
        auto other = [&](float x) {
            sm.part[nx & 1][t][half][r] = x;
            asm volatile("bar.sync %0, 64;\n" ::"r"(1 + 4 * t + quarter) : "memory");
            return sm.part[nx++ & 1][t][1 - half][r];
        };
        auto any_of_both = [&](bool x) {   // of the two warps' lanes
            uint32_t y;
            asm volatile(
                "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                : "=r"(y)
                : "r"((uint32_t)x), "r"(1 + 4 * t + quarter)
                : "memory");
            return y != 0;
        };
        for (int u = blockIdx.x; u < items; u += gridDim.x) {
            if (!w.set(a, u, paired)) continue;
            const int x2 = nu++ & 1, i = w.i0[t] + r;
            // the blocks that this tile sees, of those that the CTA walks
            KeyTiles kt(w.i0[t], max(w.i1[t], w.i0[t] + 1), BN, a.window, a.sinks);
            const int mine = w.i0[t] < w.i1[t] ? kt.count() : 0;
            float m = -INFINITY, l = 0.f;   // reference maximum (of unscaled scores) and this half's sum
            for (int b = 0; b < mine; ++b) {
                const int j0 = kt.tile(b) * BN;
                ok = ok && wait(sm.sfull[t][nb & 1], nb / 2);
                tc_fence_after_sync();
                const uint32_t tS = tS0 + 64 * (nb & 1);
                uint32_t s[32];
                tmem_ld32(tS, s);
                tmem_wait_ld();
                tmem_tie(s);
                if (!plain) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * a.scale);
                }
                // masked only where the diagonal or the window's far edge crosses the block
                if (!(j0 + BN - 1 <= w.i0[t] && (w.i0[t] + BM - 1 - j0 < a.window || j0 + BN <= a.sinks))) {
                    const int c0 = j0 + 32 * half, top = i - c0;                       // seen: columns 0 .. top that are
                    const int from = (int)max((long long)i - a.window + 1 - c0, 0LL);  // from this one on, or sinks
                    const int before = a.sinks - c0;
                    const uint32_t past = top >= 31 ? 0xffffffffu : top < 0 ? 0u : (2u << top) - 1u;
                    const uint32_t near = from > 31 ? 0u : 0xffffffffu << from;
                    const uint32_t sink = before >= 32 ? 0xffffffffu : before <= 0 ? 0u : (1u << before) - 1u;
                    const uint32_t seen = past & (near | sink);
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!((seen >> x) & 1u)) s[x] = 0xff800000u;   // -inf
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < 32; x += 2) mx[x / 2 & 3] = max3(mx[x / 2 & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (any_of_both((mb - m) * sc > kLazy)) {       // rare after the first block
                    mb = fmaxf(mb, other(mb));
                    const bool grown = (mb - m) * sc > kLazy;   // of this row alone: a row's result depends on no other
                    const float m1 = grown ? mb : m, f = grown ? ex2((m - m1) * sc) : 1.f;
                    if (b > 0) {
                        ok = ok && wait(sm.ofull[t][(nb - 1) & 1], (nb - 1) / 2);
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
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    const float2 z = fma2(make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), make_float2(sc, sc), make_float2(-base, -base));
                    const float2 p = make_float2(ex2(z.x), ex2(z.y));
                    sum[x / 2 & 1] = add2(sum[x / 2 & 1], p);
                    s[x / 2] = pack_bf16(p.x, p.y);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st16(tS, s);
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive_warp(&sm.pfull[t][nb & 1]);
                ++nb;
            }
            if (mine > 0) {
                l += other(l);
                ok = ok && wait(sm.ofull[t][(nb - 1) & 1], (nb - 1) / 2);
                tc_fence_after_sync();
                const float inv = 1.f / l;
                const size_t at = (size_t)(w.row0 + i) * a.Hq + w.h[t];
                // rows through the tile's query tile (its last S is done) and out by TMA; a last tile's straight to
                // memory, since the rows behind it are others' (16 bytes a row and store: 2 us a CTA where the
                // copy takes a quarter of that)
                const bool whole = w.i1[t] - w.i0[t] == BM;
                uint4 *out = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * D + (D / 2) * half);
#pragma unroll
                for (int x = 0; x < D / 2; x += 32) {
                    uint32_t o[32];
                    tmem_ld32(tO + x, o);
                    tmem_wait_ld();
                    tmem_tie(o);
#pragma unroll
                    for (int y = 0; y < 32; y += 8) {
                        uint4 v;
                        v.x = pack_bf16(__uint_as_float(o[y]) * inv, __uint_as_float(o[y + 1]) * inv);
                        v.y = pack_bf16(__uint_as_float(o[y + 2]) * inv, __uint_as_float(o[y + 3]) * inv);
                        v.z = pack_bf16(__uint_as_float(o[y + 4]) * inv, __uint_as_float(o[y + 5]) * inv);
                        v.w = pack_bf16(__uint_as_float(o[y + 6]) * inv, __uint_as_float(o[y + 7]) * inv);
                        if (whole)
                            *reinterpret_cast<uint4 *>(sm.q[x2][t][0] + umma_off(r, (D / 2) * half + x + y, BM)) = v;
                        else if (ok && i < w.i1[t])
                            out[(x + y) / 8] = v;
                    }
                }
                tc_fence_before_sync();
                mbar_arrive_warp(&sm.ofree[t]);
                if (whole) {
                    fence_proxy_async_smem();
                    asm volatile("bar.sync %0, 256;\n" ::"r"(9 + t) : "memory");   // the tile's eight warps
                    if (warp % 8 == 0 && ok && elect_one()) {
                        for (int x = 0; x < KH; ++x) tma_store_3d(&mo, sm.q[x2][t][x], 64 * x, w.h[t], (int)(w.row0 + w.i0[t]));
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                }
                if (ok && a.lse && half == 0 && i < w.i1[t]) a.lse[at] = (m * sc + log2f(l)) * 0.6931471805599453f;
            }
            // The tile's last S is done, its outputs have left.  (The queries of a tile without rows are given back by
            // its product warp.)
            if (warp % 8 == 0 && mine > 0) {
                if (elect_one()) mbar_arrive(&sm.qfree[x2]);
                __syncwarp();
            }
        }
    }
    if (!ok && lane == 0) atomicOr(&g_swa_fwd_status, kTimedOut);
    if (blockIdx.x == gridDim.x - 1) check_seqs(a.seq, &g_swa_fwd_status, kBadOffsets);
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
    CUtensorMap mq, mk, mv, mo;
    if (e == cudaSuccess) e = make_operand_tile_map(&mq, a.q, D, a.Hq, rows, BM);
    if (e == cudaSuccess) e = make_operand_tile_map(&mo, a.o, D, a.Hq, rows, BM);
    if (e == cudaSuccess) e = make_operand_tile_map(&mk, a.k, D, a.Hkv, rows, BN);
    if (e == cudaSuccess) e = make_operand_tile_map(&mv, a.v, D, a.Hkv, rows, BN);
    if (e != cudaSuccess) return e;
    const int paired = (a.Hq / a.Hkv) % 2 == 0;
    const int items = (int)(paired ? a.seq.n_tiles(BM) * (a.Hq / 2) : a.seq.n_tiles(2 * BM) * a.Hq), sms = sm_count();
    kern<<<items < sms ? items : sms, kThreadsTc, bytes, st>>>(a, mq, mk, mv, mo, paired, items);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swa_fwd_tc(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? fwd_t<64>(a, st) : fwd_t<128>(a, st);
}

}  // namespace carve
