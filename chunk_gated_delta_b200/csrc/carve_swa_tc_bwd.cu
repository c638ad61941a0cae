// Sliding-window attention with sink tokens, backward, on the 5th-generation tensor core (bf16;
// include/carve_mixers.h).
//
// With lse and delta_i = sum_c dO_ic o_ic from the forward's results,
//   p_ij = e^{scale q_i.k_j - lse_i},  ds_ij = p_ij (dO_i.v_j - delta_i)
//   dv_j = sum_i p_ij dO_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
// Two passes of one kernel (and, for few keys, one that joins the first's parts), so that every sum
// stays in one accumulator in a fixed order (one pass with dq summed by atomics needs 5 products
// instead of 7, but its results would depend on the order of arrival).  A unit holds 128 rows (KEYS: keys with dk, dv; else queries with dq) as two
// resident operand tiles R1, R2 and streams the other side in tiles C1, C2 of 64:
//             R1   R2   C1   C2
//   KEYS      k    v    q    dO     over the query heads of the key head
//   else      q    dO   k    v
//   S = R1 C1^T, dP = R2 C2^T   accumulators in tensor memory, two buffers
//   P, dS                       two threads a row, 32 columns each; back to tensor memory as bf16 over S, dP
//   acc1 += dS C1 (dk or dq),  acc2 += P C2 (dv)   A from tensor memory, C's rows contracted
// Roles: warps 0-7 and 8-15 form P, dS of the even and odd column tiles, warp 16 copies, warp 18 takes what
// has landed, warp 17 issues the products: S, dP of the tile after next go out while the other buffer
// is being worked on.
// Persistent: a CTA walks its units with one set of running phases; R is given back with the unit's last
// S and dP, so the next unit's rows load beside this one's last sums and epilogue.  Four column stages:
// three tiles are held by what is being computed (a fifth changes nothing).  A tile of 128 x 64 takes
// 1900 cycles: the tensor core 1280 (keys) or 1024 (queries), most of it at the rate at which shared memory
// gives S and dP their operands, and the product warp's way from one tile to the next the rest.  8
// sequences of 4096 tokens, 16 query and 4 key heads, d = 128, W = 1024: keys 780 us, queries 520 us.
#include "carve_mixers.cuh"
#include "carve_umma.cuh"

namespace carve {

__device__ int g_swa_bwd_status;   // kTimedOut, kBadOffsets

int swa_bwd_take_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_swa_bwd_status, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_swa_bwd_status, &z, sizeof(int));
    }
    return v;
}

namespace {

constexpr int BR = 128, BC = 64, kStages = 4, kWorkers = 16, kThreadsTc = (kWorkers + 3) * 32;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct BwdSmem {
    __nv_bfloat16 r[2][D / 64][BR * 64];           // R1, R2
    __nv_bfloat16 c[kStages][2][D / 64][BC * 64];  // [stage][C1, C2]
    float2 ld[kStages][BC + 2];                    // (-lse log2 e, -delta) of the columns (KEYS), from an even index on
    uint64_t rfull, rfree, cfull[kStages], cready[kStages], cfree[kStages], sfull[2], dfull[2], accfull, accfree;
    uint32_t tmem;
};

// (-lse log2 e, -delta) of every row and query head, [Hq][rows]: 16 lanes a (row, head), 16 bytes each
template <int D>
__global__ void __launch_bounds__(256) swa_rows(SwaArgs a, long long rows) {
    constexpr int L = D / 8;
    if (blockIdx.x == 0) check_seqs(a.seq, &g_swa_bwd_status, kBadOffsets);
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) / L;   // row * Hq + head
    const int x = threadIdx.x % L;
    float s = 0.f;
    if (i < rows * a.Hq) {
        const uint4 o = reinterpret_cast<const uint4 *>(a.o)[i * L + x], g = reinterpret_cast<const uint4 *>(a.dO)[i * L + x];
        const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            s += __uint_as_float(ow[y] << 16) * __uint_as_float(gw[y] << 16);
            s += __uint_as_float(ow[y] & 0xffff0000u) * __uint_as_float(gw[y] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int off = L / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (x == 0 && i < rows * a.Hq)
        reinterpret_cast<float2 *>(a.delta)[(i % a.Hq) * rows + i / a.Hq] = make_float2(-a.lse[i] * kLog2e, -s);
}

// A unit: 128 rows of one sequence and head, and its column tiles.
template <bool KEYS>
struct Unit {
    long long row0;
    int len, r0, r1, head;   // rows r0 .. r1 - 1, their head
    int n, per, c0;          // column tiles; KEYS: per query head, from tile c0
    int part, b0;            // KEYS: the part of the unit, its first tile of them all
    KeyTiles kt;
    __device__ __forceinline__ bool set(const SwaArgs &a, int u) {
        const int heads = KEYS ? a.Hkv : a.Hq;
        int s, c;
        part = 0;
        if (KEYS) {
            part = u % a.parts;
            u /= a.parts;
        }
        if (!a.seq.find(u / heads, BR, s, c, row0, len)) return false;
        head = u % heads;
        r0 = c * BR;
        r1 = min(r0 + BR, len);
        if (KEYS) {
            c0 = r0 / BC;
            per = last_query(r0, r1, len, a.window, a.sinks) / BC - c0 + 1;
            const long long all = (long long)per * (a.Hq / a.Hkv);
            b0 = (int)(all * part / a.parts);
            n = (int)(all * (part + 1) / a.parts) - b0;
        } else {
            kt = KeyTiles(r0, r1, BC, a.window, a.sinks);
            n = kt.count();
        }
        return true;
    }
    __device__ __forceinline__ int col0(int b) const { return (KEYS ? c0 + b0 + b - (b0 + b) / per * per : kt.tile(b)) * BC; }
    __device__ __forceinline__ int col_head(const SwaArgs &a, int b) const {
        const int share = a.Hq / a.Hkv;
        return KEYS ? head * share + (b0 + b) / per : head / share;
    }
};

template <int D, bool KEYS>
__global__ void __launch_bounds__(kThreadsTc, 1)
    swa_tc_bwd(SwaArgs a, const __grid_constant__ CUtensorMap mr1, const __grid_constant__ CUtensorMap mr2,
               const __grid_constant__ CUtensorMap mc1, const __grid_constant__ CUtensorMap mc2, int units, long long rows) {
    extern __shared__ __align__(16) unsigned char raw[];
    BwdSmem<D> &sm = *reinterpret_cast<BwdSmem<D> *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int KH = D / 64;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.sfull[i], 1);
            mbar_init(&sm.dfull[i], kWorkers / 2);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.cfull[i], 1);
            mbar_init(&sm.cready[i], 1);
            mbar_init(&sm.cfree[i], 1);
        }
        mbar_init(&sm.rfull, 1);
        mbar_init(&sm.rfree, 1);
        mbar_init(&sm.accfull, 1);
        mbar_init(&sm.accfree, kWorkers);
        fence_mbar_init();
    }
    if (warp == kWorkers + 1) tmem_alloc(&sm.tmem, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = sm.tmem;   // S buffers at 0, 64; dP at 128, 192; acc1 at 256, acc2 at 384
    bool ok = true;
    auto wait = [&](uint64_t &bar, int phase) {   // by a whole warp
        return mbar_wait_warp(&bar, phase & 1, kIdleWait);
    };
    Unit<KEYS> w;
    // index of a column's entry in the table [Hq][rows]
    auto col_index = [&](const Unit<KEYS> &u, int h, int c0) { return (long long)h * rows + u.row0 + c0; };
    int nu = 0, nc = 0;   // units and column tiles so far

    if (warp == kWorkers) {
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            if (!w.set(a, u) || w.n == 0) continue;
            for (int b = 0; b < w.n; ++b) {
                if (b == 0) {
                    if (nu > 0) ok = wait(sm.rfree, nu - 1);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_expect_tx(&sm.rfull, 2 * BR * D * 2);
                        for (int y = 0; y < KH; ++y) {
                            tma_load_3d(sm.r[0][y], &mr1, 64 * y, w.head, (int)w.row0 + w.r0, &sm.rfull);
                            tma_load_3d(sm.r[1][y], &mr2, 64 * y, w.head, (int)w.row0 + w.r0, &sm.rfull);
                        }
                    }
                    ++nu;
                }
                const int s = nc % kStages, c0 = w.col0(b), h = w.col_head(a, b);
                if (nc >= kStages) ok = wait(sm.cfree[s], nc / kStages - 1);
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect_tx(&sm.cfull[s], 2 * BC * D * 2 + (KEYS ? sizeof(sm.ld[0]) : 0));
                    for (int y = 0; y < KH; ++y) {
                        tma_load_3d(sm.c[s][0][y], &mc1, 64 * y, h, (int)w.row0 + c0, &sm.cfull[s]);
                        tma_load_3d(sm.c[s][1][y], &mc2, 64 * y, h, (int)w.row0 + c0, &sm.cfull[s]);
                    }
                    // rows behind the sequence are masked; those behind the table lie in the workspace's tail
                    if (KEYS) bulk_g2s(sm.ld[s], reinterpret_cast<const float2 *>(a.delta) + (col_index(w, h, c0) & ~1ll), sizeof(sm.ld[0]), &sm.cfull[s]);
                }
                ++nc;
            }
        }
        if (!ok) {   // the copies in flight land before the CTA leaves
            if (nu) wait(sm.rfull, nu - 1);
            for (int i = max(0, nc - kStages); i < nc; ++i) wait(sm.cfull[i % kStages], i / kStages);
        }
    } else if (warp == kWorkers + 1) {
        constexpr uint32_t iS = umma_idesc_bf16(BR, BC), iA = umma_idesc_bf16(BR, D) | kUmmaBmn;
        const uint64_t dr = umma_desc(smem_u32(sm.r)), dc = umma_desc(smem_u32(sm.c)), dct = umma_desc_mn(smem_u32(sm.c), BC * 128);
        // S, dP of the tile (by the elected lane)
        auto issue_s = [&](int c, int s, bool last) {
            const uint64_t cols = desc_at(dc, s * (uint32_t)sizeof(sm.c[0]));
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16(tm + 128 * y + 64 * (c & 1), desc_at(dr, BR * 128 * (KH * y + kk / 4) + 32 * (kk % 4)),
                              desc_at(cols, BC * 128 * (KH * y + kk / 4) + 32 * (kk % 4)), iS, kk > 0);
            umma_commit(&sm.sfull[c & 1]);
            if (last) umma_commit(&sm.rfree);   // the next unit's rows load beside this one's last sums
        };
        int done = 0;                    // column tiles whose S, dP were issued
        int ss = 0, sp = 0, fs = 0;      // stage and phase of the next S, dP, stage of the next sums
        auto step = [&] {
            ss = ss + 1 == kStages ? 0 : ss + 1;
            sp ^= ss == 0;
            ++done;
        };
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            if (!w.set(a, u) || w.n == 0) continue;
            const int n = w.n;
            ok = wait(sm.rfull, nu);
            for (int b = 0; b < min(2, n) && ok; ++b) {
                if (!(ok = wait(sm.cready[ss], sp))) break;
                tc_fence_after_sync();
                if (elect_one()) issue_s(nc + b, ss, b == n - 1);
                __syncwarp();
                step();
            }
            // The queue of products is short, so what this warp does between them is seen in full: the
            // tiles are taken by another warp, and the sums and the next products go out together.
            for (int b = 0; b < n && ok; ++b, ++nc) {
                const bool more = b + 2 < n;
                if (more) ok = wait(sm.cready[ss], sp);
                if (ok) ok = wait(sm.dfull[nc & 1], nc / 2);
                if (ok && b == 0 && nu > 0) ok = wait(sm.accfree, nu - 1);
                if (!ok) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t cols = desc_at(dct, fs * (uint32_t)sizeof(sm.c[0]));
#pragma unroll
                    for (int kk = 0; kk < BC / 16; ++kk)
                        umma_bf16_ta(tm + 256, tm + 128 + 64 * (nc & 1) + 8 * kk + (kk < 2 ? 0 : 16), desc_at(cols, 2048 * kk), iA,
                                     b > 0 || kk > 0);
                    if (KEYS) {
#pragma unroll
                        for (int kk = 0; kk < BC / 16; ++kk)
                            umma_bf16_ta(tm + 384, tm + 64 * (nc & 1) + 8 * kk + (kk < 2 ? 0 : 16),
                                         desc_at(cols, BC * 128 * KH + 2048 * kk), iA, b > 0 || kk > 0);
                    }
                    umma_commit(&sm.cfree[fs]);
                    if (b == n - 1) umma_commit(&sm.accfull);
                    if (more) issue_s(nc + 2, ss, b + 2 == n - 1);
                }
                __syncwarp();
                fs = fs + 1 == kStages ? 0 : fs + 1;
                if (more) step();
            }
            ++nu;
        }
        if (!ok) {   // products in flight finish before the tensor memory is freed
            for (int i = max(0, done - 2); i < done; ++i) wait(sm.sfull[i & 1], i / 2);
            for (int i = max(0, nc - kStages); i < nc; ++i) wait(sm.cfree[i % kStages], i / kStages);
        }
    } else if (warp == kWorkers + 2) {
        // takes the column tiles as they land: rows behind the sequence's end, which meet P = dS = 0 in the
        // sums, become zero
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            if (!w.set(a, u) || w.n == 0) continue;
            for (int b = 0; b < w.n; ++b, ++nc) {
                const int s = nc % kStages, there = w.len - w.col0(b);
                if (!(ok = wait(sm.cfull[s], nc / kStages))) break;
                if (there < BC) {
                    for (int y = 0; y < 2 * KH; ++y)
                        for (int i = there * 8 + lane; i < BC * 8; i += 32)
                            reinterpret_cast<uint4 *>(sm.c[s][y / KH][y % KH])[i] = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                mbar_arrive_warp(&sm.cready[s]);
            }
        }
    } else {
        const int g = warp / 8, half = (warp / 4) % 2, quarter = warp % 4, t = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;
        const uint32_t tS = tm + 64 * g + 32 * half + lanes, tP = tm + 128 + 64 * g + 32 * half + lanes;
        const float sc = a.scale * kLog2e;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            if (!w.set(a, u)) continue;
            const int row = w.r0 + t;   // of the sequence
            float2 mine = make_float2(0.f, 0.f);
            if (!KEYS && row < w.r1) mine = reinterpret_cast<const float2 *>(a.delta)[(size_t)w.head * rows + w.row0 + row];
            for (int b = 0; b < w.n && ok; ++b, ++nc) {
                if ((nc & 1) != g) continue;
                const int c0 = w.col0(b);
                ok = wait(sm.sfull[g], nc / 2);
                if (!ok) break;
                tc_fence_after_sync();
                // masked only where the diagonal, the window's far edge or the end crosses the tile
                const int i0 = KEYS ? c0 : w.r0, i1 = KEYS ? c0 + BC : w.r0 + BR, j0 = KEYS ? w.r0 : c0, j1 = KEYS ? w.r0 + BR : c0 + BC;
                const bool edge = !(j1 - 1 <= i0 && (i1 - 1 - j0 < a.window || j1 <= a.sinks) && i1 <= w.len);
                const int y = c0 + 32 * half;
                uint32_t seen = 0xffffffffu;
                if (edge) {   // bit x: column y + x
                    if (KEYS) {   // queries from this key on, below its window's end (a sink: any), below len
                        const int from = row - y;
                        const long long end = row < a.sinks ? (long long)w.len : min((long long)w.len, (long long)row + a.window);
                        const long long n = end - y;
                        seen = from <= 0 ? 0xffffffffu : from > 31 ? 0u : 0xffffffffu << from;
                        seen &= n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << (int)n) - 1u;
                    } else {      // keys up to this query, from its window's start on or sinks
                        const int top = row - y, before = a.sinks - y;
                        const long long from = (long long)row - a.window + 1 - y;
                        const uint32_t near = from <= 0 ? 0xffffffffu : from > 31 ? 0u : 0xffffffffu << (int)from;
                        const uint32_t sink = before >= 32 ? 0xffffffffu : before <= 0 ? 0u : (1u << before) - 1u;
                        seen = (top >= 31 ? 0xffffffffu : top < 0 ? 0u : (2u << top) - 1u) & (near | sink);
                    }
                }
#pragma unroll
                for (int b16 = 0; b16 < 32; b16 += 16) {
                    uint32_t s[16], d[16], pk[8], dk[8];
                    tmem_ld16(tS + b16, s);
                    tmem_ld16(tP + b16, d);
                    tmem_wait_ld();
                    tmem_tie16(s);
                    tmem_tie16(d);
                    const float2 *ld = sm.ld[nc % kStages] + 32 * half + b16 + (KEYS ? col_index(w, w.col_head(a, b), c0) & 1 : 0);
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        const float2 c = KEYS ? ld[x] : mine, c1 = KEYS ? ld[x + 1] : mine;
                        const float2 z = fma2(make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), make_float2(sc, sc), make_float2(c.x, c1.x));
                        const float2 f = add2(make_float2(__uint_as_float(d[x]), __uint_as_float(d[x + 1])), make_float2(c.y, c1.y));
                        float p0 = ex2(z.x), p1 = ex2(z.y);
                        const float2 g2 = mul2(make_float2(p0, p1), f);
                        float e0 = g2.x, e1 = g2.y;
                        if (edge) {
                            if (!((seen >> (b16 + x)) & 1u)) p0 = e0 = 0.f;
                            if (!((seen >> (b16 + x + 1)) & 1u)) p1 = e1 = 0.f;
                        }
                        pk[x / 2] = pack_bf16(p0, p1);
                        dk[x / 2] = pack_bf16(e0, e1);
                    }
                    // over columns that this thread has read
                    if (KEYS) tmem_st8(tS + b16 / 2, pk);
                    tmem_st8(tP + b16 / 2, dk);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive_warp(&sm.dfull[g]);
            }
            if (!ok) break;
            if (w.n > 0) {
                ok = wait(sm.accfull, nu);
                if (!ok) break;
                ++nu;
                tc_fence_after_sync();
            }
            // KEYS: group 0 writes dv, 1 dk, a thread half the channels; else a quarter of dq's
            constexpr int W = KEYS ? D / 2 : D / 4;
            const int x0 = W * (KEYS ? half : 2 * g + half);
            const uint32_t src = tm + lanes + x0 + (KEYS && g == 0 ? 384 : 256);
            const float f = KEYS && g == 0 ? 1.f : a.scale;
            const size_t at = ((size_t)(w.row0 + row) * (KEYS ? a.Hkv : a.Hq) + w.head) * D + x0;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(KEYS ? (g == 0 ? a.dv : a.dk) : a.dq) + at;
            float *sums = KEYS && a.parts > 1 ? a.partial + (size_t)((1 - g) * a.parts + w.part) * rows * a.Hkv * D + at : nullptr;
#pragma unroll
            for (int x = 0; x < W; x += 16) {
                uint32_t o[16];
                if (w.n > 0) {
                    tmem_ld16(src + x, o);
                    tmem_wait_ld();
                    tmem_tie16(o);
                } else {
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] = 0u;
                }
                if (sums) {
                    if (row < w.r1)
#pragma unroll
                        for (int y = 0; y < 16; y += 4)
                            *reinterpret_cast<float4 *>(sums + x + y) =
                                make_float4(__uint_as_float(o[y]) * f, __uint_as_float(o[y + 1]) * f, __uint_as_float(o[y + 2]) * f, __uint_as_float(o[y + 3]) * f);
                } else if (row < w.r1) {
#pragma unroll
                    for (int y = 0; y < 16; y += 8) {
                        uint4 v;
                        v.x = pack_bf16(__uint_as_float(o[y]) * f, __uint_as_float(o[y + 1]) * f);
                        v.y = pack_bf16(__uint_as_float(o[y + 2]) * f, __uint_as_float(o[y + 3]) * f);
                        v.z = pack_bf16(__uint_as_float(o[y + 4]) * f, __uint_as_float(o[y + 5]) * f);
                        v.w = pack_bf16(__uint_as_float(o[y + 6]) * f, __uint_as_float(o[y + 7]) * f);
                        *reinterpret_cast<uint4 *>(out + x + y) = v;
                    }
                }
            }
            tc_fence_before_sync();
            if (w.n > 0) mbar_arrive_warp(&sm.accfree);
        }
    }
    if (!ok && lane == 0) atomicOr(&g_swa_bwd_status, kTimedOut);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kWorkers + 1) tmem_dealloc(tm, 512);
}

// dk, dv of JR rows of a key head: their parts' sums, in order
constexpr int JR = 8;
template <int D>
__global__ void __launch_bounds__(2 * JR * D / 4) swa_join(SwaArgs a, long long rows) {
    constexpr int X = D / 4;
    int s, c, len;
    long long row0;
    const int u = blockIdx.x / (BR / JR), head = u % a.Hkv;
    if (!a.seq.find(u / a.Hkv, BR, s, c, row0, len)) return;
    const int z = threadIdx.x / (JR * X), r = c * BR + blockIdx.x % (BR / JR) * JR + threadIdx.x / X % JR;
    if (r >= len) return;
    const size_t per = (size_t)rows * a.Hkv * D, at = ((size_t)(row0 + r) * a.Hkv + head) * D + threadIdx.x % X * 4;
    const float *src = a.partial + (size_t)z * a.parts * per + at;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p) {
        const float4 v = *reinterpret_cast<const float4 *>(src + p * per);
        y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
    }
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(z ? a.dv : a.dk) + at) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}

template <int D, bool KEYS>
cudaError_t pass(const SwaArgs &a, const CUtensorMap &r1, const CUtensorMap &r2, const CUtensorMap &c1, const CUtensorMap &c2,
                 long long rows, cudaStream_t st) {
    auto kern = swa_tc_bwd<D, KEYS>;
    const int bytes = (int)sizeof(BwdSmem<D>) + 1024;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), bytes);
    if (e != cudaSuccess) return e;
    const int units = (int)(a.seq.n_tiles(BR) * (KEYS ? a.Hkv * a.parts : a.Hq)), sms = sm_count();
    kern<<<units < sms ? units : sms, kThreadsTc, bytes, st>>>(a, r1, r2, c1, c2, units, rows);
    return cudaGetLastError();
}

template <int D>
cudaError_t bwd_t(const SwaArgs &a, cudaStream_t st) {
    const long long rows = a.seq.cu ? a.seq.total : (long long)a.seq.N * a.seq.T;
    const void *base[4] = {a.q, a.k, a.v, a.dO};
    CUtensorMap big[4], small[4];   // boxes of 128 and 64 rows of q, k, v, dO
    for (int i = 0; i < 4; ++i) {
        const int H = i == 1 || i == 2 ? a.Hkv : a.Hq;
        cudaError_t e = make_operand_tile_map(&big[i], base[i], D, H, rows, BR);
        if (e == cudaSuccess) e = make_operand_tile_map(&small[i], base[i], D, H, rows, BC);
        if (e != cudaSuccess) return e;
    }
    swa_rows<D><<<(unsigned)((rows * a.Hq * (D / 8) + 255) / 256), 256, 0, st>>>(a, rows);
    cudaError_t e = pass<D, true>(a, big[1], big[2], small[0], small[3], rows, st);
    if (e == cudaSuccess && a.parts > 1) swa_join<D><<<(unsigned)(a.seq.n_tiles(BR) * a.Hkv * (BR / JR)), 2 * JR * D / 4, 0, st>>>(a, rows);
    if (e == cudaSuccess) e = pass<D, false>(a, big[0], big[3], small[1], small[2], rows, st);
    return e;
}

}  // namespace

// Parts that the keys' pass takes a unit's column tiles in, when the units (128 keys of a key head) leave SMs
// idle: as many as there are SMs for, of four tiles at least.  Partial sums in fp32, joined in order (1 sequence
// of 1000 tokens, 8 query and 2 key heads, window 200: pass and join 33 us from 75 us; 2 of 4000, 4 and 1 heads,
// window 1500: 156 us from 271 us).  The rule asks for sizes alone, so that the scratch can be sized without
// a device; packed calls of very many sequences have too many tile numbers for it.
int swa_bwd_parts(const SwaArgs &a) {
    const long long rows = a.seq.cu ? a.seq.total : a.seq.T, units = (a.seq.cu ? a.seq.total / BR + 1 : a.seq.n_tiles(BR)) * a.Hkv;
    const long long tiles = (a.Hq / a.Hkv) * ((rows < a.window ? rows : a.window) / BC + 2);
    if (units < 1 || a.seq.N > 4096) return 1;
    const long long parts = 148 / units < tiles / 4 ? 148 / units : tiles / 4;
    return parts < 2 ? 1 : parts > 16 ? 16 : (int)parts;
}

cudaError_t launch_swa_bwd_tc(const SwaArgs &a, cudaStream_t st) {
    return a.d == 64 ? bwd_t<64>(a, st) : bwd_t<128>(a, st);
}

}  // namespace carve
