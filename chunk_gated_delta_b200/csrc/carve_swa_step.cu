// Decoding with sliding-window attention and sink tokens (include/carve_mixers.h): the cache
// that a prompt leaves, and one token per sequence against it.
//
// Token t lives in slot t (t < sinks) or sinks + (t - sinks) mod window, so while a sequence has p
// tokens the new token's visible keys are exactly slots 0 .. min(p + 1, sinks + window) - 1 with
// the new token in its own slot: a dense range, whatever the position.  A step reads every
// visible key and value once (2 e (sinks + window) Hkv d bytes a sequence) and is bound by that.
//
// The slots of a (sequence, key head, up to 16 of its query heads) are split over a cluster of 1,
// 2, 4 or 8 CTAs of 4 warps; the CTAs' partial (maximum, sum, output) meet through distributed
// shared memory, so a step is one launch without workspace.  bf16: the products run on mma.sync
// with the query heads as the 16 rows, and keys and values go from global memory straight into
// the fragments: the channel order of a contraction is free, so a lane's 16-byte load of a key
// row holds its pairs for two k-steps, and the channel order of the output tiles is free too,
// so a lane's 16-byte loads of two value rows interleave into the pairs of eight tiles.
#include "carve_mixers.cuh"
#include "carve_mma.cuh"

namespace carve {

__device__ int g_swa_fill_bad_seqlens;   // set when a packed sequence's offsets are out of range

int swa_fill_take_bad_seqlens() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_swa_fill_bad_seqlens, sizeof(int)) != cudaSuccess) return 0;
    if (v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_swa_fill_bad_seqlens, &z, sizeof(int));
    }
    return v;
}

namespace {

// ---- fill ------------------------------------------------------------------------------------
// one warp per (sequence, slot): the newest token of the slot, if there is one
__global__ void __launch_bounds__(256) swa_fill_kernel(SwaArgs a, int row16, long long slots) {
    const long long i = (long long)blockIdx.x * 8 + threadIdx.x / 32;
    const int per = a.sinks + a.window;
    if (i >= slots) return;
    const int n = (int)(i / per), slot = (int)(i - (long long)n * per);
    long long row0;
    int len;
    a.seq.rows(n, row0, len, slot == 0 && threadIdx.x % 32 == 0 ? &g_swa_fill_bad_seqlens : nullptr);
    int t = slot;
    if (slot >= a.sinks) {
        const int back = (int)((((long long)len - 1 - slot) % a.window + a.window) % a.window);
        t = len - 1 - back;
        if (t < a.sinks) return;
    }
    if (t >= len) return;
    const size_t src = (size_t)(row0 + t) * row16, dst = (size_t)i * row16;
    for (int x = threadIdx.x % 32; x < row16; x += 32) {
        static_cast<uint4 *>(a.k_cache)[dst + x] = static_cast<const uint4 *>(a.k)[src + x];
        static_cast<uint4 *>(a.v_cache)[dst + x] = static_cast<const uint4 *>(a.v)[src + x];
    }
}

// ---- step ------------------------------------------------------------------------------------
constexpr int kWarps = 4;
constexpr int kHeads = 16;   // query heads of a CTA

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ float ld_peer(const float *p, uint32_t rank) {   // the same variable in CTA `rank`
    uint32_t addr;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(x) : "r"(addr) : "memory");
    return x;
}

template <int D>
struct StepSmem {
    float o[kWarps][kHeads][D];   // partial outputs (of warp 0 after the CTA's join)
    float m[kWarps][kHeads], l[kWarps][kHeads];
};

// This CTA's part of the slots, the pointers of its keys and values, and the new token's slot.
struct Part {
    int lo, hi, now;
    size_t cache, fresh;   // element offsets of (sequence, head) in the caches and in k, v
};
__device__ __forceinline__ Part part_of(const SwaArgs &a, int b, int hk, int rank, int parts, int D) {
    Part p;
    const long long pos = a.pos[b];
    const int per = a.sinks + a.window;
    const int n = pos < 0 ? 0 : pos + 1 < per ? (int)(pos + 1) : per;
    p.now = pos < 0 ? -1 : pos < a.sinks ? (int)pos : a.sinks + (int)((pos - a.sinks) % a.window);
    const int step = ((n + parts - 1) / parts + 15) / 16 * 16;   // whole 16-key blocks
    p.lo = min(n, rank * step);
    p.hi = min(n, p.lo + step);
    p.cache = ((size_t)b * per * a.Hkv + hk) * D;
    p.fresh = ((size_t)b * a.Hkv + hk) * D;
    return p;
}

// Joins the warps' and then the cluster's partial results and writes the outputs.
template <int D, class IO>
__device__ __forceinline__ void join(StepSmem<D> &sm, const SwaArgs &a, int b, int h0, int nh, int parts) {
    __syncthreads();
    for (int i = threadIdx.x; i < nh * D; i += kWarps * 32) {
        const int g = i / D, x = i % D;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][g]);
        const float base = m == -INFINITY ? 0.f : m;
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) o += expf(sm.m[w][g] - base) * sm.o[w][g][x];
        sm.o[0][g][x] = o;
    }
    __syncthreads();
    if (threadIdx.x < nh) {
        const int g = threadIdx.x;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][g]);
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += expf(sm.m[w][g] - base) * sm.l[w][g];
        sm.m[0][g] = m;
        sm.l[0][g] = l;
    }
    IO *out = static_cast<IO *>(a.o) + ((size_t)b * a.Hq + h0) * D;
    if (parts == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < nh * D; i += kWarps * 32) {
            const float l = sm.l[0][i / D];
            st_io(out + i, l > 0.f ? sm.o[0][i / D][i % D] / l : 0.f);
        }
        return;
    }
    cluster_sync_all();
    const int rank = (int)cluster_rank();
    for (int i = rank * kWarps * 32 + threadIdx.x; i < nh * D; i += parts * kWarps * 32) {
        const int g = i / D, x = i % D;
        float mr[8], m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            mr[r] = r < parts ? ld_peer(&sm.m[0][g], r) : -INFINITY;
            m = fmaxf(m, mr[r]);
        }
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < parts) {
                const float f = expf(mr[r] - base);
                l += f * ld_peer(&sm.l[0][g], r);
                o += f * ld_peer(&sm.o[0][g][x], r);
            }
        st_io(out + i, l > 0.f ? o / l : 0.f);
    }
    cluster_sync_all();   // no CTA leaves while another reads its shared memory
}

// the new token's key and value into its slot (first part, first head group)
template <class IO, int D>
__device__ __forceinline__ void put_token(const SwaArgs &a, const Part &p) {
    constexpr int N = D * (int)sizeof(IO) / 16;
    if (p.now < 0 || threadIdx.x >= 2 * N) return;
    const size_t dst = (p.cache + (size_t)p.now * a.Hkv * D) * sizeof(IO) / 16, src = p.fresh * sizeof(IO) / 16;
    if (threadIdx.x < N)
        static_cast<uint4 *>(a.k_cache)[dst + threadIdx.x] = static_cast<const uint4 *>(a.k)[src + threadIdx.x];
    else
        static_cast<uint4 *>(a.v_cache)[dst + threadIdx.x - N] = static_cast<const uint4 *>(a.v)[src + threadIdx.x - N];
}

// fp32: a warp takes a key at a time, its lanes the channels, the query heads in turn
template <int D>
__global__ void __launch_bounds__(kWarps * 32) swa_step_fp32(SwaArgs a, int groups, int parts) {
    __shared__ StepSmem<D> sm;
    __shared__ float q[kHeads][D];
    const int u = blockIdx.x / parts, rank = blockIdx.x % parts;
    const int grp = u % groups, hk = u / groups % a.Hkv, b = u / groups / a.Hkv;
    const int share = a.Hq / a.Hkv, nh = min(kHeads, share - grp * kHeads), h0 = hk * share + grp * kHeads;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Part p = part_of(a, b, hk, rank, parts, D);
    if (rank == 0 && grp == 0) put_token<float, D>(a, p);
    for (int i = threadIdx.x; i < nh * D; i += kWarps * 32)
        q[i / D][i % D] = static_cast<const float *>(a.q)[((size_t)b * a.Hq + h0) * D + i] * a.scale;
    for (int i = lane; i < nh * D; i += 32) sm.o[warp][i / D][i % D] = 0.f;
    if (lane < kHeads) {
        sm.m[warp][lane] = -INFINITY;
        sm.l[warp][lane] = 0.f;
    }
    __syncthreads();
    for (int j = p.lo + warp; j < p.hi; j += kWarps) {
        const float *kp = j == p.now ? static_cast<const float *>(a.k) + p.fresh
                                     : static_cast<const float *>(a.k_cache) + p.cache + (size_t)j * a.Hkv * D;
        const float *vp = j == p.now ? static_cast<const float *>(a.v) + p.fresh
                                     : static_cast<const float *>(a.v_cache) + p.cache + (size_t)j * a.Hkv * D;
        float k[D / 32], v[D / 32];
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            k[x] = kp[lane + 32 * x];
            v[x] = vp[lane + 32 * x];
        }
        for (int g = 0; g < nh; ++g) {
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) s += k[x] * q[g][lane + 32 * x];
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const float m0 = sm.m[warp][g], m1 = fmaxf(m0, s);
            const float base = m1 == -INFINITY ? 0.f : m1, f = expf(m0 - base), e = expf(s - base);
            __syncwarp();
            if (lane == 0) {
                sm.m[warp][g] = m1;
                sm.l[warp][g] = sm.l[warp][g] * f + e;
            }
#pragma unroll
            for (int x = 0; x < D / 32; ++x) sm.o[warp][g][lane + 32 * x] = sm.o[warp][g][lane + 32 * x] * f + e * v[x];
            __syncwarp();
        }
    }
    join<D, float>(sm, a, b, h0, nh, parts);
}

__device__ __forceinline__ uint32_t lo_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi_pair(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// bf16: a warp takes 16 keys at a time.  Lane (g, c): query row g (and g + 8 when WIDE).
template <int D, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32) swa_step_bf16(SwaArgs a, int groups, int parts) {
    constexpr int NQ = D / 32;   // 16-byte chunks of a row per lane quad member: chunk 4 x + c
    constexpr int NV = D / 64;   // 16-byte chunks of a value row per lane g: chunk 8 x + g
    __shared__ StepSmem<D> sm;
    const int u = blockIdx.x / parts, rank = blockIdx.x % parts;
    const int grp = u % groups, hk = u / groups % a.Hkv, b = u / groups / a.Hkv;
    const int share = a.Hq / a.Hkv, nh = min(kHeads, share - grp * kHeads), h0 = hk * share + grp * kHeads;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
    const Part p = part_of(a, b, hk, rank, parts, D);
    if (rank == 0 && grp == 0) put_token<__nv_bfloat16, D>(a, p);
    // queries as A fragments: k-step 2 x + y of chunk x has pairs (words 2 y, 2 y + 1 of the chunk)
    uint32_t qf[WIDE ? 2 : 1][NQ][4];
#pragma unroll
    for (int i = 0; i < (WIDE ? 2 : 1); ++i)
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (g + 8 * i < nh)
                w = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                     ((size_t)b * a.Hq + h0 + g + 8 * i) * D + 8 * (4 * x + c));
            qf[i][x][0] = w.x;
            qf[i][x][1] = w.y;
            qf[i][x][2] = w.z;
            qf[i][x][3] = w.w;
        }
    const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(a.k_cache) + p.cache;
    const __nv_bfloat16 *vc = static_cast<const __nv_bfloat16 *>(a.v_cache) + p.cache;
    const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(a.k) + p.fresh;
    const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(a.v) + p.fresh;
    const size_t ld = (size_t)a.Hkv * D;
    // row j of the keys or values; a slot behind the part is read as its first slot and masked
    auto row = [&](const __nv_bfloat16 *cache, const __nv_bfloat16 *fresh, int j) {
        return j == p.now ? fresh : cache + (size_t)(j < p.hi ? j : p.lo) * ld;
    };
    float o[8 * NV][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, dead[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 8 * NV; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    const float sc = a.scale * 1.4426950408889634f;   // base-2 exponentials
    uint4 kr[2][NQ], vr[4][NV];
    auto load_k = [&](int j0) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            int j = j0 + 8 * t + g;
            if (j >= p.hi && p.lo == p.now) j = p.now;   // the part's first slot may be the new token's
            const __nv_bfloat16 *r = row(kc, kn, j);
#pragma unroll
            for (int x = 0; x < NQ; ++x) kr[t][x] = __ldcs(reinterpret_cast<const uint4 *>(r + 8 * (4 * x + c)));
        }
    };
    auto load_v = [&](int j0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            int j = j0 + 2 * c + (t & 1) + 8 * (t >> 1);
            if (j >= p.hi && p.lo == p.now) j = p.now;
            const __nv_bfloat16 *r = row(vc, vn, j);
#pragma unroll
            for (int x = 0; x < NV; ++x) vr[t][x] = __ldcs(reinterpret_cast<const uint4 *>(r + 8 * (8 * x + g)));
        }
    };
    int j0 = p.lo + 16 * warp;
    if (j0 < p.hi) {
        load_k(j0);
        load_v(j0);
    }
    for (; j0 < p.hi; j0 += 16 * kWarps) {
        float s[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const uint32_t a0[4] = {qf[0][x][0], WIDE ? qf[WIDE ? 1 : 0][x][0] : 0u, qf[0][x][1], WIDE ? qf[WIDE ? 1 : 0][x][1] : 0u};
                const uint32_t a1[4] = {qf[0][x][2], WIDE ? qf[WIDE ? 1 : 0][x][2] : 0u, qf[0][x][3], WIDE ? qf[WIDE ? 1 : 0][x][3] : 0u};
                mma_bf16(s[t], a0, kr[t][x].x, kr[t][x].y);
                mma_bf16(s[t], a1, kr[t][x].z, kr[t][x].w);
            }
        const bool more = j0 + 16 * kWarps < p.hi;
        if (more) load_k(j0 + 16 * kWarps);
        // s[t][0..1]: row g, keys 8 t + 2 c, + 1; s[t][2..3]: row g + 8
        uint32_t pf[4];
#pragma unroll
        for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[t][2 * i + e];
                    x = j0 + 8 * t + 2 * c + e < p.hi ? x * sc : -INFINITY;
                    mx = fmaxf(mx, x);
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m1 = fmaxf(m[i], mx), base = m1 == -INFINITY ? 0.f : m1;
            if (__any_sync(0xffffffffu, m1 != m[i])) {
                const float f = exp2f(m[i] - base);
                l[i] *= f;
#pragma unroll
                for (int t = 0; t < 8 * NV; ++t) {
                    o[t][2 * i] *= f;
                    o[t][2 * i + 1] *= f;
                }
                m[i] = m1;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float e0 = exp2f(s[t][2 * i] - base), e1 = exp2f(s[t][2 * i + 1] - base);
                l[i] += e0 + e1;
                pf[2 * t + i] = pack_bf16(e0, e1);
            }
        }
        if (!WIDE) pf[1] = pf[3] = 0u;
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const uint32_t *r0 = reinterpret_cast<const uint32_t *>(&vr[0][x]), *r1 = reinterpret_cast<const uint32_t *>(&vr[1][x]);
            const uint32_t *r2 = reinterpret_cast<const uint32_t *>(&vr[2][x]), *r3 = reinterpret_cast<const uint32_t *>(&vr[3][x]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {   // channels 8 (8 x + g) + 2 y and + 1
                if (WIDE) {
                    mma_bf16(o[8 * x + 2 * y], pf, lo_pair(r0[y], r1[y]), lo_pair(r2[y], r3[y]));
                    mma_bf16(o[8 * x + 2 * y + 1], pf, hi_pair(r0[y], r1[y]), hi_pair(r2[y], r3[y]));
                } else {   // rows 8 .. 15 are zero: their accumulators are one shared pair
                    float t0[4] = {o[8 * x + 2 * y][0], o[8 * x + 2 * y][1], dead[0], dead[1]};
                    mma_bf16(t0, pf, lo_pair(r0[y], r1[y]), lo_pair(r2[y], r3[y]));
                    float t1[4] = {o[8 * x + 2 * y + 1][0], o[8 * x + 2 * y + 1][1], dead[0], dead[1]};
                    mma_bf16(t1, pf, hi_pair(r0[y], r1[y]), hi_pair(r2[y], r3[y]));
                    o[8 * x + 2 * y][0] = t0[0];
                    o[8 * x + 2 * y][1] = t0[1];
                    o[8 * x + 2 * y + 1][0] = t1[0];
                    o[8 * x + 2 * y + 1][1] = t1[1];
                }
            }
        }
        if (more) load_v(j0 + 16 * kWarps);
    }
    // tile 8 x + t holds rows g, g + 8 of output channels 8 (8 x + col) + t, col = 2 c, 2 c + 1
#pragma unroll
    for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
#pragma unroll
        for (int x = 0; x < NV; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < 8; t += 4)
                    *reinterpret_cast<float4 *>(&sm.o[warp][g + 8 * i][8 * (8 * x + 2 * c + e) + t]) =
                        make_float4(o[8 * x + t][2 * i + e], o[8 * x + t + 1][2 * i + e], o[8 * x + t + 2][2 * i + e],
                                    o[8 * x + t + 3][2 * i + e]);
        if (c == 0) {
            sm.m[warp][g + 8 * i] = m[i] * 0.6931471805599453f;
            sm.l[warp][g + 8 * i] = l[i];
        }
    }
    join<D, __nv_bfloat16>(sm, a, b, h0, nh, parts);
}

template <class K>
cudaError_t launch_clusters(K kern, const SwaArgs &a, int groups, int parts, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)a.seq.N * a.Hkv * groups * parts));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)parts;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, groups, parts);
}

}  // namespace

cudaError_t launch_swa_fill(bool bf16, const SwaArgs &a, cudaStream_t st) {
    const long long slots = (long long)a.seq.N * (a.sinks + a.window);
    swa_fill_kernel<<<(unsigned)((slots + 7) / 8), 256, 0, st>>>(a, a.Hkv * a.d * (bf16 ? 2 : 4) / 16, slots);
    return cudaGetLastError();
}

cudaError_t launch_swa_step(bool bf16, const SwaArgs &a, cudaStream_t st) {
    const int share = a.Hq / a.Hkv, groups = (share + kHeads - 1) / kHeads;
    const long long units = (long long)a.seq.N * a.Hkv * groups;
    // a part holds at least 64 slots (a block of 16 for each warp); more parts only while SMs are
    // without one: their join costs more than it gains beside other units (window 1024, 4 key heads,
    // 64 sequences: 29 us in one part each, 37 in two, 47 in four)
    int parts = 1;
    while (parts < 8 && units * parts < 148 && (a.sinks + a.window) / (2 * parts) >= 64) parts *= 2;
    if (!bf16) return a.d == 64 ? launch_clusters(swa_step_fp32<64>, a, groups, parts, st) : launch_clusters(swa_step_fp32<128>, a, groups, parts, st);
    if (share <= 8)
        return a.d == 64 ? launch_clusters(swa_step_bf16<64, false>, a, groups, parts, st) : launch_clusters(swa_step_bf16<128, false>, a, groups, parts, st);
    return a.d == 64 ? launch_clusters(swa_step_bf16<64, true>, a, groups, parts, st) : launch_clusters(swa_step_bf16<128, true>, a, groups, parts, st);
}

}  // namespace carve
