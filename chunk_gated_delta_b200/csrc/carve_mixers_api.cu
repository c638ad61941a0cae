// Host side of the C ABI declared in include/carve_mixers.h: argument validation, buffer sizing
// and kernel dispatch.  Nothing here allocates, frees or synchronises.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/carve_mixers.h"
#include "carve_mixers.cuh"

namespace carve {

// Whether this process has launched kernels of a mixer: carve_check reads their status words only then
// (each word is a synchronous copy of 13 us).  Never taken back: a captured graph may launch them again.
std::atomic<bool> g_gdr_used{false}, g_swa_used{false};

int gdr_take_status() {
    if (!g_gdr_used.load(std::memory_order_relaxed)) return 0;
    return (gdr_tc_fwd_take_timeout() | gdr_tc_bwd_take_timeout() ? kTimedOut : 0) |
           (gdr_take_bad_seqlens() | gdr_tc_fwd_take_bad_seqlens() | gdr_tc_bwd_take_bad_seqlens() ? kBadOffsets : 0);
}
int swa_take_status() {
    if (!g_swa_used.load(std::memory_order_relaxed)) return 0;
    return swa_fwd_take_status() | swa_bwd_take_status() | (swa_take_bad_seqlens() | swa_fill_take_bad_seqlens() ? kBadOffsets : 0);
}

}  // namespace carve

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// a required pointer (of a tensor that may be empty: `rows` == 0), and an optional one
bool ok_ptr(const void *p, long long rows = 1) { return (p != nullptr || rows == 0) && aligned16(p); }
bool ok_opt(const void *p) { return aligned16(p); }
// tensors without a channel axis (gates, offsets, positions, log-sum-exps): read by element, so
// aligned to `size`, their element
bool ok_elem(const void *p, size_t size, long long rows = 1) {
    return (p != nullptr || rows == 0) && reinterpret_cast<uintptr_t>(p) % size == 0;
}
bool ok_elem_opt(const void *p, size_t size = 4) { return reinterpret_cast<uintptr_t>(p) % size == 0; }
size_t io_bytes(int io) { return io == CARVE_IO_BF16 ? 2 : 4; }

carve_status status(cudaError_t e) { return e == cudaSuccess ? CARVE_OK : CARVE_ERR_CUDA; }

// checks of heads and sequences shared by both mixers; `heads` the larger head count, `width` the
// widest row of channels
carve_status check_common(int B, int T, int64_t total, int io, int small, int heads, bool seq, bool packed) {
    if (B < 1 || small < 1 || heads < 1) return CARVE_ERR_INVALID_ARG;
    if (io != CARVE_IO_FP32 && io != CARVE_IO_BF16) return CARVE_ERR_INVALID_ARG;
    if (heads % small != 0) return CARVE_ERR_INVALID_ARG;
    if (seq && !packed && T < 0) return CARVE_ERR_INVALID_ARG;
    if (seq && packed && total < 0) return CARVE_ERR_INVALID_ARG;
    const long long rows = !seq ? B : packed ? (long long)total : (long long)B * T;
    // token rows index as int; grids are (rows or sequences) x heads, one-dimensional
    if (rows > 0x7fffffffLL - 128) return CARVE_ERR_UNSUPPORTED;
    if ((rows / 32 + 2LL * B) * heads > (1LL << 28)) return CARVE_ERR_UNSUPPORTED;
    return CARVE_OK;
}

carve_status check(const carve_gdr_dims *d, bool seq, bool packed) {
    if (!d) return CARVE_ERR_INVALID_ARG;
    const carve_status st = check_common(d->B, d->T, d->total_tokens, d->io, d->Hk, d->Hv, seq, packed);
    if (st != CARVE_OK) return st;
    if (d->dk < 1 || d->dv < 1) return CARVE_ERR_INVALID_ARG;
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128)) return CARVE_ERR_UNSUPPORTED;
    return CARVE_OK;
}

carve_status check(const carve_swa_dims *d, bool seq, bool packed) {
    if (!d) return CARVE_ERR_INVALID_ARG;
    const carve_status st = check_common(d->B, d->T, d->total_tokens, d->io, d->Hkv, d->Hq, seq, packed);
    if (st != CARVE_OK) return st;
    if (d->d < 1 || d->window < 1 || d->sinks < 0 || !std::isfinite(d->scale)) return CARVE_ERR_INVALID_ARG;
    if (d->d != 64 && d->d != 128) return CARVE_ERR_UNSUPPORTED;
    return CARVE_OK;
}
// the cache's slots, and a launch over them
carve_status check_cache(const carve_swa_dims *d) {
    const long long slots = (long long)d->sinks + d->window;
    return slots > 0x7fffffffLL || slots * d->B > (1LL << 33) ? CARVE_ERR_UNSUPPORTED : CARVE_OK;
}

template <class D>
carve::Seqs seqs(const D *d, const int32_t *cu, bool packed) {
    return carve::Seqs{cu, packed ? (long long)d->total_tokens : 0, d->B, packed ? 0 : d->T};
}
template <class D>
long long rows_of(const D *d, bool packed) {
    return packed ? (long long)d->total_tokens : (long long)d->B * d->T;
}

carve::GdrSizes sizes(const carve_gdr_dims *d, bool packed) {
    static const int32_t dummy = 0;   // n_tiles asks only whether the call is packed
    const carve::Seqs s = seqs(d, packed ? &dummy : nullptr, packed);
    return d->io == CARVE_IO_BF16 ? carve::gdr_tc_sizes(s, d->Hv, d->dk, d->dv) : carve::gdr_simt_sizes(s, d->Hv, d->dk, d->dv);
}
size_t up(size_t n) { return (n + 255) / 256 * 256; }

carve::SwaArgs swa_args(const carve_swa_dims *d, const int32_t *cu) {
    carve::SwaArgs a{};
    a.seq = seqs(d, cu, cu != nullptr);
    a.Hq = d->Hq; a.Hkv = d->Hkv; a.d = d->d; a.window = d->window; a.sinks = d->sinks; a.scale = d->scale;
    return a;
}

// a call without rows: packed offsets are looked at all the same
carve_status no_rows(const carve::Seqs &s, cudaStream_t st) { return s.cu ? status(carve::launch_swa_check(s, st)) : CARVE_OK; }

// the backward's scratch: two floats a row and head (the CUDA-core path uses one), and the partial
// dk, dv where the keys' pass is split
int swa_parts(const carve_swa_dims *d, const carve::SwaArgs &a) { return d->io == CARVE_IO_BF16 ? carve::swa_bwd_parts(a) : 1; }
size_t swa_table_bytes(const carve_swa_dims *d, bool packed) { return up(2 * sizeof(float) * (size_t)rows_of(d, packed) * d->Hq) + 1024; }
size_t swa_partial_bytes(const carve_swa_dims *d, bool packed, int parts) {
    return parts > 1 ? up(2 * sizeof(float) * (size_t)parts * rows_of(d, packed) * d->Hkv * d->d) : 0;
}

}  // namespace

extern "C" {

size_t carve_gdr_fwd_workspace_bytes(const carve_gdr_dims *d, int packed) {
    if (check(d, true, packed != 0) != CARVE_OK) return 0;
    return up(sizes(d, packed != 0).prep) + 256;
}

size_t carve_gdr_saved_bytes(const carve_gdr_dims *d, int packed) {
    if (check(d, true, packed != 0) != CARVE_OK) return 0;
    const carve::GdrSizes s = sizes(d, packed != 0);
    return up(s.prep) + up(s.saved) + 256;
}

size_t carve_gdr_bwd_workspace_bytes(const carve_gdr_dims *d, int packed) {
    if (check(d, true, packed != 0) != CARVE_OK) return 0;
    return up(sizes(d, packed != 0).bwd) + 256;
}

carve_status carve_gdr_fwd(const carve_gdr_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, const void *g_logit, const void *w_logit,
                           const float *A_dec, const float *tau, const float *S0, void *o,
                           float *S_final, void *saved, void *workspace, void *stream) {
    const bool packed = cu_seqlens != nullptr;
    const carve_status st = check(d, true, packed);
    if (st != CARVE_OK) return st;
    const long long rows = rows_of(d, packed);
    if (!ok_elem_opt(cu_seqlens) || !ok_ptr(q, rows) || !ok_ptr(k, rows) || !ok_ptr(v, rows) ||
        !ok_elem(g_logit, io_bytes(d->io), rows) || !ok_elem(w_logit, io_bytes(d->io), rows) || !ok_ptr(o, rows) ||
        !ok_elem_opt(A_dec) || !ok_elem_opt(tau) ||
        !ok_opt(S0) || !ok_opt(S_final) || !ok_opt(saved) || !ok_opt(workspace) || (!saved && !workspace))
        return CARVE_ERR_INVALID_ARG;
    carve::g_gdr_used.store(true, std::memory_order_relaxed);
    carve::GdrArgs a{};
    a.seq = seqs(d, cu_seqlens, packed);
    a.Hk = d->Hk; a.Hv = d->Hv;
    a.q = q; a.k = k; a.v = v; a.g_logit = g_logit; a.w_logit = w_logit;
    a.A_dec = A_dec; a.tau = tau; a.S0 = S0; a.o = o; a.S_final = S_final;
    a.prep = static_cast<char *>(saved ? saved : workspace);
    if (saved) a.saved = a.prep + up(sizes(d, packed).prep);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return status(d->io == CARVE_IO_BF16 ? carve::launch_gdr_fwd_tc(d->dk, d->dv, a, saved != nullptr, cs)
                                         : carve::launch_gdr_fwd_simt(d->dk, d->dv, a, saved != nullptr, cs));
}

carve_status carve_gdr_bwd(const carve_gdr_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, const void *g_logit, const void *w_logit,
                           const float *A_dec, const float *tau, const void *saved, const void *dO,
                           const float *dS_final, void *dq, void *dk, void *dv, void *dg_logit,
                           void *dw_logit, float *dA_dec, float *dtau, float *dS0, void *workspace,
                           void *stream) {
    const bool packed = cu_seqlens != nullptr;
    const carve_status st = check(d, true, packed);
    if (st != CARVE_OK) return st;
    const long long rows = rows_of(d, packed);
    if (!ok_elem_opt(cu_seqlens) || !ok_ptr(q, rows) || !ok_ptr(k, rows) || !ok_ptr(v, rows) ||
        !ok_elem(g_logit, io_bytes(d->io), rows) || !ok_elem(w_logit, io_bytes(d->io), rows) || !ok_ptr(saved) || !ok_ptr(dO, rows) ||
        !ok_ptr(dq, rows) || !ok_ptr(dk, rows) || !ok_ptr(dv, rows) || !ok_elem(dg_logit, io_bytes(d->io), rows) ||
        !ok_elem(dw_logit, io_bytes(d->io), rows) || !ok_ptr(workspace) || !ok_opt(dS_final) || !ok_opt(dS0) || !ok_elem_opt(A_dec) ||
        !ok_elem_opt(tau) || !ok_elem_opt(dA_dec) || !ok_elem_opt(dtau) || (A_dec == nullptr) != (dA_dec == nullptr) ||
        (tau == nullptr) != (dtau == nullptr))
        return CARVE_ERR_INVALID_ARG;
    carve::g_gdr_used.store(true, std::memory_order_relaxed);
    carve::GdrArgs a{};
    a.seq = seqs(d, cu_seqlens, packed);
    a.Hk = d->Hk; a.Hv = d->Hv;
    a.q = q; a.k = k; a.v = v; a.g_logit = g_logit; a.w_logit = w_logit; a.A_dec = A_dec; a.tau = tau;
    a.dO = dO; a.dS_final = dS_final; a.dq = dq; a.dk = dk; a.dv = dv; a.dg_logit = dg_logit;
    a.dw_logit = dw_logit; a.dA_dec = dA_dec; a.dtau = dtau; a.dS0 = dS0;
    a.prep = static_cast<char *>(const_cast<void *>(saved));
    a.saved = a.prep + up(sizes(d, packed).prep);
    a.ws = static_cast<char *>(workspace);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return status(d->io == CARVE_IO_BF16 ? carve::launch_gdr_bwd_tc(d->dk, d->dv, a, cs)
                                         : carve::launch_gdr_bwd_simt(d->dk, d->dv, a, cs));
}

carve_status carve_gdr_step(const carve_gdr_dims *d, const void *q, const void *k, const void *v,
                            const void *g_logit, const void *w_logit, const float *A_dec,
                            const float *tau, float *S, void *o, void *stream) {
    const carve_status st = check(d, false, false);
    if (st != CARVE_OK) return st;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_elem(g_logit, io_bytes(d->io)) || !ok_elem(w_logit, io_bytes(d->io)) || !ok_elem_opt(A_dec) ||
        !ok_elem_opt(tau) || !ok_ptr(S) || !ok_ptr(o))
        return CARVE_ERR_INVALID_ARG;
    carve::GdrArgs a{};
    a.seq = carve::Seqs{nullptr, 0, d->B, 1};
    a.Hk = d->Hk; a.Hv = d->Hv;
    a.q = q; a.k = k; a.v = v; a.g_logit = g_logit; a.w_logit = w_logit; a.A_dec = A_dec; a.tau = tau;
    a.o = o; a.S_final = S;
    return status(carve::launch_gdr_step(d->dk, d->dv, d->io == CARVE_IO_BF16, a, static_cast<cudaStream_t>(stream)));
}

carve_status carve_swa_fwd(const carve_swa_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, void *o, float *lse, void *stream) {
    const bool packed = cu_seqlens != nullptr;
    const carve_status st = check(d, true, packed);
    if (st != CARVE_OK) return st;
    const long long rows = rows_of(d, packed);
    if (!ok_elem_opt(cu_seqlens) || !ok_ptr(q, rows) || !ok_ptr(k, rows) || !ok_ptr(v, rows) || !ok_ptr(o, rows) ||
        !ok_elem_opt(lse))
        return CARVE_ERR_INVALID_ARG;
    carve::g_swa_used.store(true, std::memory_order_relaxed);
    carve::SwaArgs a = swa_args(d, cu_seqlens);
    a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (rows == 0) return no_rows(a.seq, cs);
    return status(d->io == CARVE_IO_BF16 ? carve::launch_swa_fwd_tc(a, cs) : carve::launch_swa_fwd_simt(a, cs));
}

size_t carve_swa_bwd_workspace_bytes(const carve_swa_dims *d, int packed) {
    if (check(d, true, packed != 0) != CARVE_OK) return 0;
    static const int32_t dummy = 0;   // only whether the call is packed counts
    const carve::SwaArgs a = swa_args(d, packed ? &dummy : nullptr);
    return swa_table_bytes(d, packed != 0) + swa_partial_bytes(d, packed != 0, swa_parts(d, a)) + 256;
}

carve_status carve_swa_bwd(const carve_swa_dims *d, const int32_t *cu_seqlens, const void *q,
                           const void *k, const void *v, const void *o, const float *lse,
                           const void *dO, void *dq, void *dk, void *dv, void *workspace,
                           void *stream) {
    const bool packed = cu_seqlens != nullptr;
    const carve_status st = check(d, true, packed);
    if (st != CARVE_OK) return st;
    const long long rows = rows_of(d, packed);
    if (!ok_elem_opt(cu_seqlens) || !ok_ptr(q, rows) || !ok_ptr(k, rows) || !ok_ptr(v, rows) || !ok_ptr(o, rows) ||
        !ok_elem(lse, 4, rows) || !ok_ptr(dO, rows) || !ok_ptr(dq, rows) || !ok_ptr(dk, rows) || !ok_ptr(dv, rows) ||
        !ok_ptr(workspace))
        return CARVE_ERR_INVALID_ARG;
    carve::g_swa_used.store(true, std::memory_order_relaxed);
    carve::SwaArgs a = swa_args(d, cu_seqlens);
    if (rows == 0) return no_rows(a.seq, static_cast<cudaStream_t>(stream));
    a.q = q; a.k = k; a.v = v; a.o = const_cast<void *>(o); a.lse = const_cast<float *>(lse);
    a.dO = dO; a.dq = dq; a.dk = dk; a.dv = dv; a.delta = static_cast<float *>(workspace);
    a.parts = swa_parts(d, a);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + swa_table_bytes(d, packed));
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    return status(d->io == CARVE_IO_BF16 ? carve::launch_swa_bwd_tc(a, cs) : carve::launch_swa_bwd_simt(a, cs));
}

carve_status carve_swa_fill(const carve_swa_dims *d, const int32_t *cu_seqlens, const void *k,
                            const void *v, void *k_cache, void *v_cache, void *stream) {
    const bool packed = cu_seqlens != nullptr;
    carve_status st = check(d, true, packed);
    if (st == CARVE_OK) st = check_cache(d);
    if (st != CARVE_OK) return st;
    const long long rows = rows_of(d, packed);
    if (!ok_elem_opt(cu_seqlens) || !ok_ptr(k, rows) || !ok_ptr(v, rows) || !ok_ptr(k_cache) || !ok_ptr(v_cache))
        return CARVE_ERR_INVALID_ARG;
    carve::g_swa_used.store(true, std::memory_order_relaxed);
    carve::SwaArgs a = swa_args(d, cu_seqlens);
    if (rows == 0) return no_rows(a.seq, static_cast<cudaStream_t>(stream));
    a.k = k; a.v = v; a.k_cache = k_cache; a.v_cache = v_cache;
    return status(carve::launch_swa_fill(d->io == CARVE_IO_BF16, a, static_cast<cudaStream_t>(stream)));
}

carve_status carve_swa_step(const carve_swa_dims *d, const void *q, const void *k, const void *v,
                            void *k_cache, void *v_cache, const int64_t *pos, void *o, void *stream) {
    carve_status st = check(d, false, false);
    if (st == CARVE_OK) st = check_cache(d);
    if (st != CARVE_OK) return st;
    if (!ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(k_cache) || !ok_ptr(v_cache) || !ok_elem(pos, 8) || !ok_ptr(o))
        return CARVE_ERR_INVALID_ARG;
    carve::SwaArgs a = swa_args(d, nullptr);
    a.q = q; a.k = k; a.v = v; a.k_cache = k_cache; a.v_cache = v_cache; a.o = o;
    a.pos = reinterpret_cast<const long long *>(pos);
    return status(carve::launch_swa_step(d->io == CARVE_IO_BF16, a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
