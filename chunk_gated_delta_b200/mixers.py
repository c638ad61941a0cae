"""Binding of the mixers of include/carve_mixers.h: the scalar-gated delta rule (carve_gdr_*) and
sliding-window attention with sink tokens (carve_swa_*).

Argument checks and marshalling only, as in the package's other calls; here they are in C++
(csrc/carve_bind.cpp, _carve_bind.so), since a decoding step's kernel is shorter than they were in
Python.  Tensors are contiguous, on one CUDA device (which need not be the current one) and
launched on that device's current stream, or on `stream`.  What a call allocates (results, scratch)
belongs to the stream that it is launched on, as within `torch.cuda.stream(stream)`; inputs and
buffers that the caller brings from another stream are the caller's to order.  What does not fit
raises TypeError (a dtype) or ValueError; what the library refuses, CarveError.

    out  = carve.carve_gdr_fwd(q, k, v, g_logit, w_logit)
    g    = carve.carve_gdr_bwd(q, k, v, g_logit, w_logit, out["saved"], dO)
    o    = carve.carve_gdr_step(q1, k1, v1, g1, w1, S)                         # S in place
    out  = carve.carve_swa_fwd(q, k, v, window=512, sinks=4)
    g    = carve.carve_swa_bwd(q, k, v, out["o"], out["lse"], dO, window=512, sinks=4)
    carve.carve_swa_fill(k, v, k_cache, v_cache, window=512, sinks=4)          # after a prompt
    o    = carve.carve_swa_step(q1, k1, v1, k_cache, v_cache, pos, window=512, sinks=4)

Packed sequences: token tensors [rows, heads, channels] with cu_seqlens, int32 [N + 1] on the
device; sequence n owns rows cu[n] .. cu[n + 1].
"""
from __future__ import annotations

import ctypes

from . import _torch, load


class GdrDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "Hk", "Hv", "dk", "dv", "io")] + [("total_tokens", ctypes.c_int64)]


class SwaDims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "T", "Hq", "Hkv", "d", "window", "sinks", "io")] +
                [("scale", ctypes.c_float), ("total_tokens", ctypes.c_int64)])


_handle = None     # libcarve with this file's entry points declared (structures and sizes, for C-level use)
_ext = None        # the binding, imported with the first call


def _bind():
    global _ext
    _torch()   # its libraries, which the binding links
    load()
    try:
        from . import _carve_bind
    except ImportError as e:
        raise ImportError(f"_carve_bind.so does not load ({e}): build it with `python -m chunk_gated_delta_b200.build`") from e
    _ext = _carve_bind
    return _ext


def _lib():
    global _handle
    if _handle is None:
        lib = load()
        P, G, W = ctypes.c_void_p, ctypes.POINTER(GdrDims), ctypes.POINTER(SwaDims)
        for name, dims in (("gdr_fwd_workspace", G), ("gdr_saved", G), ("gdr_bwd_workspace", G), ("swa_bwd_workspace", W)):
            f = getattr(lib, f"carve_{name}_bytes")
            f.argtypes, f.restype = [dims, ctypes.c_int], ctypes.c_size_t
        for name, dims, n in (("gdr_fwd", G, 14), ("gdr_bwd", G, 21), ("gdr_step", G, 10), ("swa_fwd", W, 7),
                              ("swa_bwd", W, 12), ("swa_fill", W, 6), ("swa_step", W, 8)):
            f = getattr(lib, f"carve_{name}")
            f.argtypes, f.restype = [dims] + [P] * n, ctypes.c_int
        _handle = lib
    return _handle


# ---- the scalar-gated delta rule ------------------------------------------------------------
def carve_gdr_fwd(q, k, v, g_logit, w_logit, A_dec=None, tau=None, S0=None, cu_seqlens=None,
                  save_for_bwd: bool = True, out: dict | None = None, workspace=None, stream=None) -> dict:
    """The scalar-gated delta rule over [B,T,Hk,dk] q, k and [B,T,Hv,dv] v with gates [B,T,Hv] of the
    same dtype (or packed rows): a = exp(-e^A_dec softplus(g_logit + tau)), w = sigmoid(w_logit),
    S_t = a S + w (v - a S k) k^T, o = S_t q.  A_dec, tau [Hv] float32 and S0 [B,Hv,dv,dk]
    float32 are optional.  Returns dict(o, S_final[, saved]); `out` may supply preallocated
    buffers under the same keys (S_final may be S0 itself)."""
    return (_ext or _bind()).gdr_fwd(q, k, v, g_logit, w_logit, A_dec, tau, S0, cu_seqlens, bool(save_for_bwd), out, workspace, stream)


def carve_gdr_bwd(q, k, v, g_logit, w_logit, saved, dO, A_dec=None, tau=None, dS_final=None, cu_seqlens=None,
                  want_dS0: bool = True, out: dict | None = None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dO o) + sum(dS_final S_final): dict(dq, dk, dv, dg_logit, dw_logit), plus
    dS0 and, when the forward had A_dec or tau, dA_dec and dtau ([Hv], summed over all tokens)."""
    return (_ext or _bind()).gdr_bwd(q, k, v, g_logit, w_logit, saved, dO, A_dec, tau, dS_final, cu_seqlens, bool(want_dS0), out,
                                     workspace, stream)


def carve_gdr_step(q, k, v, g_logit, w_logit, S, A_dec=None, tau=None, o=None, stream=None):
    """One token of every batch element: q, k [B,Hk,dk], v [B,Hv,dv], gates [B,Hv]; S
    [B,Hv,dv,dk] float32 is updated in place.  Returns o [B,Hv,dv]."""
    return (_ext or _bind()).gdr_step(q, k, v, g_logit, w_logit, S, A_dec, tau, o, stream)


# ---- sliding-window attention with sink tokens ----------------------------------------------
def carve_swa_fwd(q, k, v, window: int, sinks: int = 0, scale=None, cu_seqlens=None, want_lse: bool = True,
                  out: dict | None = None, stream=None) -> dict:
    """Attention of [B,T,Hq,d] queries to [B,T,Hkv,d] keys and values (or packed rows): query i
    sees key j <= i where i - j < window or j < sinks.  scale defaults to d^-0.5.  Returns
    dict(o[, lse]), lse [rows, Hq] float32 for carve_swa_bwd."""
    return (_ext or _bind()).swa_fwd(q, k, v, int(window), int(sinks), scale, cu_seqlens, bool(want_lse), out, stream)


def carve_swa_bwd(q, k, v, o, lse, dO, window: int, sinks: int = 0, scale=None, cu_seqlens=None,
                  out: dict | None = None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dO o): dict(dq, dk, dv), from the forward's inputs, o and lse."""
    return (_ext or _bind()).swa_bwd(q, k, v, o, lse, dO, int(window), int(sinks), scale, cu_seqlens, out, workspace, stream)


def carve_swa_fill(k, v, k_cache, v_cache, window: int, sinks: int = 0, cu_seqlens=None, stream=None) -> None:
    """Writes the tokens of a prompt that stay visible, the first `sinks` and the last `window` of
    each sequence, into the caches [B, sinks + window, Hkv, d]: token t in slot t (t < sinks) or
    sinks + (t - sinks) mod window.  Other slots are left as they were."""
    (_ext or _bind()).swa_fill(k, v, k_cache, v_cache, int(window), int(sinks), cu_seqlens, stream)


def carve_swa_step(q, k, v, k_cache, v_cache, pos, window: int, sinks: int = 0, scale=None, o=None, stream=None):
    """One token of every batch element: q [B,Hq,d], k, v [B,Hkv,d]; pos [B] int64, the tokens that
    each sequence already has (the caller advances it).  Puts k and v into the caches and returns
    o [B,Hq,d], the attention to every visible token, this one included."""
    return (_ext or _bind()).swa_step(q, k, v, k_cache, v_cache, pos, int(window), int(sinks), scale, o, stream)
