"""Binding of the mixers of include/carve_mixers.h: the scalar-gated delta rule (carve_gdr_*) and
sliding-window attention with sink tokens (carve_swa_*).

Argument checks and marshalling only, as in the package's other calls.  Tensors are contiguous,
on one CUDA device (which need not be the current one) and launched on that device's current
stream, or on `stream`.

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

from . import CarveError, IO_BF16, IO_FP32, _check, _torch, load


class GdrDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "Hk", "Hv", "dk", "dv", "io")] + [("total_tokens", ctypes.c_int64)]


class SwaDims(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "T", "Hq", "Hkv", "d", "window", "sinks", "io")] +
                [("scale", ctypes.c_float), ("total_tokens", ctypes.c_int64)])


_t = None          # torch, imported with the first call
_handle = None     # libcarve, declared with the first call that launches


def _init():
    global _t
    if _t is None:
        _t = _torch()


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


# ---- argument checks ------------------------------------------------------------------------
# A decoding step's kernel takes a few microseconds, so a call's host side is kept as short: one
# pass of comparisons that all hold in a right call, and the messages worked out only where one
# does not (a single-token call took 21 us on the host with checks that built their messages and
# stream objects as they went).
def _io(x, what):
    if x.dtype == _t.bfloat16:
        return IO_BF16
    if x.dtype == _t.float32:
        return IO_FP32
    raise TypeError(f"{what} must be float32 or bfloat16, got {x.dtype}")


def _want(like, *specs):
    """Each (name, tensor, shape, dtype) has that shape and dtype, is contiguous and on the device of
    `like`, which must be a CUDA device; a None tensor is an argument left out."""
    dev = like.get_device()
    for name, x, shape, dtype in specs:
        if x is not None and (x.get_device() != dev or x.dtype != dtype or x.shape != shape or not x.is_contiguous()):
            _complain(like, name, x, shape, dtype)
    if dev < 0 or not like.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, got {like.device}")


def _complain(like, name, x, shape, dtype):
    if x.device != like.device:
        raise ValueError(f"{name} is on {x.device}, q (or k) on {like.device}")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rank(x, n, what):
    if x.dim() != n:
        raise ValueError(f"{what} must have {n} dimensions, got shape {tuple(x.shape)}")


def _lead(x, cu_seqlens, what):
    """(leading dimensions, B, T, rows) of a token tensor."""
    if cu_seqlens is None:
        _rank(x, 4, what)
        B, T = x.shape[:2]
        return (B, T), B, T, B * T
    _rank(x, 3, f"packed {what}")
    _rank(cu_seqlens, 1, "cu_seqlens")
    if cu_seqlens.dtype != _t.int32:
        raise TypeError(f"cu_seqlens must be torch.int32, got {cu_seqlens.dtype}")
    if cu_seqlens.device != x.device or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous tensor on the device of the tokens")
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens needs at least two offsets")
    return (x.shape[0],), cu_seqlens.numel() - 1, 0, x.shape[0]


def _heads(few, many, what):
    if few < 1 or many % few:
        raise ValueError(f"{what}: {many} heads are not a multiple of {few}")


def _addr(x):
    return None if x is None else x.data_ptr()


def _call(name, like, stream, dims, *pointers):
    """Calls libcarve with the device of `like` current, on `stream` or that device's current one."""
    dev = like.get_device()
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device != like.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {like.device}")
    else:
        handle = stream.cuda_stream
    f = getattr(_lib(), name)
    if dev == _t.cuda.current_device():
        rc = f(dims, *pointers, handle)
    else:
        with _t.cuda.device(dev):
            rc = f(dims, *pointers, handle)
    if rc:
        _check(name, rc)


def _raw_stream(dev):
    return _t._C._cuda_getCurrentRawStream(dev)


def _bytes(name, dims, packed, device):
    n = int(getattr(_lib(), name)(dims, int(packed)))
    if n == 0:
        raise CarveError(name, 1)
    return _t.empty(n, dtype=_t.uint8, device=device)


def _enough(name, buf, sized_by, dims, packed, like):
    """Checks a caller's buffer: bytes on the right device, as many as the library asks for."""
    n = int(getattr(_lib(), sized_by)(dims, int(packed)))
    if buf.device != like.device or not buf.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {like.device}")
    if buf.numel() * buf.element_size() < n:
        raise ValueError(f"{name} holds {buf.numel() * buf.element_size()} bytes, {n} are needed")


# ---- the scalar-gated delta rule ------------------------------------------------------------
def _gdr(q, k, v, g_logit, w_logit, A_dec, tau, cu_seqlens):
    _init()
    io = _io(q, "q")
    lead, B, T, rows = _lead(q, cu_seqlens, "q")
    Hk, dk = q.shape[-2:]
    _rank(v, len(lead) + 2, "v")
    Hv, dv = v.shape[-2:]
    _heads(Hk, Hv, "value heads on key heads")
    _want(q, ("q", q, lead + (Hk, dk), q.dtype), ("k", k, lead + (Hk, dk), q.dtype), ("v", v, lead + (Hv, dv), q.dtype),
          ("g_logit", g_logit, lead + (Hv,), q.dtype), ("w_logit", w_logit, lead + (Hv,), q.dtype),
          ("A_dec", A_dec, (Hv,), _t.float32), ("tau", tau, (Hv,), _t.float32))
    return GdrDims(B, T, Hk, Hv, dk, dv, io, rows)


def carve_gdr_fwd(q, k, v, g_logit, w_logit, A_dec=None, tau=None, S0=None, cu_seqlens=None,
                  save_for_bwd: bool = True, out: dict | None = None, workspace=None, stream=None) -> dict:
    """The scalar-gated delta rule over [B,T,Hk,dk] q, k and [B,T,Hv,dv] v with gates [B,T,Hv]
    (or packed rows): a = exp(-e^A_dec softplus(g_logit + tau)), w = sigmoid(w_logit),
    S_t = a S + w (v - a S k) k^T, o = S_t q.  A_dec, tau [Hv] float32 and S0 [B,Hv,dv,dk]
    float32 are optional.  Returns dict(o, S_final[, saved]); `out` may supply preallocated
    buffers under the same keys (S_final may be S0 itself)."""
    _init()
    d = _gdr(q, k, v, g_logit, w_logit, A_dec, tau, cu_seqlens)
    packed = cu_seqlens is not None
    state = (d.B, d.Hv, d.dv, d.dk)
    out = dict(out or {})
    if "o" not in out:
        out["o"] = _t.empty_like(v)
    if "S_final" not in out:
        out["S_final"] = _t.empty(state, dtype=_t.float32, device=q.device)
    _want(q, ("S0", S0, state, _t.float32), ("o", out["o"], v.shape, v.dtype),
          ("S_final", out["S_final"], state, _t.float32))
    if save_for_bwd:
        if out.get("saved") is None:
            out["saved"] = _bytes("carve_gdr_saved_bytes", d, packed, q.device)
        _enough("saved", out["saved"], "carve_gdr_saved_bytes", d, packed, q)
    elif workspace is None:
        workspace = _bytes("carve_gdr_fwd_workspace_bytes", d, packed, q.device)
    if workspace is not None:
        _enough("workspace", workspace, "carve_gdr_fwd_workspace_bytes", d, packed, q)
    _call("carve_gdr_fwd", q, stream, d, _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(g_logit), _addr(w_logit),
          _addr(A_dec), _addr(tau), _addr(S0), _addr(out["o"]), _addr(out["S_final"]),
          _addr(out["saved"] if save_for_bwd else None), _addr(workspace))
    return out


def carve_gdr_bwd(q, k, v, g_logit, w_logit, saved, dO, A_dec=None, tau=None, dS_final=None, cu_seqlens=None,
                  want_dS0: bool = True, out: dict | None = None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dO o) + sum(dS_final S_final): dict(dq, dk, dv, dg_logit, dw_logit), plus
    dS0 and, when the forward had A_dec or tau, dA_dec and dtau ([Hv], summed over all tokens)."""
    _init()
    d = _gdr(q, k, v, g_logit, w_logit, A_dec, tau, cu_seqlens)
    packed = cu_seqlens is not None
    state = (d.B, d.Hv, d.dv, d.dk)
    want = dict(dq=(q.shape, q.dtype), dk=(k.shape, q.dtype), dv=(v.shape, q.dtype),
                dg_logit=(g_logit.shape, q.dtype), dw_logit=(w_logit.shape, q.dtype))
    if want_dS0:
        want["dS0"] = (state, _t.float32)
    for key, x in (("dA_dec", A_dec), ("dtau", tau)):
        if x is not None:
            want[key] = ((d.Hv,), _t.float32)
    out = dict(out or {})
    for key, (shape, dtype) in want.items():
        if key not in out:
            out[key] = _t.empty(shape, dtype=dtype, device=q.device)
    _want(q, ("dO", dO, v.shape, v.dtype), ("dS_final", dS_final, state, _t.float32),
          *((key, out[key], *w) for key, w in want.items()))
    _enough("saved", saved, "carve_gdr_saved_bytes", d, packed, q)
    if workspace is None:
        workspace = _bytes("carve_gdr_bwd_workspace_bytes", d, packed, q.device)
    _enough("workspace", workspace, "carve_gdr_bwd_workspace_bytes", d, packed, q)
    _call("carve_gdr_bwd", q, stream, d, _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(g_logit), _addr(w_logit),
          _addr(A_dec), _addr(tau), _addr(saved), _addr(dO), _addr(dS_final), _addr(out["dq"]), _addr(out["dk"]),
          _addr(out["dv"]), _addr(out["dg_logit"]), _addr(out["dw_logit"]),
          _addr(out["dA_dec"] if A_dec is not None else None), _addr(out["dtau"] if tau is not None else None),
          _addr(out["dS0"] if want_dS0 else None), _addr(workspace))
    return out


def carve_gdr_step(q, k, v, g_logit, w_logit, S, A_dec=None, tau=None, o=None, stream=None):
    """One token of every batch element: q, k [B,Hk,dk], v [B,Hv,dv], gates [B,Hv]; S
    [B,Hv,dv,dk] float32 is updated in place.  Returns o [B,Hv,dv]."""
    _init()
    io = _io(q, "q")
    _rank(q, 3, "q")
    _rank(v, 3, "v")
    B, Hk, dk = q.shape
    Hv, dv = v.shape[-2:]
    _heads(Hk, Hv, "value heads on key heads")
    if o is None:
        o = _t.empty_like(v)
    dt, gates = q.dtype, (B, Hv)
    _want(q, ("q", q, q.shape, dt), ("k", k, q.shape, dt), ("v", v, (B, Hv, dv), dt), ("g_logit", g_logit, gates, dt),
          ("w_logit", w_logit, gates, dt), ("S", S, (B, Hv, dv, dk), _t.float32), ("A_dec", A_dec, (Hv,), _t.float32),
          ("tau", tau, (Hv,), _t.float32), ("o", o, v.shape, dt))
    _call("carve_gdr_step", q, stream, GdrDims(B, 1, Hk, Hv, dk, dv, io, 0), _addr(q), _addr(k), _addr(v), _addr(g_logit),
          _addr(w_logit), _addr(A_dec), _addr(tau), _addr(S), _addr(o))
    return o


# ---- sliding-window attention with sink tokens ----------------------------------------------
def _window(window, sinks):
    window, sinks = int(window), int(sinks)
    if not 1 <= window < 1 << 31 or not 0 <= sinks < 1 << 31:
        raise ValueError(f"window must be 1 .. 2^31 - 1 and sinks 0 .. 2^31 - 1, got {window} and {sinks}")
    return window, sinks


def _swa(q, k, v, window, sinks, scale, cu_seqlens):
    window, sinks = _window(window, sinks)
    io = _io(q, "q")
    lead, B, T, rows = _lead(q, cu_seqlens, "q")
    Hq, D = q.shape[-2:]
    _rank(k, len(lead) + 2, "k")
    Hkv = k.shape[-2]
    _heads(Hkv, Hq, "query heads on key heads")
    kv = lead + (Hkv, D)
    _want(q, ("q", q, lead + (Hq, D), q.dtype), ("k", k, kv, q.dtype), ("v", v, kv, q.dtype))
    return SwaDims(B, T, Hq, Hkv, D, window, sinks, io, D ** -0.5 if scale is None else float(scale), rows)


def carve_swa_fwd(q, k, v, window: int, sinks: int = 0, scale=None, cu_seqlens=None, want_lse: bool = True,
                  out: dict | None = None, stream=None) -> dict:
    """Attention of [B,T,Hq,d] queries to [B,T,Hkv,d] keys and values (or packed rows): query i
    sees key j <= i where i - j < window or j < sinks.  scale defaults to d^-0.5.  Returns
    dict(o[, lse]), lse [rows, Hq] float32 for carve_swa_bwd."""
    _init()
    d = _swa(q, k, v, window, sinks, scale, cu_seqlens)
    out = dict(out or {})
    if "o" not in out:
        out["o"] = _t.empty_like(q)
    if want_lse and out.get("lse") is None:
        out["lse"] = _t.empty(q.shape[:-1], dtype=_t.float32, device=q.device)
    _want(q, ("o", out["o"], q.shape, q.dtype), ("lse", out.get("lse"), q.shape[:-1], _t.float32))
    _call("carve_swa_fwd", q, stream, d, _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(out["o"]),
          _addr(out["lse"] if want_lse else None))
    return out


def carve_swa_bwd(q, k, v, o, lse, dO, window: int, sinks: int = 0, scale=None, cu_seqlens=None,
                  out: dict | None = None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dO o): dict(dq, dk, dv), from the forward's inputs, o and lse."""
    _init()
    d = _swa(q, k, v, window, sinks, scale, cu_seqlens)
    packed = cu_seqlens is not None
    out = dict(out or {})
    for key, x in (("dq", q), ("dk", k), ("dv", v)):
        if key not in out:
            out[key] = _t.empty_like(x)
    _want(q, ("o", o, q.shape, q.dtype), ("dO", dO, q.shape, q.dtype), ("lse", lse, q.shape[:-1], _t.float32),
          ("dq", out["dq"], q.shape, q.dtype), ("dk", out["dk"], k.shape, q.dtype), ("dv", out["dv"], k.shape, q.dtype))
    if workspace is None:
        workspace = _bytes("carve_swa_bwd_workspace_bytes", d, packed, q.device)
    _enough("workspace", workspace, "carve_swa_bwd_workspace_bytes", d, packed, q)
    _call("carve_swa_bwd", q, stream, d, _addr(cu_seqlens), _addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), _addr(dO),
          _addr(out["dq"]), _addr(out["dk"]), _addr(out["dv"]), _addr(workspace))
    return out


def _cache(like, k_cache, v_cache, B, Hkv, D, window, sinks):
    shape = (B, sinks + window, Hkv, D)
    return ("k_cache", k_cache, shape, like.dtype), ("v_cache", v_cache, shape, like.dtype)


def carve_swa_fill(k, v, k_cache, v_cache, window: int, sinks: int = 0, cu_seqlens=None, stream=None) -> None:
    """Writes the tokens of a prompt that stay visible, the first `sinks` and the last `window` of
    each sequence, into the caches [B, sinks + window, Hkv, d]: token t in slot t (t < sinks) or
    sinks + (t - sinks) mod window.  Other slots are left as they were."""
    _init()
    d = _swa(k, k, v, window, sinks, 1.0, cu_seqlens)
    _want(k, *_cache(k, k_cache, v_cache, d.B, d.Hkv, d.d, d.window, d.sinks))
    _call("carve_swa_fill", k, stream, d, _addr(cu_seqlens), _addr(k), _addr(v), _addr(k_cache), _addr(v_cache))


def carve_swa_step(q, k, v, k_cache, v_cache, pos, window: int, sinks: int = 0, scale=None, o=None, stream=None):
    """One token of every batch element: q [B,Hq,d], k, v [B,Hkv,d]; pos [B] int64, the tokens that
    each sequence already has (the caller advances it).  Puts k and v into the caches and returns
    o [B,Hq,d], the attention to every visible token, this one included."""
    _init()
    window, sinks = _window(window, sinks)
    io = _io(q, "q")
    _rank(q, 3, "q")
    _rank(k, 3, "k")
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    _heads(Hkv, Hq, "query heads on key heads")
    if o is None:
        o = _t.empty_like(q)
    _want(q, ("q", q, q.shape, q.dtype), ("k", k, (B, Hkv, D), q.dtype), ("v", v, (B, Hkv, D), q.dtype),
          ("pos", pos, (B,), _t.int64), ("o", o, q.shape, q.dtype), *_cache(q, k_cache, v_cache, B, Hkv, D, window, sinks))
    d = SwaDims(B, 1, Hq, Hkv, D, window, sinks, io, D ** -0.5 if scale is None else float(scale), 0)
    _call("carve_swa_step", q, stream, d, _addr(q), _addr(k), _addr(v), _addr(k_cache), _addr(v_cache), _addr(pos), _addr(o))
    return o
