"""The mixers of include/carve_mixers.h on the GPU against their plain fp64 references.

Tolerances count roundings.  u is half a step of the tensors' type relative to the value (bf16
2^-8, fp32 2^-24).

Delta rule, relative L2: fp32, 1e-5 (sums of a few hundred terms at 2^-24 each).  bf16 outputs and
gradients: the result's own rounding and one for each operand that is rounded to bf16 on the way
to it (o: start state, A, U; dq: start state, P1; dv: dU and Tm^T; dk: start state, end gradient
state, P1, P2, U, dY; gates: as dk), at most u each: 8 u = 3.2e-2 for dk and the gates, 4 u for
the others.  States: every factor is carried in two bf16 terms, 2^-16 each: 2e-5.

Window, elementwise: |error| <= c u m + the fp32 term, m the sum of the absolute values of the
result's terms (mixer_reference.window_masses).  Roundings: o and dv: p and the result, c = 2; dq,
dk: o within delta, ds, the result, c = 3.  fp32 term: sums of n terms and exponentials of scores
that are sums of d terms: (n + 4 d) 2^-24 m.
"""
import numpy as np
import pytest
import torch

import chunk_gated_delta_b200 as carve
from tests import mixer_reference as R

pytestmark = pytest.mark.gpu

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.bfloat16]
ids = {torch.float32: "fp32", torch.bfloat16: "bf16"}.get


@pytest.fixture(autouse=True)
def device_status(cuda_device):
    yield
    assert carve.carve_check() == 0


def rel(x, ref):
    d = x.double().cpu() - ref
    n = ref.norm().item()
    return d.norm().item() / n if n else d.norm().item()


def delta_inputs(T, Hk, Hv, dk, dv, dt, seed, strong=False):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x = dict(q=r(T, Hk, dk), k=r(T, Hk, dk), v=r(T, Hv, dv), g=r(T, Hv) * (4.0 if strong else 0.5) + (2.0 if strong else -3.0),
             w=r(T, Hv), dO=r(T, Hv, dv))
    for n in ("q", "k"):
        x[n] = x[n] / x[n].norm(dim=-1, keepdim=True)
    return {n: t.to(dt).double() for n, t in x.items()}   # the reference reads the rounded values


DELTA_CASES = [  # lens (None: a batch of two), Hk, Hv, dk, dv
    ((1,), 1, 1, 64, 64), ((15, 64, 1, 0, 65), 1, 2, 64, 128), ((130, 3), 2, 2, 128, 64), ((63, 128, 200), 2, 4, 128, 128),
    (None, 1, 3, 128, 128), (None, 2, 2, 64, 64)]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("case", DELTA_CASES, ids=str)
@pytest.mark.parametrize("full", [False, True], ids=["plain", "full"])
@pytest.mark.parametrize("strong", [False, True], ids=["mild", "strong"])
def test_delta_forward_backward(cuda_device, dt, case, full, strong):
    """full: amplitude, bias, start state and the last state's gradient.  Packed rows before, between
    and after hold NaN; outputs there stay as they were.  strong: log decays to -20 a step."""
    lens, Hk, Hv, dk, dv = case
    packed = lens is not None
    lens = lens if packed else (77, 77)
    N = len(lens)
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float32).double()  # noqa: E731
    A_dec, tau, S0, dS = (0.3 * r(Hv), 0.5 * r(Hv), 0.2 * r(N, Hv, dv, dk), r(N, Hv, dv, dk)) if full else (None,) * 4
    seqs = [delta_inputs(T, Hk, Hv, dk, dv, dt, 100 + n, strong) for n, T in enumerate(lens)]
    names = ("q", "k", "v", "g", "w", "dO")
    tail = 3 if packed else 0

    def lay(n):
        x = torch.cat([s[n] for s in seqs] + [torch.full((tail,) + seqs[0][n].shape[1:], float("nan"), dtype=torch.float64)])
        return (x if packed else x.unflatten(0, (N, lens[0]))).to(dt).to(cuda_device)

    dev = lambda x: None if x is None else x.float().to(cuda_device)  # noqa: E731
    q, k, v, gl, wl, dO = (lay(n) for n in names)
    cu = torch.tensor(np.cumsum((0,) + lens), dtype=torch.int32, device=cuda_device) if packed else None
    more = dict(A_dec=dev(A_dec), tau=dev(tau), cu_seqlens=cu)
    mark = torch.full_like(v, 7.0)
    out = carve.carve_gdr_fwd(q, k, v, gl, wl, S0=dev(S0), out=dict(o=mark), **more)
    lean = carve.carve_gdr_fwd(q, k, v, gl, wl, S0=dev(S0), save_for_bwd=False, **more)
    marks = {n: torch.full_like(x, 7.0) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg_logit", gl), ("dw_logit", wl))}
    gr = carve.carve_gdr_bwd(q, k, v, gl, wl, out["saved"], dO, dS_final=dev(dS), out=dict(marks), **more)
    again = carve.carve_gdr_bwd(q, k, v, gl, wl, out["saved"], dO, dS_final=dev(dS), **more)
    rows = sum(lens)
    flat = lambda x: x.flatten(0, -3) if not packed else x  # noqa: E731
    assert torch.equal(flat(lean["o"])[:rows], flat(out["o"])[:rows]) and torch.equal(lean["S_final"], out["S_final"])
    if packed:
        for x in [out["o"]] + [gr[n] for n in marks]:
            assert (x[rows:] == 7.0).all()
    for n in gr:
        a, b = (x.flatten(0, 1) if n in ("dg_logit", "dw_logit") and not packed else x for x in (gr[n], again[n]))
        if n in marks and packed:
            a, b = a[:rows], b[:rows]
        assert torch.equal(a, b), f"{n} differs between two calls"
    at, sums = 0, dict(dA_dec=0.0, dtau=0.0)
    u = U[dt]
    tol = {"o": 4 * u, "dq": 4 * u, "dv": 4 * u, "dk": 8 * u, "g": 8 * u, "w": 8 * u} if dt == torch.bfloat16 else {}
    cmp = {n: ([], []) for n in ("o", "S", "dq", "dk", "dv", "g", "w", "dS0")}
    for n, (T, s) in enumerate(zip(lens, seqs)):
        inp = dict(q=s["q"], k=s["k"], v=s["v"], g=s["g"], w=s["w"], A_dec=A_dec, tau=tau, S0=S0[n] if full else None)
        want_o, want_S = R.delta(**inp)
        wg = R.grads(R.delta, inp, (s["dO"], dS[n] if full else None)) if T or full else {}
        part = slice(at, at + T)
        pick = (lambda x: x[part]) if packed else (lambda x: x[n])   # noqa: E731
        for key, got, want in (("o", pick(out["o"]), want_o), ("S", out["S_final"][n], want_S),
                               ("dq", pick(gr["dq"]), wg.get("q")), ("dk", pick(gr["dk"]), wg.get("k")),
                               ("dv", pick(gr["dv"]), wg.get("v")), ("g", pick(gr["dg_logit"]), wg.get("g")),
                               ("w", pick(gr["dw_logit"]), wg.get("w")), ("dS0", gr["dS0"][n], wg.get("S0"))):
            if want is not None:
                cmp[key][0].append(got.double().cpu().flatten())
                cmp[key][1].append(want.flatten())
        if full:
            sums["dA_dec"], sums["dtau"] = sums["dA_dec"] + wg["A_dec"], sums["dtau"] + wg["tau"]
        at += T
    for key, (got, want) in cmp.items():
        if got:
            lim = tol.get(key, 1e-5 if dt == torch.float32 else 2e-5 if key == "S" else 4 * u)
            assert rel(torch.cat(got), torch.cat(want)) <= lim, (key, rel(torch.cat(got), torch.cat(want)), lim)
    if full:
        lim = 2e-5 if dt == torch.float32 else 8 * u
        for n, want in sums.items():
            # a sum over tokens of either sign: relative to the terms' size, sqrt(rows) of them at least
            assert rel(gr[n], want) <= 4 * lim, (n, rel(gr[n], want))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_delta_chains_over_calls_and_steps(cuda_device, dt):
    """A sequence cut into two forwards and then single steps gives the whole sequence's outputs."""
    T, Hk, Hv, d = 150, 2, 4, 128
    s = {n: x.to(dt).to(cuda_device)[None] for n, x in delta_inputs(T, Hk, Hv, d, d, dt, 5).items()}
    xs = [s[n] for n in ("q", "k", "v", "g", "w")]
    whole = carve.carve_gdr_fwd(*xs, save_for_bwd=False)
    a = carve.carve_gdr_fwd(*(x[:, :70].contiguous() for x in xs), save_for_bwd=False)
    S = a["S_final"]
    b = carve.carve_gdr_fwd(*(x[:, 70:140].contiguous() for x in xs), S0=S, save_for_bwd=False, out=dict(S_final=S))
    steps = [carve.carve_gdr_step(*(x[:, t].contiguous() for x in xs), S) for t in range(140, T)]
    o = torch.cat([a["o"], b["o"], torch.stack(steps, 1)], 1)
    lim = 1e-5 if dt == torch.float32 else 2 * 4 * U[dt]
    assert rel(o, whole["o"].double().cpu()) <= lim
    assert rel(S, whole["S_final"].double().cpu()) <= 4e-5


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("B,Hk,Hv,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 6, 128, 64), (5, 4, 4, 64, 128), (2, 16, 16, 128, 128)])
def test_delta_step(cuda_device, dt, B, Hk, Hv, dk, dv):
    s = delta_inputs(B, Hk, Hv, dk, dv, dt, 9)
    g = torch.Generator().manual_seed(10)
    S0 = torch.randn(B, Hv, dv, dk, generator=g)
    A_dec, tau = torch.randn(Hv, generator=g), torch.randn(Hv, generator=g)
    S = S0.to(cuda_device)
    xs = [s[n].to(dt).to(cuda_device) for n in ("q", "k", "v", "g", "w")]
    o = carve.carve_gdr_step(*xs, S, A_dec=A_dec.to(cuda_device), tau=tau.to(cuda_device))
    for b in range(B):
        want, last = R.delta(*(s[n][b:b + 1] for n in ("q", "k", "v", "g", "w")), A_dec.double(), tau.double(), S0[b].double())
        assert rel(o[b], want[0]) <= 4e-6 + (U[dt] if dt == torch.bfloat16 else 0)
        assert rel(S[b], last) <= 4e-6


def window_inputs(T, Hq, Hkv, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64).to(dt).double()  # noqa: E731
    return dict(q=r(T, Hq, d), k=r(T, Hkv, d), v=r(T, Hkv, d), dO=r(T, Hq, d))


def near(got, want, mass, c, n, d, dt):
    err = (got.double().cpu() - want).abs()
    lim = (c * U[dt] if dt == torch.bfloat16 else 0.0) * mass + (n + 4 * d) * 2.0 ** -24 * (mass + want.abs())
    assert (err <= lim).all(), (err - lim).max().item()


WINDOW_CASES = [  # lens (None: a batch of two), Hq, Hkv, d, window, sinks
    ((1,), 1, 1, 64, 1, 0), ((40, 0, 1, 129, 64), 2, 1, 64, 7, 3), ((300, 33), 4, 4, 128, 64, 0), ((257, 128), 6, 2, 128, 100, 5),
    ((200, 260), 2, 2, 64, 1000, 4), ((500,), 3, 1, 128, 65, 130), ((350,), 1, 1, 64, 1, 1), (None, 4, 2, 128, 128, 4),
    (None, 2, 2, 64, 33, 64)]


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("case", WINDOW_CASES, ids=str)
@pytest.mark.parametrize("scale", [None, -0.7], ids=["usual", "negative"])
def test_window_forward_backward(cuda_device, dt, case, scale):
    lens, Hq, Hkv, d, W, sinks = case
    packed = lens is not None
    lens = lens if packed else (190, 190)
    seqs = [window_inputs(T, Hq, Hkv, d, dt, 40 + n) for n, T in enumerate(lens)]
    tail = 5 if packed else 0

    def lay(n):
        x = torch.cat([s[n] for s in seqs] + [torch.full((tail,) + seqs[0][n].shape[1:], float("nan"), dtype=torch.float64)])
        return (x if packed else x.unflatten(0, (len(lens), lens[0]))).to(dt).to(cuda_device)

    q, k, v, dO = (lay(n) for n in ("q", "k", "v", "dO"))
    cu = torch.tensor(np.cumsum((0,) + lens), dtype=torch.int32, device=cuda_device) if packed else None
    at = dict(window=W, sinks=sinks, scale=scale, cu_seqlens=cu)
    out = carve.carve_swa_fwd(q, k, v, out=dict(o=torch.full_like(q, 7.0)), **at)
    marks = dict(dq=torch.full_like(q, 7.0), dk=torch.full_like(k, 7.0), dv=torch.full_like(v, 7.0))
    gr = carve.carve_swa_bwd(q, k, v, out["o"], out["lse"], dO, out=dict(marks), **at)
    again = carve.carve_swa_bwd(q, k, v, out["o"], out["lse"], dO, out={n: x.clone() for n, x in marks.items()}, **at)
    for n in gr:
        assert torch.equal(gr[n], again[n])
    rows = sum(lens)
    if packed:
        for x in [out["o"]] + list(gr.values()):
            assert (x[rows:] == 7.0).all()
    row = 0
    for n, (T, s) in enumerate(zip(lens, seqs)):
        if T:
            inp = {x: s[x] for x in ("q", "k", "v")}
            want, lse = R.window(**inp, win=W, sinks=sinks, scale=scale)
            wg = R.grads(lambda q, k, v: R.window(q, k, v, W, sinks, scale)[:1], inp, (s["dO"],))
            mass = R.window_masses(**inp, dO=s["dO"], win=W, sinks=sinks, scale=scale)
            pick = (lambda x: x[row:row + T]) if packed else (lambda x: x[n])   # noqa: E731
            near(pick(out["o"]), want, mass["o"], 2, T, d, dt)
            assert (pick(out["lse"]).double().cpu() - lse).abs().max() <= 1e-4
            near(pick(gr["dv"]), wg["v"], mass["dv"], 2, T * Hq // Hkv, d, dt)
            near(pick(gr["dq"]), wg["q"], mass["dq"], 3, T, d, dt)
            near(pick(gr["dk"]), wg["k"], mass["dk"], 3, T * Hq // Hkv, d, dt)
        row += T


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("Hq,Hkv,d,W,sinks", [(1, 1, 64, 1, 0), (4, 2, 64, 5, 3), (12, 1, 128, 70, 0), (40, 2, 64, 200, 7),
                                              (8, 8, 128, 300, 1), (4, 4, 128, 2000, 4)])
def test_window_steps_after_a_prompt(cuda_device, dt, Hq, Hkv, d, W, sinks):
    """Prompts of ragged lengths (none, shorter and longer than the window) fill the caches, then
    every sequence decodes; each step's output is the whole sequence's at that position.  Slots
    that no token has reached hold NaN."""
    lens, steps = (0, 1, 3, 90, 331), 6
    seqs = [window_inputs(T + steps, Hq, Hkv, d, dt, 60 + n) for n, T in enumerate(lens)]
    dev = lambda x: x.to(dt).to(cuda_device)  # noqa: E731
    k0, v0 = (dev(torch.cat([s[n][:T] for s, T in zip(seqs, lens)])) for n in ("k", "v"))
    kc = torch.full((len(lens), sinks + W, Hkv, d), float("nan"), dtype=dt, device=cuda_device)
    vc = kc.clone()
    cu = torch.tensor(np.cumsum((0,) + lens), dtype=torch.int32, device=cuda_device)
    carve.carve_swa_fill(k0, v0, kc, vc, window=W, sinks=sinks, cu_seqlens=cu)
    pos = torch.tensor(lens, dtype=torch.int64, device=cuda_device)
    got = []
    for i in range(steps):
        q, k, v = (dev(torch.stack([s[n][T + i] for s, T in zip(seqs, lens)])) for n in ("q", "k", "v"))
        got.append(carve.carve_swa_step(q, k, v, kc, vc, pos, window=W, sinks=sinks))
        pos += 1
    for n, (T, s) in enumerate(zip(lens, seqs)):
        want, _ = R.window(s["q"], s["k"], s["v"], W, sinks)
        mass = R.window_masses(s["q"], s["k"], s["v"], s["dO"], W, sinks)["o"]
        near(torch.stack([x[n] for x in got]), want[T:], mass[T:], 2, T + steps, d, dt)
        for t in range(T + steps):   # the newest token of each slot
            slot = t if t < sinks else sinks + (t - sinks) % W
            if t < sinks or t >= T + steps - W:
                assert torch.equal(kc[n, slot], dev(s["k"][t])) and torch.equal(vc[n, slot], dev(s["v"][t]))
        assert torch.isnan(kc[n, T + steps:]).all()   # slots beyond stay as they were


def test_step_without_a_sequence(cuda_device):
    """A negative position: zeros, and the caches untouched."""
    r = lambda *s: torch.randn(*s, device=cuda_device, dtype=torch.bfloat16)  # noqa: E731
    q, k, v, kc, vc = r(2, 4, 64), r(2, 2, 64), r(2, 2, 64), r(2, 10, 2, 64), r(2, 10, 2, 64)
    was = kc.clone(), vc.clone()
    o = carve.carve_swa_step(q, k, v, kc, vc, torch.tensor([-1, 3], device=cuda_device), window=8, sinks=2)
    assert (o[0] == 0).all() and torch.equal(kc[0], was[0][0]) and torch.equal(vc[0], was[1][0])
    assert torch.isfinite(o[1]).all() and torch.equal(kc[1, 3], k[1])


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_no_rows(cuda_device, dt):
    z = lambda *s: torch.zeros(*s, device=cuda_device, dtype=dt)  # noqa: E731
    S0 = torch.randn(2, 4, 64, 64, device=cuda_device)
    x = (z(2, 0, 2, 64), z(2, 0, 2, 64), z(2, 0, 4, 64), z(2, 0, 4), z(2, 0, 4))
    A = torch.zeros(4, device=cuda_device)
    out = carve.carve_gdr_fwd(*x, S0=S0, A_dec=A)
    assert torch.equal(out["S_final"], S0)
    g = carve.carve_gdr_bwd(*x, out["saved"], x[2], dS_final=S0, A_dec=A)
    assert torch.equal(g["dS0"], S0) and (g["dA_dec"] == 0).all()
    q, k = z(2, 0, 4, 64), z(2, 0, 2, 64)
    out = carve.carve_swa_fwd(q, k, k, window=3)
    carve.carve_swa_bwd(q, k, k, out["o"], out["lse"], q, window=3)
    kc = torch.full((2, 3, 2, 64), 7.0, device=cuda_device, dtype=dt)
    carve.carve_swa_fill(k, k, kc, kc.clone(), window=3)
    assert (kc == 7.0).all()
    cu = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    out = carve.carve_gdr_fwd(z(0, 2, 64), z(0, 2, 64), z(0, 4, 64), z(0, 4), z(0, 4), S0=S0, cu_seqlens=cu)
    assert torch.equal(out["S_final"], S0)
    carve.carve_swa_fwd(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), window=3, cu_seqlens=cu)


def test_bad_offsets_are_reported(cuda_device):
    """A sequence that leaves the rows is computed as empty, the others as usual, and the status says
    so (its code is taken here, so that the fixture finds a clean one)."""
    r = lambda *s: torch.randn(*s, device=cuda_device)  # noqa: E731
    cu = torch.tensor([0, 40, 90], dtype=torch.int32, device=cuda_device)   # 80 rows are there
    q, k, v, gl = r(80, 2, 64), r(80, 2, 64) / 8, r(80, 2, 64), r(80, 2)
    S0 = r(2, 2, 64, 64)
    out = carve.carve_gdr_fwd(q, k, v, gl, gl, S0=S0, cu_seqlens=cu, save_for_bwd=False)
    assert torch.equal(out["S_final"][1], S0[1])
    assert carve.carve_check() == 1 and carve.carve_check() == 0
    o = carve.carve_swa_fwd(q, k, v, window=9, cu_seqlens=cu, out=dict(o=torch.full_like(q, 7.0)))["o"]
    assert (o[40:] == 7.0).all() and (o[:40] != 7.0).any()
    assert carve.carve_check() == 1 and carve.carve_check() == 0


def _stack(x, dt, W, sinks, cu, S, caches, pos=None):
    """Two mixer layers of a hybrid stack on x [..., H, d]: the delta rule, then the window over its
    output, each added to its input.  pos None: a prompt; else one token."""
    unit = lambda y: (y.float() / y.float().norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    gate = lambda y, s: (y[..., 0] * s).contiguous()  # noqa: E731
    qk = unit(x)
    args = (qk, qk, x, gate(x, 0.5) - 2, gate(x, 1.0))
    if pos is None:
        out = carve.carve_gdr_fwd(*args, S0=S, cu_seqlens=cu, save_for_bwd=False, out=dict(S_final=S))
        y = x + out["o"]
        z = y + carve.carve_swa_fwd(y, y, y, window=W, sinks=sinks, cu_seqlens=cu, want_lse=False)["o"]
        carve.carve_swa_fill(y, y, *caches, window=W, sinks=sinks, cu_seqlens=cu)
        return z
    y = x + carve.carve_gdr_step(*args, S)
    return y + carve.carve_swa_step(y, y, y, *caches, pos, window=W, sinks=sinks)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_hybrid_layers_prompt_then_decode(cuda_device, dt):
    """The two mixers in series: packed prompts, then decoding from the kept state and caches under
    a replayed graph, against the prompts that already hold the decoded tokens."""
    W, sinks, H, d, steps = 24, 2, 2, 64, 5
    lens = (50, 7, 33)
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn(T + steps, H, d, generator=g).to(dt).to(cuda_device) for T in lens]
    zeros = lambda: (torch.zeros(3, H, d, d, device=cuda_device),  # noqa: E731
                     [torch.zeros(3, sinks + W, H, d, dtype=dt, device=cuda_device) for _ in range(2)])
    cut = lambda n: torch.tensor(np.cumsum([0] + [T + n for T in lens]), dtype=torch.int32, device=cuda_device)  # noqa: E731
    want = _stack(torch.cat(xs), dt, W, sinks, cut(steps), *zeros())
    S, caches = zeros()
    _stack(torch.cat([x[:T] for x, T in zip(xs, lens)]), dt, W, sinks, cut(0), S, caches)
    tok = torch.empty(3, H, d, dtype=dt, device=cuda_device)
    pos = torch.tensor(lens, dtype=torch.int64, device=cuda_device)
    keep = S.clone(), [c.clone() for c in caches]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):   # warm-up, off the default stream
        tok.copy_(xs[0][0].expand(3, -1, -1))
        _stack(tok, dt, W, sinks, None, S, caches, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = _stack(tok, dt, W, sinks, None, S, caches, pos)
        pos += 1
    S.copy_(keep[0])
    for c, was in zip(caches, keep[1]):
        c.copy_(was)
    pos.copy_(torch.tensor(lens))
    row = np.cumsum([0] + [T + steps for T in lens])
    for i in range(steps):
        tok.copy_(torch.stack([x[T + i] for x, T in zip(xs, lens)]))
        graph.replay()
        for n, T in enumerate(lens):
            ref = want[row[n] + T + i].double().cpu()
            # one rounding less or more of each layer's output, and of the sums between them
            assert rel(z[n], ref) <= (1e-5 if dt == torch.float32 else 12 * U[dt])


def test_prompt_call_is_captured_and_replayed(cuda_device):
    """Forward and backward of both mixers in one graph, replayed on new inputs, equal to eager calls."""
    dt = torch.bfloat16
    r = lambda *s: torch.randn(*s, device=cuda_device).to(dt)  # noqa: E731

    def inputs():
        k = r(1, 70, 2, 128).float()
        return [r(1, 70, 2, 128) / 11, (k / k.norm(dim=-1, keepdim=True)).to(dt), r(1, 70, 2, 128), r(1, 70, 2), r(1, 70, 2), r(1, 70, 2, 128)]

    def both(q, k, v, gl, wl, dO):
        a = carve.carve_gdr_fwd(q, k, v, gl, wl)
        b = carve.carve_swa_fwd(q, k, v, window=20, sinks=1)
        ga = carve.carve_gdr_bwd(q, k, v, gl, wl, a["saved"], dO)
        gb = carve.carve_swa_bwd(q, k, v, b["o"], b["lse"], dO, window=20, sinks=1)
        return [a["o"], a["S_final"], b["o"], *ga.values(), *gb.values()]

    held = inputs()
    both(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*held)
    for _ in range(2):
        new = inputs()
        for h, x in zip(held, new):
            h.copy_(x)
        graph.replay()
        for x, y in zip(got, both(*new)):
            assert torch.equal(x, y)


def test_two_streams_at_once(cuda_device):
    """Two calls in flight with buffers of their own give what each gives alone."""
    dt = torch.bfloat16
    xs = [window_inputs(700, 4, 2, 128, dt, s) for s in (1, 2)]
    xs = [[s[n].to(dt).to(cuda_device)[None] for n in ("q", "k", "v")] for s in xs]
    alone = [carve.carve_swa_fwd(*x, window=200, sinks=4)["o"] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [carve.carve_swa_fwd(*x, window=200, sinks=4, stream=s)["o"] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a, b)


def test_rows_of_a_window_do_not_depend_on_what_they_do_not_see(cuda_device):
    """Changing tokens outside a query's window (and no sink) changes no bit of its output."""
    for dt in TYPES:
        s = window_inputs(400, 2, 2, 64, dt, 77)
        q, k, v = (s[n].to(dt).to(cuda_device)[None] for n in ("q", "k", "v"))
        a = carve.carve_swa_fwd(q, k, v, window=50, sinks=3)["o"]
        k2, v2 = k.clone(), v.clone()
        k2[:, 100:130] = 50.0
        v2[:, 100:130] = -9.0
        b = carve.carve_swa_fwd(q, k2, v2, window=50, sinks=3)["o"]
        assert torch.equal(a[:, :100], b[:, :100]) and torch.equal(a[:, 129 + 50:], b[:, 129 + 50:])
        assert not torch.equal(a[:, 130:150], b[:, 130:150])


def _both_types(f, tensors, scalars):
    """f on bf16 tensors and, on the same values, in fp32 (other kernels)."""
    return f(*tensors, **scalars), f(*(x.float() for x in tensors), **scalars)


@pytest.mark.parametrize("lens,Hk,Hv,dk,dv", [
    ((4000,), 4, 8, 128, 128),                                   # more tiles than the GPU has processors, several heads a tile
    ((64, 128, 1, 0, 640, 63, 65, 1500, 2, 192) * 2, 2, 2, 128, 64), ((320, 321, 319) * 4, 8, 8, 64, 128),
    (None, 16, 16, 64, 64)])
def test_delta_over_many_tiles(cuda_device, lens, Hk, Hv, dk, dv):
    """Persistent work and long chains of chunks: the bf16 kernels against the fp32 ones (which the small
    cases hold to the definition), packed sequences that end on, before and behind chunk borders.
    Roundings as in the header: 4 u and 8 u, states 2e-5 and the fp32 kernels' own 1e-5."""
    packed = lens is not None
    rows = sum(lens) if packed else 1000
    lead = (rows,) if packed else (3, rows)
    g = torch.Generator(device="cuda").manual_seed(21)
    r = lambda *s: torch.randn(*lead, *s, generator=g, device=cuda_device)  # noqa: E731
    q, k, v, dO = r(Hk, dk), r(Hk, dk), r(Hv, dv), r(Hv, dv)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    gl, wl = 0.5 * r(Hv) - 3, r(Hv)
    x = [y.to(torch.bfloat16) for y in (q, k, v, gl, wl, dO)]
    N = len(lens) if packed else 3
    S0 = 0.2 * torch.randn(N, Hv, dv, dk, generator=g, device=cuda_device)
    A, tau = 0.3 * torch.randn(Hv, generator=g, device=cuda_device), 0.5 * torch.randn(Hv, generator=g, device=cuda_device)
    cu = torch.tensor(np.cumsum((0,) + lens), dtype=torch.int32, device=cuda_device) if packed else None

    def f(q, k, v, gl, wl, dO):
        more = dict(A_dec=A, tau=tau, cu_seqlens=cu)
        out = carve.carve_gdr_fwd(q, k, v, gl, wl, S0=S0, **more)
        g = carve.carve_gdr_bwd(q, k, v, gl, wl, out["saved"], dO, dS_final=S0, **more)
        return dict(o=out["o"], S=out["S_final"], **g)

    got, want = _both_types(f, x, {})
    u = U[torch.bfloat16]
    for n, lim in dict(o=4 * u, S=3e-5, dq=4 * u, dk=8 * u, dv=4 * u, dg_logit=8 * u, dw_logit=8 * u, dS0=4 * u, dA_dec=32 * u,
                       dtau=32 * u).items():
        assert rel(got[n], want[n].double().cpu()) <= lim, (n, rel(got[n], want[n].double().cpu()))


@pytest.mark.parametrize("lens,Hq,Hkv,d,W,sinks", [
    ((3000,), 8, 2, 128, 700, 4), (None, 6, 6, 64, 129, 0), ((64, 128, 1, 0, 640, 63, 65, 1500, 2, 192) * 2, 6, 2, 128, 65, 70),
    ((257, 255, 256) * 4, 4, 4, 64, 64, 1)])
def test_window_over_many_tiles(cuda_device, lens, Hq, Hkv, d, W, sinks):
    """More units than the GPU has processors, in both pairings of query tiles: the bf16 kernels against
    the fp32 ones.  Relative L2: the roundings of the header are of either sign, over sums of terms
    of either sign, so they count once each: 3 u for o, 4 u for the gradients."""
    packed = lens is not None
    rows = sum(lens) if packed else 900
    lead = (rows,) if packed else (4, rows)
    g = torch.Generator(device="cuda").manual_seed(22)
    x = [torch.randn(*lead, h, d, generator=g, device=cuda_device).to(torch.bfloat16) for h in (Hq, Hkv, Hkv, Hq)]
    cu = torch.tensor(np.cumsum((0,) + lens), dtype=torch.int32, device=cuda_device) if packed else None

    def f(q, k, v, dO):
        at = dict(window=W, sinks=sinks, cu_seqlens=cu)
        out = carve.carve_swa_fwd(q, k, v, **at)
        return dict(o=out["o"], lse=out["lse"], **carve.carve_swa_bwd(q, k, v, out["o"], out["lse"], dO, **at))

    got, want = _both_types(f, x, {})
    u = U[torch.bfloat16]
    for n, lim in dict(o=3 * u, dq=4 * u, dk=4 * u, dv=3 * u).items():
        assert rel(got[n], want[n].double().cpu()) <= lim, (n, rel(got[n], want[n].double().cpu()))
    assert (got["lse"] - want["lse"]).abs().max() <= 1e-4


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_delta_on_two_streams_at_once(cuda_device, dt):
    """Forward and backward of two inputs in flight, repeatedly, give what each gives alone."""
    def inputs(seed):
        s = delta_inputs(500, 4, 8, 128, 128, dt, seed)
        return [s[n].to(dt).to(cuda_device)[None].expand(3, -1, *(-1,) * (s[n].dim() - 1)).contiguous() for n in ("q", "k", "v", "g", "w", "dO")]

    def run(x, stream=None):
        out = carve.carve_gdr_fwd(*x[:5], stream=stream)
        return [out["o"], out["S_final"], *carve.carve_gdr_bwd(*x[:5], out["saved"], x[5], stream=stream).values()]

    xs = [inputs(s) for s in (1, 2)]
    alone = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(run(x, s))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_state_in_place_of_the_start_state(cuda_device):
    """S_final may be S0: the call then continues a state in place."""
    for dt in TYPES:
        s = delta_inputs(130, 2, 2, 64, 64, dt, 31)
        x = [s[n].to(dt).to(cuda_device)[None] for n in ("q", "k", "v", "g", "w")]
        S = torch.randn(1, 2, 64, 64, device=cuda_device)
        want = carve.carve_gdr_fwd(*x, S0=S, save_for_bwd=False)["S_final"]
        carve.carve_gdr_fwd(*x, S0=S, save_for_bwd=False, out=dict(S_final=S))
        assert torch.equal(S, want)


def test_refusals_on_the_device(cuda_device):
    """What the binding refuses with tensors on the GPU: buffers that are too small, a key in the wrong
    type, a state of the wrong shape; nothing is launched."""
    dt = torch.bfloat16
    z = lambda *s: torch.zeros(*s, device=cuda_device, dtype=dt)  # noqa: E731
    x = (z(1, 70, 2, 64), z(1, 70, 2, 64), z(1, 70, 2, 64), z(1, 70, 2), z(1, 70, 2))
    few = torch.zeros(64, dtype=torch.uint8, device=cuda_device)
    with pytest.raises(ValueError, match="bytes"):
        carve.carve_gdr_fwd(*x, out=dict(saved=few))
    with pytest.raises(ValueError, match="bytes"):
        carve.carve_gdr_fwd(*x, save_for_bwd=False, workspace=few)
    with pytest.raises(ValueError, match="bytes"):
        carve.carve_gdr_bwd(*x, few, x[2])
    with pytest.raises(TypeError, match="k must be"):
        carve.carve_gdr_fwd(x[0], x[1].float(), *x[2:])
    with pytest.raises(ValueError, match="S0 must have shape"):
        carve.carve_gdr_fwd(*x, S0=torch.zeros(1, 2, 64, 32, device=cuda_device))
    with pytest.raises(ValueError, match="is on cpu"):
        carve.carve_gdr_fwd(x[0], x[1], x[2].cpu(), *x[3:])
    with pytest.raises(carve.CarveError, match="UNSUPPORTED"):
        carve.carve_swa_fwd(z(1, 9, 2, 80), z(1, 9, 2, 80), z(1, 9, 2, 80), window=4)
    with pytest.raises(ValueError, match="lse"):
        carve.carve_swa_bwd(*x[:3], x[0], torch.zeros(1, 70, 3, device=cuda_device), x[0], window=4)
