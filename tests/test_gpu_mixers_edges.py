"""Calls of the mixers of include/carve_mixers.h that stand at an edge: very many short sequences, no
rows, other streams, tokens that reset a state.  Tolerances as in test_gpu_mixers.py, whose fp64
comparisons hold the fp32 kernels to the definition."""
import numpy as np
import pytest
import torch

import chunk_gated_delta_b200 as carve
from tests import mixer_reference as R
from tests.test_gpu_mixers import TYPES, U, delta_inputs, ids, near, rel, window_inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def device_status(cuda_device):
    yield
    assert carve.carve_check() == 0


def offsets(lens, device):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device=device)


def delta_tensors(lead, Hk, Hv, dk, dv, seed, device):
    """q, k, v, g_logit, w_logit, dO in bf16."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*lead, *s, generator=g, device=device)  # noqa: E731
    q, k = r(Hk, dk), r(Hk, dk)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    return [x.to(BF16) for x in (q, k, r(Hv, dv), 0.5 * r(Hv) - 3, r(Hv), r(Hv, dv))]


def delta_both(x, cu=None, stream=None, **more):
    out = carve.carve_gdr_fwd(*x[:5], cu_seqlens=cu, stream=stream, **more)
    g = carve.carve_gdr_bwd(*x[:5], out["saved"], x[5], cu_seqlens=cu, stream=stream, **more)
    return dict(o=out["o"], S=out["S_final"], **g)


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 1, 64, 64), (2, 4, 128, 64)])
def test_delta_gradients_of_very_many_short_sequences(cuda_device, Hk, Hv, dk, dv):
    """Thousands of items of a tile or less, so that the warps of a gradient CTA drift apart by as much as
    their hand-overs allow: the bf16 kernels against the fp32 ones, and bits from call to call."""
    g = np.random.default_rng(5)
    lens = g.integers(0, 70, 3000).tolist()
    x, cu = delta_tensors((sum(lens),), Hk, Hv, dk, dv, 31, cuda_device), offsets(lens, cuda_device)
    got, want = delta_both(x, cu), delta_both([y.float() for y in x], cu)
    u = U[BF16]
    for n, lim in dict(o=4 * u, S=3e-5, dq=4 * u, dk=8 * u, dv=4 * u, dg_logit=8 * u, dw_logit=8 * u, dS0=4 * u).items():
        assert rel(got[n], want[n].double().cpu()) <= lim, (n, rel(got[n], want[n].double().cpu()))
    for _ in range(3):
        for n, y in delta_both(x, cu).items():
            assert torch.equal(y, got[n]), n


def window_tensors(lead, Hq, Hkv, d, seed, device):
    """q, k, v, dO in bf16."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*lead, h, d, generator=g, device=device).to(BF16) for h in (Hq, Hkv, Hkv, Hq)]


@pytest.mark.parametrize("Hq,Hkv,d", [(3, 3, 64), (3, 1, 128), (2, 1, 64)])
def test_window_of_very_many_short_sequences(cuda_device, Hq, Hkv, d):
    """Thousands of units of one key block, whose second query tile is empty where heads do not pair: the
    query buffers pass from unit to unit as fast as they can.  bf16 against fp32 (3 u: see
    test_window_over_many_tiles), and bits from call to call."""
    lens = np.random.default_rng(6).integers(0, 70, 3000).tolist()
    q, k, v, _ = window_tensors((sum(lens),), Hq, Hkv, d, 32, cuda_device)
    at = dict(window=20, sinks=2, cu_seqlens=offsets(lens, cuda_device))
    got, want = carve.carve_swa_fwd(q, k, v, **at), carve.carve_swa_fwd(q.float(), k.float(), v.float(), **at)
    assert rel(got["o"], want["o"].double().cpu()) <= 3 * U[BF16]
    assert (got["lse"] - want["lse"]).abs().max() <= 1e-4
    for _ in range(10):
        again = carve.carve_swa_fwd(q, k, v, **at)
        assert torch.equal(again["o"], got["o"]) and torch.equal(again["lse"], got["lse"])


def test_states_pass_through_calls_without_rows_in_order(cuda_device):
    """Calls without tokens hand the state on, each after what the stream holds before it: a backward, a
    forward that starts from its dS0, and a forward in place, on states that change from turn to turn."""
    z = lambda *s: torch.zeros(*s, device=cuda_device, dtype=BF16)  # noqa: E731
    x = (z(40, 0, 8, 128), z(40, 0, 8, 128), z(40, 0, 8, 128), z(40, 0, 8), z(40, 0, 8))
    saved = carve.carve_gdr_fwd(*x)["saved"]
    state = torch.zeros(40, 8, 128, 128, device=cuda_device)
    mid, last = torch.empty_like(state), torch.empty_like(state)
    for i in range(1, 40):
        state += 1.0
        carve.carve_gdr_bwd(*x, saved, x[2], dS_final=state, out=dict(dS0=mid))
        carve.carve_gdr_fwd(*x, S0=mid, out=dict(S_final=last, saved=saved))
        carve.carve_gdr_fwd(*x, S0=last, out=dict(S_final=last, saved=saved))
        assert torch.equal(last, torch.full_like(last, float(i))), i


def test_delta_gradients_wait_for_the_longest_sequence(cuda_device):
    """One sequence of 60 thousand tokens beside short ones: the gradients' kernel starts on the SMs that the
    short ones leave and waits there (for 3 ms; its bounded waits begin behind that)."""
    lens = [3, 60000, 5, 64, 1]
    x, cu = delta_tensors((sum(lens),), 1, 1, 64, 64, 33, cuda_device), offsets(lens, cuda_device)
    got, want = delta_both(x, cu), delta_both([y.float() for y in x], cu)
    u = U[BF16]
    for n, lim in dict(o=4 * u, S=3e-5, dq=4 * u, dk=8 * u, dv=4 * u, dg_logit=8 * u, dw_logit=8 * u, dS0=4 * u).items():
        assert rel(got[n], want[n].double().cpu()) <= lim, (n, rel(got[n], want[n].double().cpu()))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_scratch_belongs_to_the_stream_of_the_call(cuda_device, dt):
    """Calls on `stream=`, made from the default stream, whose scratch the binding allocates: two at once, and
    memory of the scratch's size that the default stream takes and writes as soon as each call is back."""
    def inputs(seed):
        return ([y.to(dt) for y in delta_tensors((2, 1500), 2, 4, 128, 128, seed, cuda_device)],
                [y.to(dt) for y in window_tensors((1, 1500), 4, 2, 128, seed, cuda_device)])

    def prompt(x, y, kept, stream):
        out = carve.carve_gdr_fwd(*x[:5], save_for_bwd=False, stream=stream)
        return [out["o"], out["S_final"]]

    def delta(x, y, kept, stream):
        return list(carve.carve_gdr_bwd(*x[:5], kept["saved"], x[5], stream=stream).values())

    def window(x, y, kept, stream):
        return list(carve.carve_swa_bwd(*y[:3], kept["o"], kept["lse"], y[3], window=300, sinks=4, stream=stream).values())

    xs = [inputs(s) for s in (41, 42)]
    kept = [dict(carve.carve_swa_fwd(*y[:3], window=300, sinks=4), saved=carve.carve_gdr_fwd(*x[:5])["saved"]) for x, y in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for f in (prompt, delta, window):
        alone = [f(*x, kp, None) for x, kp in zip(xs, kept)]
        torch.cuda.synchronize()
        for _ in range(4):
            got, junk = [], []
            for x, kp, s in zip(xs, kept, streams):
                got.append(f(*x, kp, s))
                junk += [torch.full((n,), float("nan"), device=cuda_device) for n in (1 << 16, 1 << 19, 1 << 20, 1 << 21, 1 << 22)]
            torch.cuda.synchronize()
            for a, b in zip(alone, got):
                assert all(torch.equal(y, z) for y, z in zip(a, b)), f.__name__


def test_results_belong_to_the_stream_of_the_call(cuda_device):
    """A result's memory returns to the stream that wrote it: what the default stream allocates after the call
    and its result are gone is other memory."""
    x = delta_tensors((1, 3000), 2, 2, 128, 128, 43, cuda_device)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = carve.carve_gdr_fwd(*x[:5], save_for_bwd=False, stream=side)["o"].data_ptr()
    size = x[2].numel()
    mine = [torch.empty(size, dtype=BF16, device=cuda_device) for _ in range(8)]
    assert at not in [y.data_ptr() for y in mine]
    with torch.cuda.stream(side):
        assert at in [torch.empty(size, dtype=BF16, device=cuda_device).data_ptr()]
    torch.cuda.synchronize()


def test_streams_that_do_not_fit_are_refused(cuda_device):
    x = delta_tensors((1, 70), 2, 2, 64, 64, 44, cuda_device)

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 0

    with pytest.raises(ValueError, match="the stream is on"):
        carve.carve_gdr_fwd(*x[:5], stream=Elsewhere())
    handle = torch.cuda.Stream()
    ext = torch.cuda.ExternalStream(handle.cuda_stream)
    want = carve.carve_gdr_fwd(*x[:5])["o"]
    for s in (handle, ext, torch.cuda.default_stream()):
        torch.cuda.synchronize()
        o = carve.carve_gdr_fwd(*x[:5], stream=s)["o"]
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.cuda.current_stream() == torch.cuda.default_stream()


def test_recurrence_scratch_belongs_to_the_stream_of_the_call(cuda_device):
    """The same of carve_fwd and carve_bwd, which this file's mixers stand beside."""
    def inputs(seed):
        q, k, v, gl, wl, dO = delta_tensors((2, 1024), 4, 4, 128, 128, seed, cuda_device)
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=cuda_device)  # noqa: E731
        return (q, k, v, 0.5 * r(2, 1024, 4, 128) - 3, r(2, 1024, 4, 128), wl.float(), 0.02 * r(4, 128, 8), 0.02 * r(4, 8, 128)), dO

    def run(x, dO, stream):
        out = carve.carve_fwd(*x, chunk=64, stream=stream)
        return [out["o"], out["S_final"], *carve.carve_bwd(*x, out["saved"], dO, chunk=64, stream=stream).values()]

    xs = [inputs(s) for s in (51, 52)]
    alone = [run(*x, None) for x in xs]
    assert all(torch.equal(y, z) for y, z in zip(alone[0], run(*xs[0], None)))   # deterministic
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        got, junk = [], []
        for x, s in zip(xs, streams):
            got.append(run(*x, s))
            junk += [torch.full((n,), float("nan"), device=cuda_device) for n in (1 << 16, 1 << 19, 1 << 20, 1 << 21, 1 << 22)]
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(y, z) for y, z in zip(a, b))


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("cu", [(0, 40, 90), (0, 60, 50, 80), (-1, 40, 80), (90, 95), (0, 40, 2 ** 31 - 1)], ids=str)
def test_bad_offsets_are_reported_by_every_packed_call(cuda_device, dt, cu):
    """80 rows; a sequence that leaves them, or whose end lies before its start, counts as empty: its rows
    stay as they were, and each call is reported once."""
    N = len(cu) - 1
    cu = torch.tensor(cu, dtype=torch.int32, device=cuda_device)
    g = torch.Generator(device="cuda").manual_seed(61)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_device).to(dt)  # noqa: E731
    q, k, v, gl, dO = r(80, 2, 64), r(80, 2, 64) / 8, r(80, 2, 64), r(80, 2), r(80, 2, 64)

    def reported(f, *a, **kw):
        assert carve.carve_check() == 0
        out = f(*a, **kw)
        assert carve.carve_check() == 1 and carve.carve_check() == 0, f.__name__
        return out

    a = reported(carve.carve_gdr_fwd, q, k, v, gl, gl, cu_seqlens=cu)
    reported(carve.carve_gdr_bwd, q, k, v, gl, gl, a["saved"], dO, cu_seqlens=cu)
    marks = lambda: dict(o=torch.full_like(q, 7.0))  # noqa: E731
    b = reported(carve.carve_swa_fwd, q, k, v, window=9, sinks=1, cu_seqlens=cu, out=marks())
    grads = reported(carve.carve_swa_bwd, q, k, v, b["o"], b["lse"].nan_to_num(), dO, window=9, sinks=1, cu_seqlens=cu,
                     out={n: torch.full_like(q, 7.0) for n in ("dq", "dk", "dv")})
    kc = torch.full((N, 10, 2, 64), 7.0, dtype=dt, device=cuda_device)
    vc = kc.clone()
    reported(carve.carve_swa_fill, k, v, kc, vc, window=9, sinks=1, cu_seqlens=cu)
    at = cu.tolist()
    owned = torch.zeros(80, dtype=torch.bool)
    for n in range(N):
        good = 0 <= at[n] <= at[n + 1] <= 80
        if good:
            owned[at[n]:at[n + 1]] = True
        assert (kc[n] == 7.0).all() != good and (vc[n] == 7.0).all() != good
    for x in (b["o"], *grads.values()):
        assert (x.cpu()[~owned] == 7.0).all()


def test_bad_offsets_without_rows_are_reported(cuda_device):
    q = torch.zeros(0, 2, 64, dtype=BF16, device=cuda_device)
    kc = torch.full((2, 3, 2, 64), 7.0, dtype=BF16, device=cuda_device)
    for ends, code in (((0, 0, 0), 0), ((0, 0, 1), 1), ((-1, -1, -1), 1)):
        cu = torch.tensor(ends, dtype=torch.int32, device=cuda_device)
        o = carve.carve_swa_fwd(q, q, q, window=3, cu_seqlens=cu)
        assert carve.carve_check() == code
        carve.carve_swa_bwd(q, q, q, o["o"], o["lse"], q, window=3, cu_seqlens=cu)
        assert carve.carve_check() == code
        carve.carve_swa_fill(q, q, kc, kc.clone(), window=3, cu_seqlens=cu)
        assert carve.carve_check() == code and (kc == 7.0).all()
        gl = torch.zeros(0, 2, dtype=BF16, device=cuda_device)
        carve.carve_gdr_fwd(q, q, q, gl, gl, cu_seqlens=cu)
        assert carve.carve_check() == code


def delta_definition(q, k, v, g, w, A_dec=None, tau=None, S0=None):
    """mixer_reference.delta with a softplus whose gradient is finite for any logit (there it divides
    e^x by 1 + e^x, which is no number between 710 and 1e9)."""
    T, Hv, dv = v.shape
    q, k = (y.repeat_interleave(Hv // k.shape[1], 1) for y in (q, k))
    x = g if tau is None else g + tau
    a = torch.exp(-torch.logaddexp(x, torch.zeros_like(x)) * (1.0 if A_dec is None else torch.exp(A_dec)))
    w = torch.sigmoid(w)
    S = torch.zeros(Hv, dv, k.shape[2], dtype=torch.float64) if S0 is None else S0
    o = []
    for t in range(T):
        S = S * a[t][:, None, None]
        S = S + (w[t][:, None] * (v[t] - (S * k[t][:, None, :]).sum(-1)))[:, :, None] * k[t][:, None, :]
        o.append((S * q[t][:, None, :]).sum(-1))
    return torch.stack(o), S


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("logit", [30.0, 1e3, 1e4, 1e5, 3e38], ids=str)
@pytest.mark.parametrize("full", [False, True], ids=["plain", "full"])
def test_delta_tokens_that_reset_the_state(cuda_device, dt, logit, full):
    """Mild decays (0.95 a token) with a token in ten that clears the state: what follows it within its chunk is
    as accurate as elsewhere.  Tolerances as in test_gpu_mixers.py: fp32 1e-5; bf16 states 2e-5, results 4 u
    and 8 u."""
    T, Hk, Hv, dk, dv = 200, 2, 4, 128, 64
    s = delta_inputs(T, Hk, Hv, dk, dv, dt, 71)
    g = torch.Generator().manual_seed(72)
    r = lambda *n: torch.randn(*n, generator=g, dtype=torch.float32).double()  # noqa: E731
    s["g"] = torch.where(torch.rand(T, Hv, generator=g) < 0.1, torch.tensor(logit, dtype=dt).double(), s["g"])
    A_dec, tau, S0, dS = (0.3 * r(Hv), 0.5 * r(Hv), 0.2 * r(Hv, dv, dk), r(Hv, dv, dk)) if full else (None,) * 4
    dev = lambda x: None if x is None else x.float().to(cuda_device)  # noqa: E731
    x = [s[n].to(dt).to(cuda_device)[None] for n in ("q", "k", "v", "g", "w", "dO")]
    more = dict(A_dec=dev(A_dec), tau=dev(tau))
    out = carve.carve_gdr_fwd(*x[:5], S0=dev(S0[None]) if full else None, **more)
    gr = carve.carve_gdr_bwd(*x[:5], out["saved"], x[5], dS_final=dev(dS[None]) if full else None, **more)
    inp = dict(q=s["q"], k=s["k"], v=s["v"], g=s["g"], w=s["w"], A_dec=A_dec, tau=tau, S0=S0)
    want_o, want_S = delta_definition(**inp)
    wg = R.grads(delta_definition, inp, (s["dO"], dS))
    u, f32 = U[BF16], dt == torch.float32
    pairs = dict(o=(out["o"][0], want_o, 4 * u), S=(out["S_final"][0], want_S, 2e-5), dq=(gr["dq"][0], wg["q"], 4 * u),
                 dk=(gr["dk"][0], wg["k"], 8 * u), dv=(gr["dv"][0], wg["v"], 4 * u), dg=(gr["dg_logit"][0], wg["g"], 8 * u),
                 dw=(gr["dw_logit"][0], wg["w"], 8 * u))
    if full:   # dS0 is nearly all cleared: one rounding of each chunk's factors
        pairs.update(dS0=(gr["dS0"][0], wg["S0"], 4 * u), dA=(gr["dA_dec"], wg["A_dec"], 8 * u), dtau=(gr["dtau"], wg["tau"], 8 * u))
    for n, (got, want, lim) in pairs.items():
        lim = (8e-5 if n in ("dA", "dtau") else 1e-5) if f32 else lim
        assert rel(got, want) <= lim, (n, rel(got, want), lim)


def test_out_may_hold_none_and_refuses_what_is_no_tensor(cuda_device):
    x = delta_tensors((1, 70), 2, 2, 64, 64, 45, cuda_device)
    q, k, v, dO = window_tensors((1, 70), 2, 2, 64, 45, cuda_device)
    want = carve.carve_gdr_fwd(*x[:5])
    got = carve.carve_gdr_fwd(*x[:5], out=dict(o=None, S_final=None, saved=None))
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["S_final"], want["S_final"])
    a = carve.carve_swa_fwd(q, k, v, window=9, out=dict(o=None, lse=None))
    g = carve.carve_swa_bwd(q, k, v, a["o"], a["lse"], dO, window=9, out=dict(dq=None))
    assert torch.equal(g["dq"], carve.carve_swa_bwd(q, k, v, a["o"], a["lse"], dO, window=9)["dq"])
    for out in (dict(o=[1.0]), dict(S_final=np.zeros(3)), dict(saved="x"), [1, 2], 5):
        with pytest.raises(TypeError):
            carve.carve_gdr_fwd(*x[:5], out=out)


@pytest.mark.parametrize("Hk,Hv,dk,dv,seed", [(1, 2, 128, 128, 81), (2, 2, 64, 128, 82), (1, 1, 128, 64, 83), (2, 4, 64, 64, 84)])
@pytest.mark.parametrize("kind", ["mild", "resets"])
def test_delta_bf16_by_the_number_of_its_roundings(cuda_device, Hk, Hv, dk, dv, seed, kind):
    """A rounding to bf16 is off by at most u, evenly spread, so u / sqrt(3) in the L2 norm; n independent
    ones sqrt(n) times that, and half as much again where terms of either sign cancel.  n, the result's own
    among them: o (A) 2; dq (S0, U, P1) 4; dk (S0, dS1, U, dY, P1, P2) 7; dv (A) 2; gates' g (S0, dS1, U, dY) 5,
    w (U, dY) 3.  The gates' gradients by blocks of 16 tokens and heads too, so that a term that only some
    tokens have cannot hide; amplitude and bias against the sum of their terms' sizes."""
    T = 260
    s = delta_inputs(T, Hk, Hv, dk, dv, BF16, seed)
    g = torch.Generator().manual_seed(seed)
    r = lambda *n: torch.randn(*n, generator=g, dtype=torch.float32).double()  # noqa: E731
    if kind == "resets":
        s["g"] = torch.where(torch.rand(T, Hv, generator=g) < 0.03, torch.tensor(200.0, dtype=torch.float64), s["g"])
    A_dec, tau, S0, dS = 0.3 * r(Hv), 0.5 * r(Hv), 0.2 * r(Hv, dv, dk), r(Hv, dv, dk)
    dev = lambda x: x.float().to(cuda_device)  # noqa: E731
    x = [s[n].to(BF16).to(cuda_device)[None] for n in ("q", "k", "v", "g", "w", "dO")]
    more = dict(A_dec=dev(A_dec), tau=dev(tau))
    out = carve.carve_gdr_fwd(*x[:5], S0=dev(S0[None]), **more)
    gr = carve.carve_gdr_bwd(*x[:5], out["saved"], x[5], dS_final=dev(dS[None]), **more)
    inp = dict(q=s["q"], k=s["k"], v=s["v"], g=s["g"], w=s["w"], A_dec=A_dec, tau=tau, S0=S0)
    want_o, want_S = delta_definition(**inp)
    wg = R.grads(delta_definition, inp, (s["dO"], dS))
    u = U[BF16]
    lim = lambda n: 1.5 * (n / 3) ** 0.5 * u  # noqa: E731
    assert rel(out["S_final"][0], want_S) <= 2e-5
    for name, got, want, n in (("o", out["o"], want_o, 2), ("dq", gr["dq"], wg["q"], 4), ("dk", gr["dk"], wg["k"], 7),
                               ("dv", gr["dv"], wg["v"], 2), ("dg", gr["dg_logit"], wg["g"], 5), ("dw", gr["dw_logit"], wg["w"], 3)):
        assert rel(got[0], want) <= lim(n), (name, rel(got[0], want), lim(n))
    for name, got, want, n in (("dg", gr["dg_logit"], wg["g"], 5), ("dw", gr["dw_logit"], wg["w"], 3)):
        err = got[0].double().cpu() - want
        size = (want.square().mean(0)).sqrt()   # of a token's gradient, by head
        for t in range(0, T, 16):
            e, w = err[t:t + 16].norm(dim=0), want[t:t + 16].norm(dim=0)
            # 16 tokens spread about twice as wide as all of them; a block whose own gradients are small still
            # carries the roundings of what passes through it: half of an average token's for each
            assert (e <= 2 * lim(n) * (w + 0.5 * size * 4)).all(), (name, t, (e / (w + 2 * size)).max().item())
    softplus = torch.logaddexp(s["g"] + tau, torch.zeros(1, dtype=torch.float64))
    slope = torch.sigmoid(s["g"] + tau)
    for name, got, want, terms in (("dtau", gr["dtau"], wg["tau"], wg["g"]), ("dA", gr["dA_dec"], wg["A_dec"], wg["g"] / slope * softplus)):
        assert ((got.double().cpu() - want).abs() <= lim(5) * terms.abs().sum(0)).all(), (name, got, want)


@pytest.mark.parametrize("Hq,Hkv,d,W,sinks", [(4, 2, 128, 64, 4), (3, 3, 64, 33, 16), (2, 1, 64, 128, 1)])
def test_window_gradients_of_sinks_in_sequences_far_beyond_the_window(cuda_device, Hq, Hkv, d, W, sinks):
    """A sink's gradients sum over every query; bf16 against fp64, tolerances as in test_gpu_mixers.py."""
    lens = (1500, 700)
    seqs = [window_inputs(T, Hq, Hkv, d, BF16, 90 + n) for n, T in enumerate(lens)]
    q, k, v, dO = (torch.cat([s[n] for s in seqs]).to(BF16).to(cuda_device) for n in ("q", "k", "v", "dO"))
    at = dict(window=W, sinks=sinks, cu_seqlens=offsets(lens, cuda_device))
    out = carve.carve_swa_fwd(q, k, v, **at)
    gr = carve.carve_swa_bwd(q, k, v, out["o"], out["lse"], dO, **at)
    row = 0
    for T, s in zip(lens, seqs):
        inp = {x: s[x] for x in ("q", "k", "v")}
        want, lse = R.window(**inp, win=W, sinks=sinks)
        wg = R.grads(lambda q, k, v: R.window(q, k, v, W, sinks)[:1], inp, (s["dO"],))
        mass = R.window_masses(**inp, dO=s["dO"], win=W, sinks=sinks)
        part = slice(row, row + T)
        near(out["o"][part], want, mass["o"], 2, T, d, BF16)
        assert (out["lse"][part].double().cpu() - lse).abs().max() <= 1e-4
        near(gr["dv"][part], wg["v"], mass["dv"], 2, T * Hq // Hkv, d, BF16)
        near(gr["dq"][part], wg["q"], mass["dq"], 3, T, d, BF16)
        near(gr["dk"][part], wg["k"], mass["dk"], 3, T * Hq // Hkv, d, BF16)
        row += T


LARGEST = 2 ** 31 - 1


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("W,sinks,scale", [(LARGEST, 0, None), (1, LARGEST, None), (LARGEST, LARGEST, None), (40, 3, 0.0)], ids=str)
def test_window_arguments_at_their_ends(cuda_device, dt, W, sinks, scale):
    """The largest window and sink counts see everything before a token; scale 0 weighs all seen keys alike."""
    T, Hq, Hkv, d = 300, 2, 1, 64
    s = window_inputs(T, Hq, Hkv, d, dt, 95)
    q, k, v, dO = (s[n].to(dt).to(cuda_device)[None] for n in ("q", "k", "v", "dO"))
    at = dict(window=W, sinks=sinks, scale=scale)
    out = carve.carve_swa_fwd(q, k, v, **at)
    gr = carve.carve_swa_bwd(q, k, v, out["o"], out["lse"], dO, **at)
    inp = {x: s[x] for x in ("q", "k", "v")}
    want, lse = R.window(**inp, win=W, sinks=sinks, scale=scale)
    wg = R.grads(lambda q, k, v: R.window(q, k, v, W, sinks, scale)[:1], inp, (s["dO"],))
    mass = R.window_masses(**inp, dO=s["dO"], win=W, sinks=sinks, scale=scale)
    near(out["o"][0], want, mass["o"], 2, T, d, dt)
    assert (out["lse"][0].double().cpu() - lse).abs().max() <= 1e-4
    near(gr["dv"][0], wg["v"], mass["dv"], 2, T * Hq // Hkv, d, dt)
    near(gr["dq"][0], wg["q"], mass["dq"], 3, T, d, dt)
    near(gr["dk"][0], wg["k"], mass["dk"], 3, T * Hq // Hkv, d, dt)


@pytest.mark.parametrize("dt", TYPES, ids=ids)
def test_window_steps_at_far_positions(cuda_device, dt):
    """Positions beyond 2^32 reach the slots that they stand for: as at the small position of the same slot."""
    W, sinks, Hq, Hkv, d = 37, 3, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(97)
    r = lambda *s: torch.randn(*s, generator=g, device=cuda_device).to(dt)  # noqa: E731
    q, k, v, kc, vc = r(3, Hq, d), r(3, Hkv, d), r(3, Hkv, d), r(3, sinks + W, Hkv, d), r(3, sinks + W, Hkv, d)
    near_pos = torch.tensor([W + 5, W + 6, 2 * W + 1], device=cuda_device)
    got = []
    for far in (0, 2 ** 32 // W * W + W, 2 ** 50 // W * W):
        a, b = kc.clone(), vc.clone()
        got.append([carve.carve_swa_step(q, k, v, a, b, near_pos + far, window=W, sinks=sinks), a, b])
    for x in got[1:]:
        assert all(torch.equal(y, z) for y, z in zip(got[0], x))
    for n, p in enumerate(near_pos.tolist()):
        assert torch.equal(got[0][1][n, sinks + (p - sinks) % W], k[n])


@pytest.mark.parametrize("dt", TYPES, ids=ids)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("lens,first", [((70, 50, 30), 0), ((130, 1, 64, 3), 37)], ids=str)
def test_a_sequence_that_is_not_finite_stays_alone(cuda_device, dt, bad, lens, first):
    """Packed rows that start behind row 0; one sequence, and the rows of none, hold no finite value in any input.
    The other sequences' results keep every bit, and the rows of no sequence stay as they were."""
    cu = offsets(lens, cuda_device) + first
    total, sick = first + sum(lens) + 5, 1
    at = cu.tolist()
    Hk, Hv, dk, dv = 2, 4, 128, 64
    x = [y.to(dt) for y in delta_tensors((total,), Hk, Hv, dk, dv, 98, cuda_device)]
    y = [z.to(dt) for z in window_tensors((total,), 4, 2, 64, 98, cuda_device)]

    def spoil(t):
        t = t.clone()
        t[:first] = bad
        t[at[sick]:at[sick + 1]] = bad
        t[at[-1]:] = bad
        return t

    def run(x, y):
        mark = lambda t: torch.full_like(t, 7.0)  # noqa: E731
        out = carve.carve_gdr_fwd(*x[:5], cu_seqlens=cu, out=dict(o=mark(x[2])))
        g = carve.carve_gdr_bwd(*x[:5], out["saved"], x[5], cu_seqlens=cu, out={n: mark(x[i]) for n, i in
                                (("dq", 0), ("dk", 1), ("dv", 2), ("dg_logit", 3), ("dw_logit", 4))})
        W = dict(window=20, sinks=2, cu_seqlens=cu)
        b = carve.carve_swa_fwd(*y[:3], out=dict(o=mark(y[0])), **W)
        gb = carve.carve_swa_bwd(*y[:3], b["o"], b["lse"], y[3], out=dict(dq=mark(y[0]), dk=mark(y[1]), dv=mark(y[2])), **W)
        return [out["o"], *(g[n] for n in ("dq", "dk", "dv", "dg_logit", "dw_logit")), b["o"], *gb.values()], [out["S_final"], g["dS0"]]

    rows, states = run(x, y)
    rows2, states2 = run([spoil(t) for t in x], [spoil(t) for t in y])
    for a, b in zip(rows, rows2):
        assert (b[:first] == 7.0).all() and (b[at[-1]:] == 7.0).all()
        for n in range(len(lens)):
            if n != sick:
                assert torch.equal(a[at[n]:at[n + 1]], b[at[n]:at[n + 1]])
    for a, b in zip(states, states2):
        for n in range(len(lens)):
            assert n == sick or torch.equal(a[n], b[n])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_delta_prompts_on_many_streams_at_once(cuda_device, dk, dv):
    """Preparations and sweeps of eight calls share the SMs and their tensor memory: each call's result is what
    it is alone, and no wait runs out."""
    xs = [delta_tensors((6, 300), 4, 8, dk, dv, 110 + n, cuda_device) for n in range(8)]
    alone = [carve.carve_gdr_fwd(*x[:5], save_for_bwd=False) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        got = [carve.carve_gdr_fwd(*x[:5], save_for_bwd=False, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a["o"], b["o"]) and torch.equal(a["S_final"], b["S_final"])


def test_tensors_beyond_2_to_the_31_elements(cuda_device):
    """Packed rows, states and caches whose last elements lie behind 2^31 (caches 2^32): the last sequence's results
    are the ones that it gives alone, bit for bit."""
    H, d, tail = 16, 128, 500
    rows = 2 ** 31 // (H * d) + 4000
    first = rows - tail
    g = torch.Generator(device="cuda").manual_seed(120)

    def normal(*s):
        return torch.empty(*s, dtype=BF16, device=cuda_device).normal_(generator=g)

    last = lambda xs: [x[first:].clone() for x in xs]  # noqa: E731
    cu = offsets((first, tail), cuda_device)
    x = [normal(rows, H, d) for _ in range(3)] + [normal(rows, H), normal(rows, H), normal(rows, H, d)]
    for i in (0, 1):
        x[i] /= d ** 0.5
    at = dict(window=64, sinks=0)   # without sinks, which every query of the long sequence would see
    b = carve.carve_swa_fwd(*x[:3], cu_seqlens=cu, **at)
    gb = carve.carve_swa_bwd(*x[:3], b["o"], b["lse"], x[5], cu_seqlens=cu, **at)
    y = last(x)
    one = offsets((tail,), cuda_device)
    c = carve.carve_swa_fwd(*y[:3], cu_seqlens=one, **at)
    assert torch.equal(b["o"][first:], c["o"]) and torch.equal(b["lse"][first:], c["lse"])
    gc = carve.carve_swa_bwd(*y[:3], c["o"], c["lse"], y[5], cu_seqlens=one, **at)
    # dk, dv: a pass of few keys is summed in parts, so equal but for the rounding of the result (half a step each)
    assert torch.equal(gb["dq"][first:], gc["dq"])
    for n in ("dk", "dv"):
        assert rel(gb[n][first:], gc[n].double().cpu()) <= 2 * U[BF16], n
    del b, gb
    a = delta_both(x, cu)
    z = delta_both(y, one)
    for n in ("o", "dq", "dk", "dv", "dg_logit", "dw_logit"):
        assert torch.equal(a[n][first:], z[n]), n
    for n in ("S", "dS0"):
        assert torch.equal(a[n][1:], z[n]), n
    del a, x
    B, W, Hkv = 33, 65536 * 2, 8
    kc = torch.zeros(B, W, Hkv, d, dtype=BF16, device=cuda_device)
    assert kc.numel() > 2 ** 32
    vc = torch.zeros_like(kc)
    kc[-1].normal_(generator=g)
    vc[-1].normal_(generator=g)
    q, k, v = normal(B, 2 * Hkv, d), normal(B, Hkv, d), normal(B, Hkv, d)
    pos = torch.full((B,), W - 1, dtype=torch.int64, device=cuda_device)
    pos[:-1] = 0
    k1, v1 = kc[-1:].clone(), vc[-1:].clone()
    o = carve.carve_swa_step(q, k, v, kc, vc, pos, window=W)
    o1 = carve.carve_swa_step(q[-1:].clone(), k[-1:].clone(), v[-1:].clone(), k1, v1, pos[-1:].clone(), window=W)
    # one sequence alone may be split over more parts: a rounding of the result, and of each part's p
    assert rel(o[-1:], o1.double().cpu()) <= 2 * U[BF16]
    assert torch.equal(kc[-1:], k1) and torch.equal(vc[-1:], v1)
    del kc, vc, k1, v1
    S = torch.zeros(9000, 16, 128, 128, device=cuda_device)
    assert S.numel() > 2 ** 31
    S[-1].normal_(generator=g)
    S1 = S[-1:].clone()
    t = [normal(9000, 16, 128) / 11, normal(9000, 16, 128) / 11, normal(9000, 16, 128), normal(9000, 16), normal(9000, 16)]
    o = carve.carve_gdr_step(*t, S)
    o1 = carve.carve_gdr_step(*(y[-1:].clone() for y in t), S1)
    assert torch.equal(o[-1:], o1) and torch.equal(S[-1:], S1)
    del S, t, o
    torch.cuda.empty_cache()   # some 60 GB that the next tests do not need
