"""What the mixers' entry points refuse, and their plain references against differences: no GPU."""
import ctypes
import os
import re

import pytest
import torch

import chunk_gated_delta_b200 as carve
from chunk_gated_delta_b200 import build, mixers
from tests import mixer_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mixers._lib()


def test_every_declared_symbol_is_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "carve_mixers.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(carve_[a-z_]+)\s*\(", src)))
    assert names == ["carve_gdr_bwd", "carve_gdr_bwd_workspace_bytes", "carve_gdr_fwd", "carve_gdr_fwd_workspace_bytes",
                     "carve_gdr_saved_bytes", "carve_gdr_step", "carve_swa_bwd", "carve_swa_bwd_workspace_bytes",
                     "carve_swa_fill", "carve_swa_fwd", "carve_swa_step"]
    for n in names:
        assert hasattr(lib, n), n


P = 1 << 20   # a pointer that no refused call follows


def gdr(**kw):
    return mixers.GdrDims(**{**dict(B=2, T=50, Hk=2, Hv=4, dk=128, dv=64, io=1, total_tokens=0), **kw})


def swa(**kw):
    return mixers.SwaDims(**{**dict(B=2, T=50, Hq=4, Hkv=2, d=64, window=8, sinks=2, io=1, scale=0.1, total_tokens=0), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hk=0), 1), (dict(Hk=3), 1), (dict(Hv=0), 1), (dict(dk=0), 1), (dict(io=2), 1),
    (dict(io=-1), 1), (dict(dk=96), 2), (dict(dv=256), 2), (dict(B=1 << 16, T=1 << 16), 2), (dict(B=1 << 20, Hv=1 << 10), 2)])
def test_delta_dims_refused(lib, kw, code):
    d = gdr(**kw)
    n = [P] * 5
    assert lib.carve_gdr_fwd(d, None, *n, None, None, None, P, P, P, P, None) == code
    assert lib.carve_gdr_bwd(d, None, *n, None, None, P, P, None, P, P, P, P, P, None, None, None, P, None) == code
    for f in (lib.carve_gdr_fwd_workspace_bytes, lib.carve_gdr_saved_bytes, lib.carve_gdr_bwd_workspace_bytes):
        assert f(d, 0) == 0
    if "T" not in kw:
        assert lib.carve_gdr_step(d, *n, None, None, P, P, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(window=0), 1), (dict(sinks=-1), 1),
    (dict(io=7), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(d=80), 2), (dict(d=0), 1),
    (dict(B=1 << 16, T=1 << 16), 2)])
def test_window_dims_refused(lib, kw, code):
    d = swa(**kw)
    assert lib.carve_swa_fwd(d, None, P, P, P, P, P, None) == code
    assert lib.carve_swa_bwd(d, None, P, P, P, P, P, P, P, P, P, P, None) == code
    assert lib.carve_swa_fill(d, None, P, P, P, P, None) == code
    assert lib.carve_swa_bwd_workspace_bytes(d, 0) == 0
    if "T" not in kw:
        assert lib.carve_swa_step(d, P, P, P, P, P, P, P, None) == code


def test_cache_beyond_its_limit_is_refused(lib):
    big = swa(window=(1 << 31) - 1, sinks=(1 << 31) - 1)
    assert lib.carve_swa_fill(big, None, P, P, P, P, None) == 2
    assert lib.carve_swa_step(big, P, P, P, P, P, P, P, None) == 2


def test_null_and_misaligned_pointers_are_refused(lib):
    bad = P + 8
    for at in range(5):
        for x in (None, bad if at < 3 else P + 1):   # gates need their element's alignment only
            n = [P] * 5
            n[at] = x
            assert lib.carve_gdr_fwd(gdr(), None, *n, None, None, None, P, P, P, P, None) == 1
            assert lib.carve_gdr_step(gdr(), *n, None, None, P, P, None) == 1
    n = [P] * 5
    assert lib.carve_gdr_fwd(gdr(), None, *n, None, None, None, P, P, None, None, None) == 1   # no buffer at all
    assert lib.carve_gdr_fwd(gdr(), P + 2, *n, None, None, None, P, P, P, P, None) == 1
    for A, dA in ((P, None), (None, P)):   # a parameter without its gradient
        assert lib.carve_gdr_bwd(gdr(), None, *n, A, None, P, P, None, P, P, P, P, P, dA, None, None, P, None) == 1
        assert lib.carve_gdr_bwd(gdr(), None, *n, None, A, P, P, None, P, P, P, P, P, None, dA, None, P, None) == 1
    assert lib.carve_swa_fwd(swa(), None, P, None, P, P, None, None) == 1
    assert lib.carve_swa_fwd(swa(), None, P, P, P, P, P + 2, None) == 1
    assert lib.carve_swa_step(swa(), P, P, P, P, P, P + 4, P, None) == 1
    assert lib.carve_swa_bwd(swa(), None, P, P, P, P, None, P, P, P, P, P, None) == 1
    assert lib.carve_swa_step(swa(), P, P, P, P, None, P, P, None) == 1
    assert lib.carve_swa_step(swa(), P, P, P, P, P, None, P, None) == 1


def test_buffers_grow_with_the_tokens_not_with_the_longest_sequence(lib):
    many = gdr(B=1000, total_tokens=4000)
    one = gdr(B=1, total_tokens=4000)
    assert lib.carve_gdr_saved_bytes(many, 1) <= 1200 * lib.carve_gdr_saved_bytes(one, 1) / 60
    assert ctypes.sizeof(mixers.GdrDims) == 40 and ctypes.sizeof(mixers.SwaDims) == 48


def _delta_args(**kw):
    t = dict(q=torch.zeros(2, 5, 2, 64), k=torch.zeros(2, 5, 2, 64), v=torch.zeros(2, 5, 4, 128),
             g_logit=torch.zeros(2, 5, 4), w_logit=torch.zeros(2, 5, 4))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,err", [
    (dict(), ValueError),                                             # not on a GPU
    (dict(q=torch.zeros(2, 5, 2, 64, dtype=torch.float16)), TypeError),
    (dict(k=torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)), TypeError),
    (dict(k=torch.zeros(2, 6, 2, 64)), ValueError),
    (dict(v=torch.zeros(2, 5, 3, 128)), ValueError),
    (dict(g_logit=torch.zeros(2, 5, 2)), ValueError),
    (dict(q=torch.zeros(2, 5, 64, 2).transpose(2, 3)), ValueError),   # strided
    (dict(A_dec=torch.zeros(4, dtype=torch.float64)), TypeError),
    (dict(cu_seqlens=torch.tensor([0, 5])), ValueError),              # packed rows have 3 dimensions
])
def test_delta_tensors_refused(kw, err):
    with pytest.raises(err):
        carve.carve_gdr_fwd(**_delta_args(**kw))


@pytest.mark.parametrize("kw,err", [
    (dict(), ValueError), (dict(window=0), ValueError), (dict(window=1 << 31), ValueError), (dict(sinks=-1), ValueError),
    (dict(k=torch.zeros(2, 5, 3, 64)), ValueError), (dict(v=torch.zeros(2, 5, 2, 128)), ValueError),
    (dict(v=torch.zeros(2, 5, 2, 64, dtype=torch.bfloat16)), TypeError)])
def test_window_tensors_refused(kw, err):
    t = dict(q=torch.zeros(2, 5, 4, 64), k=torch.zeros(2, 5, 2, 64), v=torch.zeros(2, 5, 2, 64), window=4, sinks=1)
    t.update(kw)
    with pytest.raises(err):
        carve.carve_swa_fwd(**t)


def test_packed_offsets_refused():
    t = dict(q=torch.zeros(5, 2, 64), k=torch.zeros(5, 2, 64), v=torch.zeros(5, 2, 64), window=4)
    for cu, err in ((torch.tensor([0, 5]), TypeError), (torch.tensor([0], dtype=torch.int32), ValueError),
                    (torch.zeros(2, 2, dtype=torch.int32), ValueError)):
        with pytest.raises(err):
            carve.carve_swa_fwd(cu_seqlens=cu, **t)


def test_cache_shapes_refused():
    t = dict(q=torch.zeros(2, 4, 64), k=torch.zeros(2, 2, 64), v=torch.zeros(2, 2, 64), window=8, sinks=2)
    pos = torch.zeros(2, dtype=torch.int64)
    good = torch.zeros(2, 10, 2, 64)
    for kc, p, err in ((torch.zeros(2, 9, 2, 64), pos, ValueError), (good, pos.int(), TypeError),
                       (good.bfloat16(), pos, TypeError), (good, pos, ValueError)):   # the last: not on a GPU
        with pytest.raises(err):
            carve.carve_swa_step(k_cache=kc, v_cache=good, pos=p, **t)


def _difference(f, inputs, cot, grads, seed):
    """Central differences along a random direction in every input at once against the gradient."""
    gen = torch.Generator().manual_seed(seed)
    dirs = {n: torch.randn(x.shape, generator=gen, dtype=torch.float64) for n, x in inputs.items()}

    def at(e):
        return sum((c * o).sum() for c, o in zip(cot, f(**{n: x + e * dirs[n] for n, x in inputs.items()}))).item()

    e = 1e-5   # truncation ~ e^2, cancellation ~ 1e-16 / e: both ~ 1e-10 of the values
    got = (at(e) - at(-e)) / (2 * e)
    want = sum((grads[n] * dirs[n]).sum().item() for n in inputs)
    assert abs(got - want) <= 1e-7 * max(1.0, abs(want))


def test_delta_reference_against_differences():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = dict(q=r(9, 1, 4), k=0.5 * r(9, 1, 4), v=r(9, 2, 3), g=r(9, 2), w=r(9, 2), A_dec=r(2), tau=r(2), S0=r(2, 3, 4))
    cot = (r(9, 2, 3), r(2, 3, 4))
    _difference(R.delta, x, cot, R.grads(R.delta, x, cot), 4)


def test_window_reference_against_differences():
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x = dict(q=r(12, 2, 4), k=r(12, 1, 4), v=r(12, 1, 4))
    f = lambda q, k, v: R.window(q, k, v, 3, 2)[:1]  # noqa: E731
    cot = (r(12, 2, 4),)
    _difference(f, x, cot, R.grads(f, x, cot), 6)


def test_declared_arguments_match_the_header(lib):
    """As many argument types as the C prototype has parameters: one too few would pass half a pointer."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "carve_mixers.h")).read(), flags=re.S)
    protos = dict(re.findall(r"\b(carve_[a-z_]+)\s*\(([^)]*)\)\s*;", src))
    assert len(protos) == 11
    for name, params in protos.items():
        assert len(getattr(lib, name).argtypes) == len(params.split(",")), name
