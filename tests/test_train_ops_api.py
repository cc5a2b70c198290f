"""Refusals of the layer norm, rotary position and orthogonalisation entry points (no GPU): every bad
argument is turned down on the host before anything is enqueued."""
import ctypes

import pytest
import torch

from linear_attention_split_b200 import build, ttt

FAKE = ctypes.c_void_p(0x100000)      # 16-byte aligned, never dereferenced: checks fail first
MISALIGNED = ctypes.c_void_p(0x100008)
ODD = ctypes.c_void_p(0x100001)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    build.build()
    return ttt.lib()


def test_new_entry_points_are_declared(L):
    names = set(ttt.declared_functions())
    for n in ("ttt_layernorm", "ttt_layernorm_bwd", "ttt_layernorm_bwd_workspace_bytes", "ttt_rope", "ttt_orthogonalize",
              "ttt_orthogonalize_workspace_bytes", "ttt_linear_fullbatch_orth",
              "ttt_linear_fullbatch_orth_workspace_bytes"):
        assert n in names and hasattr(L, n)


@pytest.mark.parametrize("change,want", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(gamma=None), INVALID), (dict(x=MISALIGNED), INVALID),
    (dict(gamma=MISALIGNED), INVALID), (dict(beta=MISALIGNED), INVALID), (dict(rows=0), INVALID), (dict(C=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(dt=2), INVALID),
    (dict(C=16385), UNSUPPORTED)])
def test_layernorm_refusals(L, change, want):
    a = dict(x=FAKE, gamma=FAKE, beta=None, y=FAKE, rows=4, C=64, eps=1e-6, dt=1) | change
    assert L.ttt_layernorm(a["x"], a["gamma"], a["beta"], a["y"], a["rows"], a["C"], a["eps"], a["dt"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(dy=None), INVALID), (dict(dx=MISALIGNED), INVALID), (dict(dgamma=None), INVALID),
    (dict(dgamma=MISALIGNED), INVALID), (dict(dbeta=MISALIGNED), INVALID), (dict(rows=-2), INVALID),
    (dict(eps=-0.5), INVALID), (dict(C=20000), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nb=8), WORKSPACE),
    (dict(ws=MISALIGNED), INVALID)])
def test_layernorm_bwd_refusals(L, change, want):
    a = dict(dy=FAKE, x=FAKE, gamma=FAKE, dx=FAKE, dgamma=FAKE, dbeta=None, rows=4, C=64, eps=1e-6, dt=1, ws=FAKE,
             nb=1 << 30) | change
    assert L.ttt_layernorm_bwd(a["dy"], a["x"], a["gamma"], a["dx"], a["dgamma"], a["dbeta"], a["rows"], a["C"], a["eps"],
                               a["dt"], a["ws"], a["nb"], None) == want


def rope(L, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=None, pb=0, grid=(4, 4), dims=(32, 32), B=1, H=2, N=16, d=64, base=1e4,
         strides=None, dt=1, axes=None):
    ints = lambda v: None if v is None else (ctypes.c_int * max(1, len(v)))(*v)  # noqa: E731
    st = None if strides is None else (ctypes.c_longlong * 12)(*strides)
    n = len(dims) if axes is None else axes
    return L.ttt_rope(q, k, qo, ko, pos, pb, ints(grid), ints(dims), n, B, H, N, d, base, 0, 0, st, dt, None)


DENSE = (2048, 1024, 64)


@pytest.mark.parametrize("change,want", [
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID), (dict(ko=None), INVALID),
    (dict(q=ODD), INVALID), (dict(dt=9), INVALID), (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(d=0), INVALID),
    (dict(axes=0), INVALID), (dict(dims=(31, 33)), INVALID), (dict(dims=(32, 34)), INVALID), (dict(dims=(0, 64)), INVALID),
    (dict(dims=(-2, 64)), INVALID), (dict(grid=(4, 5)), INVALID), (dict(grid=(0, 16)), INVALID), (dict(grid=(-4, -4)), INVALID),
    (dict(grid=(1 << 20, 1 << 20)), INVALID), (dict(grid=None), INVALID), (dict(pos=FAKE), INVALID),
    (dict(pos=ctypes.c_void_p(0x100002), grid=None), INVALID), (dict(base=0.0), INVALID), (dict(base=NAN), INVALID),
    (dict(base=-2.0), INVALID), (dict(d=514), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(H=65536), UNSUPPORTED),
    (dict(dims=(2,) * 5, grid=(16, 1, 1, 1, 1)), UNSUPPORTED),
    # an output that addresses an element twice, a negative stride, in place with other strides
    (dict(strides=DENSE * 2 + (2048, 0, 64) + DENSE, B=1), INVALID),
    (dict(strides=DENSE * 2 + (2048, 1024, 63) + DENSE), INVALID),
    (dict(strides=(2048, -1024, 64) + DENSE * 3), INVALID),
    (dict(strides=(2048, 64, 128) + DENSE * 3), INVALID)])
def test_rope_refusals(L, change, want):
    assert rope(L, **change) == want


def orth(L, x=FAKE, out=FAKE, U=1, m=8, n=8, steps=5, coef=ttt.NS_COEF, eps=1e-7, scale=1.0, dt=0, ws=FAKE, nb=1 << 30):
    return L.ttt_orthogonalize(x, out, U, m, n, steps, *coef, eps, scale, dt, ws, nb, None)


@pytest.mark.parametrize("change,want", [
    (dict(x=None), INVALID), (dict(out=MISALIGNED), INVALID), (dict(U=0), INVALID), (dict(m=-1), INVALID), (dict(n=0), INVALID),
    (dict(steps=0), INVALID), (dict(steps=65), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(coef=(NAN, 0.0, 0.0)), INVALID), (dict(dt=5), INVALID),
    (dict(coef=(4.0, 0.0, 0.0)), UNSUPPORTED), (dict(coef=(3.4445, 4.775, 2.0315)), UNSUPPORTED),
    (dict(coef=(2.0, -40.0, 39.0)), UNSUPPORTED), (dict(U=65536), UNSUPPORTED), (dict(m=32769), UNSUPPORTED),
    (dict(ws=None, m=80, n=80), WORKSPACE), (dict(nb=16, n=257), WORKSPACE), (dict(ws=MISALIGNED), INVALID)])
def test_orthogonalize_refusals(L, change, want):
    assert orth(L, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(q=None), INVALID), (dict(q=MISALIGNED), INVALID), (dict(w0=None), INVALID), (dict(wst=MISALIGNED), INVALID),
    (dict(B=0), INVALID), (dict(N=-1), INVALID), (dict(eta=NAN), INVALID), (dict(eps=-1.0), INVALID), (dict(steps=0), INVALID),
    (dict(d=129), UNSUPPORTED), (dict(coef=(9.0, 0.0, 0.0)), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(nb=100), WORKSPACE), (dict(ws=MISALIGNED), INVALID)])
def test_linear_orth_refusals(L, change, want):
    a = dict(q=FAKE, w0=FAKE, wst=None, B=1, H=1, N=16, d=64, eta=0.1, steps=5, coef=ttt.NS_COEF, eps=1e-7, ws=FAKE,
             nb=1 << 40) | change
    assert L.ttt_linear_fullbatch_orth(a["q"], FAKE, FAKE, a["w0"], FAKE, a["wst"], a["B"], a["H"], a["N"], a["d"],
                                       a["eta"], a["steps"], *a["coef"], a["eps"], 1, a["ws"], a["nb"], None) == want


def test_workspace_queries(L):
    assert L.ttt_layernorm_bwd_workspace_bytes(0, 64, 1) == 0
    assert L.ttt_layernorm_bwd_workspace_bytes(1, 64, 1) >= 2 * 64 * 4
    assert L.ttt_orthogonalize_workspace_bytes(1, 0, 4, 0) == 0
    assert L.ttt_orthogonalize_workspace_bytes(3, 64, 256, 0) == 0  # a block's shared memory holds it
    assert L.ttt_orthogonalize_workspace_bytes(1, 65, 65, 0) > 0
    assert L.ttt_orthogonalize_workspace_bytes(1, 257, 64, 1) > 0
    assert L.ttt_linear_fullbatch_orth_workspace_bytes(1, 1, 16, 64, 1) > 0


def test_binding_refuses_before_the_library():
    x, g = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError):  # not CUDA tensors
        ttt.layernorm(x, g)
    q = torch.zeros(1, 2, 16, 64)
    with pytest.raises(ValueError):  # neither grid nor positions
        ttt.rope(q, q, (32, 32))
    with pytest.raises(ValueError):  # both
        ttt.rope(q, q, (32, 32), grid=(4, 4), pos=torch.zeros(16, 2))
    with pytest.raises(ValueError):  # one size per axis
        ttt.rope(q, q, (32, 32), grid=(16,))
    with pytest.raises(ValueError):  # shapes differ
        ttt.rope(q, torch.zeros(1, 1, 16, 64), (32, 32), grid=(4, 4))
    with pytest.raises(TypeError):
        ttt.rope(q, q.double(), (32, 32), grid=(4, 4))
    with pytest.raises(TypeError):
        ttt.rope(q.half(), q.half(), (32, 32), grid=(4, 4))
    with pytest.raises(ValueError):  # features not adjacent
        ttt.rope(q.transpose(2, 3), q.transpose(2, 3), (8, 8), grid=(8, 8))
