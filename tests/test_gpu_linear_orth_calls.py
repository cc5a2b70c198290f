"""Calls of the orthogonalised TTT-Linear step that its documentation allows (GPU): other steps, coefficients and
floors, values that are not finite, explicit streams and workspaces, graphs that share a workspace."""
import pytest
import torch

from linear_attention_split_b200 import inputs, ttt
from test_gpu_orth import steps64
from tolerance import assert_close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def draw(B, H, N, d, dtype, seed=0):
    return {n: t.to(DEV) for n, t in inputs.linear_inputs(B, H, N, d, dtype=dtype, seed=seed).items()}


def call(g, **kw):
    return ttt.linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], with_w_star=True, **kw)


def want64(g, eta, **kw):
    q, k, v, w0 = (g[n].double() for n in ("q", "k", "v", "w0"))
    w = w0 - eta * steps64((k.mT @ (k @ w0 - v)) / k.shape[2], **kw)
    return q @ w, w


@pytest.mark.parametrize("N,d,dtype", [(300, 64, "bf16"), (300, 64, "f32"), (150, 40, "bf16"), (150, 33, "f32"), (200, 96, "bf16"), (200, 100, "f32")])
@pytest.mark.parametrize("kw", [dict(steps=1), dict(steps=2), dict(steps=8), dict(coef=(2.0, -1.5, 0.5), steps=6), dict(coef=(1.5, -0.5, 0.0), steps=4),
                                dict(eps=10.0), dict(steps=1, coef=(1.0, 0.0, 0.0))])
def test_other_arguments(N, d, dtype, kw):
    g = draw(2, 2, N, d, dtype, seed=N + d)
    out, w = call(g, eta=-0.3, **kw)
    ro, rw = want64(g, -0.3, **kw)
    assert_close(out, ro.cpu().numpy(), DT[dtype], "O")
    assert_close(w, rw.cpu().numpy(), torch.float32, "W*")


@pytest.mark.parametrize("N,d,dtype", [(300, 64, "bf16"), (1500, 64, "f32"), (150, 40, "bf16"), (200, 96, "bf16"), (200, 100, "f32")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_values_stay_in_their_unit(N, d, dtype, bad):
    g = draw(3, 2, N, d, dtype, seed=1)
    out, w = call(g)
    for name in ("k", "v"):
        x = dict(g)
        x[name] = g[name].clone()
        x[name][1, 0, N - 1, d - 1] = bad
        o, s = call(x)
        assert o[1, 0].isnan().all() and s[1, 0].isnan().all()
        for b, h in [(0, 0), (0, 1), (1, 1), (2, 0), (2, 1)]:
            assert torch.equal(o[b, h], out[b, h]) and torch.equal(s[b, h], w[b, h])
    x = dict(g, q=g["q"].clone())
    x["q"][2, 1, N // 2, 3] = bad  # a query: its row alone
    o, s = call(x)
    assert torch.equal(s, w)
    row = torch.zeros(3, 2, N, dtype=torch.bool, device=DEV)
    row[2, 1, N // 2] = True
    assert torch.equal(o[~row], out[~row]) and not o[row].isfinite().any()
    x = dict(g, w0=g["w0"].clone())
    x["w0"][1, 0, 0] = bad  # a head: all its units
    o, s = call(x)
    assert torch.equal(o[:, 0], out[:, 0]) and torch.equal(s[:, 0], w[:, 0]) and not s[:, 1].isfinite().any()


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (48, "bf16"), (64, "f32"), (96, "f32")])
def test_explicit_streams_and_workspaces(d, dtype):
    cases = [draw(2, 3, 400, d, dtype, seed=s) for s in (1, 2)]
    want = [call(g)[0] for g in cases]
    nb = ttt.ttt_linear_fullbatch_orth_workspace_bytes(2, 3, 400, d, ttt._DT[DT[dtype]])
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w) for w in want]
    spaces = [torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV) for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):  # both at once, each on a stream and workspace of its own
        for g, o, st, ws in zip(cases, outs, streams, spaces):
            ttt.ttt_linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], o, workspace=ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for ws in (spaces[0][:nb - 1], torch.empty(nb, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            g = cases[0]
            ttt.ttt_linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], outs[0], workspace=ws)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (48, "bf16"), (96, "f32")])
def test_graphs_that_share_a_workspace(d, dtype):
    # one after the other on one stream: each finds what the other left
    cases = [draw(2, 3, 400, d, dtype, seed=3), draw(1, 2, 150, d, dtype, seed=4)]
    want = [call(g)[0] for g in cases]
    nb = max(ttt.ttt_linear_fullbatch_orth_workspace_bytes(*g["q"].shape, ttt._DT[DT[dtype]]) for g in cases)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.zeros_like(w) for w in want], []
    torch.cuda.synchronize()
    for g, o in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ttt.ttt_linear_fullbatch_orth(g["q"], g["k"], g["v"], g["w0"], o, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("U,m,n,dt", [(1, 130, 257, torch.bfloat16), (2, 300, 200, torch.float32), (1, 1024, 1024, torch.bfloat16)])
def test_orthogonalize_in_graphs_that_share_a_workspace(U, m, n, dt):
    g = torch.Generator(device=DEV).manual_seed(m)
    xs = [torch.randn(U, m, n, generator=g, device=DEV).to(dt) for _ in range(2)]
    want = [ttt.orthogonalize(x) for x in xs]
    ws = torch.full((ttt.ttt_orthogonalize_workspace_bytes(U, m, n, ttt._DT[dt]),), 0xFF, dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.zeros_like(x) for x in xs], []
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ttt.ttt_orthogonalize(x, o, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
