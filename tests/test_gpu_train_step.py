"""A training step made of the new operators and the layer (GPU): norm, projection, rotary positions,
TTT-Linear, its backward pass, the way back, and the orthogonalised update of the inner weights --
eagerly, on another stream, and captured into a graph -- against autograd in 64 bits."""
import math

import pytest
import torch

from linear_attention_split_b200 import ttt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS, ETA, DIMS, GRID = 1e-6, 1.0, (32, 32), (9, 11)
B, H, D = 2, 2, 64
N, C = GRID[0] * GRID[1], H * D


def draw(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(B, N, C).to(DEV), gamma=(1 + 0.1 * r(C)).to(DEV), beta=(0.1 * r(C)).to(DEV),
                w=(r(C, 3 * C) / math.sqrt(C * D)).to(DEV), w0=(r(H, D, D) / math.sqrt(D)).to(DEV),
                dout=(r(B, H, N, D) / math.sqrt(D)).to(DEV))


def step(s):
    """One pass; everything the library computes, in fp32."""
    y = ttt.layernorm(s["x"], s["gamma"], s["beta"], EPS)
    qkv = (y.view(-1, C) @ s["w"]).view(B, N, 3, H, D)
    q, k = ttt.rope(qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2), DIMS, grid=GRID)
    v = qkv[:, :, 2].transpose(1, 2).contiguous()
    out = ttt.linear_fullbatch(q, k, v, s["w0"], ETA)
    dq, dk, dv, dw0 = ttt.linear_fullbatch_bwd(q, k, v, s["w0"], s["dout"], ETA)
    dqkv = torch.empty_like(qkv)
    ttt.ttt_rope(dq, dk, dqkv[:, :, 0].transpose(1, 2), dqkv[:, :, 1].transpose(1, 2), DIMS, grid=GRID, inverse=True)
    dqkv[:, :, 2].copy_(dv.transpose(1, 2))
    dy = (dqkv.view(-1, 3 * C) @ s["w"].t()).view(B, N, C)
    dw = y.view(-1, C).t() @ dqkv.view(-1, 3 * C)
    dx, dgamma, dbeta = ttt.layernorm_bwd(dy, s["x"], s["gamma"], EPS)
    return dict(out=out, dx=dx, dgamma=dgamma, dbeta=dbeta, dw=dw, dw0=dw0, upd0=ttt.orthogonalize(dw0),
                upd=ttt.orthogonalize(dw))


def rotate64(x):
    pos = torch.stack(torch.meshgrid(*[torch.arange(n, device=DEV).double() for n in GRID], indexing="ij"), -1).view(N, 2)
    parts, at = [], 0
    for a, w in enumerate(DIMS):
        ang = pos[:, a, None] * 10000.0 ** (-2.0 * torch.arange(w // 2, device=DEV).double() / w)
        x1, x2 = x[..., at:at + w // 2], x[..., at + w // 2:at + w]
        parts += [x1 * ang.cos() - x2 * ang.sin(), x2 * ang.cos() + x1 * ang.sin()]
        at += w
    return torch.cat(parts, -1)


def orth64(x):
    x = x / torch.linalg.matrix_norm(x)[..., None, None]
    a, b, c = ttt.NS_COEF
    for _ in range(5):
        g = x @ x.mT
        x = a * x + (b * g + c * g @ g) @ x
    return x


def step64(s):
    t = {n: v.double().requires_grad_() for n, v in s.items() if n != "dout"}
    xc = t["x"] - t["x"].mean(-1, keepdim=True)
    y = xc / (xc.square().mean(-1, keepdim=True) + EPS).sqrt() * t["gamma"] + t["beta"]
    qkv = (y @ t["w"]).view(B, N, 3, H, D).permute(2, 0, 3, 1, 4)
    q, k, v = rotate64(qkv[0]), rotate64(qkv[1]), qkv[2]
    w = t["w0"] - ETA / N * (k.mT @ k @ t["w0"] - k.mT @ v)
    out = q @ w
    g = torch.autograd.grad(out, [t[n] for n in ("x", "gamma", "beta", "w", "w0")], s["dout"].double())
    r = dict(zip(("dx", "dgamma", "dbeta", "dw", "dw0"), g), out=out.detach())
    return r | dict(upd0=orth64(r["dw0"]), upd=orth64(r["dw"]))


def check(got, s):
    # fp32 throughout.  Each link is within 1e-5 of its own norm, a chain of at most eight of them and the
    # products' sums within 1e-4; an orthogonal factor magnifies its input's error by up to
    # 3.4445^5 / (0.7 sqrt(r)) = 87 at r = 64, so 2e-3 bounds it with an input good to 2e-5.
    want = step64(s)
    for n, w in want.items():
        rel = ((got[n].double() - w).norm() / w.norm()).item()
        assert rel <= (2e-3 if n.startswith("upd") else 1e-4), (n, rel)


def test_training_step():
    s = draw()
    check(step(s), s)
    assert ttt.device_error() == 0


def test_training_step_on_another_stream():
    s = draw(1)
    want = step(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(s)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], want[n]) for n in want)


def test_training_step_captured_and_replayed():
    s = draw(2)
    step(s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):  # two graphs, each with scratch of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(s))
        graphs.append(g)
    for seed in (3, 4):
        new = draw(seed)
        for n in s:
            s[n].copy_(new[n])
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        want = step(new)
        for o in outs:
            assert all(torch.equal(o[n], want[n]) for n in want)
        check(outs[0], new)


def test_calls_on_two_streams_at_once():
    a, b = draw(5), draw(6)
    wa, wb = step(a), step(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            ga = step(a)
        with torch.cuda.stream(s2):
            gb = step(b)
    torch.cuda.synchronize()
    assert all(torch.equal(ga[n], wa[n]) for n in wa) and all(torch.equal(gb[n], wb[n]) for n in wb)


def test_explicit_stream_with_scratch_of_its_own():
    s = draw(7)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    x = torch.randn(1, 200, 300, device=DEV)
    want = ttt.orthogonalize(x)
    dy = torch.randn(B, N, C, device=DEV)
    wdx = ttt.layernorm_bwd(dy, s["x"], s["gamma"], EPS)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        out, dx, dg, db = torch.empty_like(x), torch.empty_like(dy), torch.empty_like(s["gamma"]), torch.empty_like(s["gamma"])
        torch.cuda.synchronize()
        ttt.ttt_orthogonalize(x, out, stream=stream)
        ttt.ttt_layernorm_bwd(dy, s["x"], s["gamma"], dx, dg, db, EPS, stream=stream)
        junk = [torch.full((1 << 20,), 3.0, device=DEV) for _ in range(8)]  # takes freed scratch of the current stream
        side.synchronize()
        assert torch.equal(out, want) and all(torch.equal(p, q) for p, q in zip((dx, dg, db), wdx))
        del junk


def test_calls_from_threads():
    # the binding releases the interpreter lock during a call, so these overlap on the host as well
    import threading

    cases = [draw(seed) for seed in range(20, 24)]
    want = [step(s) for s in cases]
    torch.cuda.synchronize()
    got, failed = [None] * len(cases), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got[i] = step(cases[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    # the projections are torch's own products, whose kernels may differ by thread; everything else is bitwise
    for g, w in zip(got, want):
        for n in w:
            assert torch.allclose(g[n], w[n], rtol=1e-3, atol=1e-4 * w[n].abs().max().item()), n


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from linear_attention_split_b200 import ttt
x = torch.randn(300, 96, device="cuda"); gamma = torch.ones(96, device="cuda"); dy = torch.randn_like(x)
q = torch.randn(2, 3, 20, 64, device="cuda").bfloat16(); w0 = torch.randn(3, 64, 64, device="cuda") / 8
m, h = torch.randn(1, 200, 150, device="cuda"), torch.randn(1, 200, 150, device="cuda").bfloat16()
def run():
    a, b = ttt.rope(q, q, (32, 32), grid=(4, 5))
    return [ttt.layernorm(x, gamma), *ttt.layernorm_bwd(dy, x, gamma), a, b, ttt.orthogonalize(m), ttt.orthogonalize(h),
            ttt.orthogonalize(w0), *ttt.linear_fullbatch_orth(a, b, q, w0, with_w_star=True)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = run()
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
assert all(torch.equal(s, t) for s, t in zip(captured, run()))
assert ttt.device_error() == 0
print("captured first")
"""


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
