"""Rotary positions with several axes against complex rotations in 64 bits (GPU).

Tolerance.  The fraction of a turn is rounded to fp32 once (2^-26 turns at most: 9.4e-8 in the angle),
sincospi is good to 2 steps (2.4e-7), the two products and their sum round three times (1.8e-7):
below 5.5e-7 (|x| + |y|) of the pair, plus half a step of the output's type (bf16 2^-8).
"""
import math

import pytest
import torch

from linear_attention_split_b200 import ttt

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def coords(grid):
    axes = torch.meshgrid(*[torch.arange(n, dtype=torch.float64) for n in grid], indexing="ij")
    return torch.stack([a.reshape(-1) for a in axes], 1).to(DEV)


def rotate(x, dims, pos, base=10000.0, interleaved=False, inverse=False):
    """(result, |x| + |y| of each element's pair) in 64 bits; pos [N, axes] or [B, N, axes]."""
    x = x.double()
    pos = pos.double()
    pos = pos[None] if pos.dim() == 2 else pos
    out, size, at = x.clone(), torch.zeros_like(x), 0
    for a, s in enumerate(dims):
        for j in range(s // 2):
            i1, i2 = (at + 2 * j, at + 2 * j + 1) if interleaved else (at + j, at + j + s // 2)
            ang = pos[:, :, a] * base ** (-2.0 * j / s) * (-1 if inverse else 1)
            c, n = ang.cos()[:, None], ang.sin()[:, None]
            out[..., i1] = x[..., i1] * c - x[..., i2] * n
            out[..., i2] = x[..., i2] * c + x[..., i1] * n
            size[..., i1] = size[..., i2] = x[..., i1].abs() + x[..., i2].abs()
        at += s
    return out, size


def check(got, x, *args, **kw):
    want, size = rotate(x, *args, **kw)
    tol = HALF[x.dtype] * want.abs() + 5.5e-7 * size
    assert ((got.double() - want).abs() <= tol).all(), (got.double() - want).abs().max().item()


def draw(shape, dt, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dt).to(DEV)


CASES = [  # B, H, grid, dims, d
    (1, 1, (1,), (2,), 2), (1, 6, (14, 14), (32, 32), 64), (2, 3, (7, 5), (20, 12), 32), (2, 1, (3, 4, 5), (16, 24, 24), 64),
    (1, 2, (5, 9), (22, 42), 64), (3, 2, (17,), (48,), 64), (2, 2, (2, 2, 2, 2), (2, 4, 6, 8), 33), (1, 1, (80, 81), (24, 24), 48),
    (4, 12, (8, 6, 6), (32, 48, 48), 128), (1, 3, (9, 7), (6, 10), 17), (2, 2, (11,), (512,), 512), (1, 64, (2, 3), (64, 64), 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,grid,dims,d", CASES)
def test_rope_on_a_grid(B, H, grid, dims, d, interleaved, dtype):
    N = math.prod(grid)
    q, k = draw((B, H, N, d), DT[dtype], 1), draw((B, H, N, d), DT[dtype], 2)
    for inverse in (False, True):
        a, b = ttt.rope(q, k, dims, grid=grid, interleaved=interleaved, inverse=inverse)
        for got, x in ((a, q), (b, k)):
            check(got, x, dims, coords(grid), interleaved=interleaved, inverse=inverse)
    assert torch.equal(ttt.rope(q, None, dims, grid=grid, interleaved=interleaved, inverse=True), a)
    assert ttt.device_error() == 0


@pytest.mark.parametrize("batched", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_at_given_positions(batched, dtype):
    B, H, N, d, dims = 3, 2, 77, 64, (20, 30)
    q, k = draw((B, H, N, d), DT[dtype], 3), draw((B, H, N, d), DT[dtype], 4)
    g = torch.Generator().manual_seed(7)
    pos = (torch.rand(*((B, N, 2) if batched else (N, 2)), generator=g) * 2e5 - 1e5).to(DEV)
    pos[..., 0, :] = 0.0
    pos[..., 1, :] = 16777216.0
    for il in (False, True):
        a, b = ttt.rope(q, k, dims, pos=pos, interleaved=il, base=500.0)
        for got, x in ((a, q), (b, k)):
            check(got, x, dims, pos, interleaved=il, base=500.0)
            assert torch.equal(got[:, :, 0], x[:, :, 0])  # position zero turns nothing


STRIDES = ["qkv", "qkv_odd", "offset", "expand", "head_slice"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", STRIDES)
def test_rope_strides(layout, dtype):
    B, H, N, d, dims, dt = 2, 3, 35, 24, (12, 8), DT[dtype]
    if layout == "qkv":
        t = draw((B, N, 3, H, d), dt)
        q, k = t[:, :, 0].transpose(1, 2), t[:, :, 1].transpose(1, 2)
    elif layout == "qkv_odd":  # rows of an odd length: no vector is aligned
        t = draw((B, N, 2 * H * d + 1), dt)
        q = t[..., 1:1 + H * d].unflatten(-1, (H, d)).transpose(1, 2)
        k = t[..., 1 + H * d:].unflatten(-1, (H, d)).transpose(1, 2)
    elif layout == "offset":
        t = draw((B * H * N * d + 3,), dt)
        q, k = t[1:1 + B * H * N * d].view(B, H, N, d), t[3:].view(B, H, N, d)
    elif layout == "expand":  # one head's features for all heads
        q, k = draw((B, 1, N, d), dt).expand(B, H, N, d), draw((1, 1, 1, d), dt, 2).expand(B, H, N, d)
    else:
        q, k = draw((B, 2 * H, N, d + 8), dt)[:, ::2, :, 4:4 + d], draw((B, H, 2 * N, d), dt, 2)[:, :, ::2]
    for il in (False, True):
        want = ttt.rope(q.contiguous(), k.contiguous(), dims, grid=(5, 7), interleaved=il)
        check(want[0], q.contiguous(), dims, coords((5, 7)), interleaved=il)
        got = ttt.rope(q, k, dims, grid=(5, 7), interleaved=il)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # into a strided output, whose gaps stay as they were
        big = torch.full((B, N, 2, H, d + 1), 7.0, dtype=dt, device=DEV)
        qo, ko = big[:, :, 0, :, :d].transpose(1, 2), big[:, :, 1, :, :d].transpose(1, 2)
        ttt.ttt_rope(q, k, qo, ko, dims, grid=(5, 7), interleaved=il)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]) and (big[..., d] == 7.0).all()


@pytest.mark.parametrize("dims", [(32, 32), (24, 24), (22, 6), (2, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_and_back(dims, interleaved):
    t = draw((2, 30, 3, 2, 64), torch.float32)
    q, k = t[:, :, 0].transpose(1, 2), t[:, :, 1].transpose(1, 2)
    want = ttt.rope(q, k, dims, grid=(5, 6), interleaved=interleaved)
    before = t.clone()
    ttt.ttt_rope(q, k, q, k, dims, grid=(5, 6), interleaved=interleaved)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(t[:, :, 2], before[:, :, 2])
    ttt.ttt_rope(q, k, q, k, dims, grid=(5, 6), interleaved=interleaved, inverse=True)
    assert (t - before).abs().max() <= 2 * 5.5e-7 * 2 * before.abs().max()


def test_rope_backward_is_the_transpose():
    q, g = draw((2, 2, 12, 16), torch.float32, 1), draw((2, 2, 12, 16), torch.float32, 2)
    pos = torch.rand(12, 1, generator=torch.Generator().manual_seed(1)).to(DEV) * 50
    fwd, bwd = ttt.rope(q, None, (12,), pos=pos), ttt.rope_bwd(g, None, (12,), pos=pos)
    x = q.double().requires_grad_()
    grad, = torch.autograd.grad(rotate(x, (12,), pos)[0], x, g.double())
    size = rotate(g, (12,), pos)[1]
    assert ((bwd.double() - grad).abs() <= 2.0 ** -24 * grad.abs() + 5.5e-7 * size).all()
    lhs, rhs = (fwd.double() * g.double()).sum(), (q.double() * bwd.double()).sum()
    assert (lhs - rhs).abs() <= 2 * 5.5e-7 * 2 * (q.abs().double().sum() * g.abs().max())


def test_rope_nonfinite_stays_in_its_pair():
    q = draw((1, 2, 9, 32), torch.bfloat16)
    clean = ttt.rope(q, None, (16, 16), grid=(3, 3))
    q[0, 1, 4, 3] = float("inf")
    got = ttt.rope(q, None, (16, 16), grid=(3, 3))
    touched = torch.zeros_like(got, dtype=torch.bool)
    touched[0, 1, 4, [3, 11]] = True
    assert torch.equal(got[~touched], clean[~touched])


def test_rope_refusals_on_tensors():
    q = draw((1, 2, 9, 32), torch.float32)
    with pytest.raises(ttt.TTTError):
        ttt.rope(q, None, (15, 17), grid=(3, 3))
    with pytest.raises(ttt.TTTError):
        ttt.rope(q, None, (16, 16), grid=(3, 4))
    with pytest.raises(ttt.TTTError):  # an output that holds an element twice
        ttt.ttt_rope(q, None, q[:, :1].expand(1, 2, 9, 32), None, (16, 16), grid=(3, 3))
    with pytest.raises(ValueError):
        ttt.rope(q, None, (16, 16), pos=torch.zeros(8, 2, device=DEV))
    with pytest.raises(ValueError):
        ttt.rope(q, None, (16, 16), pos=torch.zeros(9, 2))


def test_rope_past_32_bit_offsets():
    # a line of tokens whose last ones lie behind what a 32-bit element offset reaches; far positions as well
    N, d = (1 << 25) + 11, 64
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free device memory")
    q = torch.empty(1, 1, N, d, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(5))
    got = ttt.rope(q, None, (64,), grid=(N,))
    at = torch.tensor([0, 1, 12345, (1 << 25) - 1, 1 << 25, N - 1], device=DEV)
    check(got[:, :, at], q[:, :, at], (64,), at[:, None].double())
