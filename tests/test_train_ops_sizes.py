"""Sizes that the library's 32-bit integers cannot hold are turned down by the binding (no GPU: the checks go by
the tensors' descriptions, and tensors of the meta device have no memory)."""
import pytest
import torch

from linear_attention_split_b200 import ttt

TOO_LARGE = "below 2\\^31"
BF, F32 = torch.bfloat16, torch.float32


def meta(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("rows", [2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40])
def test_layernorm_rows(rows):
    x, g = meta(rows, 8), meta(8, dtype=F32)
    for call in (lambda: ttt.layernorm(x, g), lambda: ttt.layernorm(x.view(2, rows // 2, 8) if rows % 2 == 0 else x, g),
                 lambda: ttt.layernorm_bwd(x, x, g), lambda: ttt.ttt_layernorm(x, g, None, x),
                 lambda: ttt.ttt_layernorm_bwd(x, x, g, x, g)):
        with pytest.raises(ValueError, match=TOO_LARGE):
            call()


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 1, 1), (2 ** 16, 2 ** 16, 2, 2), (1, 2 ** 32 + 4, 1), (1, 1, 2 ** 32 + 4)])
def test_orthogonalize_matrices(shape):
    x = meta(*shape)
    for call in (lambda: ttt.orthogonalize(x), lambda: ttt.ttt_orthogonalize(x, x)):
        with pytest.raises(ValueError, match=TOO_LARGE):
            call()


@pytest.mark.parametrize("shape", [(1, 1, 2 ** 32 + 16, 4), (2 ** 32 + 1, 1, 16, 4), (1, 2 ** 32 + 1, 16, 4)])
def test_rope_sizes(shape):
    q = meta(*shape)
    for kw in (dict(grid=(16,)), dict(grid=(shape[2],)), dict(pos=meta(shape[2], 1, dtype=F32))):
        with pytest.raises(ValueError, match=TOO_LARGE):
            ttt.rope(q, q, (4,), **kw)


@pytest.mark.parametrize("dims,grid", [((2 ** 32 + 4,), (16,)), ((4,), (2 ** 32 + 16,)), ((-2 ** 32 + 4,), (16,))])
def test_rope_axes(dims, grid):
    q = meta(1, 1, 16, 4)
    with pytest.raises(ValueError, match=TOO_LARGE):
        ttt.rope(q, q, dims, grid=grid)


@pytest.mark.parametrize("B,H,N,d", [(1, 1, 2 ** 32 + 16, 8), (2 ** 32 + 1, 1, 4, 8)])
def test_linear_orth_sizes(B, H, N, d):
    q, w0 = meta(B, H, N, d), meta(H, d, d, dtype=F32)
    with pytest.raises(ValueError, match=TOO_LARGE):
        ttt.linear_fullbatch_orth(q, q, q, w0)


def test_steps():
    # past the description checks, which need no device here: the arguments are given as a call finds them
    x, args = meta(2, 4, 4), (2, 4, 4, 1, 0)
    with pytest.raises(ValueError, match=TOO_LARGE):
        ttt._orthogonalize(x, x, 2 ** 32 + 5, ttt.NS_COEF, 1e-7, 1.0, None, None, args)


def test_workspace_queries():
    for call in (lambda: ttt.ttt_layernorm_bwd_workspace_bytes(2 ** 32 + 5, 8, 1),
                 lambda: ttt.ttt_orthogonalize_workspace_bytes(2 ** 32 + 1, 80, 80, 0),
                 lambda: ttt.ttt_linear_fullbatch_orth_workspace_bytes(1, 1, 2 ** 32 + 16, 64, 1)):
        with pytest.raises(ValueError, match=TOO_LARGE):
            call()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("C", [1, 8, 64, 384, 1000, 16384])
def test_layernorm_bwd_workspace_of_the_most_rows(C, dtype):
    # two blocks an SM at most, of which each leaves two rows of C sums
    few = ttt.ttt_layernorm_bwd_workspace_bytes(2 ** 24, C, dtype)
    assert 0 < few <= 2 * 256 * 2 * C * 4
    for rows in (2 ** 31 - 600, 2 ** 31 - 512, 2 ** 31 - 256, 2 ** 31 - 2, 2 ** 31 - 1):
        assert ttt.ttt_layernorm_bwd_workspace_bytes(rows, C, dtype) == few


def test_rope_axes_are_taken_by_value(monkeypatch):
    # widths and grid sizes held in integer tensors that change between calls
    seen = []
    monkeypatch.setattr(ttt, "_sig_device", lambda *sigs: 0)
    monkeypatch.setattr(ttt, "_call", lambda fn, dev, stream, *args: seen.append((list(args[6]), list(args[7]))))
    monkeypatch.setattr(ttt, "lib", lambda: type("L", (), {"ttt_rope": None}))
    q = meta(1, 2, 12, 8)
    dims, grid = (torch.tensor(4), torch.tensor(2)), (torch.tensor(3), torch.tensor(4))
    ttt.rope(q, q, dims, grid=grid)
    dims[1].fill_(4)
    grid[0].fill_(6)
    grid[1].fill_(2)
    ttt.rope(q, q, dims, grid=grid)
    assert seen == [([3, 4], [4, 2]), ([6, 2], [4, 4])]
    for bad in ((4.0, 2.0), ("4", "2")):  # also after the same whole numbers were taken
        with pytest.raises(TypeError):
            ttt.rope(q, q, bad, grid=(3, 4))
    ttt._rope_args.cache_clear()
