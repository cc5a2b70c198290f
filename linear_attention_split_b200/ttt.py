"""Thin Python binding of libttt_b200.so (the C ABI declared in include/ttt.h).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels.
PyTorch provides device memory and streams.  The functions carry the C names and take
torch CUDA tensors; ``*_workspace_bytes`` mirror the C queries.  If the library has not
been built this module raises on first use -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import operator
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libttt_b200.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "ttt.h")

TTT_F32, TTT_BF16 = 0, 1
_DT = {torch.float32: TTT_F32, torch.bfloat16: TTT_BF16}

STATUS = {0: "TTT_OK", 1: "TTT_ERR_INVALID_ARG", 2: "TTT_ERR_UNSUPPORTED", 3: "TTT_ERR_WORKSPACE",
          4: "TTT_ERR_CUDA", 5: "TTT_ERR_TIMEOUT"}


class TTTError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}: "
                         f"{lib().ttt_status_string(status).decode()}")


_lib = None


def lib():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m linear_attention_split_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.ttt_status_string.restype = ctypes.c_char_p
        L.ttt_status_string.argtypes = [i]
        L.ttt_version.restype = i
        L.ttt_version.argtypes = []
        L.ttt_kernel_launch_count.restype = ctypes.c_ulonglong
        L.ttt_kernel_launch_count.argtypes = []
        L.ttt_device_error.restype = i
        L.ttt_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.ttt_debug_set_wait_limit.restype = i
        L.ttt_debug_set_wait_limit.argtypes = [ctypes.c_longlong]
        L.ttt_debug_arm_fault.restype = i
        L.ttt_debug_arm_fault.argtypes = [ctypes.c_uint]
        L.ttt_linear_fullbatch_workspace_bytes.restype = sz
        L.ttt_linear_fullbatch_workspace_bytes.argtypes = [i, i, i, i, i]
        L.ttt_linear_fullbatch.restype = i
        L.ttt_linear_fullbatch.argtypes = [p, p, p, p, p, p, i, i, i, i, f, i, p, sz, p]
        L.ttt_vit3_block_workspace_bytes.restype = sz
        L.ttt_vit3_block_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.ttt_vit3_block.restype = i
        L.ttt_vit3_block.argtypes = [p, p, p, p, p, p, i, i, i, i, i, f, i, p, sz, p]
        L.ttt_linear_fullbatch_bwd_workspace_bytes.restype = sz
        L.ttt_linear_fullbatch_bwd_workspace_bytes.argtypes = [i, i, i, i, i]
        L.ttt_linear_fullbatch_bwd.restype = i
        L.ttt_linear_fullbatch_bwd.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, f, i, p, sz, p]
        L.ttt_dwconv_fullbatch_workspace_bytes.restype = sz
        L.ttt_dwconv_fullbatch_workspace_bytes.argtypes = [i, i, i, i, i]
        L.ttt_dwconv_fullbatch.restype = i
        L.ttt_dwconv_fullbatch.argtypes = [p, p, p, p, p, p, i, i, i, i, f, i, p, sz, p]
        L.ttt_mlp_fullbatch_workspace_bytes.restype = sz
        L.ttt_mlp_fullbatch_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.ttt_mlp_fullbatch.restype = i
        L.ttt_mlp_fullbatch.argtypes = [p, p, p, p, p, p, p, p, i, i, i, i, i, f, i, p, sz, p]
        L.ttt_linear_chunked_bidir_workspace_bytes.restype = sz
        L.ttt_linear_chunked_bidir_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.ttt_linear_chunked_bidir.restype = i
        L.ttt_linear_chunked_bidir.argtypes = [p, p, p, p, p, i, i, i, i, i, f, i, p, sz, p]
        L.ttt_linear_chunked_workspace_bytes.restype = sz
        L.ttt_linear_chunked_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        L.ttt_linear_chunked.restype = i
        L.ttt_linear_chunked.argtypes = [p, p, p, p, p, i, i, i, i, i, f, i, i, p, sz, p]
        L.ttt_linear_minibatch_workspace_bytes.restype = sz
        L.ttt_linear_minibatch_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        L.ttt_linear_minibatch.restype = i
        L.ttt_linear_minibatch.argtypes = [p, p, p, p, p, p, i, i, i, i, i, i, f, i, p, sz, p]
        L.ttt_linear_chunked_conv_workspace_bytes.restype = sz
        L.ttt_linear_chunked_conv_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
        L.ttt_linear_chunked_conv.restype = i
        L.ttt_linear_chunked_conv.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, i, f, i, i, p, sz, p]
        L.ttt_linear_chunked_bidir_noalloc.restype = i
        L.ttt_linear_chunked_bidir_noalloc.argtypes = [p, p, p, p, p, i, i, i, i, i, f, i, p]
        L.ttt_linear_chunked_bidir_noalloc_max_bytes.restype = sz
        L.ttt_linear_chunked_bidir_noalloc_max_bytes.argtypes = []
        L.ttt_layernorm.restype = i
        L.ttt_layernorm.argtypes = [p, p, p, p, i, i, f, i, p]
        L.ttt_layernorm_bwd_workspace_bytes.restype = sz
        L.ttt_layernorm_bwd_workspace_bytes.argtypes = [i, i, i]
        L.ttt_layernorm_bwd.restype = i
        L.ttt_layernorm_bwd.argtypes = [p, p, p, p, p, p, i, i, f, i, p, sz, p]
        L.ttt_rope.restype = i
        L.ttt_rope.argtypes = [p, p, p, p, p, i, p, p, i, i, i, i, i, ctypes.c_double, i, i, p, i, p]
        L.ttt_orthogonalize_workspace_bytes.restype = sz
        L.ttt_orthogonalize_workspace_bytes.argtypes = [i, i, i, i]
        L.ttt_orthogonalize.restype = i
        L.ttt_orthogonalize.argtypes = [p, p, i, i, i, i, f, f, f, f, f, i, p, sz, p]
        L.ttt_linear_fullbatch_orth_workspace_bytes.restype = sz
        L.ttt_linear_fullbatch_orth_workspace_bytes.argtypes = [i, i, i, i, i]
        L.ttt_linear_fullbatch_orth.restype = i
        L.ttt_linear_fullbatch_orth.argtypes = [p, p, p, p, p, p, i, i, i, i, f, i, f, f, f, f, i, p, sz, p]
        _lib = L
    return _lib


def declared_functions() -> list[str]:
    """Names of the functions include/ttt.h declares."""
    with open(HEADER_PATH) as fh:
        text = fh.read()
    return sorted(set(re.findall(r"\b(ttt_[a-z0-9_]+)\s*\(", text)))


# ----------------------------------------------------------------------- helpers -------
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype(*ts):
    dt = ts[0].dtype
    for t in ts:
        if t.dtype != dt:
            raise TypeError("q, k, v and out must share one dtype")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
    if dt not in _DT:
        raise TypeError(f"unsupported dtype {dt}")
    return _DT[dt]


def _weights(*ws):
    for w in ws:
        if w is None:
            continue
        if w.dtype != torch.float32 or not w.is_cuda or not w.is_contiguous():
            raise ValueError("inner weights must be contiguous fp32 CUDA tensors")


def _workspace(nbytes, workspace, device):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    return workspace, workspace.numel() * workspace.element_size()


def _check(fn, rc):
    if rc != 0:
        raise TTTError(fn, rc)


# ----------------------------------------------------------------------- entry points --
def ttt_linear_fullbatch_workspace_bytes(B, H, N, d, dtype):
    return lib().ttt_linear_fullbatch_workspace_bytes(B, H, N, d, dtype)


def ttt_linear_fullbatch(q, k, v, w0, out, w_star=None, eta=1.0, workspace=None, stream=None):
    """q, k, v, out [B,H,N,d] (fp32 or bf16); w0 [H,d,d] fp32; w_star [B,H,d,d] fp32 or None."""
    dt = _dtype(q, k, v, out)
    _weights(w0, w_star)
    B, H, N, d = q.shape
    ws, nbytes = _workspace(ttt_linear_fullbatch_workspace_bytes(B, H, N, d, dt), workspace, q.device)
    rc = lib().ttt_linear_fullbatch(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(out), _ptr(w_star), B, H, N,
                                    d, float(eta), dt, _ptr(ws), nbytes, _stream(stream))
    _check("ttt_linear_fullbatch", rc)
    return out


def ttt_vit3_block_workspace_bytes(B, Hg, Wg, C, H, dtype):
    return lib().ttt_vit3_block_workspace_bytes(B, Hg, Wg, C, H, dtype)


def ttt_vit3_block(x, wqkvg, w0, wc, wo, y, Hg, Wg, H, eta=1.0, workspace=None, stream=None):
    """The ViT^3 TTT block: x, y [B, Hg*Wg, C]; wqkvg [C, 4C] and wo [2C, C] in x's dtype;
    w0 [H, C/H, C/H] and wc [C, 3, 3] fp32."""
    dt = _dtype(x, wqkvg, wo, y)
    _weights(w0, wc)
    B, N, C = x.shape
    if N != Hg * Wg:
        raise ValueError("N must equal Hg * Wg")
    ws, nbytes = _workspace(ttt_vit3_block_workspace_bytes(B, Hg, Wg, C, H, dt), workspace, x.device)
    rc = lib().ttt_vit3_block(_ptr(x), _ptr(wqkvg), _ptr(w0), _ptr(wc), _ptr(wo), _ptr(y), B, Hg, Wg, C, H,
                              float(eta), dt, _ptr(ws), nbytes, _stream(stream))
    _check("ttt_vit3_block", rc)
    return y


def vit3_block(x, wqkvg, w0, wc, wo, Hg, Wg, H, eta=1.0):
    y = torch.empty_like(x)
    return ttt_vit3_block(x, wqkvg, w0, wc, wo, y, Hg, Wg, H, eta)


def ttt_linear_fullbatch_bwd_workspace_bytes(B, H, N, d, dtype):
    return lib().ttt_linear_fullbatch_bwd_workspace_bytes(B, H, N, d, dtype)


def ttt_linear_fullbatch_bwd(q, k, v, w0, dout, dq, dk, dv, dw0, eta=1.0, workspace=None, stream=None):
    """Gradients of the full-batch TTT-Linear layer: dq, dk, dv [B,H,N,d] (dtype of q), dw0 [H,d,d] fp32."""
    dt = _dtype(q, k, v, dout, dq, dk, dv)
    _weights(w0, dw0)
    B, H, N, d = q.shape
    ws, nbytes = _workspace(ttt_linear_fullbatch_bwd_workspace_bytes(B, H, N, d, dt), workspace, q.device)
    rc = lib().ttt_linear_fullbatch_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(dout), _ptr(dq), _ptr(dk),
                                        _ptr(dv), _ptr(dw0), B, H, N, d, float(eta), dt, _ptr(ws), nbytes,
                                        _stream(stream))
    _check("ttt_linear_fullbatch_bwd", rc)
    return dq, dk, dv, dw0


def ttt_dwconv_fullbatch_workspace_bytes(B, Hg, Wg, C, dtype):
    return lib().ttt_dwconv_fullbatch_workspace_bytes(B, Hg, Wg, C, dtype)


def ttt_dwconv_fullbatch(q, k, v, w0, out, w_star=None, eta=1.0, workspace=None, stream=None):
    """q, k, v, out [B,Hg,Wg,C] channels-last; w0 [C,3,3] fp32; w_star [B,C,3,3] fp32 or None."""
    dt = _dtype(q, k, v, out)
    _weights(w0, w_star)
    B, Hg, Wg, C = q.shape
    ws, nbytes = _workspace(ttt_dwconv_fullbatch_workspace_bytes(B, Hg, Wg, C, dt), workspace, q.device)
    rc = lib().ttt_dwconv_fullbatch(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(out), _ptr(w_star), B, Hg, Wg,
                                    C, float(eta), dt, _ptr(ws), nbytes, _stream(stream))
    _check("ttt_dwconv_fullbatch", rc)
    return out


def ttt_mlp_fullbatch_workspace_bytes(B, H, N, d, hidden, dtype):
    return lib().ttt_mlp_fullbatch_workspace_bytes(B, H, N, d, hidden, dtype)


def ttt_mlp_fullbatch(q, k, v, w1, w2, out, w1_star=None, w2_star=None, eta=1.0, workspace=None,
                      stream=None):
    """q, k, v, out [B,H,N,d]; w1 [H,d,h], w2 [H,h,d] fp32; optional fp32 updated weights."""
    dt = _dtype(q, k, v, out)
    _weights(w1, w2, w1_star, w2_star)
    B, H, N, d = q.shape
    hidden = w1.shape[2]
    ws, nbytes = _workspace(ttt_mlp_fullbatch_workspace_bytes(B, H, N, d, hidden, dt), workspace, q.device)
    rc = lib().ttt_mlp_fullbatch(_ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(w2), _ptr(out), _ptr(w1_star),
                                 _ptr(w2_star), B, H, N, d, hidden, float(eta), dt, _ptr(ws), nbytes,
                                 _stream(stream))
    _check("ttt_mlp_fullbatch", rc)
    return out


def ttt_linear_chunked_bidir_workspace_bytes(B, H, N, d, chunk, dtype):
    return lib().ttt_linear_chunked_bidir_workspace_bytes(B, H, N, d, chunk, dtype)


def ttt_linear_chunked_bidir(q, k, v, w0, out, chunk, eta=1.0, workspace=None, stream=None):
    """q, k, v, out [B,H,N,d]; w0 [H,d,d] fp32; N % chunk == 0."""
    dt = _dtype(q, k, v, out)
    _weights(w0)
    B, H, N, d = q.shape
    ws, nbytes = _workspace(ttt_linear_chunked_bidir_workspace_bytes(B, H, N, d, chunk, dt), workspace,
                            q.device)
    rc = lib().ttt_linear_chunked_bidir(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(out), B, H, N, d,
                                        int(chunk), float(eta), dt, _ptr(ws), nbytes, _stream(stream))
    _check("ttt_linear_chunked_bidir", rc)
    return out


def ttt_linear_chunked_workspace_bytes(B, H, N, d, chunk, direction, dtype):
    return lib().ttt_linear_chunked_workspace_bytes(B, H, N, d, chunk, direction, dtype)


def ttt_linear_chunked(q, k, v, w0, out, chunk, eta=1.0, direction=0, workspace=None, stream=None):
    """One-way (direction +1 raster, -1 reverse) or bidirectional (0) chunked scan."""
    dt = _dtype(q, k, v, out)
    _weights(w0)
    B, H, N, d = q.shape
    ws, nbytes = _workspace(ttt_linear_chunked_workspace_bytes(B, H, N, d, chunk, direction, dt), workspace,
                            q.device)
    rc = lib().ttt_linear_chunked(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(out), B, H, N, d, int(chunk),
                                  float(eta), int(direction), dt, _ptr(ws), nbytes, _stream(stream))
    _check("ttt_linear_chunked", rc)
    return out


def ttt_linear_minibatch_workspace_bytes(B, H, N, d, chunk, epochs, dtype):
    return lib().ttt_linear_minibatch_workspace_bytes(B, H, N, d, chunk, epochs, dtype)


def ttt_linear_minibatch(q, k, v, w0, out, chunk, epochs=1, w_final=None, eta=1.0, workspace=None, stream=None):
    """`epochs` epochs of mini-batch inner training (chunks of `chunk` tokens), then out = Q W_final."""
    dt = _dtype(q, k, v, out)
    _weights(w0, w_final)
    B, H, N, d = q.shape
    ws, nbytes = _workspace(ttt_linear_minibatch_workspace_bytes(B, H, N, d, chunk, epochs, dt), workspace,
                            q.device)
    rc = lib().ttt_linear_minibatch(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(out), _ptr(w_final), B, H, N, d,
                                    int(chunk), int(epochs), float(eta), dt, _ptr(ws), nbytes, _stream(stream))
    _check("ttt_linear_minibatch", rc)
    return out


def ttt_linear_chunked_conv_workspace_bytes(B, H, Hg, Wg, d, chunk, direction, dtype):
    return lib().ttt_linear_chunked_conv_workspace_bytes(B, H, Hg, Wg, d, chunk, direction, dtype)


def ttt_linear_chunked_conv(q, k, v, w0, wk, wv, out, Hg, Wg, chunk, eta=1.0, direction=0, workspace=None,
                            stream=None):
    """Chunked scan on (Q, conv3x3(K; wk), conv3x3(V; wv)) over the Hg x Wg token grid."""
    dt = _dtype(q, k, v, out)
    _weights(w0, wk, wv)
    B, H, N, d = q.shape
    if N != Hg * Wg:
        raise ValueError("N must equal Hg * Wg")
    ws, nbytes = _workspace(ttt_linear_chunked_conv_workspace_bytes(B, H, Hg, Wg, d, chunk, direction, dt),
                            workspace, q.device)
    rc = lib().ttt_linear_chunked_conv(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(wk), _ptr(wv), _ptr(out), B, H,
                                       Hg, Wg, d, int(chunk), float(eta), int(direction), dt, _ptr(ws), nbytes,
                                       _stream(stream))
    _check("ttt_linear_chunked_conv", rc)
    return out


def ttt_linear_chunked_bidir_noalloc(q, k, v, w0, out, chunk, eta=1.0, stream=None):
    """The chunked scan without a workspace argument: for callers that may not allocate
    device memory at call time.  Its scratch is a fixed array inside the library's device
    image (ttt_linear_chunked_bidir_noalloc_max_bytes() long); calls that overlap on the GPU
    race on it."""
    dt = _dtype(q, k, v, out)
    _weights(w0)
    B, H, N, d = q.shape
    rc = lib().ttt_linear_chunked_bidir_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(out), B, H, N, d,
                                                int(chunk), float(eta), dt, _stream(stream))
    _check("ttt_linear_chunked_bidir_noalloc", rc)
    return out


NS_COEF = (3.4445, -4.7750, 2.0315)  # the usual quintic of the Newton-Schulz steps


# The checks of arguments below go by what a check can depend on: each tensor's type, shape, strides and
# device.  A function that has passed them once for such a description keeps what it found (functools.lru_cache;
# nothing is kept by a tensor's identity or address, and a refusal is not kept), which is most of a call's host time.
def _sig(t):
    return None if t is None else (t.dtype, t.shape, t.stride(), t.get_device())


def _sig_dense(sig):
    want = 1
    for n, st in zip(reversed(sig[1]), reversed(sig[2])):
        if n != 1 and st != want:
            return 0 in sig[1]
        want *= n
    return True


def _sig_device(*sigs):
    """The index of the device, which has to be one CUDA device."""
    dev = sigs[0][3]
    if any(s is not None and s[3] != dev for s in sigs):
        raise ValueError("tensors must be on one device")
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    return dev


def _sig_type(*sigs):
    """The library's type of dense tensors of one dtype and shape."""
    dtype, shape = sigs[0][:2]
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    for s in sigs:
        if s[0] is not dtype:
            raise TypeError("tensors must share one dtype")
        if s[1] != shape:
            raise ValueError("tensors must have one shape")
        if not _sig_dense(s):
            raise ValueError("tensors must be contiguous CUDA tensors")
    return _DT[dtype]


def _sig_int(*sizes):
    """Sizes fit the library's int: ctypes would cut them to 32 bits without a word."""
    if any(not -2 ** 31 <= n < 2 ** 31 for n in sizes):
        raise ValueError(f"sizes have to be below 2^31, got {sizes}")
    return sizes


def _sig_vector(sig, C, name):
    if sig is not None and (sig[0] is not torch.float32 or tuple(sig[1]) != (C,) or not _sig_dense(sig)):
        raise ValueError(f"{name} must be a contiguous fp32 tensor [C]")


@functools.lru_cache(maxsize=512)
def _scratch_bytes(query, dev, *args):
    """A workspace query's answer, kept by its arguments and the device whose SM count it may go by."""
    with torch.cuda.device(dev):
        return getattr(lib(), query)(*args)


def _scratch(nbytes, workspace, dev, stream):
    """(pointer, size, owner) of the caller's workspace, or of one allocated on the stream that uses it."""
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous and on the tensors' device")
        size = workspace.numel() * workspace.element_size()
        if size < nbytes:
            raise ValueError("workspace too small")
        return workspace.data_ptr() or None, size, workspace
    if nbytes == 0:
        return None, 0, None
    if stream is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(s):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws.data_ptr(), nbytes, ws


def _call(fn, dev, stream, *args):
    """Call a C entry point with `dev` current, on `stream` (default: dev's current stream)."""
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(dev)
    else:
        st = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, st)
    if rc != 0:
        raise TTTError(fn.__name__, rc)


def _at(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=512)
def _norm_args(x, gamma, beta, *like_x):
    """(rows, C, type, device) of a layer norm of x [..., C] with vectors gamma, beta [C]."""
    dt = _sig_type(x, *like_x)
    shape = x[1]
    C = shape[-1] if len(shape) else 0
    _sig_vector(gamma, C, "gamma")
    _sig_vector(beta, C, "beta")
    return *_sig_int(math.prod(shape[:-1]) if C else 0, C), dt, _sig_device(x, gamma, beta, *like_x)


def _layernorm(x, gamma, beta, y, eps, stream, args):
    rows, C, dt, dev = args
    _call(lib().ttt_layernorm, dev, stream, x.data_ptr(), gamma.data_ptr(), _at(beta), y.data_ptr(), rows, C, eps, dt)
    return y


def _layernorm_bwd(dy, x, gamma, dx, dgamma, dbeta, eps, workspace, stream, args):
    rows, C, dt, dev = args
    ws, nbytes, _keep = _scratch(_scratch_bytes("ttt_layernorm_bwd_workspace_bytes", dev, rows, C, dt), workspace, dev, stream)
    _call(lib().ttt_layernorm_bwd, dev, stream, dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), dx.data_ptr(), dgamma.data_ptr(),
          _at(dbeta), rows, C, eps, dt, ws, nbytes)
    return dx, dgamma, dbeta


def ttt_layernorm(x, gamma, beta, y, eps=1e-6, stream=None):
    """Layer norm over the last axis: x, y [..., C] (y may be x); gamma, beta [C] fp32, beta may be None."""
    return _layernorm(x, gamma, beta, y, eps, stream, _norm_args(_sig(x), _sig(gamma), _sig(beta), _sig(y)))


def ttt_layernorm_bwd_workspace_bytes(rows, C, dtype):
    return lib().ttt_layernorm_bwd_workspace_bytes(*_sig_int(rows, C), dtype)


def ttt_layernorm_bwd(dy, x, gamma, dx, dgamma, dbeta=None, eps=1e-6, workspace=None, stream=None):
    """Gradients of ttt_layernorm: dx [..., C] (may be dy or x), dgamma and dbeta [C] fp32 (dbeta may be None)."""
    args = _norm_args(_sig(x), _sig(gamma), _sig(dgamma), _sig(dy), _sig(dx))
    _norm_args(_sig(x), _sig(gamma), _sig(dbeta))
    return _layernorm_bwd(dy, x, gamma, dx, dgamma, dbeta, eps, workspace, stream, args)


@functools.lru_cache(maxsize=512)
def _rope_args(q, k, q_out, k_out, pos, dims, grid):
    """The library's arguments behind the tensors' pointers; an output without a description is dense."""
    if (grid is None) == (pos is None):
        raise ValueError("give either grid or pos")
    dtype, shape = q[:2]
    if len(shape) != 4:
        raise ValueError("q, k and their outputs must be [B, H, N, d]")
    if dtype not in _DT:
        raise TypeError(f"unsupported dtype {dtype}")
    B, H, N, d = _sig_int(*shape)
    _sig_int(*dims, *(grid or ()))
    strides = []
    for t in (q, k, q_out, k_out):
        if t is None:
            strides += [H * N * d, N * d, d]
            continue
        if t[0] is not dtype:
            raise TypeError("q, k and their outputs must share one dtype")
        if t[1] != shape:
            raise ValueError("q, k and their outputs must have one shape")
        if t[2][3] != 1 and d != 1:
            raise ValueError("the features of a head must be adjacent")
        strides += t[2][:3]
    dev = _sig_device(q, k, q_out, k_out, pos)
    axes = len(dims)
    if grid is not None and len(grid) != axes:
        raise ValueError("grid and dims must have one length")
    batched = 0
    if pos is not None:
        batched = int(len(pos[1]) == 3)
        if pos[0] is not torch.float32 or not _sig_dense(pos) or tuple(pos[1]) != ((B, N, axes) if batched else (N, axes)):
            raise ValueError("pos must be contiguous fp32 [N, axes] or [B, N, axes]")
    ints = ctypes.c_int * max(axes, 1)
    return (batched, None if grid is None else ints(*grid), ints(*dims), axes, B, H, N, d), (ctypes.c_longlong * 12)(*strides), \
        _DT[dtype], dev


def _rope(q, k, q_out, k_out, pos, base, interleaved, inverse, stream, args):
    sizes, strides, dt, dev = args
    _call(lib().ttt_rope, dev, stream, q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out), _at(pos), *sizes, base, interleaved,
          inverse, strides, dt)


def _whole(sizes):
    """Plain integers, which is what the checks' answers are kept by (an integer tensor would go by its identity)."""
    return None if sizes is None else tuple(map(operator.index, sizes))


def ttt_rope(q, k, q_out, k_out, dims, grid=None, pos=None, base=10000.0, interleaved=False, inverse=False, stream=None):
    """Rotary positions: q, k and their outputs [B, H, N, d], any strides with adjacent features (k, k_out may be
    None; an output may be its own input).  dims: the even widths of the axes' sections.  Either grid, the sizes of
    the token grid, or pos, fp32 [N, axes] or [B, N, axes].  inverse: turn back, which is the backward pass."""
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    args = _rope_args(_sig(q), _sig(k), _sig(q_out), _sig(k_out), _sig(pos), _whole(dims), _whole(grid))
    _rope(q, k, q_out, k_out, pos, base, interleaved, inverse, stream, args)
    return q_out, k_out


def ttt_orthogonalize_workspace_bytes(U, m, n, dtype):
    return lib().ttt_orthogonalize_workspace_bytes(*_sig_int(U, m, n), dtype)


def ttt_orthogonalize(x, out, steps=5, coef=NS_COEF, eps=1e-7, scale=1.0, workspace=None, stream=None):
    """out = scale * the Newton-Schulz steps of each matrix of x [..., m, n] (out may be x)."""
    return _orthogonalize(x, out, steps, coef, eps, scale, workspace, stream, _orth_args(_sig(x), _sig(out)))


@functools.lru_cache(maxsize=512)
def _orth_args(x, *like_x):
    """(U, m, n, type, device) of matrices [..., m, n]."""
    dt = _sig_type(x, *like_x)
    if len(x[1]) < 2:
        raise ValueError("x must be [..., m, n]")
    m, n = x[1][-2:]
    return *_sig_int(math.prod(x[1][:-2]), m, n), dt, _sig_device(x, *like_x)


def _orthogonalize(x, out, steps, coef, eps, scale, workspace, stream, args):
    U, m, n, dt, dev = args
    _sig_int(steps)
    a, b, c = coef
    ws, nbytes, _keep = _scratch(_scratch_bytes("ttt_orthogonalize_workspace_bytes", dev, U, m, n, dt), workspace, dev, stream)
    _call(lib().ttt_orthogonalize, dev, stream, x.data_ptr(), out.data_ptr(), U, m, n, steps, a, b, c, eps, scale, dt, ws, nbytes)
    return out


def ttt_linear_fullbatch_orth_workspace_bytes(B, H, N, d, dtype):
    return lib().ttt_linear_fullbatch_orth_workspace_bytes(*_sig_int(B, H, N, d), dtype)


def ttt_linear_fullbatch_orth(q, k, v, w0, out, w_star=None, eta=0.1, steps=5, coef=NS_COEF, eps=1e-7, workspace=None,
                              stream=None):
    """TTT-Linear whose inner step goes along the orthogonalised gradient; tensors as for ttt_linear_fullbatch."""
    B, H, N, d, dt, dev = _linear_orth_args(_sig(q), _sig(k), _sig(v), _sig(out), _sig(w0), _sig(w_star))
    _sig_int(steps)
    a, b, c = coef
    ws, nbytes, _keep = _scratch(_scratch_bytes("ttt_linear_fullbatch_orth_workspace_bytes", dev, B, H, N, d, dt), workspace, dev,
                                 stream)
    _call(lib().ttt_linear_fullbatch_orth, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), w0.data_ptr(), out.data_ptr(),
          _at(w_star), B, H, N, d, eta, steps, a, b, c, eps, dt, ws, nbytes)
    return out


@functools.lru_cache(maxsize=512)
def _linear_orth_args(q, k, v, out, w0, w_star):
    dt = _sig_type(q, k, v, out)
    if len(q[1]) != 4:
        raise ValueError("q, k, v and out must be [B, H, N, d]")
    B, H, N, d = _sig_int(*q[1])
    for w, shape in ((w0, (H, d, d)), (w_star, (B, H, d, d))):
        if w is not None and (w[0] is not torch.float32 or tuple(w[1]) != shape or not _sig_dense(w)):
            raise ValueError("w0 must be [H, d, d] and w_star [B, H, d, d], contiguous fp32")
    return B, H, N, d, dt, _sig_device(q, k, v, out, w0, w_star)


TTT_FAULT_SKIP_LOAD = 0x1


def debug_set_wait_limit(cycles: int) -> None:
    """Bounded-wait limit (SM cycles) of kernels launched afterwards; <= 0 restores the default."""
    _check("ttt_debug_set_wait_limit", lib().ttt_debug_set_wait_limit(int(cycles)))


def debug_arm_fault(bits: int) -> None:
    """Arm (bits != 0) or clear (0) the simulated lost-transfer test hook."""
    _check("ttt_debug_arm_fault", lib().ttt_debug_arm_fault(int(bits)))


def kernel_launch_count() -> int:
    return int(lib().ttt_kernel_launch_count())


def device_error() -> int:
    """Synchronise and return (and clear) the device error bits; raises on a timeout."""
    bits = ctypes.c_uint(0)
    rc = lib().ttt_device_error(ctypes.byref(bits))
    if rc != 0:
        raise TTTError("ttt_device_error", rc)
    return bits.value


# ----------------------------------------------------------------------- conveniences --
def linear_fullbatch(q, k, v, w0, eta=1.0, with_w_star=False):
    out = torch.empty_like(q)
    ws = torch.empty((q.shape[0], q.shape[1], q.shape[3], q.shape[3]), dtype=torch.float32,
                     device=q.device) if with_w_star else None
    ttt_linear_fullbatch(q, k, v, w0, out, ws, eta)
    return (out, ws) if with_w_star else out


def linear_fullbatch_bwd(q, k, v, w0, dout, eta=1.0):
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dw0 = torch.empty_like(w0)
    return ttt_linear_fullbatch_bwd(q, k, v, w0, dout, dq, dk, dv, dw0, eta)


def dwconv_fullbatch(q, k, v, w0, eta=1.0, with_w_star=False):
    out = torch.empty_like(q)
    ws = torch.empty((q.shape[0], q.shape[3], 3, 3), dtype=torch.float32,
                     device=q.device) if with_w_star else None
    ttt_dwconv_fullbatch(q, k, v, w0, out, ws, eta)
    return (out, ws) if with_w_star else out


def mlp_fullbatch(q, k, v, w1, w2, eta=1.0, with_w_star=False):
    out = torch.empty_like(q)
    B, H, _, d = q.shape
    h = w1.shape[2]
    w1s = torch.empty((B, H, d, h), dtype=torch.float32, device=q.device) if with_w_star else None
    w2s = torch.empty((B, H, h, d), dtype=torch.float32, device=q.device) if with_w_star else None
    ttt_mlp_fullbatch(q, k, v, w1, w2, out, w1s, w2s, eta)
    return (out, w1s, w2s) if with_w_star else out


def linear_chunked(q, k, v, w0, chunk, eta=1.0, direction=0):
    out = torch.empty_like(q)
    ttt_linear_chunked(q, k, v, w0, out, chunk, eta, direction)
    return out


def linear_minibatch(q, k, v, w0, chunk, epochs=1, eta=1.0, with_w_final=False):
    out = torch.empty_like(q)
    wf = torch.empty((q.shape[0], q.shape[1], q.shape[3], q.shape[3]), dtype=torch.float32,
                     device=q.device) if with_w_final else None
    ttt_linear_minibatch(q, k, v, w0, out, chunk, epochs, wf, eta)
    return (out, wf) if with_w_final else out


def linear_chunked_conv(q, k, v, w0, wk, wv, Hg, Wg, chunk, eta=1.0, direction=0):
    out = torch.empty_like(q)
    ttt_linear_chunked_conv(q, k, v, w0, wk, wv, out, Hg, Wg, chunk, eta, direction)
    return out


def linear_chunked_bidir(q, k, v, w0, chunk, eta=1.0):
    out = torch.empty_like(q)
    ttt_linear_chunked_bidir(q, k, v, w0, out, chunk, eta)
    return out


def layernorm(x, gamma, beta=None, eps=1e-6):
    args = _norm_args(_sig(x), _sig(gamma), _sig(beta))
    return _layernorm(x, gamma, beta, torch.empty_like(x), eps, None, args)


def layernorm_bwd(dy, x, gamma, eps=1e-6, with_dbeta=True):
    """(dx, dgamma, dbeta); dbeta is None without with_dbeta."""
    args = _norm_args(_sig(x), _sig(gamma), None, _sig(dy))
    return _layernorm_bwd(dy, x, gamma, torch.empty_like(x), torch.empty_like(gamma),
                          torch.empty_like(gamma) if with_dbeta else None, eps, None, None, args)


def rope(q, k=None, dims=None, grid=None, pos=None, base=10000.0, interleaved=False, inverse=False):
    """q and k turned to their positions, each contiguous [B, H, N, d]; without k, q alone."""
    args = _rope_args(_sig(q), _sig(k), None, None, _sig(pos), _whole(dims), _whole(grid))
    q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    k_out = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
    _rope(q, k, q_out, k_out, pos, base, interleaved, inverse, None, args)
    return q_out if k is None else (q_out, k_out)


def rope_bwd(dq, dk=None, dims=None, grid=None, pos=None, base=10000.0, interleaved=False):
    """Gradients of q and k from those of rope's outputs: the rotation turned back."""
    return rope(dq, dk, dims, grid, pos, base, interleaved, inverse=True)


def orthogonalize(x, steps=5, coef=NS_COEF, eps=1e-7, scale=1.0):
    return _orthogonalize(x, torch.empty_like(x), steps, coef, eps, scale, None, None, _orth_args(_sig(x)))


def linear_fullbatch_orth(q, k, v, w0, eta=0.1, steps=5, coef=NS_COEF, eps=1e-7, with_w_star=False):
    out = torch.empty_like(q)
    ws = torch.empty((q.shape[0], q.shape[1], q.shape[3], q.shape[3]), dtype=torch.float32,
                     device=q.device) if with_w_star else None
    ttt_linear_fullbatch_orth(q, k, v, w0, out, ws, eta, steps, coef, eps)
    return (out, ws) if with_w_star else out
