"""Python binding of the C ABI in include/fa.h (argument marshalling only).

The ``fa_*`` functions mirror the C entry points one to one: they take torch
tensors that already live on the GPU, check dtype/shape/contiguity, and pass raw
pointers, sizes and the current CUDA stream to libfa_b200.so. Every arithmetic
step runs in the library's kernels; there is no CPU or PyTorch fallback.

``forward``, ``backward`` and ``attention`` are conveniences on top: they allocate
outputs (and the backward workspace) with torch and call the entry points;
``attention`` is differentiable through ``FlashAttentionFunction``.

Operation (see include/fa.h): O = softmax(scale * Q K^T [causal mask]) V and
LSE = natural-log log-sum-exp per query row, for [B, H, N, d] tensors, d in
{64, 128}; backward gives dQ, dK, dV of the loss <dO, O>.
"""
from __future__ import annotations

import contextlib
import functools
import math

import torch

from ._lib import FAError, check, lib

__all__ = [
    "FAError", "fa_forward", "fa_backward", "fa_backward_workspace_size",
    "fa_backward_preprocess", "fa_backward_main", "fa_backward_dq_convert",
    "fa_backward_noalloc", "fa_forward_f16", "fa_backward_f16", "fa_forward_masked",
    "fa_backward_masked", "fa_forward_dropout", "fa_backward_dropout", "fa_forward_f32",
    "fa_backward_f32", "fa_forward_scored", "fa_backward_scored", "fa_forward_scored_f16",
    "fa_backward_scored_f16", "fa_backward_scored_workspace_size", "fa_cache4_append",
    "fa_cache4_read", "fa_cache4_attend", "fa_cache4_append_f16", "fa_cache4_read_f16",
    "fa_cache4_attend_f16", "fa_cache4_workspace_size",
    "fa_get_status", "fa_watchdog_selftest", "fa_version", "fa_dropout_rate",
    "fa_launch_plan",
    "forward", "backward", "attention", "FlashAttentionFunction", "cache4_empty",
    "cache4_append", "cache4_read", "cache4_attend",
]


_Tensor, _Stream = torch.Tensor, torch.cuda.Stream
_current_device = torch.cuda.current_device
_current_gpu = torch._C._cuda_getDevice  # the same without initialising CUDA: a GPU tensor has


def _one_device(*args):
    """A context that makes current the one CUDA device of a call's tensors (and
    stream): the library launches on the current device, and a stream left as None
    is that device's current stream. Arguments on two different GPUs raise."""
    devs = set()
    for a in args:
        dev = getattr(a, "device", None)
        if isinstance(dev, torch.device) and dev.type == "cuda" and dev.index is not None:
            devs.add(dev)
    if len(devs) > 1:
        raise ValueError("the tensors of one call must be on one GPU, got "
                         + ", ".join(sorted(str(x) for x in devs)))
    return torch.cuda.device(devs.pop()) if devs else contextlib.nullcontext()


def _on_one_device(fn):
    @functools.wraps(fn)
    def call(*args, **kwargs):
        # The common case, everything on the current GPU, without a context to enter.
        index = -1
        for a in (*args, *kwargs.values()) if kwargs else args:
            if isinstance(a, _Tensor):
                i = a.get_device()  # -1 on the CPU
            elif isinstance(a, _Stream):
                i = a.device.index
            else:
                continue
            if i != index and i >= 0:
                if index >= 0:
                    break
                index = i
        else:
            if index < 0 or index == _current_gpu():
                return fn(*args, **kwargs)
        with _one_device(*args, *kwargs.values()):
            return fn(*args, **kwargs)
    return call


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(_current_device())
    return int(getattr(stream, "cuda_stream", stream))


def _shape(t: torch.Tensor):
    if t.dim() != 4:
        raise ValueError(f"expected a [B, H, N, d] tensor, got shape {tuple(t.shape)}")
    return tuple(t.shape)


def _need(name: str, t: torch.Tensor, dtype: torch.dtype, shape) -> int:
    if (isinstance(t, _Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def fa_version() -> str:
    return lib().fa_version().decode()


@functools.lru_cache(maxsize=1024)  # a function of its arguments alone
def fa_backward_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_backward_workspace_size(B, H, N, d))


@functools.lru_cache(maxsize=1024)
def fa_backward_scored_workspace_size(B: int, H: int, Hkv: int, N: int, d: int) -> int:
    """Bytes of workspace that fa_backward_scored makes use of."""
    return int(lib().fa_backward_scored_workspace_size(B, H, Hkv, N, d))


@functools.lru_cache(maxsize=1024)
def fa_cache4_workspace_size(B: int, H: int, Hkv: int, Nq: int, d: int, max_len: int,
                             window_left: int = -1) -> int:
    """Bytes of workspace that fa_cache4_attend needs."""
    return int(lib().fa_cache4_workspace_size(B, H, Hkv, Nq, d, max_len, window_left))


@_on_one_device
def fa_forward(Q, K, V, O, LSE, scale: float, causal: bool, stream=None) -> None:
    B, H, N, d = _shape(Q)
    bf = torch.bfloat16
    args = [_need("Q", Q, bf, (B, H, N, d)), _need("K", K, bf, (B, H, N, d)),
            _need("V", V, bf, (B, H, N, d)), _need("O", O, bf, (B, H, N, d)),
            _need("LSE", LSE, torch.float32, (B, H, N))]
    check("fa_forward", lib().fa_forward(*args, B, H, N, d, float(scale), int(bool(causal)),
                                         _stream(stream)))


@_on_one_device
def fa_forward_f16(Q, K, V, O, LSE, scale: float, causal: bool, stream=None) -> None:
    B, H, N, d = _shape(Q)
    h = torch.float16
    args = [_need("Q", Q, h, (B, H, N, d)), _need("K", K, h, (B, H, N, d)),
            _need("V", V, h, (B, H, N, d)), _need("O", O, h, (B, H, N, d)),
            _need("LSE", LSE, torch.float32, (B, H, N))]
    check("fa_forward_f16", lib().fa_forward_f16(*args, B, H, N, d, float(scale),
                                                 int(bool(causal)), _stream(stream)))


def _block_mask(block_mask, N: int):
    """Device pointer of a [ceil(N/128)]^2 uint8/bool CUDA tensor, or None."""
    if block_mask is None:
        return None
    T = (N + 127) // 128
    if not isinstance(block_mask, torch.Tensor) or not block_mask.is_cuda:
        raise ValueError("block_mask must be a CUDA tensor")
    if block_mask.dtype not in (torch.uint8, torch.bool):
        raise TypeError("block_mask must be uint8 or bool")
    if tuple(block_mask.shape) != (T, T) or not block_mask.is_contiguous():
        raise ValueError(f"block_mask must be a contiguous [{T}, {T}] tensor")
    return block_mask.data_ptr()


def _bound(n) -> int:
    """A window's side as the library takes it: 32 bits, -1 for none."""
    n = int(n)
    return n if -1 <= n < 2**31 else max(-1, min(n, 2**31 - 1))


def _window(window):
    if window is None:
        return -1, -1
    left, right = window
    return _bound(left), _bound(right)


@_on_one_device
def fa_forward_masked(Q, K, V, O, LSE, scale: float, causal: bool, window=None,
                      block_mask=None, stream=None) -> None:
    """fa_forward with a sliding window (left, right) (negative = unbounded side)
    and/or a 128 x 128 block mask, both ANDed with causal."""
    B, H, N, d = _shape(Q)
    bf = torch.bfloat16
    args = [_need("Q", Q, bf, (B, H, N, d)), _need("K", K, bf, (B, H, N, d)),
            _need("V", V, bf, (B, H, N, d)), _need("O", O, bf, (B, H, N, d)),
            _need("LSE", LSE, torch.float32, (B, H, N))]
    wl, wr = _window(window)
    check("fa_forward_masked", lib().fa_forward_masked(
        *args, B, H, N, d, float(scale), int(bool(causal)), wl, wr, _block_mask(block_mask, N),
        _stream(stream)))


@_on_one_device
def fa_backward_masked(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool, workspace,
                       window=None, block_mask=None, stream=None) -> None:
    ptrs, (B, H, N, d), ws, nbytes = _bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace,
                                               torch.bfloat16)
    wl, wr = _window(window)
    check("fa_backward_masked", lib().fa_backward_masked(
        *ptrs, B, H, N, d, float(scale), int(bool(causal)), wl, wr, _block_mask(block_mask, N),
        ws, nbytes, _stream(stream)))


def fa_launch_plan(B: int, H: int, N: int, d: int, causal: bool = False) -> dict:
    """How a plain call of this shape is distributed on the current GPU (launches
    nothing): ``fwd_persistent`` / ``bwd_persistent`` (persistent kernels, CTAs walking
    a list of tiles) and ``bwd_split`` (key tiles run as two CTAs)."""
    import ctypes
    fp, bp, bs = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    check("fa_launch_plan", lib().fa_launch_plan(B, H, N, d, int(causal), ctypes.addressof(fp),
                                                 ctypes.addressof(bp), ctypes.addressof(bs)))
    return {"fwd_persistent": bool(fp.value), "bwd_persistent": bool(bp.value),
            "bwd_split": bs.value}


def fa_dropout_rate(p: float) -> float:
    """The drop probability the dropout calls apply for ``p``: p rounded down to a
    multiple of 1/256. Raises ValueError for a rate they refuse (outside [0, 1), or
    in (0, 1/256), which would round down to no dropout)."""
    r = float(lib().fa_dropout_rate(float(p)))
    if r < 0:
        raise ValueError(f"dropout rate {p} is outside [0, 1) or below 1/256")
    return r


def _dropout(dropout):
    """(p, seed, offset, head_base) from dropout = (p, seed, offset) or (p, seed, offset,
    head_base); head_base (default 0) as for fa_forward_dropout_heads."""
    if dropout is None:
        return 0.0, 0, 0, 0
    p, seed, offset, *rest = dropout
    if len(rest) > 1:
        raise ValueError("dropout is (p, seed, offset) or (p, seed, offset, head_base)")
    head_base = int(rest[0]) if rest else 0
    return float(p), int(seed) & ((1 << 64) - 1), int(offset) & 0xFFFFFFFF, head_base


@_on_one_device
def fa_forward_dropout(Q, K, V, O, LSE, scale: float, causal: bool, dropout, window=None,
                       block_mask=None, stream=None) -> None:
    """fa_forward_masked with dropout=(p, seed, offset) on P (Philox-4x32-10 mask, one
    byte per element; the drop rate is p rounded down to a multiple of 1/256). A fourth
    element, head_base, draws the masks of heads head_base + b*H + h of a larger
    problem (fa_forward_dropout_heads)."""
    B, H, N, d = _shape(Q)
    bf = torch.bfloat16
    args = [_need("Q", Q, bf, (B, H, N, d)), _need("K", K, bf, (B, H, N, d)),
            _need("V", V, bf, (B, H, N, d)), _need("O", O, bf, (B, H, N, d)),
            _need("LSE", LSE, torch.float32, (B, H, N))]
    wl, wr = _window(window)
    p, seed, offset, head_base = _dropout(dropout)
    common = (*args, B, H, N, d, float(scale), int(bool(causal)), wl, wr,
              _block_mask(block_mask, N), p, seed, offset)
    if head_base:
        check("fa_forward_dropout_heads",
              lib().fa_forward_dropout_heads(*common, head_base, _stream(stream)))
    else:
        check("fa_forward_dropout", lib().fa_forward_dropout(*common, _stream(stream)))


@_on_one_device
def fa_backward_dropout(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool, workspace,
                        dropout, window=None, block_mask=None, stream=None) -> None:
    ptrs, (B, H, N, d), ws, nbytes = _bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace,
                                               torch.bfloat16)
    wl, wr = _window(window)
    p, seed, offset, head_base = _dropout(dropout)
    common = (*ptrs, B, H, N, d, float(scale), int(bool(causal)), wl, wr,
              _block_mask(block_mask, N), p, seed, offset)
    if head_base:
        check("fa_backward_dropout_heads", lib().fa_backward_dropout_heads(
            *common, head_base, ws, nbytes, _stream(stream)))
    else:
        check("fa_backward_dropout", lib().fa_backward_dropout(
            *common, ws, nbytes, _stream(stream)))


@_on_one_device
def fa_forward_f32(Q, K, V, O, LSE, scale: float, causal: bool, stream=None) -> None:
    B, H, N, d = _shape(Q)
    f = torch.float32
    args = [_need("Q", Q, f, (B, H, N, d)), _need("K", K, f, (B, H, N, d)),
            _need("V", V, f, (B, H, N, d)), _need("O", O, f, (B, H, N, d)),
            _need("LSE", LSE, f, (B, H, N))]
    check("fa_forward_f32", lib().fa_forward_f32(*args, B, H, N, d, float(scale),
                                                 int(bool(causal)), _stream(stream)))


def _bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, dtype):
    B, H, N, d = _shape(Q)
    s4 = (B, H, N, d)
    ptrs = [_need("Q", Q, dtype, s4), _need("K", K, dtype, s4), _need("V", V, dtype, s4),
            _need("O", O, dtype, s4), _need("dO", dO, dtype, s4),
            _need("LSE", LSE, torch.float32, (B, H, N)),
            _need("dQ", dQ, dtype, s4), _need("dK", dK, dtype, s4), _need("dV", dV, dtype, s4)]
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ptrs, (B, H, N, d), workspace.data_ptr(), workspace.numel() * workspace.element_size()


@_on_one_device
def fa_backward(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool, workspace,
                stream=None) -> None:
    ptrs, (B, H, N, d), ws, nbytes = _bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace,
                                               torch.bfloat16)
    check("fa_backward", lib().fa_backward(*ptrs, B, H, N, d, float(scale), int(bool(causal)),
                                           ws, nbytes, _stream(stream)))


def _ws(workspace):
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


@_on_one_device
def fa_backward_preprocess(O, dO, LSE, scale: float, causal: bool, workspace, stream=None):
    B, H, N, d = _shape(O)
    bf = torch.bfloat16
    ws, nbytes = _ws(workspace)
    check("fa_backward_preprocess", lib().fa_backward_preprocess(
        _need("O", O, bf, (B, H, N, d)), _need("dO", dO, bf, (B, H, N, d)),
        _need("LSE", LSE, torch.float32, (B, H, N)), B, H, N, d, float(scale),
        int(bool(causal)), ws, nbytes, _stream(stream)))


@_on_one_device
def fa_backward_main(Q, K, V, dO, dK, dV, scale: float, causal: bool, workspace, stream=None):
    B, H, N, d = _shape(Q)
    s4, bf = (B, H, N, d), torch.bfloat16
    ws, nbytes = _ws(workspace)
    check("fa_backward_main", lib().fa_backward_main(
        _need("Q", Q, bf, s4), _need("K", K, bf, s4), _need("V", V, bf, s4),
        _need("dO", dO, bf, s4), _need("dK", dK, bf, s4), _need("dV", dV, bf, s4),
        B, H, N, d, float(scale), int(bool(causal)), ws, nbytes, _stream(stream)))


@_on_one_device
def fa_backward_dq_convert(dQ, scale: float, workspace, stream=None):
    B, H, N, d = _shape(dQ)
    ws, nbytes = _ws(workspace)
    check("fa_backward_dq_convert", lib().fa_backward_dq_convert(
        _need("dQ", dQ, torch.bfloat16, (B, H, N, d)), B, H, N, d, float(scale), ws, nbytes,
        _stream(stream)))


@_on_one_device
def fa_backward_noalloc(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool,
                        stream=None) -> None:
    """fa_backward for callers that cannot allocate device memory: the workspace
    is a fixed 32 MiB array inside the library (one per GPU). Shapes needing more
    raise FAError (FA_ERR_UNSUPPORTED). Calls on one GPU share the array, so they
    must not overlap: keep them on one stream. The first call on a GPU does a
    one-time look-up of the array's address; make it before any stream capture."""
    B, H, N, d = _shape(Q)
    s4, bf = (B, H, N, d), torch.bfloat16
    ptrs = [_need("Q", Q, bf, s4), _need("K", K, bf, s4), _need("V", V, bf, s4),
            _need("O", O, bf, s4), _need("dO", dO, bf, s4),
            _need("LSE", LSE, torch.float32, (B, H, N)),
            _need("dQ", dQ, bf, s4), _need("dK", dK, bf, s4), _need("dV", dV, bf, s4)]
    check("fa_backward_noalloc", lib().fa_backward_noalloc(
        *ptrs, B, H, N, d, float(scale), int(bool(causal)), _stream(stream)))


@_on_one_device
def fa_backward_f16(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool, workspace,
                    stream=None) -> None:
    ptrs, (B, H, N, d), ws, nbytes = _bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace,
                                               torch.float16)
    check("fa_backward_f16", lib().fa_backward_f16(*ptrs, B, H, N, d, float(scale),
                                                   int(bool(causal)), ws, nbytes,
                                                   _stream(stream)))


@_on_one_device
def fa_backward_f32(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool, workspace,
                    stream=None) -> None:
    ptrs, (B, H, N, d), ws, nbytes = _bwd_args(Q, K, V, O, dO, LSE, dQ, dK, dV, workspace,
                                               torch.float32)
    check("fa_backward_f32", lib().fa_backward_f32(*ptrs, B, H, N, d, float(scale),
                                                   int(bool(causal)), ws, nbytes,
                                                   _stream(stream)))


def _shared_heads(Q, K):
    """(B, H, Hkv, N, d) of a call whose K/V heads are shared by groups of query heads."""
    B, H, N, d = _shape(Q)
    Hkv = _shape(K)[1]
    if Hkv < 1 or H % Hkv:
        raise ValueError(f"{H} query heads cannot share {Hkv} K/V heads evenly")
    return B, H, Hkv, N, d


def _device_array(name, t, dtype, shape):
    """Device pointer of a contiguous CUDA tensor, or None for None."""
    return None if t is None else _need(name, t, dtype, shape)


def _score(B, H, softcap, slopes, documents, prefix):
    """The C arguments softcap, slopes, documents, n_docs, prefix."""
    if slopes is None and documents is None and prefix is None:
        return 0.0 if softcap is None else float(softcap), None, None, 1, None
    n_docs = 1
    if documents is not None:
        if documents.dim() != 2 or documents.shape[1] < 2:
            raise ValueError("documents must be a [B, documents + 1] tensor of offsets, got shape "
                             f"{tuple(documents.shape)}")
        n_docs = int(documents.shape[1]) - 1
    if prefix is not None and prefix.dim() == 1 and documents is None:
        prefix = prefix.unsqueeze(1)
    return (0.0 if softcap is None else float(softcap),
            _device_array("slopes", slopes, torch.float32, (H,)),
            _device_array("documents", documents, torch.int32, (B, n_docs + 1)), n_docs,
            _device_array("prefix", prefix, torch.int32, (B, n_docs)))


def _forward_scored(name, dtype, Q, K, V, O, LSE, scale, causal, window, softcap, slopes,
                    documents, prefix, stream):
    B, H, Hkv, N, d = _shared_heads(Q, K)
    sq, sk = (B, H, N, d), (B, Hkv, N, d)
    args = (_need("Q", Q, dtype, sq), _need("K", K, dtype, sk), _need("V", V, dtype, sk),
            _need("O", O, dtype, sq), _need("LSE", LSE, torch.float32, (B, H, N)))
    wl, wr = _window(window)
    status = getattr(lib(), name)(
        *args, B, H, Hkv, N, d, float(scale), int(bool(causal)), wl, wr,
        *_score(B, H, softcap, slopes, documents, prefix), _stream(stream))
    if status:
        check(name, status)


def _backward_scored(name, dtype, Q, K, V, O, dO, LSE, dQ, dK, dV, scale, causal, workspace,
                     window, softcap, slopes, documents, prefix, stream):
    B, H, Hkv, N, d = _shared_heads(Q, K)
    sq, sk = (B, H, N, d), (B, Hkv, N, d)
    ptrs = [_need("Q", Q, dtype, sq), _need("K", K, dtype, sk), _need("V", V, dtype, sk),
            _need("O", O, dtype, sq), _need("dO", dO, dtype, sq),
            _need("LSE", LSE, torch.float32, (B, H, N)),
            _need("dQ", dQ, dtype, sq), _need("dK", dK, dtype, sk), _need("dV", dV, dtype, sk)]
    ws, nbytes = _ws(workspace)
    wl, wr = _window(window)
    check(name, getattr(lib(), name)(
        *ptrs, B, H, Hkv, N, d, float(scale), int(bool(causal)), wl, wr,
        *_score(B, H, softcap, slopes, documents, prefix), ws, nbytes, _stream(stream)))


@_on_one_device
def fa_forward_scored(Q, K, V, O, LSE, scale: float, causal: bool, window=None, softcap=None,
                      slopes=None, documents=None, prefix=None, stream=None) -> None:
    """fa_forward with shaped scores (bf16): capped at ``softcap`` by a tanh, lowered by
    ``slopes[h] * |i - j|``, within ``documents`` and with a ``prefix`` that every query
    of the document sees; K and V may have fewer heads than Q."""
    _forward_scored("fa_forward_scored", torch.bfloat16, Q, K, V, O, LSE, scale, causal, window,
                    softcap, slopes, documents, prefix, stream)


@_on_one_device
def fa_forward_scored_f16(Q, K, V, O, LSE, scale: float, causal: bool, window=None, softcap=None,
                          slopes=None, documents=None, prefix=None, stream=None) -> None:
    _forward_scored("fa_forward_scored_f16", torch.float16, Q, K, V, O, LSE, scale, causal,
                    window, softcap, slopes, documents, prefix, stream)


@_on_one_device
def fa_backward_scored(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool, workspace,
                       window=None, softcap=None, slopes=None, documents=None, prefix=None,
                       stream=None) -> None:
    _backward_scored("fa_backward_scored", torch.bfloat16, Q, K, V, O, dO, LSE, dQ, dK, dV, scale,
                     causal, workspace, window, softcap, slopes, documents, prefix, stream)


@_on_one_device
def fa_backward_scored_f16(Q, K, V, O, dO, LSE, dQ, dK, dV, scale: float, causal: bool,
                           workspace, window=None, softcap=None, slopes=None, documents=None,
                           prefix=None, stream=None) -> None:
    _backward_scored("fa_backward_scored_f16", torch.float16, Q, K, V, O, dO, LSE, dQ, dK, dV,
                     scale, causal, workspace, window, softcap, slopes, documents, prefix, stream)


def _cache4(codes, params, page_table, dtype, B, Hkv, d):
    """(codes, params, page table pointers), (page, n_pages, max_pages)."""
    if not isinstance(codes, _Tensor) or codes.dim() != 5:
        raise ValueError("codes must be a [pages, 2, K/V heads, page, d / 2] tensor")
    n_pages, _, _, page, _ = codes.shape
    if not isinstance(page_table, _Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [B, pages per sequence] tensor")
    max_pages = page_table.shape[1]
    return ((_need("codes", codes, torch.uint8, (n_pages, 2, Hkv, page, d // 2)),
             _need("params", params, dtype, (n_pages, 2, Hkv, page, 2)),
             _need("page_table", page_table, torch.int32, (B, max_pages))),
            (page, n_pages, max_pages))


def _cache4_rows(name, dtype, K, V, codes, params, page_table, positions, counts, stream):
    shape = B, Hkv, n, d = _shape(K)
    k, v = _need("K", K, dtype, shape), _need("V", V, dtype, shape)
    ptrs, sizes = _cache4(codes, params, page_table, dtype, B, Hkv, d)
    status = getattr(lib(), name)(
        k, v, *ptrs, _need("positions", positions, torch.int32, (B,)),
        None if counts is None else _need("counts", counts, torch.int32, (B,)), B, Hkv, n, d, *sizes,
        _stream(stream))
    if status:
        check(name, status)


def _cache4_attend(name, dtype, Q, O, LSE, codes, params, page_table, lengths, max_len, scale,
                   window_left, softcap, slopes, workspace, stream):
    shape = B, H, Nq, d = _shape(Q)
    Hkv = codes.shape[2] if codes.dim() == 5 else 0
    q, o = _need("Q", Q, dtype, shape), _need("O", O, dtype, shape)
    lse = _need("LSE", LSE, torch.float32, (B, H, Nq))
    ptrs, sizes = _cache4(codes, params, page_table, dtype, B, Hkv, d)
    ws, nbytes = (None, 0) if workspace is None else _ws(workspace)
    status = getattr(lib(), name)(
        q, o, lse, *ptrs, _need("lengths", lengths, torch.int32, (B,)), B, H, Hkv, Nq, d, *sizes,
        int(max_len), float(scale), _bound(window_left), 0.0 if softcap is None else float(softcap),
        None if slopes is None else _need("slopes", slopes, torch.float32, (H,)), ws, nbytes,
        _stream(stream))
    if status:
        check(name, status)


@_on_one_device
def fa_cache4_append(K, V, codes, params, page_table, positions, counts=None,
                     stream=None) -> None:
    """K, V (bf16 [B, Hkv, n, d]) into a 4-bit cache at positions[b] .. of sequence b."""
    _cache4_rows("fa_cache4_append", torch.bfloat16, K, V, codes, params, page_table, positions,
                 counts, stream)


@_on_one_device
def fa_cache4_append_f16(K, V, codes, params, page_table, positions, counts=None,
                         stream=None) -> None:
    _cache4_rows("fa_cache4_append_f16", torch.float16, K, V, codes, params, page_table,
                 positions, counts, stream)


@_on_one_device
def fa_cache4_read(K, V, codes, params, page_table, positions, counts=None, stream=None) -> None:
    """Rows of a 4-bit cache into K, V (bf16 [B, Hkv, n, d])."""
    _cache4_rows("fa_cache4_read", torch.bfloat16, K, V, codes, params, page_table, positions,
                 counts, stream)


@_on_one_device
def fa_cache4_read_f16(K, V, codes, params, page_table, positions, counts=None,
                       stream=None) -> None:
    _cache4_rows("fa_cache4_read_f16", torch.float16, K, V, codes, params, page_table, positions,
                 counts, stream)


@_on_one_device
def fa_cache4_attend(Q, O, LSE, codes, params, page_table, lengths, max_len: int, scale: float,
                     window_left: int = -1, softcap=None, slopes=None, workspace=None,
                     stream=None) -> None:
    """The last Nq tokens of each sequence over a 4-bit cache (bf16)."""
    _cache4_attend("fa_cache4_attend", torch.bfloat16, Q, O, LSE, codes, params, page_table,
                   lengths, max_len, scale, window_left, softcap, slopes, workspace, stream)


@_on_one_device
def fa_cache4_attend_f16(Q, O, LSE, codes, params, page_table, lengths, max_len: int,
                         scale: float, window_left: int = -1, softcap=None, slopes=None,
                         workspace=None, stream=None) -> None:
    _cache4_attend("fa_cache4_attend_f16", torch.float16, Q, O, LSE, codes, params, page_table,
                   lengths, max_len, scale, window_left, softcap, slopes, workspace, stream)


@_on_one_device
def fa_get_status(stream=None) -> int:
    """Synchronises the stream; returns the library status code (0 = ok, 4 = a
    kernel's bounded wait ran out since the last call)."""
    return int(lib().fa_get_status(_stream(stream)))


@_on_one_device
def fa_watchdog_selftest(timeout_ms: int, stream=None) -> None:
    check("fa_watchdog_selftest", lib().fa_watchdog_selftest(int(timeout_ms), _stream(stream)))


# ---------------------------------------------------------------- conveniences


def _default_scale(d: int, scale):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _masked(window, block_mask) -> bool:
    return window is not None or block_mask is not None


def _scored(q, k, window, block_mask, dropout, softcap, slopes, documents, prefix) -> bool:
    """Whether a call takes the scored entry points; windows of f16 tensors do as well."""
    return (softcap is not None or slopes is not None or documents is not None
            or prefix is not None or (k.dim() == 4 and k.shape[1] != q.shape[1])
            or (q.dtype == torch.float16 and window is not None and block_mask is None
                and dropout is None))


def _check_scored(q, block_mask, dropout) -> str:
    """The suffix of the scored entry points for q's type; refuses what they do not take."""
    if block_mask is not None or dropout is not None:
        raise ValueError("block_mask and dropout do not combine with softcap, slopes, documents, "
                         "prefix or shared K/V heads")
    if q.dtype is torch.bfloat16:
        return ""
    if q.dtype is not torch.float16:
        raise TypeError("softcap, slopes, documents, prefix and shared K/V heads are supported "
                        "for bf16 and f16 inputs")
    return "_f16"


def forward(q, k, v, causal: bool = False, scale=None, window=None, block_mask=None,
            dropout=None, softcap=None, slopes=None, documents=None, prefix=None):
    """(O, LSE) for bf16, f16 or fp32 q, k, v of shape [B, H, N, d] on the GPU.
    ``window`` / ``block_mask`` as for fa_forward_masked and ``dropout`` = (p, seed,
    offset) as for fa_forward_dropout (bf16 only; ``window`` f16 too).

    Shaped scores (bf16 and f16, see fa_forward_scored in include/fa.h): ``softcap`` caps
    the scores by c * tanh(s / c); ``slopes`` (fp32 [H]) subtracts slopes[h] * |i - j|;
    ``documents`` (int32 [B, M + 1]) holds the offsets of each row's documents, between
    which nothing is seen; ``prefix`` (int32 [B, M], [B] without documents) the number of
    first tokens that every query of the document sees. k and v may have fewer heads than
    q (a divisor): query head h uses head h // (H // Hkv)."""
    B, H, N, d = _shape(q)
    scale = _default_scale(d, scale)
    o = torch.empty_like(q)
    lse = q.new_empty((B, H, N), dtype=torch.float32)
    if _scored(q, k, window, block_mask, dropout, softcap, slopes, documents, prefix):
        fn = fa_forward_scored_f16 if _check_scored(q, block_mask, dropout) else fa_forward_scored
        fn(q, k, v, o, lse, scale, causal, window, softcap, slopes, documents, prefix)
    elif dropout is not None:
        if q.dtype != torch.bfloat16:
            raise TypeError("dropout is supported for bf16 inputs")
        fa_forward_dropout(q, k, v, o, lse, scale, causal, dropout, window, block_mask)
    elif _masked(window, block_mask):
        if q.dtype != torch.bfloat16:
            raise TypeError("window and block_mask are supported for bf16 inputs")
        fa_forward_masked(q, k, v, o, lse, scale, causal, window, block_mask)
    elif q.dtype == torch.bfloat16:
        fa_forward(q, k, v, o, lse, scale, causal)
    elif q.dtype == torch.float16:
        fa_forward_f16(q, k, v, o, lse, scale, causal)
    elif q.dtype == torch.float32:
        fa_forward_f32(q, k, v, o, lse, scale, causal)
    else:
        raise TypeError(f"unsupported dtype {q.dtype}: bf16, f16 or fp32")
    return o, lse


def workspace_for(q) -> torch.Tensor:
    B, H, N, d = _shape(q)
    n = max(1, fa_backward_workspace_size(B, H, N, d))
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def backward(q, k, v, o, lse, do, causal: bool = False, scale=None, workspace=None,
             window=None, block_mask=None, dropout=None, softcap=None, slopes=None,
             documents=None, prefix=None):
    """(dQ, dK, dV) of the loss <dO, O> (same masks, dropout and scores as the forward)."""
    B, H, N, d = _shape(q)
    scale = _default_scale(d, scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    scored = _scored(q, k, window, block_mask, dropout, softcap, slopes, documents, prefix)
    if workspace is not None:
        ws = workspace
    elif scored:
        ws = q.new_empty(max(1, fa_backward_scored_workspace_size(B, H, _shared_heads(q, k)[2], N, d)),
                         dtype=torch.uint8)
    else:
        ws = workspace_for(q)
    if scored:
        fn = (fa_backward_scored_f16 if _check_scored(q, block_mask, dropout)
              else fa_backward_scored)
        fn(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws, window, softcap, slopes,
           documents, prefix)
    elif dropout is not None:
        if q.dtype != torch.bfloat16:
            raise TypeError("dropout is supported for bf16 inputs")
        fa_backward_dropout(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws, dropout, window,
                            block_mask)
    elif _masked(window, block_mask):
        if q.dtype != torch.bfloat16:
            raise TypeError("window and block_mask are supported for bf16 inputs")
        fa_backward_masked(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws, window,
                           block_mask)
    elif q.dtype == torch.bfloat16:
        fa_backward(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws)
    elif q.dtype == torch.float16:
        fa_backward_f16(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws)
    elif q.dtype == torch.float32:
        fa_backward_f32(q, k, v, o, do, lse, dq, dk, dv, scale, causal, ws)
    else:
        raise TypeError(f"unsupported dtype {q.dtype}: bf16, f16 or fp32")
    return dq, dk, dv


_SLOPES_CONSTANT = "slopes are constants: they have no gradient"


class FlashAttentionFunction(torch.autograd.Function):
    """Differentiable exact attention through the library's forward and backward."""

    @staticmethod
    def forward(ctx, q, k, v, causal: bool = False, scale=None, window=None, block_mask=None,
                dropout=None, softcap=None, slopes=None, documents=None, prefix=None):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o, lse = forward(q, k, v, causal, scale, window, block_mask, dropout, softcap, slopes,
                         documents, prefix)
        ctx.save_for_backward(q, k, v, o, lse, slopes, documents, prefix)
        ctx.causal, ctx.scale, ctx.window, ctx.block_mask = causal, scale, window, block_mask
        ctx.dropout = dropout  # the backward regenerates the same keep mask
        ctx.softcap = softcap
        return o

    @staticmethod
    def backward(ctx, do):
        if ctx.needs_input_grad[9]:
            raise ValueError(_SLOPES_CONSTANT)
        q, k, v, o, lse, slopes, documents, prefix = ctx.saved_tensors
        dq, dk, dv = backward(q, k, v, o, lse, do.contiguous(), ctx.causal, ctx.scale,
                              window=ctx.window, block_mask=ctx.block_mask,
                              dropout=ctx.dropout, softcap=ctx.softcap, slopes=slopes,
                              documents=documents, prefix=prefix)
        return (dq, dk, dv) + (None,) * (len(ctx.needs_input_grad) - 3)


def attention(q, k, v, causal: bool = False, scale=None, window=None, block_mask=None,
              dropout=None, softcap=None, slopes=None, documents=None, prefix=None):
    """Differentiable attention; ``dropout`` = (p, seed, offset): pass a new offset (or
    seed) per call to draw a new mask. ``softcap``, ``slopes``, ``documents`` and
    ``prefix`` as for ``forward``; slopes are constants, and those that require a gradient are
    refused unless autograd is off.

    A backward pass may be captured into a CUDA graph, but not while an eager graph of the same
    leaves is alive (drop its outputs first): autograd would tie the captured pass to the
    eager one's stream, which ends the process."""
    if slopes is not None and slopes.requires_grad and torch.is_grad_enabled():
        raise ValueError(_SLOPES_CONSTANT)
    return FlashAttentionFunction.apply(q, k, v, causal, scale, window, block_mask, dropout,
                                        softcap, slopes, documents, prefix)


# ---------------------------------------------------------------- 4-bit cache


def _cache4_suffix(dtype) -> str:
    if dtype is torch.bfloat16:
        return ""
    if dtype is not torch.float16:
        raise TypeError(f"the 4-bit cache serves bf16 and f16 models, not {dtype}")
    return "_f16"


def cache4_empty(n_pages: int, kv_heads: int, page: int, d: int, dtype=torch.bfloat16,
                 device="cuda"):
    """(codes, params) of a cache of n_pages pages of ``page`` tokens (16, 32, 64, 128 or
    256) for K and V of kv_heads heads; see fa_cache4_append in include/fa.h."""
    _cache4_suffix(dtype)
    if page not in (16, 32, 64, 128, 256):
        raise ValueError(f"a page holds 16, 32, 64, 128 or 256 tokens, not {page}")
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    return (torch.empty(n_pages, 2, kv_heads, page, d // 2, dtype=torch.uint8, device=device),
            torch.empty(n_pages, 2, kv_heads, page, 2, dtype=dtype, device=device))


@_on_one_device
def cache4_append(codes, params, k, v, page_table, positions, counts=None) -> None:
    """Puts k, v ([B, kv heads, n, d], bf16 or f16) into the cache: token t of sequence b at
    position positions[b] + t, for t < counts[b] (all n without counts)."""
    _cache4_rows("fa_cache4_append" + _cache4_suffix(k.dtype), k.dtype, k, v, codes, params,
                 page_table, positions, counts, None)


@_on_one_device
def cache4_read(codes, params, page_table, positions, n: int, counts=None):
    """(k, v), [B, kv heads, n, d], as the cache holds them at positions[b] .. positions[b] +
    n - 1; zeros behind counts[b]."""
    shape = (page_table.shape[0], codes.shape[2], n, 2 * codes.shape[4])
    k, v = params.new_empty(shape), params.new_empty(shape)
    _cache4_rows("fa_cache4_read" + _cache4_suffix(params.dtype), params.dtype, k, v, codes,
                 params, page_table, positions, counts, None)
    return k, v


@_on_one_device
def cache4_attend(q, codes, params, page_table, lengths, scale=None, window_left: int = -1,
                  softcap=None, slopes=None, max_len=None):
    """(O, LSE) of the last tokens q ([B, H, n, d]; n = 1 when decoding) of sequences of
    ``lengths`` tokens (int32 [B], these tokens included) over a 4-bit cache. Scores as for
    ``forward``, causal. ``max_len``: a bound on the lengths known on the host (default: what
    the page table has room for); a close one gives a better cut of the work."""
    B, H, n, d = _shape(q)
    room = page_table.shape[1] * codes.shape[3]
    max_len = room if max_len is None else min(int(max_len), room)
    o = torch.empty_like(q)
    lse = q.new_empty((B, H, n), dtype=torch.float32)
    window_left = _bound(window_left)
    nbytes = fa_cache4_workspace_size(B, H, codes.shape[2], n, d, max_len, window_left)
    ws = q.new_empty(nbytes, dtype=torch.uint8) if nbytes else None
    _cache4_attend("fa_cache4_attend" + _cache4_suffix(q.dtype), q.dtype, q, o, lse, codes, params,
                   page_table, lengths, max_len, _default_scale(d, scale), window_left, softcap,
                   slopes, ws, None)
    return o, lse
