"""Expert selection, MXFP4 products and gradient clipping: the binding of these entry points (``include/nvfp4moe.h``
documents each) for PyTorch tensors.

At decode sizes a call takes a few microseconds on the GPU, so the binding's own time counts: arguments are checked
once, pointers and the raw stream go to ctypes as integers, and the device and stream are switched only where they are
not the current ones."""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import (BF16, F32, GROUP_MAX, LAYOUT_GEMM, LAYOUT_LOGICAL, MXFP4_SCALE_FLOOR, SCORE_SOFTMAX, Grad, Mxfp4Tensor,
               Nvfp4Error, SelectConfig, _check, lib)

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)  # storage of BF16 bits
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _elsewhere(t, stream):
    """Whether `t`'s device or `stream` is not the current one (then the call runs again inside _there)."""
    if not t.is_cuda:
        raise ValueError(f"a GPU tensor is needed, got one on {t.device}")
    return stream is not None or t.device.index != torch._C._cuda_getDevice()


@contextlib.contextmanager
def _there(stream, t, *others):
    """`t`'s device and `stream` (default: that device's current one) made current, so that outputs are allocated
    where they are used.  The call's tensors count as in use on a stream that is named: their memory, which belongs to
    another stream, is not handed out again before the call's work is done, even if the caller drops them."""
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    with torch.cuda.device(t.device), torch.cuda.stream(stream):
        yield
    if stream is not None:
        for each in (t, *others):
            if each is not None:
                each.record_stream(stream)


def _raw_stream(t):
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _need(where, t, name, dtypes, shape, device, contiguous=True):
    """ValueError unless t has one of the types, the shape, the device and (by default) contiguous elements."""
    if t.dtype not in dtypes or t.shape != shape or t.device != device:
        raise ValueError(f"{where}: {name} must be {' or '.join(str(d) for d in dtypes)} of shape {tuple(shape)} on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")


def _ld(where, t, name):
    """Elements from one row of a matrix to the next; ValueError unless its columns are consecutive."""
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1 and rows:
        raise ValueError(f"{where}: {name} must have consecutive columns, got strides {(ld, step)}")
    return ld if rows > 1 else cols  # (a single row's stride means nothing)


@functools.lru_cache(256)
def _select_config(*fields):
    """A pointer to the SelectConfig of these values."""
    return ctypes.pointer(SelectConfig(*fields))


def router_logits(x, w_router, out=None, stream=None):
    """nvfp4moe_router_logits: x [T,H] BF16, w_router [E,H] BF16 -> logits [T,E] f32 (router_topk's)."""
    if _elsewhere(x, stream):
        with _there(stream, x, w_router, out):
            return router_logits(x, w_router, out)
    T, H = x.shape
    E = w_router.shape[0]
    _need("router_logits", x, "x", _BF16, (T, H), x.device)
    _need("router_logits", w_router, "w_router", _BF16, (E, H), x.device)
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=x.device)
    else:
        _need("router_logits", out, "out", (torch.float32,), (T, E), x.device)
    _check(lib().nvfp4moe_router_logits(x.data_ptr(), T, H, w_router.data_ptr(), E, out.data_ptr(), _raw_stream(x)),
           "nvfp4moe_router_logits")
    return out


def _logits(where, logits, bias):
    """Checks logits and bias; the logits' type as the library names it, and their row stride."""
    kind = _TYPES.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        raise ValueError(f"{where}: logits must be a matrix of float32 or bfloat16, got {logits.dtype} "
                         f"{tuple(logits.shape)}")
    if bias is not None:
        _need(where, bias, "bias", (torch.float32,), logits.shape[1:], logits.device)
    return kind, _ld(where, logits, "logits")


def router_select(logits, k: int, bias=None, score: int = SCORE_SOFTMAX, renormalize: bool = True, scale: float = 1.0,
                  n_groups: int = 1, top_groups: int = 1, group_score: int = GROUP_MAX, out=None, stream=None):
    """nvfp4moe_router_select: logits [T,E] f32 or bf16 (rows may be strided), bias [E] f32 -> (ids [T,k] int32,
    probs [T,k] f32); `out` may hold the two, preallocated."""
    kind, ld = _logits("router_select", logits, bias)
    T, E = logits.shape
    if _elsewhere(logits, stream):
        with _there(stream, logits, bias, *(out or ())):
            return router_select(logits, k, bias, score, renormalize, scale, n_groups, top_groups, group_score, out)
    if out is None:
        ids = torch.empty((T, max(k, 0)), dtype=torch.int32, device=logits.device)
        probs = torch.empty((T, max(k, 0)), dtype=torch.float32, device=logits.device)
    else:
        ids, probs = out
        _need("router_select", ids, "out ids", (torch.int32,), (T, k), logits.device)
        _need("router_select", probs, "out probs", (torch.float32,), (T, k), logits.device)
    cfg = _select_config(E, k, score, 1 if renormalize else 0, scale, n_groups, top_groups, group_score, kind)
    st = lib().nvfp4moe_router_select(cfg, logits.data_ptr(), ld, T, None if bias is None else bias.data_ptr(),
                                      ids.data_ptr(), probs.data_ptr(), _raw_stream(logits))
    _check(st, "nvfp4moe_router_select")
    return ids, probs


def router_select_backward(logits, ids, dprobs, bias=None, score: int = SCORE_SOFTMAX, renormalize: bool = True,
                           scale: float = 1.0, out=None, stream=None):
    """nvfp4moe_router_select_backward: router_select's logits, bias and ids, and dprobs [T,k] f32 -> dlogits [T,E]
    of the logits' type."""
    kind, ld = _logits("router_select_backward", logits, bias)
    T, E = logits.shape
    k = ids.shape[-1]
    _need("router_select_backward", ids, "ids", (torch.int32,), (T, k), logits.device)
    _need("router_select_backward", dprobs, "dprobs", (torch.float32,), (T, k), logits.device)
    if _elsewhere(logits, stream):
        with _there(stream, logits, ids, dprobs, bias, out):
            return router_select_backward(logits, ids, dprobs, bias, score, renormalize, scale, out)
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    else:
        _need("router_select_backward", out, "out", (logits.dtype,), (T, E), logits.device, contiguous=False)
    cfg = _select_config(E, k, score, 1 if renormalize else 0, scale, 1, 1, GROUP_MAX, kind)
    st = lib().nvfp4moe_router_select_backward(cfg, logits.data_ptr(), ld, T,
                                               None if bias is None else bias.data_ptr(), ids.data_ptr(),
                                               dprobs.data_ptr(), out.data_ptr(), _ld("router_select_backward", out, "out"),
                                               _raw_stream(logits))
    _check(st, "nvfp4moe_router_select_backward")
    return out


def mxfp4_quantize(x, scale_round: int = MXFP4_SCALE_FLOOR, out=None, stream=None):
    """nvfp4moe_mxfp4_quantize, logical layout: x [rows, cols] BF16 (rows may be strided) -> (codes [rows, cols/2]
    uint8, scales [rows, cols/32] uint8)."""
    rows, cols = x.shape
    _need("mxfp4_quantize", x, "x", _BF16, (rows, cols), x.device, contiguous=False)
    if _elsewhere(x, stream):
        with _there(stream, x, *(out or ())):
            return mxfp4_quantize(x, scale_round, out)
    if out is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    else:
        codes, scales = out
        _need("mxfp4_quantize", codes, "out codes", (torch.uint8,), (rows, cols // 2), x.device)
        _need("mxfp4_quantize", scales, "out scales", (torch.uint8,), (rows, cols // 32), x.device)
    q = Mxfp4Tensor(codes.data_ptr(), scales.data_ptr(), 1, rows, cols, LAYOUT_LOGICAL)
    _check(lib().nvfp4moe_mxfp4_quantize(x.data_ptr(), _ld("mxfp4_quantize", x, "x"), q, scale_round, _raw_stream(x)),
           "nvfp4moe_mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, out=None, stream=None):
    """nvfp4moe_mxfp4_dequantize, logical layout: codes [rows, cols/2], scales [rows, cols/32] uint8 -> [rows, cols]
    bfloat16."""
    rows, half = codes.shape
    cols = 2 * half
    _need("mxfp4_dequantize", codes, "codes", (torch.uint8,), (rows, half), codes.device)
    _need("mxfp4_dequantize", scales, "scales", (torch.uint8,), (rows, cols // 32), codes.device)
    if _elsewhere(codes, stream):
        with _there(stream, codes, scales, out):
            return mxfp4_dequantize(codes, scales, out)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=codes.device)
    else:
        _need("mxfp4_dequantize", out, "out", _BF16, (rows, cols), codes.device, contiguous=False)
    q = Mxfp4Tensor(codes.data_ptr(), scales.data_ptr(), 1, rows, cols, LAYOUT_LOGICAL)
    _check(lib().nvfp4moe_mxfp4_dequantize(q, out.data_ptr(), _ld("mxfp4_dequantize", out, "out"), _raw_stream(codes)),
           "nvfp4moe_mxfp4_dequantize")
    return out


class Mxfp4Weights:
    """Caller-owned MXFP4 weights of n_mats matrices [rows, cols], in the products' layout."""

    def __init__(self, n_mats: int, rows: int, cols: int, device="cuda"):
        self.shape = (n_mats, rows, cols)
        q = Mxfp4Tensor(None, None, n_mats, rows, cols, LAYOUT_GEMM)
        nc, ns = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().nvfp4moe_mxfp4_bytes(q, ctypes.byref(nc), ctypes.byref(ns)), "nvfp4moe_mxfp4_bytes")
        self.codes = torch.empty((nc.value,), dtype=torch.uint8, device=device)
        self.scales = torch.empty((ns.value,), dtype=torch.uint8, device=device)
        self.Wq = Mxfp4Tensor(self.codes.data_ptr(), self.scales.data_ptr(), n_mats, rows, cols, LAYOUT_GEMM)

    def quantize_from(self, w, scale_round: int = MXFP4_SCALE_FLOOR, stream=None):
        """nvfp4moe_mxfp4_quantize: BF16 w [n_mats, rows, cols] -> these buffers, in place."""
        _need("Mxfp4Weights.quantize_from", w, "w", _BF16, self.shape, self.codes.device)
        if _elsewhere(w, stream):
            with _there(stream, w, self.codes, self.scales):
                return self.quantize_from(w, scale_round)
        _check(lib().nvfp4moe_mxfp4_quantize(w.data_ptr(), self.shape[2], self.Wq, scale_round, _raw_stream(w)),
               "nvfp4moe_mxfp4_quantize")
        return self

    def dequantize(self, stream=None):
        """nvfp4moe_mxfp4_dequantize: the values, [n_mats, rows, cols] bfloat16."""
        if _elsewhere(self.codes, stream):
            with _there(stream, self.codes, self.scales):
                return self.dequantize()
        out = torch.empty(self.shape, dtype=torch.bfloat16, device=self.codes.device)
        _check(lib().nvfp4moe_mxfp4_dequantize(self.Wq, out.data_ptr(), self.shape[2], _raw_stream(out)),
               "nvfp4moe_mxfp4_dequantize")
        return out


def mxfp4_workspace_bytes(M: int, K: int, n_mats: int = 1) -> int:
    n = lib().nvfp4moe_mxfp4_workspace_bytes(M, K, n_mats)
    if n == 0:
        raise Nvfp4Error(2, "nvfp4moe_mxfp4_workspace_bytes")
    return n


def mxfp4_alloc_workspace(M: int, K: int, n_mats: int = 1, device="cuda"):
    return torch.empty((mxfp4_workspace_bytes(M, K, n_mats),), dtype=torch.uint8, device=device)


def _mxfp4_product(where, x, offsets, W, scale_round, workspace, out, stream):
    E, N, K = W.shape
    M = x.shape[0]
    device = W.codes.device
    _need(where, x, "x", _BF16, (M, K), device, contiguous=False)
    if offsets is not None:
        _need(where, offsets, "offsets", (torch.int32,), (E + 1,), device)
    if _elsewhere(x, stream):
        with _there(stream, x, offsets, W.codes, W.scales, workspace, out):
            return _mxfp4_product(where, x, offsets, W, scale_round, workspace, out, None)
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=device)
    else:
        _need(where, out, "out", _BF16, (M, N), device, contiguous=False)
    if workspace is None:
        workspace = mxfp4_alloc_workspace(M, K, E, device)
    else:
        _need(where, workspace, "workspace", (torch.uint8,), (workspace.numel(),), device)
    ldx = _ld(where, x, "x")
    a = (W.Wq, out.data_ptr(), _ld(where, out, "out"), scale_round, workspace.data_ptr(), workspace.numel(), _raw_stream(x))
    if offsets is None:
        st = lib().nvfp4moe_mxfp4_linear(x.data_ptr(), M, ldx, *a)
    else:
        st = lib().nvfp4moe_mxfp4_grouped_linear(x.data_ptr(), M, ldx, offsets.data_ptr(), *a)
    _check(st, where)
    return out


def mxfp4_linear(x, W: Mxfp4Weights, scale_round: int = MXFP4_SCALE_FLOOR, workspace=None, out=None, stream=None):
    """nvfp4moe_mxfp4_linear: x [M,K] BF16 (rows may be strided), W one [N,K] matrix -> out [M,N] BF16.
    `workspace` (mxfp4_alloc_workspace) may be shared by calls that follow each other on one stream; `out` may not share
    elements with x."""
    return _mxfp4_product("nvfp4moe_mxfp4_linear", x, None, W, scale_round, workspace, out, stream)


def mxfp4_grouped_linear(x, offsets, W: Mxfp4Weights, scale_round: int = MXFP4_SCALE_FLOOR, workspace=None, out=None,
                         stream=None):
    """nvfp4moe_mxfp4_grouped_linear: x [R,K] BF16 with expert e's rows in [offsets[e], offsets[e+1]) (int32, on the
    GPU), W of E matrices [N,K] -> out [R,N] BF16; rows outside the offsets are not written."""
    return _mxfp4_product("nvfp4moe_mxfp4_grouped_linear", x, offsets, W, scale_round, workspace, out, stream)


class GradSet:
    """The tensors that clip_grad_norm works on: FP32 or BF16, contiguous, on one GPU.  `out` (default: in place)
    receives the clipped ones.  Holds the tensors and their plan on the GPU; make a new one if they move.  Making one
    copies the plan to the GPU and waits for the copy: once, before the steps, for gradients that stay where they are,
    and outside a graph's capture."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if not self.grads or len(self.out) != len(self.grads):
            raise ValueError("GradSet: needs at least one gradient, and an output for each")
        self.device = self.grads[0].device
        for g, o in zip(self.grads, self.out):
            _need("GradSet", g, "a gradient", tuple(_TYPES), g.shape, self.device)
            _need("GradSet", o, "an output", (g.dtype,), g.shape, self.device)
        if self.device.type != "cuda":
            raise ValueError(f"GradSet: GPU tensors are needed, got some on {self.device}")
        table = (Grad * len(self.grads))(*[Grad(g.data_ptr(), o.data_ptr(), g.numel(), _TYPES[g.dtype])
                                           for g, o in zip(self.grads, self.out)])
        size, n = ctypes.c_size_t(), ctypes.c_int64()
        _check(lib().nvfp4moe_grad_plan_bytes(table, len(table), ctypes.byref(size), ctypes.byref(n)),
               "nvfp4moe_grad_plan_bytes")
        self.n_chunks = n.value
        host = torch.empty((size.value // 8,), dtype=torch.int64)
        _check(lib().nvfp4moe_grad_plan(table, len(table), host.data_ptr(), size.value), "nvfp4moe_grad_plan")
        self.plan = host.to(self.device)


def clip_grad_norm(grads: GradSet, max_norm: float, stream=None):
    """nvfp4moe_clip_grad_norm: the global norm (float64 [1], on the GPU); the set's outputs hold the gradients scaled
    to at most max_norm (unchanged if the norm is not finite).  max_norm = inf takes the norm only."""
    if _elsewhere(grads.plan, stream):
        with _there(stream, grads.plan, *grads.grads, *grads.out):
            return clip_grad_norm(grads, max_norm)
    words = lib().nvfp4moe_clip_workspace_bytes() // 8
    buf = torch.empty((1 + words,), dtype=torch.float64, device=grads.device)  # the norm, then the partial sums
    at = buf.data_ptr()
    _check(lib().nvfp4moe_clip_grad_norm(grads.plan.data_ptr(), grads.n_chunks, max_norm, at, at + 8, 8 * words,
                                         _raw_stream(buf)), "nvfp4moe_clip_grad_norm")
    return buf[:1]
