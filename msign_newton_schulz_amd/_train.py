"""ctypes binding of the training-block operators (include/msign_train.h).

Argument marshalling only, as in `_binding`: torch provides device memory and
the stream, every step of the computation runs in the HIP library, and there
is no fallback.  Outputs are queued on the current stream of the inputs'
device.  Nothing here records an autograd graph: a gradient is a call of its
own, and a forward call that an autograd graph leads into warns.
"""

from __future__ import annotations

import ctypes
import warnings
from typing import Optional, Tuple

import torch

from ._binding import _STATUS, MsignError, _load

_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTIVATIONS = {"silu": 0, "gelu": 1}  # FFN_SILU, FFN_GELU
MAX_TOP = 1024  # DISTILL_MAX_TOP
_FAR = 1 << 21  # the products' largest pitch


class _Block(ctypes.Structure):
    """ffn_block_t"""
    _fields_ = [("tokens", ctypes.c_int64), ("dim", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p),
                ("ldx", ctypes.c_int64), ("ld_gate", ctypes.c_int64), ("ld_up", ctypes.c_int64),
                ("ld_down", ctypes.c_int64)]


_lib = None


def _library():
    global _lib
    if _lib is not None:
        return _lib
    lib = _load()
    i64, i32, sz, vp, f = ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    bp = ctypes.POINTER(_Block)
    lib.ffn_forward_workspace_bytes.argtypes = [bp]
    lib.ffn_forward_workspace_bytes.restype = sz
    lib.ffn_backward_workspace_bytes.argtypes = [bp, vp, i64]
    lib.ffn_backward_workspace_bytes.restype = sz
    lib.ffn_forward.argtypes = [bp, vp, i64, vp, vp, i64, vp, sz, vp]
    lib.ffn_forward.restype = ctypes.c_int
    lib.ffn_backward.argtypes = [bp, vp, i64, vp, vp, i64, vp, vp, vp, vp, vp, sz, vp]
    lib.ffn_backward.restype = ctypes.c_int
    lib.add_rms_norm.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, i64, i32, i32, f, vp]
    lib.add_rms_norm.restype = ctypes.c_int
    lib.add_rms_norm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.add_rms_norm_backward_workspace_bytes.restype = sz
    lib.add_rms_norm_backward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, i64, i64, i32, i32, vp, sz, vp]
    lib.add_rms_norm_backward.restype = ctypes.c_int
    lib.distill_topk.argtypes = [vp, i64, vp, i32, vp, i32, vp, i64, vp, vp, i64, i64, i64, f, i32, vp]
    lib.distill_topk.restype = ctypes.c_int
    lib.msign_train_last_error.argtypes = []
    lib.msign_train_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _dtype(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _same_device(first: torch.Tensor, *others):
    if not first.is_cuda:
        raise ValueError("tensors must live on a GPU device")
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:  # (-1 on the CPU)
            raise ValueError("tensors must live on one GPU device")
    return first.device


def _like(t: torch.Tensor) -> torch.Tensor:
    """Contiguous memory of t's shape and dtype (half the host time of
    torch.empty, where t's own layout will do)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _matrix(t: torch.Tensor, most: int = 1 << 36):
    """t as [rows, last dim] with unit stride along a row and rows that do
    not overlap, at most `most` elements apart, a view where the strides allow
    it and else a copy: (tensor, address, rows, cols, pitch)."""
    cols = t.shape[-1]
    if t.is_contiguous():
        rows = t.shape[0] if t.dim() == 2 else _prod(t.shape[:-1])
        return t, t.data_ptr(), rows, cols, cols or 1
    if t.dim() != 2:
        t = t.reshape(-1, cols)
    if (cols > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and not cols <= t.stride(0) <= most):
        t = t.contiguous()
    rows = t.shape[0]
    return t, t.data_ptr(), rows, cols, t.stride(0) if rows > 1 else cols


def _prod(shape) -> int:
    n = 1
    for s in shape:
        n *= s
    return n


def _launch(device, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream."""
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device.index))
    if st != 0:
        raise MsignError(st, _library().msign_train_last_error().decode())


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the handle alone, without a Stream object around it, where torch offers it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _no_graph(name: str, gradient: str, *tensors) -> None:
    """Warns where autograd would expect a graph from `name`'s inputs to its
    outputs."""
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            warnings.warn(f"{name} records no autograd graph, so no gradient reaches its inputs through its outputs: "
                          f"call {gradient} for it, under torch.no_grad() or with detached tensors", stacklevel=3)
            return


def _scratch(nbytes: int, device, workspace: Optional[torch.Tensor]):
    """(pointer, bytes, owner) of a workspace of at least nbytes."""
    if nbytes == (1 << 64) - 1:
        raise MsignError(3, "invalid sizes for the workspace query")
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the inputs' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _block(x, w_gate, w_up, w_down, activation):
    """Checked operands of a feed-forward block: the struct, its device and
    the tensors that it points into."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    if x.dim() < 1 or w_gate.dim() != 2 or w_up.dim() != 2 or w_down.dim() != 2:
        raise ValueError("x needs a last dimension, the weights two")
    hidden, dim = w_gate.shape
    if x.shape[-1] != dim or w_up.shape != w_gate.shape or w_down.shape != (dim, hidden):
        raise ValueError("shapes must be x [..., dim], w_gate and w_up [hidden, dim], w_down [dim, hidden]")
    dtype = x.dtype
    if w_gate.dtype != dtype or w_up.dtype != dtype or w_down.dtype != dtype:
        raise ValueError("x and the weights must share one dtype")
    device = _same_device(x, w_gate, w_up, w_down)
    x, px, tokens, _, ldx = _matrix(x, _FAR)
    w_gate, pg, _, _, ldg = _matrix(w_gate, _FAR)
    w_up, pu, _, _, ldu = _matrix(w_up, _FAR)
    w_down, pd, _, _, ldd = _matrix(w_down, _FAR)
    b = _Block(tokens, dim, hidden, _dtype(x), act, px, pg, pu, pd, ldx, ldg, ldu, ldd)
    return b, device, (x, w_gate, w_up, w_down)


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, *,
              activation: str = "silu", save: bool = False, workspace: Optional[torch.Tensor] = None):
    """Gated feed-forward block (C ABI `ffn_forward`): g = x Wg^T, u = x Wu^T,
    y = (a(g) * u) Wd^T with a = "silu" or "gelu" (tanh form).

    x [..., dim], w_gate and w_up [hidden, dim], w_down [dim, hidden], one
    dtype (float32, bfloat16 or float16).  Returns y [..., dim], or with
    `save` (y, g, u), where g and u [..., hidden] are what
    `gated_ffn_backward` takes.  Sums are in float32; a(g) * u is rounded
    once to the dtype for the second product (with float16, values past 65504
    become infinite).  No autograd graph is recorded."""
    lib = _library()
    b, device, owners = _block(x, w_gate, w_up, w_down, activation)
    _no_graph("gated_ffn", "gated_ffn_backward", x, w_gate, w_up, w_down)
    y = _like(x)
    g = u = None
    pg = pu = None
    if save:
        g = torch.empty(x.shape[:-1] + (b.hidden,), dtype=x.dtype, device=device)
        u = torch.empty_like(g)
        pg, pu = g.data_ptr(), u.data_ptr()
    ws, nbytes, owner = _scratch(lib.ffn_forward_workspace_bytes(b), device, workspace)
    _launch(device, lib.ffn_forward, b, y.data_ptr(), b.dim or 1, pg, pu, b.hidden or 1, ws, nbytes)
    return (y, g, u) if save else y


def gated_ffn_backward(dy: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                       w_down: torch.Tensor, g: torch.Tensor, u: torch.Tensor, *, activation: str = "silu",
                       workspace: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of `gated_ffn` (C ABI `ffn_backward`) from dy, the gradient of
    y, and the saved g and u: (dx, dw_gate, dw_up, dw_down).  Sums are in
    float32; a(g) * u and the gradients of g and u are rounded once to the
    dtype for the products that take them."""
    lib = _library()
    b, device, owners = _block(x, w_gate, w_up, w_down, activation)
    if dy.shape != x.shape or g.shape != x.shape[:-1] + (b.hidden,) or u.shape != g.shape:
        raise ValueError("dy must have x's shape, g and u [..., hidden]")
    if dy.dtype != x.dtype or g.dtype != x.dtype or u.dtype != x.dtype:
        raise ValueError("dy, g and u must have x's dtype")
    _same_device(x, dy, g, u)
    dy, pdy, _, _, ld_dy = _matrix(dy, _FAR)
    g, pg, _, _, ld_act = _matrix(g, _FAR)
    u, pu, _, _, ld_u = _matrix(u, _FAR)
    if ld_act != ld_u:
        g, pg, _, _, ld_act = _matrix(g.contiguous())
        u, pu, _, _, ld_u = _matrix(u.contiguous())
    dx, dwg, dwu, dwd = _like(x), _like(w_gate), _like(w_gate), _like(w_down)
    ws, nbytes, owner = _scratch(lib.ffn_backward_workspace_bytes(b, pdy, ld_dy), device, workspace)
    _launch(device, lib.ffn_backward, b, pdy, ld_dy, pg, pu, ld_act, dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(),
            dwd.data_ptr(), ws, nbytes)
    return dx, dwg, dwu, dwd


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                 eps: float = 1e-6) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Root-mean-square norm with the residual's addition (C ABI
    `add_rms_norm`) over the last dimension: h = x + residual,
    rstd = (mean(h^2) + eps)^(-1/2), y = h rstd weight.

    Returns (y, h, rstd): y and h in x's dtype (h is x itself without a
    residual), rstd float32 with x's shape without the last dimension.
    weight [dim] may have another dtype than x.  No autograd graph is
    recorded: `add_rms_norm_backward` takes h and rstd."""
    lib = _library()
    shape = x.shape
    if x.dim() < 1 or weight.dim() != 1 or weight.shape[0] != shape[-1]:
        raise ValueError("x must be [..., dim] and weight [dim]")
    if residual is not None and (residual.shape != shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and dtype")
    device = _same_device(x, weight, residual)
    _no_graph("add_rms_norm", "add_rms_norm_backward", x, weight, residual)
    w = weight.contiguous()
    x2, px, rows, dim, ldx = _matrix(x)
    y = _like(x)
    h, pr, ldr, ph = x, None, 0, None
    if residual is not None:
        r2, pr, _, _, ldr = _matrix(residual)
        h = torch.empty_like(y)
        ph = h.data_ptr()
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    _launch(device, lib.add_rms_norm, px, ldx, pr, ldr, w.data_ptr(), y.data_ptr(), ph, rstd.data_ptr(), rows, dim,
            _dtype(x), _dtype(w), eps)
    return y, h, rstd


def add_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor, *,
                          dh: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of `add_rms_norm` (C ABI `add_rms_norm_backward`): (dx,
    dweight).  dx is the gradient of x and of the residual alike; dh, if
    given, is the gradient that reaches h by the residual path."""
    lib = _library()
    shape, dtype = h.shape, h.dtype
    if h.dim() < 1 or weight.dim() != 1 or weight.shape[0] != shape[-1]:
        raise ValueError("h must be [..., dim] and weight [dim]")
    if dy.shape != shape or dy.dtype != dtype or (dh is not None and (dh.shape != shape or dh.dtype != dtype)):
        raise ValueError("dy and dh must have h's shape and dtype")
    if rstd.shape != shape[:-1] or rstd.dtype != torch.float32:
        raise ValueError("rstd must be float32 with h's shape without the last dimension")
    device = _same_device(h, dy, dh, rstd, weight)
    w, s = weight.contiguous(), rstd.contiguous()
    dy2, pdy, rows, dim, ld_dy = _matrix(dy)
    h2, ph, _, _, ldh = _matrix(h)
    pdh, ld_dh = None, 0
    if dh is not None:
        dh2, pdh, _, _, ld_dh = _matrix(dh)
    dx, dw = _like(h), _like(weight)
    ws, nbytes, owner = _scratch(lib.add_rms_norm_backward_workspace_bytes(rows, dim), device, workspace)
    _launch(device, lib.add_rms_norm_backward, pdy, ld_dy, ph, ldh, s.data_ptr(), w.data_ptr(), pdh, ld_dh,
            dx.data_ptr(), dw.data_ptr(), rows, dim, _dtype(h), _dtype(w), ws, nbytes)
    return dx, dw


def _distill(logits, indices, teacher, temperature, grad, out):
    lib = _library()
    if logits.dim() < 1 or indices.dim() != logits.dim() or indices.shape[:-1] != logits.shape[:-1]:
        raise ValueError("logits must be [..., vocab] and indices [..., top] with the same leading dimensions")
    if teacher.shape != indices.shape:
        raise ValueError("teacher must have the shape of indices")
    if indices.dtype not in (torch.int32, torch.int64):
        raise TypeError("indices must be int32 or int64")
    device = _same_device(logits, indices, teacher, grad, out)
    idx, t = indices.contiguous(), teacher.contiguous()
    z, pz, rows, vocab, ldz = _matrix(logits)
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=device)
    pgrad, stride, pout = None, 0, None
    if out is not None:
        pgrad, pout = grad.data_ptr(), out.data_ptr()
        stride = grad.stride(0) if grad.dim() and rows > 1 else 0
    _launch(device, lib.distill_topk, pz, ldz, idx.data_ptr(), 1 if idx.dtype == torch.int64 else 0, t.data_ptr(),
            _dtype(t), pgrad, stride, loss.data_ptr(), pout, rows, vocab, idx.shape[-1], temperature, _dtype(z))
    return loss


def distill_topk(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor, *,
                 temperature: float = 1.0) -> torch.Tensor:
    """Distillation loss of each row of logits [..., vocab] against a teacher's
    top logits (C ABI `distill_topk`): with p = softmax(teacher / tau) over the
    row's entries and q = softmax(logits / tau) over the vocabulary,
    tau^2 sum_k p_k (log p_k - log q[indices_k]).

    indices [..., top] (int32 or int64; entries outside 0 .. vocab - 1, such
    as -1, are padding) and teacher [..., top] of any float dtype.  Returns
    float32 [...]; a row with padding only has loss 0.  No autograd graph is
    recorded: `distill_topk_grad` gives the logits' gradient."""
    _no_graph("distill_topk", "distill_topk_grad", logits, teacher)
    return _distill(logits, indices, teacher, temperature, None, None)


def distill_topk_grad(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor, grad: torch.Tensor, *,
                      temperature: float = 1.0, out: Optional[torch.Tensor] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """`distill_topk` and the gradient of sum(grad * loss) in one pass:
    (loss, dlogits).  grad is float32 [...], or one value for all rows (a
    tensor without dimensions); rows whose grad is 0 get zeros.  `out` takes
    dlogits: contiguous, with the shape and dtype of logits, and may be
    logits itself."""
    if grad.dtype != torch.float32:
        raise TypeError("grad must be float32")
    if grad.dim() > 0:
        if grad.shape != logits.shape[:-1]:
            raise ValueError("grad must have the logits' leading dimensions, or none")
        if grad.dim() > 1:
            grad = grad.reshape(-1)
        if grad.shape[0] > 1 and grad.stride(0) < 0:
            grad = grad.contiguous()
    if out is None:
        out = _like(logits)
    elif out.shape != logits.shape or out.dtype != logits.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous with the shape and dtype of logits")
    return _distill(logits, indices, teacher, temperature, grad, out), out
