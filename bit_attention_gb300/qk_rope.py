"""Queries and keys on their way into attention: per-head norms and the rotary
position rotation in one pass, with gradients.  Thin Python binding of the C
ABI in ``include/sage_rope.h``; every step runs in the CUDA kernels of
``_build/libsagefp4.so``, there is no fallback, and a failed call raises.

``sage_rope_*`` mirror the C entry points; ``forward`` and ``backward`` take
torch tensors, and ``norm_rope`` is the differentiable form (a
``torch.autograd.Function`` where a gradient is wanted, ``forward`` itself
where none is).
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import threading

from . import sage_fp4 as _fp4
from .sage_fp4 import EINVAL, LAYOUTS, SageFp4Error, sage_fp4_strides

_HEADER = os.path.join(os.path.dirname(_fp4._HEADER), "sage_rope.h")
_lock = threading.Lock()
_declared = set()


class sage_rope_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "Hq", "Hk", "D", "rot", "interleaved", "norm", "weight_f32",
                                              "max_pos")]
    _fields_ += [("eps", ctypes.c_float), ("pos_b_stride", ctypes.c_int64)]
    _fields_ += [(n, ctypes.c_void_p) for n in ("positions", "cos_sin", "q_weight", "k_weight", "status")]


def header_functions() -> list:
    """Names of the functions declared in include/sage_rope.h."""
    text = open(_HEADER).read()
    return sorted(set(re.findall(r"^[a-z_ 0-9\*]+?\b(sage_rope_[a-z_0-9]+)\s*\(", text, re.M)))


def lib() -> ctypes.CDLL:
    L = _fp4.load()
    if id(L) not in _declared:
        with _lock:
            vp, sz = ctypes.c_void_p, ctypes.c_size_t
            dp, sp = ctypes.POINTER(sage_rope_desc), ctypes.POINTER(sage_fp4_strides)
            sig = {
                "sage_rope_fwd": (ctypes.c_int, [dp] + [vp, sp] * 4 + [vp]),
                "sage_rope_workspace_bytes": (sz, [dp]),
                "sage_rope_bwd": (ctypes.c_int, [dp] + [vp, sp] * 6 + [vp, vp, vp, sz, vp]),
                "sage_rope_get_status": (ctypes.c_int, [vp, vp]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype, fn.argtypes = res, args
            _declared.add(id(L))
    return L


# ------------------------------------------------------------- raw entry points
def sage_rope_fwd(desc, q_ptr, q_strides, k_ptr, k_strides, qo_ptr, qo_strides, ko_ptr, ko_strides, stream) -> int:
    """Strides: sage_fp4_strides or None (contiguous [B, N, H, D])."""
    return lib().sage_rope_fwd(desc, q_ptr, q_strides, k_ptr, k_strides, qo_ptr, qo_strides, ko_ptr, ko_strides, stream)


def sage_rope_workspace_bytes(desc) -> int:
    return lib().sage_rope_workspace_bytes(desc)


def sage_rope_bwd(desc, gq_ptr, gq_strides, gk_ptr, gk_strides, q_ptr, q_strides, k_ptr, k_strides, dq_ptr, dq_strides,
                  dk_ptr, dk_strides, dqw_ptr, dkw_ptr, ws_ptr, ws_bytes, stream) -> int:
    return lib().sage_rope_bwd(desc, gq_ptr, gq_strides, gk_ptr, gk_strides, q_ptr, q_strides, k_ptr, k_strides, dq_ptr,
                               dq_strides, dk_ptr, dk_strides, dqw_ptr, dkw_ptr, ws_ptr, ws_bytes, stream)


def sage_rope_get_status(status_ptr, stream) -> int:
    return lib().sage_rope_get_status(status_ptr, stream)


# ------------------------------------------------------------- the table of angles
class RopeTable:
    """cos and sin of every position's angles and the status word of the calls
    that use them.  ``cos_sin``: float32 CUDA tensor [positions, rot], cos of
    pair i at column i, sin at rot / 2 + i."""

    def __init__(self, cos_sin):
        import torch
        if cos_sin.dtype != torch.float32 or not cos_sin.is_cuda or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise SageFp4Error(EINVAL, "cos_sin must be a contiguous float32 CUDA tensor [positions, rot]")
        if cos_sin.shape[1] % 16 or not 16 <= cos_sin.shape[1] <= 128:
            raise SageFp4Error(EINVAL, f"rot must be a multiple of 16 from 16 to 128, not {cos_sin.shape[1]}")
        self.cos_sin = cos_sin
        self.positions, self.rot = cos_sin.shape
        self.status = torch.zeros(4, dtype=torch.int32, device=cos_sin.device)
        self.status_ptr, self.cos_sin_ptr = self.status.data_ptr(), cos_sin.data_ptr()

    def get_status(self, stream=None) -> int:
        """Synchronise, return the status word (EINDEX: a position was outside
        the table) and reset it to 0."""
        import torch
        with torch.cuda.device(self.cos_sin.device):
            return sage_rope_get_status(self.status_ptr, _fp4._stream(stream))


def rope_table(positions: int, rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               trained: int | None = None, device=None) -> RopeTable:
    """The table of `positions` positions for `rot` rotated channels, made in 64 bits.

    The angle of pair i at position p is p * base^(-2 i / rot).  scaling:
    None; "linear": every angle divided by `factor` (position interpolation);
    "yarn": pairs that turn more than 32 times over the `trained` positions
    keep their angle, pairs that turn less than once are divided by `factor`,
    those between go linearly (in turns, as the method was published; some programs
    let the ramp run over the pair's index, which wants a RopeTable of one's own)
    from one to the other, and cos and sin are multiplied by 0.1 ln(factor) + 1."""
    import torch
    if positions < 1 or not math.isfinite(base) or base <= 0:
        raise SageFp4Error(EINVAL, f"positions {positions}, base {base}")
    if not (math.isfinite(factor) and factor > 0) or scaling not in (None, "linear", "yarn"):
        raise SageFp4Error(EINVAL, f"scaling {scaling!r} with factor {factor}")
    if scaling == "yarn" and (trained is None or trained < 1 or factor < 1):
        raise SageFp4Error(EINVAL, "yarn scaling needs the number of trained positions and a factor of 1 or more")
    dev = device or "cuda"
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    size = 1.0
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        keep = ((trained * inv / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        inv = inv * keep + inv / factor * (1.0 - keep)
        size = 0.1 * math.log(factor) + 1.0
    angle = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv
    return RopeTable(torch.cat([angle.cos() * size, angle.sin() * size], 1).float())


# ------------------------------------------------------------- torch conveniences
def _dims(x, layout: str, name: str):
    """(B, N, H, D) and strides of a bf16 CUDA tensor: 4-D in `layout` ("NHD" =
    [B, N, H, D], "HND" = [B, H, N, D]) or 3-D [N, H, D] ("NHD"; B = 1)."""
    import torch
    shape, stride = x.shape, x.stride()
    if x.dtype != torch.bfloat16 or not x.is_cuda or len(shape) not in (3, 4) or (stride[-1] != 1 and x.numel()):
        raise SageFp4Error(EINVAL, f"{name} must be a 3-D or 4-D bf16 CUDA tensor with a contiguous last axis")
    if layout == "NHD":
        if len(shape) == 3:
            n, h, d = shape
            sn, sh, _ = stride
            b, sb = 1, 0
        else:
            b, n, h, d = shape
            sb, sn, sh, _ = stride
    elif layout == "HND" and len(shape) == 4:
        b, h, n, d = shape
        sb, sh, sn, _ = stride
    else:
        raise SageFp4Error(EINVAL, f"layout must be one of {LAYOUTS} (NHD for 3-D tensors), not {layout!r}")
    # the stride of an axis of one element is anything
    return (b, n, h, d), sage_fp4_strides(sb if b > 1 else 0, sh if h > 1 else 0, sn if n > 1 else 0)


class _Call:
    """A checked call: the C description of q, k and what goes with them."""
    __slots__ = ("desc", "dq", "dk", "sq", "sk", "q", "k", "ndim", "dev", "device", "workspace")

    def __init__(self, q, k, positions, table, q_weight, k_weight, eps, interleaved, layout):
        import torch
        dq, self.sq = _dims(q, layout, "q")
        dk, self.sk = _dims(k, layout, "k")
        dev = q.get_device()
        B, N, Hq, D = dq
        Hk = dk[2]
        if dk != (B, N, Hk, D) or q.dim() != k.dim():
            raise SageFp4Error(EINVAL, f"q has shape {tuple(q.shape)}, k has {tuple(k.shape)}")
        ps = positions.shape
        if positions.dtype != torch.int32 or not positions.is_contiguous() or (ps != (N,) and ps != (B, N)):
            raise SageFp4Error(EINVAL, f"positions must be a contiguous int32 CUDA tensor [N] or [B, N] = {(B, N)}")
        if table.rot > D:
            raise SageFp4Error(EINVAL, f"the table rotates {table.rot} channels, a head has {D}")
        norm, f32 = q_weight is not None, False
        if norm != (k_weight is not None):
            raise SageFp4Error(EINVAL, "give both norm weights or neither")
        if norm:
            f32 = q_weight.dtype == torch.float32
            for w, nm in ((q_weight, "q_weight"), (k_weight, "k_weight")):
                if w.dtype != (torch.float32 if f32 else torch.bfloat16) or w.shape != (D,) or not w.is_contiguous():
                    raise SageFp4Error(EINVAL, f"{nm} must be a contiguous CUDA tensor [{D}], bf16 or float32 like the other")
            _on(dev, k, positions, table.cos_sin, q_weight, k_weight)
        else:
            _on(dev, k, positions, table.cos_sin)
        qp, kp, pp = q.data_ptr(), k.data_ptr(), positions.data_ptr()
        wqp, wkp = (q_weight.data_ptr(), k_weight.data_ptr()) if norm else (None, None)
        self.desc = sage_rope_desc(B, N, Hq, Hk, D, table.rot, bool(interleaved), norm, f32, table.positions, eps,
                                   N if len(ps) == 2 else 0, pp, table.cos_sin_ptr, wqp, wkp, table.status_ptr)
        self.dq, self.dk, self.q, self.k, self.ndim, self.dev, self.device = dq, dk, qp, kp, q.dim(), dev, q.device
        self.workspace = None

    def shape(self, dims, layout: str):
        b, n, h, d = dims
        if self.ndim == 3:
            return (n, h, d)
        return (b, n, h, d) if layout == "NHD" else (b, h, n, d)

    def new(self, dims, layout: str):
        """A new contiguous tensor and its strides (None: the C ABI's contiguous [B, N, H, D])."""
        import torch
        x = torch.empty(self.shape(dims, layout), dtype=torch.bfloat16, device=self.device)
        return x, self.dense(dims, layout)

    def dense(self, dims, layout: str):
        if layout == "NHD":
            return None
        _, n, h, d = dims
        return sage_fp4_strides(h * n * d, n * d, d)

    def gradient(self, g, dims, layout: str, name: str):
        """A gradient as the kernels read it, and its strides: contiguous, or any
        strides with a contiguous last axis and aligned rows (broadcast ones
        too), else a copy."""
        import torch
        if g.shape != self.shape(dims, layout) or g.dtype != torch.bfloat16 or g.get_device() != self.dev:
            raise SageFp4Error(EINVAL, f"{name} must be a bf16 tensor {self.shape(dims, layout)} on {self.device}")
        if g.data_ptr() % 16:
            g = g.clone(memory_format=torch.contiguous_format)
        if g.is_contiguous():
            return g, self.dense(dims, layout)
        if g.stride(-1) != 1 or any(s % 8 for s, n in zip(g.stride()[:-1], g.shape) if n > 1):
            return g.clone(memory_format=torch.contiguous_format), self.dense(dims, layout)
        return g, _dims(g, layout, name)[1]

    def forward(self, table, out_layout: str, out, stream, tensors):
        if out is None:
            if out_layout not in LAYOUTS or (self.ndim == 3 and out_layout != "NHD"):
                raise SageFp4Error(EINVAL, f"out_layout must be one of {LAYOUTS} (NHD for 3-D tensors), not {out_layout!r}")
            (qo, sqo), (ko, sko) = self.new(self.dq, out_layout), self.new(self.dk, out_layout)
        else:
            qo, ko = out
            (dqo, sqo), (dko, sko) = _dims(qo, out_layout, "out"), _dims(ko, out_layout, "out")
            if dqo != self.dq or dko != self.dk:
                raise SageFp4Error(EINVAL, f"out has sizes {dqo}, {dko}, the inputs {self.dq}, {self.dk}")
            _on(self.dev, qo, ko)
            _fp4._own_elements(qo, "out")
            _fp4._own_elements(ko, "out")
            self.in_place(qo, sqo, ko, sko)
        _fp4._call(lib().sage_rope_fwd, "sage_rope_fwd", self.dev, stream, (qo, ko, table.cos_sin, table.status, *tensors),
                   self.desc, self.q, self.sq, self.k, self.sk, qo.data_ptr(), sqo, ko.data_ptr(), sko)
        return qo, ko

    def in_place(self, qo, sqo, ko, sko):
        """Refuse results that start where another tensor does, but for each input's
        own place and strides."""
        if not qo.numel() or not ko.numel():
            return
        qp, kp = qo.data_ptr(), ko.data_ptr()
        same = lambda a, b: (a.b, a.h, a.n) == (b.b, b.h, b.n)  # noqa: E731
        if qp == kp or qp == self.k or kp == self.q or (qp == self.q and not same(sqo, self.sq)) or \
                (kp == self.k and not same(sko, self.sk)):
            raise SageFp4Error(EINVAL, "out shares memory with q or k other than in place")

    def backward(self, gq, gk, table, layout: str, grad_layout: str, stream, tensors):
        import torch
        gq, sgq = self.gradient(gq, self.dq, grad_layout, "gq")
        gk, sgk = self.gradient(gk, self.dk, grad_layout, "gk")
        (dq, sdq), (dk, sdk) = self.new(self.dq, layout), self.new(self.dk, layout)
        dwq = dwk = dwqp = dwkp = None
        if self.desc.norm:
            D = self.dq[3]
            dwq = torch.empty(D, dtype=torch.float32, device=self.device)
            dwk = torch.empty(D, dtype=torch.float32, device=self.device)
            dwqp, dwkp = dwq.data_ptr(), dwk.data_ptr()
        if self.workspace is None:
            self.workspace = lib().sage_rope_workspace_bytes(self.desc)
            if self.workspace == 0:
                raise SageFp4Error(EINVAL, f"sizes {self.dq}, {self.dk}")
        ws = torch.empty(self.workspace, dtype=torch.uint8, device=self.device)
        _fp4._call(lib().sage_rope_bwd, "sage_rope_bwd", self.dev, stream,
                   (dq, dk, dwq, dwk, ws, gq, gk, table.cos_sin, table.status, *tensors),
                   self.desc, gq.data_ptr(), sgq, gk.data_ptr(), sgk, self.q, self.sq, self.k, self.sk, dq.data_ptr(), sdq,
                   dk.data_ptr(), sdk, dwqp, dwkp, ws.data_ptr(), self.workspace)
        return dq, dk, dwq, dwk


def _on(device: int, *tensors) -> None:
    for t in tensors:
        if t.get_device() != device:
            raise SageFp4Error(EINVAL, f"tensors on cuda:{device} and {t.device}")


def _places(q, k, positions, q_weight, k_weight):
    """Address and strides of every tensor."""
    wq, wk = (None, None) if q_weight is None else (q_weight.data_ptr(), q_weight.stride()), \
        (None, None) if k_weight is None else (k_weight.data_ptr(), k_weight.stride())
    return (q.data_ptr(), q.stride(), k.data_ptr(), k.stride(), positions.data_ptr(), positions.stride(), *wq, *wk)


def forward(q, k, positions, table: RopeTable, q_weight=None, k_weight=None, eps: float = 1e-6,
            interleaved: bool = False, layout: str = "NHD", out_layout: str | None = None, out=None, stream=None):
    """Norms and rotation of bf16 q and k -> new tensors (q', k').

    q, k: [B, N, H, D] (layout "NHD"), [B, H, N, D] ("HND") or [tokens, H, D],
    any strides with a contiguous last axis and 16-byte aligned rows (slices of
    a packed projection); q and k may have different numbers of heads.
    positions: int32 [N] or [B, N].  table: the angles (rope_table).  q_weight,
    k_weight: the norms' weights [D], bf16 or float32; without them the heads
    are rotated only.  interleaved: pairs (2i, 2i + 1) instead of (i, i + rot/2).
    out_layout: layout of the results (the inputs' by default; "HND" is what
    the attention calls take).  out: (q', k') to write, the inputs themselves
    among the choices (each in its own place, with its own strides; no other memory
    is shared).  Asynchronous; a position outside the table gives zeros
    and EINDEX in table.get_status()."""
    call = _Call(q, k, positions, table, q_weight, k_weight, eps, interleaved, layout)
    return call.forward(table, layout if out_layout is None else out_layout, out, stream,
                        (q, k, positions, q_weight, k_weight))


def backward(gq, gk, q, k, positions, table: RopeTable, q_weight=None, k_weight=None, eps: float = 1e-6,
             interleaved: bool = False, layout: str = "NHD", grad_layout: str | None = None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of the forward with the same
    arguments, from the gradients gq, gk of its results (bf16, in grad_layout,
    its out_layout).  dq and dk are new contiguous tensors in `layout`; the
    weights' gradients are float32 [D], None without weights."""
    call = _Call(q, k, positions, table, q_weight, k_weight, eps, interleaved, layout)
    gl = layout if grad_layout is None else grad_layout
    if gl not in LAYOUTS or (call.ndim == 3 and gl != "NHD"):
        raise SageFp4Error(EINVAL, f"grad_layout must be one of {LAYOUTS} (NHD for 3-D tensors), not {gl!r}")
    return call.backward(gq, gk, table, layout, gl, stream, (q, k, positions, q_weight, k_weight))


def _autograd_function():
    import torch

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, positions, q_weight, k_weight, table, eps, interleaved, layout, out_layout):
            call = _Call(q, k, positions, table, q_weight, k_weight, eps, interleaved, layout)
            ctx.save_for_backward(q, k, positions, q_weight, k_weight, table.cos_sin)
            ctx.call, ctx.table, ctx.args = call, table, (eps, interleaved, layout)
            ctx.places = _places(q, k, positions, q_weight, k_weight)
            ctx.out_layout = layout if out_layout is None else out_layout
            return call.forward(table, ctx.out_layout, None, None, ())

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, gq, gk):
            *saved, _ = ctx.saved_tensors
            call = ctx.call
            if _places(*saved) != ctx.places:  # saved tensors that hooks have moved
                q, k, positions, q_weight, k_weight = saved
                call = _Call(q, k, positions, ctx.table, q_weight, k_weight, *ctx.args)
            dq, dk, dwq, dwk = call.backward(gq, gk, ctx.table, ctx.args[2], ctx.out_layout, None, ())
            if dwq is not None and not call.desc.weight_f32:
                dwq, dwk = dwq.to(torch.bfloat16), dwk.to(torch.bfloat16)
            return dq, dk, None, dwq, dwk, None, None, None, None, None

    return NormRope


_fn = None


def _tangents(*tensors) -> bool:
    """Whether one of them has a forward-mode tangent (which the autograd function refuses)."""
    from torch.autograd import forward_ad
    if forward_ad._current_level < 0:  # as nearly always: no call for each tensor
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def norm_rope(q, k, positions, table: RopeTable, q_weight=None, k_weight=None, eps: float = 1e-6,
              interleaved: bool = False, layout: str = "NHD", out_layout: str | None = None):
    """Norms and rotation of q and k (see ``forward``), differentiable in q, k
    and the norms' weights (backward only: forward-mode tangents are refused)."""
    import torch
    global _fn
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or (
            q_weight is not None and q_weight.requires_grad) or (k_weight is not None and k_weight.requires_grad)) or \
            _tangents(q, k, q_weight, k_weight):
        if _fn is None:
            _fn = _autograd_function()
        return _fn.apply(q, k, positions, q_weight, k_weight, table, eps, interleaved, layout, out_layout)
    return forward(q, k, positions, table, q_weight, k_weight, eps, interleaved, layout, out_layout)
