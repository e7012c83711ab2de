"""The layer's training form: layer norm, tokens into expert order and back,
the routing's gradient and AdamW, each with its backward pass.

The same thin ctypes marshalling as the package's other calls (C names, device
pointers, the current CUDA stream of the tensors' device), over the training
section of ``include/moe_api.h``.  Outputs may be passed in; else torch
allocates them.  Tensors are contiguous CUDA tensors of one device.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

__all__ = [
    "MoeTokenShape", "MoeTokenMap", "MoeAdamwTensors", "moe_layer_norm", "moe_layer_norm_backward",
    "layer_norm_workspace", "moe_layer_norm_workspace_bytes", "moe_token_map", "moe_token_map_workspace_bytes",
    "token_map_workspace", "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
    "moe_route_backward", "moe_adamw", "adamw_tensors",
]

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
STATE_F32, STATE_MXFP8 = 0, 1

_P, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class _NormShape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("cols", _I32), ("dtype", _I32), ("w_dtype", _I32), ("eps", _F)]


class _TokenShape(ctypes.Structure):
    _fields_ = [(n, _I32) for n in ("T", "E_global", "E_local", "expert_offset", "top_k", "num_shared", "hidden",
                                    "dtype")]


class _AdamwTensor(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("p", "g", "m", "v", "m_scale", "v_scale")] + [("n", _I64)]


class _AdamwConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
               [("step", _I64), ("seed", ctypes.c_uint64), ("g_dtype", _I32), ("state", _I32)]


SIGS = {
    "moe_layer_norm_workspace_bytes": [_I64, _I32, _P],
    "moe_layer_norm": [_P] * 10,
    "moe_layer_norm_backward": [_P] * 11 + [_SZ, _P],
    "moe_token_map_workspace_bytes": [_P, _P],
    "moe_token_map": [_P] * 6 + [_SZ, _P],
    "moe_permute": [_P] * 5,
    "moe_permute_backward": [_P] * 5,
    "moe_unpermute": [_P] * 6,
    "moe_unpermute_backward": [_P] * 8,
    "moe_route_backward": [_P, _P, _F] + [_P] * 6,
    "moe_adamw": [_P, _I32, _P, _P, _P],
}


def _call(name, *args):
    from . import _call as call

    return call(name, *args)


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(name, t, dtype=None, shape=None, device=None):
    """A contiguous CUDA tensor of the given type, shape and device; None passes."""
    if t is None:
        return
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s: expected a contiguous CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s: expected a tensor on %s, got %s" % (name, device, t.device))


def _rows_dtype(name, t):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError("%s: expected bfloat16, float16 or float32, got %s" % (name, t.dtype))
    return d


# ------------------------------------------------------------------ layer norm
def _norm_args(x, weight, bias, eps):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("layer norm: expected rows of at least one column")
    cols = x.shape[-1]
    rows = x.numel() // cols
    dtype = w_dtype = _rows_dtype("x", x)
    for n, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if t.dtype != x.dtype and t.dtype != torch.float32:
                raise ValueError("%s: expected float32 or the rows' type, got %s" % (n, t.dtype))
            _check(n, t, None, (cols,), x.device)
            w_dtype = _DTYPES[t.dtype]
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias: expected one type, got %s and %s" % (weight.dtype, bias.dtype))
    return _NormShape(rows, cols, dtype, w_dtype, eps), rows, cols


def moe_layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5, y=None, h=None, mean=None, rstd=None):
    """Layer norm of h = x + residual over the last dimension: (y, h, mean, rstd),
    with mean and rstd fp32 [rows] for the backward pass.  Without a residual h is x."""
    _check("x", x)
    s, rows, _ = _norm_args(x, weight, bias, eps)
    for n, t in (("residual", residual), ("y", y), ("h", h)):
        _check(n, t, x.dtype, x.shape, x.device)
    for n, t in (("mean", mean), ("rstd", rstd)):
        _check(n, t, torch.float32, (rows,), x.device)
    if y is None:
        y = torch.empty_like(x)
    if residual is None:
        h = x
    elif h is None:
        h = torch.empty_like(x)
    if mean is None:
        mean = torch.empty(rows, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    _call("moe_layer_norm", ctypes.byref(s), x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(bias),
          h.data_ptr(), y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _stream(x))
    return y, h, mean, rstd


def moe_layer_norm_workspace_bytes(rows: int, cols: int) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_layer_norm_workspace_bytes", rows, cols, ctypes.byref(n))
    return n.value


def layer_norm_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """Scratch of moe_layer_norm_backward (torch allocates, 256-byte aligned)."""
    return torch.empty(moe_layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=device)


def moe_layer_norm_backward(dy, h, mean, rstd, weight=None, dh=None, bias_grad=True, dx=None, dweight=None,
                            dbias=None, ws=None):
    """(dx, dweight, dbias) of moe_layer_norm.  dh: the gradient that reaches h beside the norm, added to dx.
    dweight (fp32) is None without a weight, dbias (fp32) without bias_grad."""
    _check("h", h)
    s, rows, cols = _norm_args(h, weight, None, 0.0)
    for n, t in (("dy", dy), ("dh", dh), ("dx", dx)):
        _check(n, t, h.dtype, h.shape, h.device)
    for n, t in (("mean", mean), ("rstd", rstd)):
        _check(n, t, torch.float32, (rows,), h.device)
    for n, t in (("dweight", dweight), ("dbias", dbias)):
        _check(n, t, torch.float32, (cols,), h.device)
    _check("ws", ws, torch.uint8, None, h.device)
    if dx is None:
        dx = torch.empty_like(h)
    if weight is None:
        dweight = None
    elif dweight is None:
        dweight = torch.empty(cols, dtype=torch.float32, device=h.device)
    if not bias_grad:
        dbias = None
    elif dbias is None:
        dbias = torch.empty(cols, dtype=torch.float32, device=h.device)
    if ws is None and (dweight is not None or dbias is not None):
        ws = layer_norm_workspace(rows, cols, h.device)
    _call("moe_layer_norm_backward", ctypes.byref(s), dy.data_ptr(), h.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
          _ptr(weight), _ptr(dh), dx.data_ptr(), _ptr(dweight), _ptr(dbias), _ptr(ws),
          0 if ws is None else ws.numel(), _stream(h))
    return dx, dweight, dbias


# ------------------------------------------------------------------ tokens <-> rows
@dataclasses.dataclass
class MoeTokenShape:
    """Shape of the training form's token calls (see moe_token_shape in moe_api.h; the rows' type is the tensors')."""
    T: int
    E_global: int
    E_local: int
    expert_offset: int
    top_k: int
    num_shared: int
    hidden: int

    @property
    def kp(self):
        return self.top_k + self.num_shared

    def c(self, dtype: int = 0) -> _TokenShape:
        return _TokenShape(self.T, self.E_global, self.E_local, self.expert_offset, self.top_k, self.num_shared,
                           self.hidden, dtype)


@dataclasses.dataclass
class MoeTokenMap:
    """a_map int32 [T*k'] (row -> slot), c_map int32 [T, k'] (slot -> row or -1),
    expert_offsets int32 [E_local + num_shared + 1]."""
    a_map: torch.Tensor
    c_map: torch.Tensor
    expert_offsets: torch.Tensor


def moe_token_map_workspace_bytes(shape: MoeTokenShape) -> int:
    n = ctypes.c_size_t(0)
    s = shape.c()
    _call("moe_token_map_workspace_bytes", ctypes.byref(s), ctypes.byref(n))
    return n.value


def token_map_workspace(shape: MoeTokenShape, device="cuda") -> torch.Tensor:
    """Scratch of moe_token_map (torch allocates, 256-byte aligned)."""
    return torch.empty(moe_token_map_workspace_bytes(shape), dtype=torch.uint8, device=device)


def moe_token_map(shape: MoeTokenShape, topk_ids, ws=None, maps: MoeTokenMap = None) -> MoeTokenMap:
    """Sorts the slots of topk_ids int32 [T, k'] by expert (the maps of moe_sort, in buffers of their own)."""
    dev, kp, n = topk_ids.device, shape.kp, shape.T * shape.kp
    _check("topk_ids", topk_ids, torch.int32, (shape.T, kp))
    Et = shape.E_local + shape.num_shared
    if maps is None:
        maps = MoeTokenMap(torch.empty(n, dtype=torch.int32, device=dev),
                           torch.empty((shape.T, kp), dtype=torch.int32, device=dev),
                           torch.empty(Et + 1, dtype=torch.int32, device=dev))
    else:
        _check("a_map", maps.a_map, torch.int32, (n,), dev)
        _check("c_map", maps.c_map, torch.int32, (shape.T, kp), dev)
        _check("expert_offsets", maps.expert_offsets, torch.int32, (Et + 1,), dev)
    _check("ws", ws, torch.uint8, None, dev)
    if ws is None:
        ws = token_map_workspace(shape, dev)
    s = shape.c()
    _call("moe_token_map", ctypes.byref(s), topk_ids.data_ptr(), maps.a_map.data_ptr(), maps.c_map.data_ptr(),
          maps.expert_offsets.data_ptr(), ws.data_ptr(), ws.numel(), _stream(topk_ids))
    return maps


def _tokens(shape, maps, tokens, rows):
    """Checks token-major and row-major operands (name, tensor) against the shape: (C shape, dtype, device)."""
    first = (tokens + rows)[0][1]
    dt, dev = first.dtype, first.device
    d = _rows_dtype((tokens + rows)[0][0], first)
    for n, t in tokens:
        _check(n, t, dt, (shape.T, shape.hidden), dev)
    for n, t in rows:
        _check(n, t, dt, (shape.T * shape.kp, shape.hidden), dev)
    _check("c_map", maps.c_map, torch.int32, (shape.T, shape.kp), dev)
    return shape.c(d), dt, dev


def moe_permute(shape: MoeTokenShape, x, maps: MoeTokenMap, rows=None):
    """x [T, H] -> rows [T*k', H] in expert order; rows from expert_offsets[-1] on are not touched."""
    s, dt, dev = _tokens(shape, maps, [("x", x)], [("rows", rows)])
    if rows is None:
        rows = torch.empty((shape.T * shape.kp, shape.hidden), dtype=dt, device=dev)
    _call("moe_permute", ctypes.byref(s), x.data_ptr(), maps.c_map.data_ptr(), rows.data_ptr(), _stream(x))
    return rows


def moe_permute_backward(shape: MoeTokenShape, drows, maps: MoeTokenMap, dx=None):
    """Gradient of moe_permute: the sum of each token's rows."""
    s, dt, dev = _tokens(shape, maps, [("dx", dx)] if dx is not None else [], [("drows", drows)])
    if dx is None:
        dx = torch.empty((shape.T, shape.hidden), dtype=dt, device=dev)
    _call("moe_permute_backward", ctypes.byref(s), drows.data_ptr(), maps.c_map.data_ptr(), dx.data_ptr(),
          _stream(drows))
    return dx


def moe_unpermute(shape: MoeTokenShape, rows, topk_w, maps: MoeTokenMap, out=None):
    """rows [T*k', H] in expert order -> out [T, H], weighted with topk_w fp32 [T, k'] and summed per token."""
    s, dt, dev = _tokens(shape, maps, [("out", out)] if out is not None else [], [("rows", rows)])
    _check("topk_w", topk_w, torch.float32, (shape.T, shape.kp), dev)
    if out is None:
        out = torch.empty((shape.T, shape.hidden), dtype=dt, device=dev)
    _call("moe_unpermute", ctypes.byref(s), rows.data_ptr(), topk_w.data_ptr(), maps.c_map.data_ptr(),
          out.data_ptr(), _stream(rows))
    return out


def moe_unpermute_backward(shape: MoeTokenShape, dout, rows, topk_w, maps: MoeTokenMap, dy=None, dw=None):
    """Gradients of moe_unpermute: (dy [T*k', H] of the rows, dw fp32 [T, k'] of the weights).  dy may be rows;
    rows from expert_offsets[-1] on are not touched."""
    s, dt, dev = _tokens(shape, maps, [("dout", dout)], [("rows", rows), ("dy", dy)])
    _check("topk_w", topk_w, torch.float32, (shape.T, shape.kp), dev)
    _check("dw", dw, torch.float32, (shape.T, shape.kp), dev)
    if dy is None:
        dy = torch.empty_like(rows)
    if dw is None:
        dw = torch.empty_like(topk_w)
    _call("moe_unpermute_backward", ctypes.byref(s), dout.data_ptr(), rows.data_ptr(), topk_w.data_ptr(),
          maps.c_map.data_ptr(), dy.data_ptr(), dw.data_ptr(), _stream(rows))
    return dy, dw


# ------------------------------------------------------------------ routing gradient
def moe_route_backward(shape: MoeTokenShape, topk_ids, topk_w, dtopk_w, shared_logit=None, shared_scale=1.0,
                       dlogits=None, dshared=None):
    """Gradient of moe_route: (dlogits fp32 [T, E_global], dshared fp32 [T, num_shared] or None)."""
    dev, kp = topk_ids.device, shape.kp
    _check("topk_ids", topk_ids, torch.int32, (shape.T, kp))
    _check("topk_w", topk_w, torch.float32, (shape.T, kp), dev)
    _check("dtopk_w", dtopk_w, torch.float32, (shape.T, kp), dev)
    _check("dlogits", dlogits, torch.float32, (shape.T, shape.E_global), dev)
    _check("dshared", dshared, torch.float32, (shape.T, shape.num_shared), dev)
    _check("shared_logit", shared_logit, torch.bfloat16, (shape.T, shape.num_shared), dev)
    if dlogits is None:
        dlogits = torch.empty((shape.T, shape.E_global), dtype=torch.float32, device=dev)
    if not shape.num_shared:
        dshared = None
    elif dshared is None:
        dshared = torch.empty((shape.T, shape.num_shared), dtype=torch.float32, device=dev)
    s = shape.c()
    _call("moe_route_backward", ctypes.byref(s), _ptr(shared_logit), shared_scale, topk_ids.data_ptr(),
          topk_w.data_ptr(), dtopk_w.data_ptr(), dlogits.data_ptr(), _ptr(dshared), _stream(topk_ids))
    return dlogits, dshared


# ------------------------------------------------------------------ AdamW
class MoeAdamwTensors:
    """The tensors of moe_adamw, checked once: lists of params (fp32), grads (bf16
    or fp32) and states, entry i of each belonging together.  States are fp32 m and
    v, or uint8 E4M3 codes of m and sqrt(v) with uint8 E8M0 scales (one per 32
    elements).  The object holds the tensors; gradients are read from these
    buffers at every step (accumulate into them, or build another object)."""

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None):
        mx = m_scale is not None
        if mx != (v_scale is not None):
            raise ValueError("m_scale and v_scale: expected both or none")
        lists = [params, grads, m, v] + ([m_scale, v_scale] if mx else [])
        if any(len(x) != len(params) for x in lists):
            raise ValueError("expected lists of one length, got %s" % [len(x) for x in lists])
        self.params, self.grads, self.m, self.v, self.m_scale, self.v_scale = params, grads, m, v, m_scale, v_scale
        self.state = STATE_MXFP8 if mx else STATE_F32
        self.device = params[0].device if params else torch.device("cuda")
        g_dtype = grads[0].dtype if grads else torch.float32
        if g_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("grads: expected bfloat16 or float32, got %s" % g_dtype)
        self.g_dtype = _DTYPES[g_dtype]
        s_dtype = torch.uint8 if mx else torch.float32
        for i, p in enumerate(params):
            _check("params[%d]" % i, p, torch.float32, None, self.device)
            _check("grads[%d]" % i, grads[i], g_dtype, p.shape, self.device)
            _check("m[%d]" % i, m[i], s_dtype, p.shape, self.device)
            _check("v[%d]" % i, v[i], s_dtype, p.shape, self.device)
            if mx:
                blocks = ((p.numel() + 31) // 32,)
                _check("m_scale[%d]" % i, m_scale[i], torch.uint8, blocks, self.device)
                _check("v_scale[%d]" % i, v_scale[i], torch.uint8, blocks, self.device)
        self._c = (_AdamwTensor * len(params))(*[
            _AdamwTensor(*[x[i].data_ptr() for x in lists], *([] if mx else [None, None]), p.numel())
            for i, p in enumerate(params)])


def adamw_tensors(params, grads, mxfp8: bool = False) -> MoeAdamwTensors:
    """MoeAdamwTensors with zero states, fp32 or MXFP8."""
    if not mxfp8:
        return MoeAdamwTensors(params, grads, [torch.zeros_like(p) for p in params],
                               [torch.zeros_like(p) for p in params])
    codes = [[torch.zeros_like(p, dtype=torch.uint8) for p in params] for _ in range(2)]
    scales = [[torch.zeros((p.numel() + 31) // 32, dtype=torch.uint8, device=p.device) for p in params]
              for _ in range(2)]
    return MoeAdamwTensors(params, grads, codes[0], codes[1], scales[0], scales[1])


def moe_adamw(tensors: MoeAdamwTensors, step: int, lr: float, betas=(0.9, 0.999), eps: float = 1e-8,
              weight_decay: float = 0.01, grad_scale=None, seed: int = 0):
    """One AdamW step (step counts from 1) on the tensors, in place.  grad_scale: fp32 device tensor of one element
    that multiplies the gradients (not finite: the step is skipped).  seed: of the MXFP8 states' rounding, another
    one each step."""
    if grad_scale is not None:
        _check("grad_scale", grad_scale, torch.float32, None, tensors.device)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale: expected one element")
    c = _AdamwConfig(lr, betas[0], betas[1], eps, weight_decay, step, seed, tensors.g_dtype, tensors.state)
    _call("moe_adamw", tensors._c, len(tensors.params), ctypes.byref(c), _ptr(grad_scale),
          torch.cuda.current_stream(tensors.device).cuda_stream)
