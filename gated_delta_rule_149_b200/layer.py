"""The operators around the recurrence in a GDN layer, and the layer's run of them.

gdn_rotary turns and normalises q and k on their way from a projection to gdn_forward, gdn_gated_norm takes
gdn_forward's output to the next projection; each has its gradients.  gdn_layer_forward and gdn_layer_backward
run them together.  As in gdn.py, these functions check arguments and pass pointers; the work is in the
library's kernels.
"""
from typing import NamedTuple, Optional

import torch

from .gdn import GDN_FP32, View, _check, _ptr, _run, gdn_backward, gdn_forward, load_library

GDN_ROTARY_HALF = 16
GDN_ROTARY_L2 = 32

_DTYPES = {torch.bfloat16: 0, torch.float32: GDN_FP32}


def _rows(t, name, shape, dtype, device):
    """A [B,H,T,d] tensor of any strides with contiguous rows, as a gdn_view."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    sb, sh, st, sd = t.stride()
    if sd != 1 and shape[3] != 1:
        raise ValueError(f"{name}: rows (the last dimension) must be contiguous")
    return View(t.data_ptr(), sb, sh, st)


def _shape(t, name):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B,H,T,d], got {tuple(t.shape)}")
    if t.device.type != "cuda":
        raise ValueError("runs on CUDA tensors only")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return t.shape


def _heads_first(like, shape):
    """An empty [B,H,T,d] tensor, and its gdn_view."""
    B, H, T, d = shape
    t = like.new_empty(shape)
    return t, View(t.data_ptr(), H * T * d, T * d, d)


def _tokens_first(like, shape):
    """An empty [B,T,H,d] tensor, and the gdn_view of its [B,H,T,d] transpose."""
    B, H, T, d = shape
    t = like.new_empty((B, T, H, d))
    return t, View(t.data_ptr(), T * H * d, d, H * d)


def _turns(axes, grid, start, positions, theta, eps, shape, device):
    """The arguments both directions of gdn_rotary share, from positions on."""
    B, H, T, d = shape
    if len(axes) != 3:
        raise ValueError(f"axes must be three dims (time, height, width), got {axes}")
    pos, sb = None, 0
    if positions is not None:
        if positions.dtype != torch.int32:
            raise TypeError(f"positions: expected torch.int32, got {positions.dtype}")
        if tuple(positions.shape) not in ((T, 3), (1, T, 3), (B, T, 3)):
            raise ValueError(f"positions: expected shape ({T}, 3) or ({B}, {T}, 3), got {tuple(positions.shape)}")
        if positions.device != device:
            raise ValueError(f"positions: expected device {device}, got {positions.device}")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        pos, sb = positions.data_ptr(), T * 3 if positions.dim() == 3 and positions.shape[0] > 1 else 0
        grid = (0, 0)
    elif grid is None:
        raise ValueError("either grid (height, width) or positions is needed")
    return (pos, sb, B, H, T, d, *axes, *grid, start, theta, eps)


def gdn_rotary(q, k=None, *, axes, grid=None, start=0, positions=None, theta=10000.0, half=False, l2norm=False,
               eps=1e-6, stream=None):
    """Rotates q (and k) [B,H,T,d] by positions on up to three axes; returns contiguous [B,H,T,d] tensors.

    q, k: bf16 or fp32, any strides with contiguous rows (views of a projection's
    [B,T,H,d] memory, for instance); k may be None, and the result is then q's
    alone.  axes: dims of the time, height and width axes, even, summing to d.
    Positions: `positions` int32 [T,3] or [B,T,3], or the tokens' places in
    frames of grid = (height, width) tokens, counted from token number `start`.
    Pair i of an axis of n dims turns by position * theta^(-2i/n).  Pairs are
    neighbours, or (p, p + d/2) with half=True.  l2norm=True divides each row by
    sqrt(|x|^2 + eps) first.
    """
    shape = _shape(q, "q")
    dev, lib = q.device, load_library()
    how = _turns(axes, grid, start, positions, theta, eps, shape, dev)
    mode = _DTYPES[q.dtype] | (GDN_ROTARY_HALF if half else 0) | (GDN_ROTARY_L2 if l2norm else 0)
    vq = _rows(q, "q", shape, q.dtype, dev)
    vk = None if k is None else _rows(k, "k", shape, q.dtype, dev)

    def call(handle):
        yq, to_q = _heads_first(q, shape)
        yk, to_k = (None, None) if k is None else _heads_first(q, shape)
        _check(lib.gdn_rotary(vq, vk, to_q, to_k, *how, mode, handle))
        return yq if k is None else (yq, yk)

    return _run(dev, stream, call)


def gdn_rotary_backward(dq, dk=None, q=None, k=None, *, axes, grid=None, start=0, positions=None, theta=10000.0,
                        half=False, l2norm=False, eps=1e-6, stream=None):
    """Gradients of gdn_rotary's inputs from those of its outputs.

    dq, dk [B,H,T,d] of any strides with contiguous rows; q, k: the inputs of
    gdn_rotary, needed (and read) with l2norm=True only.  The other arguments are
    the forward call's.  Returns [B,H,T,d] tensors in [B,T,H,d] memory, the layout
    of a projection's gradient (dq's alone without dk).
    """
    shape = _shape(dq, "dq")
    dev, lib = dq.device, load_library()
    how = _turns(axes, grid, start, positions, theta, eps, shape, dev)
    mode = _DTYPES[dq.dtype] | (GDN_ROTARY_HALF if half else 0) | (GDN_ROTARY_L2 if l2norm else 0)
    vg = [_rows(dq, "dq", shape, dq.dtype, dev), None if dk is None else _rows(dk, "dk", shape, dq.dtype, dev)]
    vx = [None, None]
    if l2norm:
        if q is None or (dk is not None and k is None):
            raise ValueError("with l2norm the gradients need gdn_rotary's inputs q (and k)")
        vx[0] = _rows(q, "q", shape, dq.dtype, dev)
        if dk is not None:
            vx[1] = _rows(k, "k", shape, dq.dtype, dev)

    def call(handle):
        yq, to_q = _tokens_first(dq, shape)
        yk, to_k = (None, None) if dk is None else _tokens_first(dq, shape)
        _check(lib.gdn_rotary_backward(*vg, *vx, to_q, to_k, *how, mode, handle))
        return yq.transpose(1, 2) if dk is None else (yq.transpose(1, 2), yk.transpose(1, 2))

    return _run(dev, stream, call)


def _weight(weight, H, dv, device):
    if weight is None:
        return 0
    if weight.dtype != torch.float32:
        raise TypeError(f"weight: expected torch.float32, got {weight.dtype}")
    if weight.shape not in ((dv,), (H, dv)):
        raise ValueError(f"weight: expected shape ({dv},) or ({H}, {dv}), got {tuple(weight.shape)}")
    if weight.device != device:
        raise ValueError(f"weight: expected device {device}, got {weight.device}")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    return int(weight.dim() == 2)


def gdn_gated_norm(o, gate=None, weight=None, *, eps=1e-5, stream=None):
    """y = weight * o / sqrt(mean(o^2) + eps) * silu(gate) per head, as [B,T,H*dv] for the output projection.

    o [B,H,T,dv] (gdn_forward's output) and gate [B,H,T,dv] or None: bf16 or fp32,
    any strides with contiguous rows (gate is usually a view of [B,T,H,dv]
    memory).  weight: fp32 [dv] or [H,dv], or None for 1.
    """
    shape = _shape(o, "o")
    B, H, T, dv = shape
    dev, lib = o.device, load_library()
    per_head = _weight(weight, H, dv, dev)
    vo = _rows(o, "o", shape, o.dtype, dev)
    vg = None if gate is None else _rows(gate, "gate", shape, o.dtype, dev)

    def call(handle):
        y = o.new_empty((B, T, H * dv))
        _check(lib.gdn_gated_norm(vo, vg, _ptr(weight), per_head, View(y.data_ptr(), T * H * dv, dv, H * dv), B, H, T, dv,
                                  eps, _DTYPES[o.dtype], handle))
        return y

    return _run(dev, stream, call)


def gdn_gated_norm_backward(dy, o, gate=None, weight=None, *, eps=1e-5, stream=None):
    """Gradients of gdn_gated_norm from dy [B,T,H*dv]: do (contiguous [B,H,T,dv], as gdn_backward takes it), dgate
    ([B,H,T,dv] in [B,T,H,dv] memory; None without gate) and dweight (fp32, shape of weight; None without).  An
    expanded input's gradient comes per element, like any other's."""
    shape = _shape(o, "o")
    B, H, T, dv = shape
    dev, lib = o.device, load_library()
    per_head = _weight(weight, H, dv, dev)
    if dy.shape != (B, T, H * dv):
        raise ValueError(f"dy: expected shape {(B, T, H * dv)}, got {tuple(dy.shape)}")
    if dy.dtype != o.dtype:
        raise TypeError(f"dy: expected {o.dtype}, got {dy.dtype}")
    if dy.device != dev:
        raise ValueError(f"dy: expected device {dev}, got {dy.device}")
    sb, st, sd = dy.stride()
    if sd != 1 and H * dv != 1:
        raise ValueError("dy: rows (the last dimension) must be contiguous")
    vdy = View(dy.data_ptr(), sb, dv, st)
    vo = _rows(o, "o", shape, o.dtype, dev)
    vg = None if gate is None else _rows(gate, "gate", shape, o.dtype, dev)

    def call(handle):
        do, to_o = _heads_first(o, shape)
        dgate, to_g = (None, None) if gate is None else _tokens_first(o, shape)
        dw = None if weight is None else torch.empty_like(weight)
        _check(lib.gdn_gated_norm_backward(vdy, vo, vg, _ptr(weight), per_head, to_o, to_g, _ptr(dw), B, H, T, dv, eps,
                                           _DTYPES[o.dtype], handle))
        return do, None if gate is None else dgate.transpose(1, 2), dw

    return _run(dev, stream, call)


class LayerSaved(NamedTuple):
    """What gdn_layer_backward needs of a gdn_layer_forward call: its inputs, the rotated q and k, and o."""
    q_in: torch.Tensor
    k_in: torch.Tensor
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    beta: torch.Tensor
    decay: torch.Tensor
    state_in: Optional[torch.Tensor]
    o: torch.Tensor
    gate: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bidi: bool
    norm_eps: float
    rotary: dict


def gdn_layer_forward(q, k, v, beta, decay, gate=None, weight=None, state_in=None, *, axes, grid=None, start=0,
                      positions=None, theta=10000.0, half=False, l2norm=True, eps=1e-6, norm_eps=1e-5, bidi=False,
                      recurrent=False, stream=None):
    """A GDN layer between its projections: gdn_rotary on q and k, gdn_forward, gdn_gated_norm.

    q, k, gate: [B,H,T,d] views of the projections; v contiguous [B,H,T,dv]; beta,
    decay, state_in as gdn_forward; the keywords as gdn_rotary (l2norm=True here:
    the recurrence wants unit keys), norm_eps for the read-out's norm, recurrent as
    gdn_forward (bf16 with other sizes than dk = 128, dv = 64 or 128 needs it).
    Returns y [B,T,H*dv], the final state, and what gdn_layer_backward needs.
    """
    how = dict(axes=axes, grid=grid, start=start, positions=positions, theta=theta, half=half, l2norm=l2norm, eps=eps)
    qr, kr = gdn_rotary(q, k, **how, stream=stream)
    o, state = _run(q.device, stream, lambda _: gdn_forward(qr, kr, v, beta, decay, state_in, bidi=bidi, recurrent=recurrent,
                                                              stream=stream))
    y = gdn_gated_norm(o, gate, weight, eps=norm_eps, stream=stream)
    return y, state, LayerSaved(q, k, qr, kr, v, beta, decay, state_in, o, gate, weight, bidi, norm_eps, how)


def gdn_layer_backward(dy, saved, dstate=None, *, stream=None):
    """Gradients of gdn_layer_forward's inputs from dy [B,T,H*dv] and dstate (of the final state, or None): a dict of
    q, k, v, beta, decay, gate, weight, state_in (None where the input was None)."""
    s = saved
    do, dgate, dweight = gdn_gated_norm_backward(dy, s.o, s.gate, s.weight, eps=s.norm_eps, stream=stream)
    dq, dk, dv, db, da, ds = gdn_backward(s.q, s.k, s.v, s.beta, s.decay, do, s.state_in, dstate, bidi=s.bidi,
                                          stream=stream)
    dq, dk = gdn_rotary_backward(dq, dk, s.q_in, s.k_in, **s.rotary, stream=stream)
    return dict(q=dq, k=dk, v=dv, beta=db, decay=da, gate=dgate, weight=dweight,
                state_in=None if s.state_in is None else ds)
