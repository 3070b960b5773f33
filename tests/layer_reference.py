"""The layer's operators and their gradients in 64 bits, written from their definitions (test side only)."""
import math

import torch


def rotary(x, axes, theta, half, positions, l2norm, eps):
    """y = Rot(angle) x / sqrt(|x|^2 + eps); positions [B or 1, T, 3]."""
    x = x.double()
    d = x.shape[-1]
    angle = torch.cat([positions[..., a:a + 1].double() * torch.tensor([theta ** (-2.0 * i / n) for i in range(n // 2)],
                                                                     dtype=torch.float64, device=x.device)
                       for a, n in enumerate(axes) if n], -1)[:, None]
    if l2norm:
        x = x / ((x * x).sum(-1, keepdim=True) + eps).sqrt()
    at = (torch.arange(d // 2), torch.arange(d // 2) + d // 2) if half else (torch.arange(0, d, 2), torch.arange(1, d, 2))
    a, b = x[..., at[0]], x[..., at[1]]
    y = torch.empty_like(x)
    y[..., at[0]] = a * angle.cos() - b * angle.sin()
    y[..., at[1]] = a * angle.sin() + b * angle.cos()
    return y


def grid_positions(T, grid, start):
    n = torch.arange(start, start + T, dtype=torch.int64)
    h, w = grid
    return torch.stack([n // (h * w), n // w % h, n % w], -1)[None]


def gated_norm(o, gate, weight, eps):
    """[B,H,T,dv] -> [B,T,H*dv]."""
    o = o.double()
    y = o / ((o * o).mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * (weight.double() if weight.dim() == 1 else weight.double()[:, None])
    if gate is not None:
        y = y * gate.double() * torch.sigmoid(gate.double())
    return y.transpose(1, 2).flatten(2)


def recurrence(q, k, v, beta, decay, state_in=None, bidi=False):
    """gdn_forward token by token; differentiable.  Returns o and the state(s)."""
    q, k, v, beta, decay = (x.double() for x in (q, k, v, beta, decay))
    if bidi:
        o, s = recurrence(q, k, v, beta, decay, state_in)
        r, z = recurrence(q.flip(2), k.flip(2), v.flip(2), beta.flip(2), decay.flip(2))
        return o + r.flip(2), torch.stack([s, z])
    B, H, T, dk = q.shape
    h = q.new_zeros(B, H, dk, v.shape[-1]) if state_in is None else state_in.double()
    out = []
    for t in range(T):
        kt, a, b = k[:, :, t, :, None], decay[:, :, t, None, None], beta[:, :, t, None, None]
        h = a * (h - b * kt @ (kt.mT @ h)) + b * kt @ v[:, :, t, None, :]
        out.append((q[:, :, t, None, :] @ h)[:, :, 0])
    return torch.stack(out, 2), h


def gradients(outputs, given, inputs):
    """Gradients of sum <given, output> with respect to the inputs (zero where there is no path)."""
    total = sum((g.double() * o).sum() for g, o in zip(given, outputs) if g is not None)
    got = torch.autograd.grad(total, inputs, allow_unused=True)
    return [torch.zeros_like(x) if g is None else g for g, x in zip(got, inputs)]


def recurrence_gradients(q, k, v, beta, decay, do, state_in=None, dstate=None, bidi=False):
    """(dq, dk, dv, dbeta, ddecay, dstate_in) in 64 bits."""
    leaves = [x.detach().double().clone().requires_grad_() for x in (q, k, v, beta, decay)]
    B, H, _, dk = q.shape
    s0 = (torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device=q.device) if state_in is None
          else state_in.detach().double().clone()).requires_grad_()
    out = recurrence(*leaves, s0, bidi)
    return gradients(out, (do, dstate), leaves + [s0])


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def close(x, ref, dtype, noise, what=""):
    """Each value within half a step of its type of the reference, plus `noise`: fp32 arithmetic's part, relative to
    the scale tensor or number it is a product with."""
    err = (x.double() - ref).abs()
    bound = HALF_STEP[dtype] * ref.abs() + noise
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).max()):.3e} over"


def rel(x, ref):
    n = float(ref.norm())
    d = float((x.double() - ref).norm())
    return d / n if n else (0.0 if d == 0 else math.inf)
