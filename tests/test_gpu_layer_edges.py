"""gdn_rotary and gdn_gated_norm at the ends of their ranges: closed gates, far positions, rows written behind element 2^31.

Tolerances as in test_gpu_layer_ops.py: half a step of the type, and fp32's part as FINE = 2^-20."""
import ctypes

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200 import (gdn_backward, gdn_forward, gdn_gated_norm, gdn_gated_norm_backward, gdn_layer_backward,
                                       gdn_layer_forward, gdn_rotary, gdn_rotary_backward, load_library)
from gated_delta_rule_149_b200.gdn import GDNError, View
from test_gpu_layer_ops import BF16, FINE, FP32, norms, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_gates_that_nearly_close(dtype):
    """Gates of -5 to -87, value by value: with rows of ones n = 1 / sqrt(1 + eps), y = n silu(g) and dgate = dy n silu'(g),
    whose terms s and g s (1 - s) add up to no less than three quarters of the larger below -5.  The sigmoid is within 2^-21 of itself,
    a few roundings follow: 2^-20.  For bf16 7e-8 |g| more, 2^-17 at most, and the rounding of the results, 2^-9, which is half of
    its tolerance of 2^-8."""
    T, dv, eps = 512, 64, 1e-5
    g = torch.linspace(-87.0, -5.0, T * dv, dtype=torch.float64).to(dtype).view(1, 1, T, dv).cuda()
    o, dy = torch.ones_like(g), torch.ones(1, T, dv, dtype=dtype, device="cuda")
    y = gdn_gated_norm(o, g, eps=eps).view(-1).double()
    dg = gdn_gated_norm_backward(dy, o, g, eps=eps)[1].reshape(-1).double()
    x = g.double().view(-1)
    n, s = (1 + eps) ** -0.5, torch.sigmoid(x)
    tol = FINE + (ref.HALF_STEP[BF16] if dtype == BF16 else 0)
    off = (y / (n * x * s) - 1).abs().max()
    assert off <= tol, f"y: {off:.3e}"
    off = (dg / (n * (s + x * s * (1 - s))) - 1).abs().max()
    assert off <= tol, f"dgate: {off:.3e}"


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_gates_without_bounds(dtype):
    """silu as the formula has it at the ends: inf at inf, NaN at -inf (inf * 0) and NaN, 0 far below, the gate far above."""
    g = torch.zeros(1, 1, 6, 64, dtype=dtype, device="cuda")
    for t, x in enumerate((float("inf"), float("-inf"), float("nan"), -3e38, 2e38, 100.0)):
        g[0, 0, t] = x
    y = gdn_gated_norm(torch.ones_like(g), g, eps=1e-5).view(6, 64).float()
    assert torch.isposinf(y[0]).all() and y[1:3].isnan().all() and (y[3] == 0).all()
    want = g[0, 0, 4:].double() * (1 + 1e-5) ** -0.5
    ref.close(y[4:], want, dtype, FINE * want)


@pytest.mark.parametrize("grid,start", [((1, 1), 2 ** 31 - 40), ((64, 128), 2 ** 40), ((1 << 12, 1 << 13), 2 ** 52 - 2 ** 25)])
def test_rotary_far_positions(grid, start):
    """A grid's positions up to the largest that int32 positions have, and token numbers far beyond: three roundings to 53
    bits and the power's own error leave 3 * 2^-52 of the angle, 2^-19 at 2^31 (see the neighbouring int32 test), and fp32's part."""
    T, d = 40, 96
    q = normal(1, 2, T, d, seed=3)
    y = gdn_rotary(q, axes=(32, 32, 32), grid=grid, start=start)
    want = ref.rotary(q.cpu(), (32, 32, 32), 10000.0, False, ref.grid_positions(T, grid, start), False, 1e-6)
    ref.close(y.cpu(), want, FP32, 4 * FINE * norms(q).cpu())


def test_rotary_repeated_positions_turn_equal_rows_equally():
    B, H, T, d = 2, 3, 6, 64
    pos = torch.randint(-10 ** 6, 10 ** 6, (B, T, 3), generator=torch.Generator().manual_seed(5), dtype=torch.int64).to(torch.int32)
    pos[:, 1] = pos[:, 0]
    q = normal(B, H, T, d, seed=4)
    q[:, :, 1] = q[:, :, 0]
    y = gdn_rotary(q, axes=(24, 20, 20), positions=pos.cuda(), l2norm=True)
    assert torch.equal(y[:, :, 0], y[:, :, 1])
    assert not torch.equal(y[:, :, 0], y[:, :, 2])


def test_outputs_behind_element_2_to_31():
    """The C entry points with outputs whose second batch starts behind element 2^31 of a buffer: written there and nowhere
    near; read there by the gradients."""
    lib = load_library()
    B, H, T, d, far = 2, 2, 5, 128, 2 ** 31
    room = torch.full((far + 2 ** 14,), 7.0, dtype=BF16, device="cuda")
    big = room.as_strided((B, H, T, d), (far, T * d + 8, d, 1), storage_offset=16)
    to = View(big.data_ptr(), far, T * d + 8, d)
    mine = torch.zeros_like(room, dtype=torch.bool)
    mine.as_strided((B, H, T, d), (far, T * d + 8, d, 1), storage_offset=16).fill_(True)
    x, g, w = normal(B, H, T, d, dtype=BF16, seed=1), normal(B, H, T, d, dtype=BF16, seed=2), normal(d, seed=3)
    frm, gate = (View(t.data_ptr(), H * T * d, T * d, d) for t in (x, g))
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)

    def wrote(want):
        assert torch.equal(big, want)
        for a in range(0, room.numel(), 2 ** 29):          # what lies between the rows is as it was
            assert bool(((room[a:a + 2 ** 29] == 7.0) | mine[a:a + 2 ** 29]).all())

    how = (None, 0, B, H, T, d, 44, 42, 42, 2, 2, 0, 1e4, 1e-6, 32, stream)
    assert lib.gdn_rotary(frm, None, to, None, *how) == 0
    wrote(gdn_rotary(x, axes=(44, 42, 42), grid=(2, 2), l2norm=True))
    big.fill_(0)
    assert lib.gdn_gated_norm(frm, gate, w.data_ptr(), 0, to, B, H, T, d, 1e-5, 0, stream) == 0
    wrote(gdn_gated_norm(x, g, w).view(B, T, H, d).transpose(1, 2))
    dy = normal(B, T, H * d, dtype=BF16, seed=4)
    vdy = View(dy.data_ptr(), T * H * d, d, H * d)
    do, dg, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    vdo, vdg = (View(t.data_ptr(), H * T * d, T * d, d) for t in (do, dg))
    want = gdn_gated_norm_backward(dy, x, g, w)
    big.copy_(x)                                           # read behind 2^31
    assert lib.gdn_gated_norm_backward(vdy, to, gate, w.data_ptr(), 0, vdo, vdg, dw.data_ptr(), B, H, T, d, 1e-5, 0, stream) == 0
    assert torch.equal(do, want[0]) and torch.equal(dg, want[1]) and torch.equal(dw, want[2])
    big.fill_(0)                                           # written behind 2^31
    assert lib.gdn_gated_norm_backward(vdy, frm, gate, w.data_ptr(), 0, to, vdg, dw.data_ptr(), B, H, T, d, 1e-5, 0, stream) == 0
    wrote(want[0])


@pytest.mark.parametrize("dk,dv", [(64, 32), (96, 96)])
def test_layer_at_sizes_of_the_recurrent_form(dk, dv):
    """bf16 at sizes that gdn_forward takes in its recurrent form and gdn_backward in its only one: the layer is the chain of
    its calls, forward and back."""
    B, H, T = 1, 3, 70
    q, k = (normal(B, T, H, dk, dtype=BF16, seed=i).transpose(1, 2) for i in (1, 2))
    v, gate = normal(B, H, T, dv, dtype=BF16, seed=3), normal(B, T, H, dv, dtype=BF16, seed=4).transpose(1, 2)
    beta, decay = torch.sigmoid(normal(B, H, T, seed=5)), torch.sigmoid(2 + normal(B, H, T, seed=6))
    w = 1 + 0.1 * normal(dv, seed=7)
    how = dict(axes=(dk - 32, 16, 16), grid=(4, 5))
    with pytest.raises(GDNError):
        gdn_layer_forward(q, k, v, beta, decay, gate, w, **how)
    y, state, saved = gdn_layer_forward(q, k, v, beta, decay, gate, w, recurrent=True, **how)
    qr, kr = gdn_rotary(q, k, l2norm=True, **how)
    o, st = gdn_forward(qr, kr, v, beta, decay, recurrent=True)
    assert torch.equal(st, state) and torch.equal(y, gdn_gated_norm(o, gate, w))
    dy = normal(B, T, H * dv, dtype=BF16, seed=8)
    got = gdn_layer_backward(dy, saved)
    do, dg, dw = gdn_gated_norm_backward(dy, o, gate, w)
    dq, dk_, dv_, db, da, _ = gdn_backward(qr, kr, v, beta, decay, do)
    dq, dk_ = gdn_rotary_backward(dq, dk_, q, k, l2norm=True, **how)
    for name, x in dict(q=dq, k=dk_, v=dv_, beta=db, decay=da, gate=dg, weight=dw).items():
        assert torch.equal(got[name], x), name
    assert got["state_in"] is None
