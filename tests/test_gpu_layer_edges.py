"""gdn_rotary and gdn_gated_norm at the ends of their ranges: closed gates, far positions, rows written behind element 2^31.

Tolerances as in test_gpu_layer_ops.py: half a step of the type, and fp32's part as FINE = 2^-20."""
import ctypes

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200 import gdn_gated_norm, gdn_gated_norm_backward, gdn_rotary, load_library
from gated_delta_rule_149_b200.gdn import View
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
