"""gdn_backward where gates, scales and values are at their ends, and where a block takes more than one chunk.

Tolerances as in test_gpu_backward.py (rel-L2 1e-5, and 2^-8 for outputs of bf16 type) unless a test derives its own."""
import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200 import gdn_backward
from test_gpu_backward import NAMES, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,dk", [("fp32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("which", ["q", "k", "v", "beta", "decay"])
def test_nan_in_an_input_shows(dtype, dk, which):
    """A NaN at token 70 of one head: every gradient that the definition makes NaN is NaN, and the other heads, also those
    whose chunks the same block takes (200 chunks), are untouched."""
    a = make(1, 50, 200, dk, 64, dtype, 67, False, True)
    clean = run(a, False)
    i = ["q", "k", "v", "beta", "decay"].index(which)
    a[i][(0, 0, 70) + ((3,) if a[i].dim() == 4 else ())] = float("nan")
    got = run(a, False)
    want = ref.recurrence_gradients(*(x[:, :1] for x in a), False)
    seen = False
    for name, x, y, w in zip(NAMES, got, clean, want):
        assert torch.equal(x[0, 1:], y[0, 1:]), name
        assert (x[0, 0].cpu().isnan() | ~w[0, 0].isnan()).all(), name
        seen = seen or bool(w.isnan().any())
    assert seen


@pytest.mark.parametrize("dtype,dk", [("fp32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("power", [40, 0, -13, -23, -30, -40])
@pytest.mark.parametrize("bidi", [False, True])
def test_gradient_of_a_strong_decay_at_any_scale(dtype, dk, power, bidi):
    """The gradients are linear in do and dstate.  At a decay of 0 (2^-120) or 1e-35 the products that contain it are
    about 2^-120 of them, and the decay's gradient is their sum over the decay: the same 1e-5, held by these tokens alone
    as well, whatever the scale of do and dstate."""
    a = make(1, 2, 150, dk, 64, dtype, 29, bidi, True, shift=0.0)
    a[4][:, :, 70] = 0.0
    a[4][:, :, 100] = 1e-35
    a[4][:, :, 130] = 1e-20
    a[5], a[7] = a[5] * 2.0 ** power, a[7] * 2.0 ** power
    got = run(a, bidi)
    want = ref.recurrence_gradients(*a[:6], a[6], a[7], bidi)
    for name, x, y in zip(NAMES, got, want):
        tol = 1e-5 + (2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0)
        assert ref.rel(x.cpu(), y) <= tol, name
    for t in (70, 100, 130):
        e = ref.rel(got[4][:, :, t].cpu(), want[4][:, :, t])
        assert e <= 1e-5, f"ddecay at token {t}: rel-L2 {e:.3e}"
