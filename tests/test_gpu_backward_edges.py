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
