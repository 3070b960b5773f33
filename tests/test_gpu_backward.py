"""gdn_backward against the recurrence's definition in 64 bits, token by token.

Tolerances (rel-L2): fp32 outputs 1e-5, the library's bar for fp32 arithmetic; outputs of bf16 type half a step of
the type on every value, 2^-8, and that."""
import os
import subprocess
import sys

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200 import gdn_backward, gdn_forward
from gated_delta_rule_149_b200.inputs import make_custom

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dbeta", "ddecay", "dstate_in")


def make(B, H, T, dk, dv, dtype, seed, bidi, state, shift=0.0, **kw):
    inp = make_custom(B, H, T, dk, dv, dtype=dtype, seed=seed, bidi=bidi, state0=state, decay_shift=shift, **kw)
    g = torch.Generator().manual_seed(seed + 1000)
    do = torch.randn(inp.v.shape, generator=g).to(inp.v.dtype)
    ds = torch.randn(((2,) if bidi else ()) + (B, H, dk, dv), generator=g) if state else None
    return [inp.q, inp.k, inp.v, inp.beta, inp.decay, do, inp.state0, ds]


def run(args, bidi):
    return gdn_backward(*(None if x is None else x.cuda() for x in args), bidi=bidi)


def check(args, bidi, got=None):
    got = got or run(args, bidi)
    want = ref.recurrence_gradients(*args[:6], args[6], args[7], bidi)
    for name, x, y in zip(NAMES, got, want):
        tol = 1e-5 + (2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0)
        e = ref.rel(x.cpu(), y)
        assert e <= tol, f"{name}: rel-L2 {e:.3e} > {tol:.3e}"


@pytest.mark.parametrize("T", [1, 2, 5, 63, 64, 65, 200])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("bidi", [False, True])
def test_fp32_lengths(T, d, bidi):
    check(make(1, 2, T, d, d, "fp32", T + d, bidi, True), bidi)


@pytest.mark.parametrize("T", [1, 64, 129, 300])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("bidi", [False, True])
def test_bf16_lengths(T, dv, bidi):
    check(make(2, 2, T, 128, dv, "bf16", T + dv, bidi, True, shift=2.0), bidi)


@pytest.mark.parametrize("dk,dv,dtype", [(32, 128, "fp32"), (96, 64, "fp32"), (128, 96, "fp32"), (64, 32, "bf16"), (96, 96, "bf16")])
def test_rectangular(dk, dv, dtype):
    check(make(2, 3, 77, dk, dv, dtype, dk + dv, True, True), True)


@pytest.mark.parametrize("dtype,dk", [("fp32", 32), ("bf16", 128)])
def test_without_states(dtype, dk):
    """No entry state and no gradient of the final one; the gradient of the (zero) entry state all the same."""
    check(make(1, 3, 150, dk, dk, dtype, 3, False, False), False)
    check(make(1, 3, 150, dk, dk, dtype, 4, True, False), True)


@pytest.mark.parametrize("dtype,dk", [("fp32", 64), ("bf16", 128)])
@pytest.mark.parametrize("shift", [-6.0, 8.0])
def test_slow_and_strong_decay(dtype, dk, shift):
    """Decays about 0.998 (the state remembers the sequence) and about 3e-4 (ten tokens span 2^-120)."""
    check(make(1, 2, 260, dk, 64, dtype, 17, True, True, shift=shift), True)


@pytest.mark.parametrize("dtype,dk", [("fp32", 32), ("bf16", 128)])
def test_gates_at_their_ends(dtype, dk):
    """beta of exactly 0 and 1, decay of exactly 1; with unit keys beta = 1 overwrites."""
    a = make(1, 2, 140, dk, 64, dtype, 23, False, True, shift=-3.0)
    a[3][:, :, ::3] = 0.0
    a[3][:, :, 1::3] = 1.0
    a[4][:, :, ::5] = 1.0
    check(a, False)


@pytest.mark.parametrize("dtype,dk", [("fp32", 32), ("bf16", 128)])
def test_decay_of_zero_forgets(dtype, dk):
    """A decay of 0 acts as 2^-120: nothing passes it either way, and its own gradient, <dH_t, (I - b k k^T) H_{t-1}>,
    is what the definition gives at 0."""
    a = make(1, 2, 150, dk, 64, dtype, 29, False, True, shift=0.0)
    a[4][:, :, 70] = 0.0
    check(a, False)


def test_equal_keys():
    """The same key at every token, decay 1, beta 1/2: the triangular systems at their worst conditioned."""
    a = make(1, 1, 128, 64, 32, "fp32", 31, False, True)
    a[1][:] = a[1][:, :, :1]
    a[3][:] = 0.5
    a[4][:] = 1.0
    check(a, False)


def test_zero_gradients_and_zero_inputs():
    a = make(1, 2, 100, 128, 128, "bf16", 37, True, True)
    got = run([*a[:5], torch.zeros_like(a[5]), a[6], None], True)
    assert all((x == 0).all() for x in got)
    z = [torch.zeros_like(x) for x in a[:4]] + [torch.ones_like(a[4]), a[5], None, None]
    got = run(z, True)
    assert all(torch.isfinite(x).all() and (x == 0).all() for x in got)


def test_differences_of_the_forward_call():
    """<gradient, u> against central differences of gdn_forward itself (fp32): (L(x + e u) - L(x - e u)) / 2e with e = 2^-6
    has a truncation error of e^2/6 of the third derivative's term and a rounding error of about 1e-6 |L| / e: 1e-3 of
    |grad| |u| at these sizes."""
    a = make(1, 1, 40, 32, 32, "fp32", 41, False, True, shift=-2.0)
    got = run(a, False)
    dev = [None if x is None else x.cuda() for x in a]

    def loss(i, e, u):
        x = list(dev)
        x[i] = x[i] + e * u
        o, s = gdn_forward(*x[:5], x[6])
        return float((dev[5].double() * o.double()).sum() + (dev[7].double() * s.double()).sum())

    for i, g in zip((0, 1, 2, 3, 4, 6), got):
        u = torch.randn(g.shape, generator=torch.Generator().manual_seed(i)).cuda()
        u *= 0.2 * float(dev[i].norm()) / float(u.norm())
        e = 2.0 ** -6
        diff = (loss(i, e, u) - loss(i, -e, u)) / (2 * e)
        want = float((g.double() * u.double()).sum())
        assert abs(diff - want) <= 1e-3 * float(g.norm() * u.norm()), i


def test_many_heads_and_repeats():
    """More heads than one block row, the same result on every call, and inputs left as they were."""
    a = make(5, 9, 70, 128, 64, "bf16", 43, True, True)
    before = [None if x is None else x.clone() for x in a]
    dev = [None if x is None else x.cuda() for x in a]
    one, two = gdn_backward(*dev, bidi=True), gdn_backward(*dev, bidi=True)
    assert all(torch.equal(x, y) for x, y in zip(one, two))
    assert all(x is None or torch.equal(x, y.cpu()) for x, y in zip(before, dev))
    check(a, True, one)


def test_own_stream_and_graphs():
    a = make(1, 4, 200, 128, 128, "bf16", 47, True, True)
    dev = [x.cuda() for x in a]
    want = gdn_backward(*dev, bidi=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gdn_backward(*dev, bidi=True, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = gdn_backward(*dev, bidi=True)
        graphs.append((graph, out))
    dev[5].copy_(torch.randn(dev[5].shape, generator=torch.Generator().manual_seed(1)))
    want = gdn_backward(*dev, bidi=True)
    for _ in range(2):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(x, y) for x, y in zip(want, out))


FIRST_IN_CAPTURE = """
import torch
from gated_delta_rule_149_b200 import gdn_backward
x = [torch.randn(1, 2, 100, 128, device="cuda").bfloat16() for _ in range(4)]
g = [torch.rand(1, 2, 100, device="cuda") for _ in range(2)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = gdn_backward(0.1 * x[0], 0.1 * x[1], x[2], *g, x[3])
graph.replay()
want = gdn_backward(0.1 * x[0], 0.1 * x[1], x[2], *g, x[3])
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, want))
print("same")
"""


def test_first_call_of_a_process_inside_a_capture():
    """The library's pool of device memory comes into being on first use, which may be within a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once():
    """Two different calls in flight on two streams share no state."""
    calls = [[None if x is None else x.cuda() for x in make(1, 4, 700, 128, 128, "bf16", seed, True, True, shift=2.0)] for seed in (51, 52)]
    want = [gdn_backward(*c, bidi=True) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for _ in range(3):
        got = [gdn_backward(*c, bidi=True, stream=s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(w, g))


@pytest.mark.parametrize("T,heads", [(64 * 100, 230)])
def test_heads_in_several_passes(T, heads):
    """More heads and chunks than one pass's workspace holds (6 GiB): each head as in a call of its own.  The two calls may
    take other forms of the chains, which add in another order: within fp32's rounding of one another (1e-5)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k = (torch.nn.functional.normalize(n(1, heads, T, 128), dim=-1).bfloat16() for _ in range(2))
    v, do = n(1, heads, T, 128).bfloat16(), n(1, heads, T, 128).bfloat16()
    beta, decay = torch.sigmoid(n(1, heads, T)), torch.sigmoid(3 + n(1, heads, T))
    s0, ds = 0.1 * n(1, heads, 128, 128), n(1, heads, 128, 128)
    whole = gdn_backward(q, k, v, beta, decay, do, s0, ds)
    for at in (0, heads // 2 - 1, heads // 2, heads - 1):
        one = gdn_backward(*(x[:, at:at + 1].contiguous() for x in (q, k, v, beta, decay, do, s0, ds)))
        for name, x, y in zip(NAMES, whole, one):
            tol = 1e-5 + (2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0)
            assert ref.rel(x[:, at:at + 1].double(), y.double()) <= tol, (name, at)


@pytest.mark.parametrize("dtype,dk", [("fp32", 64), ("bf16", 128)])
def test_non_finite_values_stay_in_their_chunk(dtype, dk):
    """A NaN in do at token 70: what the definition keeps apart from it stays finite outside tokens 64 .. 127, and another
    head is untouched."""
    a = make(1, 2, 200, dk, 64, dtype, 61, False, True)
    clean = run(a, False)
    a[5][0, 0, 70, 3] = float("nan")
    got = run(a, False)
    for name, x, y in zip(NAMES, got, clean):
        assert torch.equal(x[0, 1], y[0, 1]), name
        if name == "dq":
            assert torch.equal(x[0, 0, :64], y[0, 0, :64]) and torch.equal(x[0, 0, 128:], y[0, 0, 128:])
        elif name != "dstate_in":
            assert torch.equal(x[0, 0, 128:], y[0, 0, 128:]), name


def test_many_short_scans_and_one_long():
    """The chains' two forms: more scans than SMs, and a few."""
    check(make(3, 30, 20, 128, 128, "bf16", 71, True, True), True)
    check(make(1, 1, 1500, 128, 64, "bf16", 72, False, True, shift=-2.0), False)
    check(make(2, 40, 33, 64, 64, "fp32", 73, True, True), True)


def test_refuses_what_it_does_not_take():
    a = [None if x is None else x.cuda() for x in make(1, 2, 10, 64, 64, "fp32", 1, False, True)]
    for i in range(8):
        bad = list(a)
        bad[i] = a[i][..., :5, :] if a[i].dim() == 4 else a[i][..., :5]
        with pytest.raises(ValueError):
            gdn_backward(*bad)
        bad[i] = a[i].double()
        with pytest.raises(TypeError):
            gdn_backward(*bad)
    with pytest.raises(ValueError):
        gdn_backward(*a, bidi=True)                      # dstate without the reverse scan's half
