"""gdn_backward where gates, scales and values are at their ends, and where a block takes more than one chunk.

Tolerances as in test_gpu_backward.py (rel-L2 1e-5, and 2^-8 for outputs of bf16 type) unless a test derives its own."""
import time

import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200 import gdn, gdn_backward, gdn_device_status
from gated_delta_rule_149_b200.gdn import GDNError
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


@pytest.mark.parametrize("dtype,dk,dv", [("fp32", 32, 32), ("bf16", 64, 32), ("bf16", 128, 64)])
@pytest.mark.parametrize("T,low,high", [(1, 1e-30, 1e-30), (3, 1e-12, 1.1e-12), (64, 0.25, 0.35), (64, 0.99, 1.0)])
def test_products_of_strong_decays(dtype, dk, dv, T, low, high):
    """With keys of zero the state only decays, so dstate_in = prod a dstate and da_t = prod_{s != t} a_s <dstate, state>
    value by value.  A token's log2 is off by 2^-25 at most (its fraction's last place), 2^x by 2^-22 of itself for an
    exponent split exactly, and a few roundings follow: T 2^-25 + 2^-20 together.  A result under 2^-126 (1e-36 times an
    entry of dstate near 0) has fp32's spacing there, 2^-149, and no more bits: that much is added."""
    a = make(1, 3, T, dk, dv, dtype, 5, False, True)
    for x in (a[0], a[1], a[5]):
        x.zero_()
    g = torch.Generator().manual_seed(T)
    a[4] = low + (high - low) * torch.rand(1, 3, T, generator=g)
    a[6] = torch.zeros_like(a[6])
    a[6][..., 3, 5] = 1.0                                # one entry: the inner product is one product
    a[7] = torch.randn(a[7].shape, generator=g)
    got = run(a, False)
    prod = a[4].double().prod(-1)
    tol = T * 2.0 ** -25 + 2.0 ** -20
    want = [prod[..., None] / a[4].double() * a[7][..., 3, 5].double()[..., None], prod[..., None, None] * a[7].double()]
    for name, x, y in zip(NAMES[4:], got[4:], want):
        off = (((x.cpu().double() - y).abs() - 2.0 ** -149).clamp(min=0) / y.abs()).max()
        assert off <= tol, f"{name}: {off:.3e} > {tol:.3e}"


@pytest.mark.parametrize("dk", [64, 128])
def test_pair_products_keep_fp32_where_they_cancel(dk):
    """Two tokens with opposite unit keys: dq_1 = (E_10 - E_11) k_0 = -(v_1 . do_1) k_0, where E_10 = do_1 . v_0 in [1, 2) has 24
    bits (three parts of 8) and the difference is 1.5 * 2^-14.  The sums' truncation is at most 2^-23 of each of the
    four products and three orders of terms, twice: 2^-20 covers it.  Pairs held in 16 bits would leave up to 2^-17."""
    H, dv = 64, 64
    a = make(1, H, 2, dk, dv, "bf16", 3, False, False)
    q, k, v, beta, decay, do = a[:6]
    for x in (k, v, do):
        x.zero_()
    beta.fill_(1.0)
    decay.fill_(1.0)
    k[:, :, 0, 0], k[:, :, 1, 0] = 1.0, -1.0
    v[:, :, 0, :3] = (1 + torch.randint(0, 115, (1, H, 3), generator=torch.Generator().manual_seed(1)) / 128.0).bfloat16()
    v[:, :, 1, 3] = 1.5
    for c, power in enumerate((0, -8, -16, -14)):
        do[:, :, 1, c] = 2.0 ** power
    dq = run(a, False)[0].cpu().double()
    want = torch.zeros_like(dq)
    want[:, :, 1, 0] = -1.5 * 2.0 ** -14
    off = (dq - want).abs().max()
    assert off <= 2.0 ** -20 + 2.0 ** -9 * 1.5 * 2.0 ** -14, f"{off:.3e}"


@pytest.mark.parametrize("dtype,dk,dv,H,T,bidi,code", [
    ("bf16", 128, 128, 2, 300, False, 192), ("bf16", 128, 32, 2, 300, True, 192), ("bf16", 128, 64, 100, 130, True, 192),
    ("fp32", 64, 64, 2, 200, True, 128), ("fp32", 128, 96, 80, 130, False, 128)])
def test_waits_run_out_and_the_next_call_is_correct(dtype, dk, dv, H, T, bidi, code):
    """Head 0's walks wait for what never comes (128) and so do, on tcgen05, its first chunk's gradients (64): the waits run out
    after 20 ms, the blocks let their copies and products end and leave, the status says so once, and a clean call is right.
    With few heads and with many (both forms of the walks), one step of dv and several."""
    a = make(1, H, T, dk, dv, dtype, 7, bidi, True, shift=1.0)
    dev = [x.cuda() for x in a]
    gdn_device_status()
    gdn.debug_wait_limit(20_000_000)
    gdn.debug_stall(1)
    try:
        start = time.perf_counter()
        gdn_backward(*dev, bidi=bidi)
        with pytest.raises(GDNError) as err:
            gdn_device_status()
        took = time.perf_counter() - start
    finally:
        gdn.debug_stall(-1)
        gdn.debug_wait_limit(0)
    assert err.value.code == -5 and f"code {code})" in str(err.value)
    assert took < 10.0
    gdn_device_status()
    got = gdn_backward(*dev, bidi=bidi)
    gdn_device_status()
    part = [x[:, :2] for x in dev[:7]] + [dev[7][..., :2, :, :]]
    for name, x, y in zip(NAMES, got, ref.recurrence_gradients(*part, bidi)):
        tol = 1e-5 + (2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0)
        assert ref.rel(x[:, :2], y) <= tol, name


@pytest.mark.parametrize("dk,dv,H,T,dtype,bidi", [
    (128, 32, 160, 130, "bf16", True), (128, 64, 160, 130, "bf16", True), (96, 96, 160, 130, "bf16", True),
    (128, 128, 160, 130, "bf16", True), (128, 128, 160, 200, "bf16", False), (128, 96, 150, 65, "bf16", False),
    (64, 32, 160, 70, "fp32", True), (128, 96, 80, 70, "fp32", True)])
def test_more_chunks_than_sms(dk, dv, H, T, dtype, bidi):
    """The chunk gradients' blocks take two to four chunks each, in one and in both directions, with one to four steps of
    32 columns; the chains' blocks of 64 columns have an odd number of 32 to fill.  The definition in 64 bits on the GPU."""
    a = [None if x is None else x.cuda() for x in make(1, H, T, dk, dv, dtype, dk + dv + T, bidi, True, shift=1.0)]
    got = gdn_backward(*a, bidi=bidi)
    for h in range(0, H, 32):
        part = [x[:, h:h + 32] for x in a[:7]] + [a[7][..., h:h + 32, :, :]]
        want = ref.recurrence_gradients(*part, bidi)
        for name, x, y in zip(NAMES, got, want):
            tol = 1e-5 + (2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0)
            e = ref.rel(x[:, h:h + 32], y)
            assert e <= tol, f"{name}, heads {h} ..: rel-L2 {e:.3e}"
