"""gdn_rotary and gdn_gated_norm, forward and backward, against their definitions in 64 bits.

Tolerances: each value within half a step of its type of the reference, plus fp32's part.  Rotary: a value is at
most about ten fp32 roundings (two products and a sum, the sine and cosine at two units each, the row's factor) of
terms no larger than the row's norm times the factor: 2^-20 of that.  Gated norm: the same count on terms no larger
than the row's largest |w n silu(g)| (forward) or r |dn| (backward); the sigmoid is within 2^-21 of itself."""
import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200 import (gdn_backward, gdn_forward, gdn_gated_norm, gdn_gated_norm_backward, gdn_layer_backward,
                                       gdn_layer_forward, gdn_rotary, gdn_rotary_backward)

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
FINE = 2.0 ** -20


def normal(*shape, dtype=FP32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def norms(x):
    return x.double().norm(dim=-1, keepdim=True)


# ------------------------------------------------------------------ rotary
def split(d):
    side = 2 * (d // 6)
    return (d - 2 * side, side, side)


@pytest.mark.parametrize("B,H,T,d,dtype,half,l2", [
    (1, 1, 1, 2, FP32, False, False), (1, 1, 1, 2, BF16, True, True), (2, 3, 7, 32, FP32, False, True),
    (1, 2, 65, 64, BF16, False, True), (2, 5, 33, 96, BF16, True, True), (1, 16, 9, 128, BF16, False, True),
    (3, 1, 100, 128, FP32, True, False), (1, 3, 17, 256, BF16, False, True), (2, 2, 30, 50, BF16, False, True),
    (1, 2, 31, 34, FP32, True, True), (1, 2, 31, 254, BF16, False, False), (1, 4, 5, 16, BF16, True, True),
    (1, 20, 1, 128, BF16, False, True)])
def test_rotary_both_ways(B, H, T, d, dtype, half, l2):
    grid, start = (3, 5), 1234567
    axes = split(d)
    qk = normal(B, T, 2, H, d, dtype=dtype, seed=T + d)
    q, k = qk[:, :, 0].transpose(1, 2), qk[:, :, 1].transpose(1, 2)
    how = dict(axes=axes, grid=grid, start=start, half=half, l2norm=l2, eps=1e-6)
    pos = ref.grid_positions(T, grid, start)
    got = gdn_rotary(q, k, **how)
    gq, gk = normal(B, H, T, d, dtype=dtype, seed=1), normal(B, H, T, d, dtype=dtype, seed=2)
    back = gdn_rotary_backward(gq, gk, q if l2 else None, k if l2 else None, **how)
    for x, y, g, dx in zip((q, k), got, (gq, gk), back):
        leaf = x.detach().cpu().double().requires_grad_()
        want = ref.rotary(leaf, axes, 10000.0, half, pos, l2, 1e-6)
        assert y.is_contiguous() and y.shape == x.shape and dx.transpose(1, 2).is_contiguous()
        scale = (norms(x).cpu() ** 2 + 1e-6).sqrt()
        ref.close(y.cpu(), want.detach(), dtype, FINE * (1.0 if l2 else norms(x).cpu()), "forward")
        want_dx, = ref.gradients((want,), (g.cpu(),), (leaf,))
        ref.close(dx.cpu(), want_dx, dtype, 2 * FINE * norms(g).cpu() / (scale if l2 else 1.0), "backward")


@pytest.mark.parametrize("shared", [False, True])
def test_rotary_explicit_positions_q_alone_and_uneven_axes(shared):
    """Positions far out, negative and repeated; one axis without a pair; q without k."""
    B, H, T, d = 2, 3, 40, 64
    axes = (0, 14, 50)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (1 if shared else B, T, 3), generator=torch.Generator().manual_seed(2), dtype=torch.int64)
    pos[:, 1] = pos[:, 0]
    pos = pos.to(torch.int32)
    q = normal(B, H, T, d, seed=3)
    given = (pos[0] if shared else pos).cuda()
    y = gdn_rotary(q, axes=axes, positions=given, theta=500.0)
    want = ref.rotary(q.cpu(), axes, 500.0, False, pos, False, 1e-6)
    # an angle of 2^31 radians is 3e8 turns: 2^-53 of that, and the frequency's own 2^-53, leave about 2^-22 of a radian
    ref.close(y.cpu(), want, FP32, 4 * FINE * norms(q).cpu())
    assert torch.equal(y[:, :, 0] if shared else y[:1, :, 0], (y if shared else y[:1])[:, :, 0])
    g = normal(B, H, T, d, seed=4)
    back = gdn_rotary_backward(g, axes=axes, positions=given, theta=500.0)
    turned = gdn_rotary(back, axes=axes, positions=given, theta=500.0)      # Rot Rot^T = 1
    ref.close(turned.cpu(), g.double().cpu(), FP32, 4 * FINE * norms(g).cpu())


@pytest.mark.parametrize("offset,pitch", [(0, 128), (1, 130), (4, 132), (8, 136)])
def test_rotary_strides_and_alignment(offset, pitch):
    """Rows on and off 16-byte boundaries, gaps between rows, broadcast batches: the same values on every path."""
    H, T, d = 2, 37, 128
    room = normal(offset + H * T * pitch, dtype=BF16, seed=9)
    q = room[offset:].as_strided((2, H, T, d), (0, T * pitch, pitch, 1), storage_offset=offset)
    how = dict(axes=(44, 42, 42), grid=(4, 4), l2norm=True)
    y = gdn_rotary(q, **how)
    ref.close(y.cpu(), ref.rotary(q.cpu(), (44, 42, 42), 10000.0, False, ref.grid_positions(T, (4, 4), 0), True, 1e-6), BF16, FINE)
    assert torch.equal(y[0], y[1])
    clean = gdn_rotary(q.contiguous(), **how)
    # the two paths add a row's squares in another order: one step apart at most
    ref.close(y.float().cpu(), clean.double().cpu(), BF16, 2.0 ** -8 * clean.abs().double().cpu() + FINE)


def test_rotary_chunks_continue_the_sequence():
    q = normal(1, 4, 100, 128, dtype=BF16, seed=5)
    how = dict(axes=(44, 42, 42), grid=(3, 7), l2norm=True)
    whole = gdn_rotary(q, **how)
    parts = [gdn_rotary(q[:, :, a:b], start=a, **how) for a, b in ((0, 1), (1, 64), (64, 100))]
    assert torch.equal(torch.cat(parts, 2), whole)


def test_rotary_zero_rows_and_non_finite_rows_stay_apart():
    q = normal(1, 2, 8, 64, seed=6)
    clean = gdn_rotary(q, axes=(24, 20, 20), grid=(2, 2), l2norm=True)
    q[0, 0, 3] = 0
    q[0, 1, 5, 7] = float("nan")
    q[0, 0, 6, 0] = float("inf")
    y = gdn_rotary(q, axes=(24, 20, 20), grid=(2, 2), l2norm=True)
    assert (y[0, 0, 3] == 0).all() and y[0, 1, 5].isnan().all()
    keep = torch.ones(2, 8, dtype=torch.bool)
    keep[0, 3] = keep[1, 5] = keep[0, 6] = False
    assert torch.equal(y[0][keep], clean[0][keep])


# ------------------------------------------------------------------ gated norm
@pytest.mark.parametrize("B,H,T,dv,dtype,gate,weight", [
    (1, 1, 1, 1, FP32, True, "shared"), (1, 16, 1, 128, BF16, True, "shared"), (2, 3, 65, 64, BF16, True, "head"),
    (2, 3, 65, 64, FP32, False, "shared"), (1, 2, 200, 80, FP32, True, "head"), (3, 5, 19, 33, BF16, True, "shared"),
    (1, 2, 50, 256, BF16, True, "none"), (2, 2, 50, 255, FP32, False, "none"), (1, 4, 1000, 32, BF16, True, "head"),
    (1, 3, 700, 96, FP32, True, "shared")])
def test_gated_norm_both_ways(B, H, T, dv, dtype, gate, weight):
    o = normal(B, H, T, dv, dtype=dtype, seed=dv)
    g = normal(B, T, H, dv, dtype=dtype, seed=dv + 1).transpose(1, 2) * 4 if gate else None
    w = None if weight == "none" else 1 + 0.3 * normal(*((H, dv) if weight == "head" else (dv,)), seed=2)
    dy = normal(B, T, H * dv, dtype=dtype, seed=7)
    y = gdn_gated_norm(o, g, w, eps=1e-5)
    do, dg, dw = gdn_gated_norm_backward(dy, o, g, w, eps=1e-5)
    leaves = [None if x is None else x.detach().cpu().double().requires_grad_() for x in (o, g, w)]
    want = ref.gated_norm(*leaves, 1e-5)
    ref.close(y.cpu(), want.detach(), dtype, 4 * FINE * want.detach().abs() + 1e-30, "y")
    there = [x for x in leaves if x is not None]
    grads = iter(ref.gradients((want,), (dy.cpu(),), there))
    wdo, wdg, wdw = (None if x is None else next(grads) for x in leaves)
    # do: terms r |dn| and r n mean(dn n), both at most the norm of r dn over the row
    act = torch.ones(()) if g is None else (g.double() * torch.sigmoid(g.double())).cpu()
    dn = dy.cpu().double().view(B, T, H, dv).transpose(1, 2) * act * (1.0 if w is None else (leaves[2].detach() if w.dim() == 1 else leaves[2].detach()[:, None]))
    r = 1 / ((o.cpu().double() ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
    ref.close(do.cpu(), wdo, dtype, 4 * FINE * norms(r * dn), "do")
    assert do.is_contiguous()
    if g is None:
        assert dg is None
    else:
        # s + g s (1 - s) crosses zero: its error goes with its terms, at most 1.3 together
        n = r * o.cpu().double() * (1.0 if w is None else (leaves[2].detach() if w.dim() == 1 else leaves[2].detach()[:, None]))
        ref.close(dg.cpu(), wdg, dtype, 4 * FINE * 1.3 * (dy.cpu().double().view(B, T, H, dv).transpose(1, 2) * n).abs(), "dgate")
        assert dg.transpose(1, 2).is_contiguous()
    if w is None:
        assert dw is None
    else:
        # sums of up to B H T fp32 terms: each carries 4 FINE, and a sum in a tree of serial runs no more than 64 long
        # per block adds at most (64 + 32 + rows per thread) half steps
        terms = (dn / (1.0 if w.dim() == 0 else (leaves[2].detach() if w.dim() == 1 else leaves[2].detach()[:, None])) * r * o.cpu().double()).abs()
        ref.close(dw.cpu(), wdw, FP32, (4 * FINE + 128 * 2.0 ** -24) * terms.sum((0, 2) if w.dim() == 2 else (0, 1, 2)), "dweight")
        again = gdn_gated_norm_backward(dy, o, g, w, eps=1e-5)[2]
        assert torch.equal(again, dw)


def test_gated_norm_extreme_gates_and_zero_rows():
    """A gate far below zero closes (0, not NaN), one far above lets through; a row of zeros stays zero, its gradient is
    dn / sqrt(eps)."""
    o = normal(1, 1, 4, 64, seed=3)
    o[0, 0, 1] = 0
    g = torch.zeros_like(o)
    g[0, 0, 0], g[0, 0, 2], g[0, 0, 3] = -200.0, 200.0, -3e38
    y = gdn_gated_norm(o, g, eps=1e-4).view(4, 64)
    assert (y[0] == 0).all() and (y[1] == 0).all() and (y[3] == 0).all()
    want = ref.gated_norm(o.cpu(), g.cpu(), None, 1e-4).view(4, 64)
    ref.close(y[2].cpu(), want[2], FP32, 4 * FINE * want[2].abs())
    g[0, 0, 1] = 1.0
    dy = torch.ones(1, 4, 64, device="cuda")
    do, dg, _ = gdn_gated_norm_backward(dy, o, g, eps=1e-4)
    assert torch.isfinite(do).all() and torch.isfinite(dg).all() and (dg[0, 0, 1] == 0).all()
    silu = float(torch.sigmoid(torch.tensor(1.0, dtype=torch.float64)))
    assert torch.allclose(do[0, 0, 1].cpu().double(), torch.full((64,), silu * 100.0, dtype=torch.float64), rtol=1e-5)


def test_gated_norm_strided_inputs():
    """o token-major, gate a slice of a wider projection, dy rows apart, rows off 16-byte boundaries."""
    B, H, T, dv = 2, 3, 21, 64
    o = normal(B, T, H, dv, dtype=BF16, seed=1).transpose(1, 2)
    wide = normal(B, T, H * dv * 2 + 3, dtype=BF16, seed=2)
    for off in (0, 3):
        g = wide[:, :, off:off + H * dv].unflatten(2, (H, dv)).transpose(1, 2)
        dy = wide[:, :, H * dv:2 * H * dv]
        w = 1 + normal(dv, seed=4) * 0.1
        y = gdn_gated_norm(o, g, w)
        want = ref.gated_norm(o.cpu(), g.cpu(), w.cpu(), 1e-5)
        ref.close(y.cpu(), want, BF16, 4 * FINE * want.abs())
        a = gdn_gated_norm_backward(dy, o, g, w)
        b = gdn_gated_norm_backward(dy.contiguous(), o.contiguous(), g.contiguous(), w)
        for x, z in zip(a, b):
            # rows off 16-byte boundaries are summed in another order
            ref.close(x.float().cpu(), z.double().cpu(), x.dtype, (2.0 ** -8 if x.dtype == BF16 else 0) * z.double().abs().cpu() + 1e-4 * float(z.abs().max()))


# ------------------------------------------------------------------ streams, devices, graphs
def test_own_stream_and_graph_replays():
    q = normal(1, 4, 300, 128, dtype=BF16, seed=1)
    o, g = normal(1, 4, 300, 128, dtype=BF16, seed=2), normal(1, 4, 300, 128, dtype=BF16, seed=3)
    w = torch.ones(128, device="cuda")
    how = dict(axes=(44, 42, 42), grid=(5, 5), l2norm=True)
    dy = normal(1, 300, 512, dtype=BF16, seed=4)
    want = [gdn_rotary(q, **how), *gdn_gated_norm_backward(dy, o, g, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [gdn_rotary(q, **how, stream=side), *gdn_gated_norm_backward(dy, o, g, w, stream=side)]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):                                   # two graphs, each with its own workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = [gdn_rotary(q, **how), *gdn_gated_norm_backward(dy, o, g, w)]
        graphs.append((graph, out))
    q.copy_(normal(1, 4, 300, 128, dtype=BF16, seed=8))
    dy.copy_(normal(1, 300, 512, dtype=BF16, seed=9))
    want = [gdn_rotary(q, **how), *gdn_gated_norm_backward(dy, o, g, w)]
    for _ in range(2):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_offsets_beyond_32_bits():
    """Rows that start behind element 2^31 of a buffer: read and written where they are."""
    room = torch.zeros(2 ** 31 + 4096, dtype=BF16, device="cuda")
    d, T = 128, 3
    q = room.as_strided((2, 1, T, d), (2 ** 31, 2 ** 20, d, 1))
    q.copy_(normal(2, 1, T, d, dtype=BF16, seed=3))
    how = dict(axes=(44, 42, 42), grid=(2, 2), l2norm=True)
    assert torch.equal(gdn_rotary(q, **how), gdn_rotary(q.contiguous(), **how))
    assert torch.equal(gdn_gated_norm(q), gdn_gated_norm(q.contiguous()))


# ------------------------------------------------------------------ the layer
@pytest.mark.parametrize("bidi", [False, True])
@pytest.mark.parametrize("dtype,H,T,dk,dv", [(FP32, 2, 70, 32, 64), (BF16, 2, 130, 128, 128)])
def test_layer_runs_and_its_gradients(dtype, H, T, dk, dv, bidi):
    """rotary -> recurrence -> gated norm and back.  fp32: against the layer's definition in 64 bits.  bf16: against the
    same chain with the tensors that the layer itself rounds (rotated q and k, o, do, dq, dk) taken as rounded."""
    B = 2
    qk = normal(B, T, 2, H, dk, dtype=dtype, seed=1)
    q, k = qk[:, :, 0].transpose(1, 2), qk[:, :, 1].transpose(1, 2)
    v, gate = normal(B, H, T, dv, dtype=dtype, seed=2), normal(B, T, H, dv, dtype=dtype, seed=3).transpose(1, 2)
    beta, decay = torch.sigmoid(normal(B, H, T, seed=4)), torch.sigmoid(2 + normal(B, H, T, seed=5))
    w, s0 = 1 + 0.1 * normal(dv, seed=6), 0.1 * normal(B, H, dk, dv, seed=7)
    side = 2 * (dk // 6)
    how = dict(axes=(dk - 2 * side, side, side), grid=(4, 5), start=40)
    y, state, saved = gdn_layer_forward(q, k, v, beta, decay, gate, w, s0, bidi=bidi, **how)
    dy = normal(B, T, H * dv, dtype=dtype, seed=8)
    ds = normal(*state.shape, seed=9)
    got = gdn_layer_backward(dy, saved, ds)
    if dtype == FP32:
        names = ("q", "k", "v", "beta", "decay", "gate", "weight", "state_in")
        leaves = [x.detach().cpu().double().requires_grad_() for x in (q, k, v, beta, decay, gate, w, s0)]
        pos = ref.grid_positions(T, (4, 5), 40)
        turned = [ref.rotary(x, how["axes"], 10000.0, False, pos, True, 1e-6) for x in leaves[:2]]
        o, s = ref.recurrence(*turned, *leaves[2:5], leaves[7], bidi)
        out = ref.gated_norm(o, leaves[5], leaves[6], 1e-5)
        assert ref.rel(y.cpu(), out.detach()) <= 1e-5 and ref.rel(state.cpu(), s.detach()) <= 1e-5
        for name, x in zip(names, ref.gradients((out, s), (dy.cpu(), ds.cpu()), leaves)):
            assert ref.rel(got[name].cpu(), x) <= 2e-5, name
    else:
        qr, kr = gdn_rotary(q, k, l2norm=True, **how)
        o, st = gdn_forward(qr, kr, v, beta, decay, s0, bidi=bidi)
        assert torch.equal(y, gdn_gated_norm(o, gate, w)) and torch.equal(st, state)
        do, dg, dw = gdn_gated_norm_backward(dy, o, gate, w)
        dq, dk_, dv_, db, da, dsi = gdn_backward(qr, kr, v, beta, decay, do, s0, ds, bidi=bidi)
        dq, dk_ = gdn_rotary_backward(dq, dk_, q, k, l2norm=True, **how)
        for name, x in dict(q=dq, k=dk_, v=dv_, beta=db, decay=da, gate=dg, weight=dw, state_in=dsi).items():
            assert torch.equal(got[name], x), name


def test_layer_streams_chunk_by_chunk():
    """A sequence in three chunks with the state carried gives the whole sequence's output."""
    H, T, d = 2, 192, 64
    q, k, v = (normal(1, H, T, d, seed=i) for i in range(3))
    beta, decay = torch.sigmoid(normal(1, H, T, seed=4)), torch.sigmoid(2 + normal(1, H, T, seed=5))
    how = dict(axes=(24, 20, 20), grid=(3, 4))
    whole, _, _ = gdn_layer_forward(q, k, v, beta, decay, **how)
    state, parts = None, []
    for a, b in ((0, 1), (1, 100), (100, 192)):
        cut = [x[:, :, a:b].contiguous() for x in (q, k, v, beta, decay)]
        y, state, _ = gdn_layer_forward(*cut, state_in=state, start=a, **how)
        parts.append(y)
    assert ref.rel(torch.cat(parts, 1).cpu(), whole.double().cpu()) <= 1e-6
