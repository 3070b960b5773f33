"""Without a GPU: the reference gradients against differences of the fp64 oracle, and every refusal of the new entry
points (all of them on the host, before anything is launched)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import layer_reference as ref
from gated_delta_rule_149_b200.inputs import make_custom

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_149_b200 import build, gdn
    build.build()
    return gdn.load_library()


def test_header_declares_and_library_exports(lib):
    src = open(os.path.join(ROOT, "include", "gdn.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    for name in ("gdn_backward", "gdn_rotary", "gdn_rotary_backward", "gdn_gated_norm", "gdn_gated_norm_backward"):
        assert re.search(r"^int %s\(" % name, src, flags=re.M) and hasattr(lib, name)


# ------------------------------------------------------------------ the reference itself
@pytest.mark.parametrize("bidi", [False, True])
def test_reference_gradients_are_differences_of_the_oracle(oracle_mod, bidi):
    """d/de L(x + e u) at e = 0, L = <do, o> + <dstate, state>: central differences of the C oracle, whose error is
    e^2 L''' / 6 + eps L / e, about 1e-8 of the largest term at e = 1e-4 with values of order one."""
    inp = make_custom(1, 2, 9, 32, 32, dtype="fp32", seed=5, state0=True, decay_shift=0.0)
    x = [t.double() for t in (inp.q, inp.k, inp.v, inp.beta, inp.decay, inp.state0)]
    g = torch.Generator().manual_seed(6)
    do = torch.randn(inp.v.shape, generator=g, dtype=torch.float64)
    ds = torch.randn(((2,) if bidi else ()) + tuple(inp.state0.shape), generator=g, dtype=torch.float64)
    grads = ref.recurrence_gradients(*x[:5], do, x[5], ds, bidi)

    def loss(vals):
        o, s = oracle_mod.gdn_forward(*(t.numpy() for t in vals[:5]), vals[5].numpy(), bidi=bidi)
        return float((do * torch.from_numpy(o)).sum() + (ds * torch.from_numpy(s)).sum())

    for i, name in enumerate(("q", "k", "v", "beta", "decay", "state_in")):
        u = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        e = 1e-4
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + e * u, x[i] - e * u
        diff = (loss(up) - loss(down)) / (2 * e)
        want = float((grads[i] * u).sum())
        scale = float(grads[i].norm() * u.norm())
        assert abs(diff - want) <= 1e-6 * scale, f"{name}: {diff} against {want}"


def test_reference_rotary_preserves_norms_and_relative_positions():
    g = torch.Generator().manual_seed(1)
    x, y = (torch.randn(1, 1, 1, 12, generator=g, dtype=torch.float64) for _ in range(2))
    at = lambda *p: torch.tensor([[p]])  # noqa: E731
    for half in (False, True):
        turn = lambda z, p: ref.rotary(z, (4, 4, 4), 100.0, half, p, False, 1e-6)  # noqa: E731,B023
        assert torch.allclose(turn(x, at(3, 5, 7)).norm(), x.norm(), rtol=1e-14)
        a = (turn(x, at(3, 5, 7)) * turn(y, at(1, 9, 2))).sum()
        b = (turn(x, at(13, 15, 17)) * turn(y, at(11, 19, 12))).sum()
        assert torch.allclose(a, b, rtol=1e-12)
        assert torch.equal(turn(x, at(0, 0, 0)), x)


# ------------------------------------------------------------------ refusals
P, PM = 0x10000, 0x10001


def view(data=P, sb=1 << 20, sh=1 << 12, st=1 << 8):
    from gated_delta_rule_149_b200.gdn import View
    return View(data, sb, sh, st)


def bwd(lib, null=None, bad=None, B=1, H=1, T=64, dk=128, dv=128, mode=0):
    names = ("q", "k", "v", "beta", "decay", "state_in", "dout", "dstate", "dq", "dk", "dv", "dbeta", "ddecay", "dstate_in")
    p = [ctypes.c_void_p(None if n == null else P + 8 if n == bad else P) for n in names]
    return lib.gdn_backward(*p, B, H, T, dk, dv, mode, None)


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "decay", "dout", "dq", "dk", "dv", "dbeta", "ddecay"])
def test_backward_null(lib, name):
    assert bwd(lib, null=name) == -1 and b"non-NULL" in lib.gdn_last_error()


@pytest.mark.parametrize("name", ["q", "beta", "state_in", "dout", "dstate", "dq", "dbeta", "dstate_in"])
def test_backward_misaligned(lib, name):
    assert bwd(lib, bad=name) == -3 and b"aligned" in lib.gdn_last_error()


@pytest.mark.parametrize("kw,code", [(dict(T=0), -1), (dict(B=-1), -1), (dict(mode=8), -1), (dict(mode=16), -1), (dict(mode=4), -2),
                                     (dict(dk=48), -2), (dict(dv=160), -2), (dict(B=256, H=256), -2), (dict(T=2 ** 31 - 1), -2)])
def test_backward_sizes_and_modes(lib, kw, code):
    assert bwd(lib, **kw) == code


ROT = dict(pos=None, psb=0, B=2, H=2, T=4, d=32, axes=(12, 10, 10), gh=2, gw=2, start=0, theta=1e4, eps=1e-6, mode=0)


def rot(lib, back=False, q=True, k=True, dq=True, dk=True, yq=True, yk=True, **kw):
    c = {**ROT, **kw}
    made = lambda x: view() if x is True else None if x is None else x  # noqa: E731
    tail = (c["pos"], c["psb"], c["B"], c["H"], c["T"], c["d"], *c["axes"], c["gh"], c["gw"], c["start"], c["theta"], c["eps"],
            c["mode"], None)
    if back:
        return lib.gdn_rotary_backward(*(made(x) for x in (dq, dk, q, k, yq, yk)), *tail)
    return lib.gdn_rotary(*(made(x) for x in (q, k, yq, yk)), *tail)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(yq=None), -1), (dict(yk=None), -1), (dict(k=None), -1), (dict(q=view(0)), -1),
    (dict(q=view(PM)), -3), (dict(yk=view(PM)), -3), (dict(q=view(sb=-1)), -1), (dict(q=view(st=1 << 62)), -1),
    (dict(yq=view(st=8)), -1), (dict(yq=view(sh=0)), -1),
    (dict(B=0), -1), (dict(H=0), -1), (dict(T=0), -1), (dict(B=300, H=300), -2), (dict(T=2 ** 31 - 1), -2), (dict(d=31), -2), (dict(d=0, axes=(0, 0, 0)), -2),
    (dict(d=258, axes=(258, 0, 0)), -2), (dict(axes=(12, 10, 8)), -1), (dict(axes=(11, 11, 10)), -1), (dict(axes=(-2, 24, 10)), -1),
    (dict(gh=0), -1), (dict(gw=-1), -1), (dict(start=-1), -1), (dict(start=(1 << 52) + 1), -1), (dict(theta=0.0), -1),
    (dict(theta=float("nan")), -1), (dict(theta=float("inf")), -1), (dict(eps=0.0, mode=32), -1), (dict(eps=float("nan"), mode=32), -1),
    (dict(mode=1), -1), (dict(mode=64), -1), (dict(pos=0x10002), -3), (dict(pos=P, psb=-1), -1),
])
def test_rotary_refuses(lib, kw, code):
    assert rot(lib, **kw) == code and lib.gdn_last_error()


@pytest.mark.parametrize("kw,code", [(dict(dq=None), -1), (dict(dk=None), -1), (dict(mode=32, q=None), -1), (dict(mode=32, k=None), -1),
                                     (dict(dk=view(PM)), -3), (dict(yq=view(st=2)), -1)])
def test_rotary_backward_refuses(lib, kw, code):
    assert rot(lib, back=True, **kw) == code


def norm(lib, back=False, o=True, gate=True, y=True, dy=True, dout=True, dgate=True, weight=P, dweight=P, per_head=0, B=2, H=2, T=4,
         dv=32, eps=1e-5, mode=0):
    made = lambda x: view() if x is True else None if x is None else x  # noqa: E731
    if back:
        return lib.gdn_gated_norm_backward(made(dy), made(o), made(gate), weight, per_head, made(dout), made(dgate), dweight, B, H, T,
                                           dv, eps, mode, None)
    return lib.gdn_gated_norm(made(o), made(gate), weight, per_head, made(y), B, H, T, dv, eps, mode, None)


@pytest.mark.parametrize("kw,code", [
    (dict(o=None), -1), (dict(y=None), -1), (dict(o=view(PM)), -3), (dict(gate=view(PM)), -3), (dict(y=view(st=31)), -1),
    (dict(weight=P + 2), -3), (dict(eps=0.0), -1), (dict(eps=float("inf")), -1), (dict(dv=0), -2), (dict(dv=257), -2),
    (dict(T=0), -1), (dict(B=65536), -2), (dict(mode=1), -1), (dict(mode=32), -1),
])
def test_gated_norm_refuses(lib, kw, code):
    assert norm(lib, **kw) == code and lib.gdn_last_error()


@pytest.mark.parametrize("kw,code", [(dict(dy=None), -1), (dict(dout=None), -1), (dict(dgate=None), -1), (dict(gate=None), -1),
                                     (dict(weight=None), -1), (dict(dweight=P + 1), -3), (dict(dout=view(sh=3)), -1)])
def test_gated_norm_backward_refuses(lib, kw, code):
    assert norm(lib, back=True, **kw) == code


def test_python_refuses_cpu_tensors_and_wrong_types():
    from gated_delta_rule_149_b200 import gdn_backward, gdn_gated_norm, gdn_gated_norm_backward, gdn_rotary, gdn_rotary_backward
    x, g = torch.zeros(1, 1, 4, 32), torch.zeros(1, 1, 4)
    with pytest.raises(ValueError):
        gdn_backward(x, x, x, g, g, x)
    with pytest.raises(ValueError):
        gdn_backward(x[0], x, x, g, g, x)
    with pytest.raises(ValueError):
        gdn_rotary(x, axes=(12, 10, 10), grid=(2, 2))
    with pytest.raises(ValueError):
        gdn_rotary_backward(x, axes=(12, 10, 10), grid=(2, 2))
    with pytest.raises(ValueError):
        gdn_gated_norm(x)
    with pytest.raises(ValueError):
        gdn_gated_norm_backward(torch.zeros(1, 4, 32), x)


def test_reference_matches_oracle_forward(oracle_mod):
    inp = make_custom(1, 2, 11, 32, 64, dtype="fp32", seed=3, state0=True, decay_shift=0.0)
    for bidi in (False, True):
        o, s = ref.recurrence(inp.q, inp.k, inp.v, inp.beta, inp.decay, inp.state0, bidi)
        o2, s2 = oracle_mod.gdn_forward(*(t.numpy() for t in (inp.q, inp.k, inp.v, inp.beta, inp.decay, inp.state0)), bidi=bidi)
        assert np.abs(o.numpy() - o2).max() < 1e-12 and np.abs(s.numpy() - s2).max() < 1e-12
