"""The operators that train a Gated-Delta-Net layer, as a user's program calls them.

    rotary   gdn_rotary / gdn_rotary_backward: q and k of a projection, rotated by (time, height, width)
             positions, L2-normalised if wanted, laid out head-major as gdn_forward takes them.
    norm     gdn_gated_norm / gdn_gated_norm_backward: the read-out of gdn_forward, normalised per head,
             scaled, gated with SiLU, laid out token-major as the output projection takes it.
    gdn      gdn_backward: the gradients of gdn_forward.

A case names the operator (``op``), the direction where there are two, sizes, type and form.
"""
import math

import torch

own = False

C = 64   # tokens per chunk of the recurrence's plain form


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the small fp32 workload's shape (4 frames of 8x8 tokens): launch latency counts
        dict(name="rotary_small_fp32", op="rotary", back=False, B=1, H=2, T=256, d=32, dtype="fp32", h=8, w=8, start=0,
             half=False, l2=True, pos=False),
        # one streaming chunk, 3 latent frames of 30x52 tokens, starting at frame 9 of the clip
        dict(name="rotary_480p_chunk", op="rotary", back=False, B=1, H=16, T=4680, d=128, dtype="bf16", h=30, w=52,
             start=14040, half=False, l2=True, pos=False),
        # explicit positions (a packed batch of images), rotation of halves, ragged sizes
        dict(name="rotary_positions_odd", op="rotary", back=True, B=3, H=5, T=1009, d=96, dtype="bf16", h=0, w=0, start=0,
             half=True, l2=False, pos=True),
        # the gradient of the whole 720p clip, 21 frames of 45x80 tokens
        dict(name="rotary_720p_backward", op="rotary", back=True, B=2, H=16, T=75600, d=128, dtype="bf16", h=45, w=80,
             start=0, half=False, l2=True, pos=False),
        # a single token of 16 heads: latency only
        dict(name="norm_one_token", op="norm", back=False, B=1, H=16, T=1, d=128, dtype="bf16", gate=True, per_head=False),
        # one streaming chunk
        dict(name="norm_480p_chunk", op="norm", back=False, B=1, H=16, T=4680, d=128, dtype="bf16", gate=True, per_head=False),
        # fp32, sizes that fill no tile, a weight per head
        dict(name="norm_backward_odd_fp32", op="norm", back=True, B=3, H=5, T=1009, d=80, dtype="fp32", gate=True, per_head=True),
        # the gradient of the whole 720p clip
        dict(name="norm_720p_backward", op="norm", back=True, B=2, H=16, T=75600, d=128, dtype="bf16", gate=True, per_head=False),
        # the small fp32 workload
        dict(name="gdn_small_fp32", op="gdn", B=1, H=2, T=256, d=32, dv=32, dtype="fp32", bidi=False, state=False, shift=0.0, frame=0),
        # one streaming chunk with the carried state, decay per frame
        dict(name="gdn_480p_chunk", op="gdn", B=1, H=16, T=4680, d=128, dv=128, dtype="bf16", bidi=False, state=True, shift=2.0,
             frame=1560),
        # a ragged batch of clips, long memory (decay near 1), values half as wide as keys
        dict(name="gdn_ragged_dv64", op="gdn", B=3, H=5, T=1009, d=128, dv=64, dtype="bf16", bidi=True, state=True, shift=-4.0,
             frame=0),
        # a full clip, both directions, gates per token
        dict(name="gdn_bidi_clip_480p", op="gdn", B=1, H=16, T=32760, d=128, dv=128, dtype="bf16", bidi=True, state=False, shift=2.0,
             frame=0),
    ]


def _size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "norm", "gdn"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    B, H, T = rng.randint(1, 3), rng.randint(1, 20), _size(rng, 1, 75600)
    if op == "rotary":
        d = 2 * rng.randint(4, 64) if rng.random() < 0.4 else rng.choice([32, 64, 96, 128])
        cap = 2 * 16 * 75600 * 64 // (2 if dtype == "fp32" else 1)
        T = max(1, min(T, cap // (B * H * d)))
        pos = rng.random() < 0.3
        return dict(op=op, back=rng.random() < 0.5, B=B, H=H, T=T, d=d, dtype=dtype, h=0 if pos else rng.randint(1, 60),
                    w=0 if pos else rng.randint(1, 100), start=0 if pos else rng.randint(0, 200000), half=rng.random() < 0.4,
                    l2=rng.random() < 0.6, pos=pos)
    if op == "norm":
        d = rng.randint(8, 128) if rng.random() < 0.4 else rng.choice([32, 64, 96, 128])
        cap = 2 * 16 * 75600 * 64 // (2 if dtype == "fp32" else 1)
        T = max(1, min(T, cap // (B * H * d)))
        return dict(op=op, back=rng.random() < 0.5, B=B, H=H, T=T, d=d, dtype=dtype, gate=rng.random() < 0.8,
                    per_head=rng.random() < 0.4)
    bidi = rng.random() < 0.5
    d, dv = (rng.choice([32, 64, 96, 128]), rng.choice([32, 64, 96, 128])) if dtype == "fp32" else (128, rng.choice([64, 128]))
    T = max(1, min(T, 16 * 8000 // (B * H * (2 if bidi else 1))))
    return dict(op=op, B=B, H=H, T=T, d=d, dv=dv, dtype=dtype, bidi=bidi, state=rng.random() < 0.5,
                shift=rng.choice([2.0, 0.0, -4.0]), frame=rng.choice([0, 0, 260]))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["B"] * case["H"] * case["T"]
    d = case["d"]
    if case["op"] == "rotary":
        moved = 6 if case["back"] and case["l2"] else 4          # q and k: read (gradient and input), written
        pos = case["B"] * case["T"] * 3 * 4 if case["pos"] else 0
        return {"bytes": n * d * e * moved + pos, "flops": n * d * (14 if case["l2"] else 6)}
    if case["op"] == "norm":
        gate = 1 if case["gate"] else 0
        moved = 3 + 2 * gate if case["back"] else 2 + gate       # dy, o, gate read, do, dgate written; or o, gate, y
        return {"bytes": n * d * e * moved + 4 * d * (2 if case["back"] else 1), "flops": n * d * (30 if case["back"] else 12)}
    dv, dirs = case["dv"], 2 if case["bidi"] else 1
    states = case["B"] * case["H"] * d * dv * 4 * ((dirs + 2) if case["state"] else 1)
    # q, k, v, do read; dq, dk, dv written; gates and their gradients.  Products with a dk x dv state, per token
    # and direction: S k, k u^T (forward), q do^T, H do, dS^T k, dS u, H x, k x^T (backward).
    return {"bytes": n * ((4 * d + 3 * dv) * e + 16) + states, "flops": 16 * d * dv * n * dirs}


# ------------------------------------------------------------------ inputs
def _axes(d):
    """The usual split of a head's d/2 rotation pairs: a third each for height and width, the rest for time."""
    side = 2 * (d // 6)
    return (d - 2 * side, side, side)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[case["dtype"]]
    B, H, T, d = case["B"], case["H"], case["T"], case["d"]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case)
    if case["op"] == "rotary":
        qk = normal(B, T, 2, H, d)                               # one projection holds q and k, token-major
        s["q"], s["k"] = qk[:, :, 0].transpose(1, 2), qk[:, :, 1].transpose(1, 2)
        if case["back"]:
            s["dq"], s["dk"] = normal(B, H, T, d), normal(B, H, T, d)
        s["axes"] = _axes(d)
        s["positions"] = None
        if case["pos"]:
            s["positions"] = torch.randint(0, 100000, (B, T, 3), generator=g, device=dev, dtype=torch.int32)
    elif case["op"] == "norm":
        s["o"] = normal(B, H, T, d)
        s["gate_t"] = normal(B, T, H, d).transpose(1, 2) if case["gate"] else None
        s["weight"] = 1.0 + 0.1 * normal(*((H, d) if case["per_head"] else (d,)), dtype=torch.float32)
        if case["back"]:
            s["dy"] = normal(B, T, H * d)
    else:
        dv = case["dv"]
        unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
        s["q"], s["k"] = unit(normal(B, H, T, d, dtype=torch.float32)), unit(normal(B, H, T, d, dtype=torch.float32))
        s["v"], s["do"] = normal(B, H, T, dv), normal(B, H, T, dv)
        s["beta"] = torch.sigmoid(normal(B, H, T, dtype=torch.float32))
        f = case["frame"] or 1
        raw = normal(B, H, -(-T // f), dtype=torch.float32)
        decay = torch.exp(-torch.nn.functional.softplus(raw + case["shift"]))
        s["decay"] = decay.repeat_interleave(f, dim=-1)[..., :T].contiguous()
        s["state_in"] = 0.02 * normal(B, H, d, dv, dtype=torch.float32) if case["state"] else None
        lead = (2,) if case["bidi"] else ()
        s["dstate"] = normal(*lead, B, H, d, dv, dtype=torch.float32) if case["state"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import gated_delta_rule_149_b200 as gdn
        if s["op"] == "rotary":
            how = dict(axes=s["axes"], grid=None if s["pos"] else (s["h"], s["w"]), start=s["start"], positions=s["positions"],
                       theta=10000.0, half=s["half"], l2norm=s["l2"], eps=1e-6)
            if s["back"]:
                return gdn.gdn_rotary_backward(s["dq"], s["dk"], s["q"] if s["l2"] else None, s["k"] if s["l2"] else None, **how)
            return gdn.gdn_rotary(s["q"], s["k"], **how)
        if s["op"] == "norm":
            if s["back"]:
                return gdn.gdn_gated_norm_backward(s["dy"], s["o"], s["gate_t"], s["weight"], eps=1e-5)
            return gdn.gdn_gated_norm(s["o"], s["gate_t"], s["weight"], eps=1e-5)
        return gdn.gdn_backward(s["q"], s["k"], s["v"], s["beta"], s["decay"], s["do"], s["state_in"], s["dstate"], bidi=s["bidi"])
    if s["op"] == "rotary":
        return _plain_rotary(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    return _plain_gdn(s)


# ------------------------------------------------------------------ rotary, plain form
def _angles(s):
    """[B or 1, 1, T, d/2] angles in 64 bits: position of the pair's axis times theta^(-2 i / d_axis)."""
    T, axes = s["T"], s["axes"]
    dev = s["q"].device
    if s["pos"]:
        at = s["positions"].double()
    else:
        t = torch.arange(T, device=dev) + s["start"]
        at = torch.stack([t // (s["h"] * s["w"]), (t // s["w"]) % s["h"], t % s["w"]], dim=-1).double()[None]
    parts = [at[..., a:a + 1] * 10000.0 ** (-torch.arange(0, n, 2, device=dev, dtype=torch.float64) / max(n, 1))
             for a, n in enumerate(axes)]
    return torch.cat(parts, dim=-1)[:, None]


def _pairs(x, half):
    d = x.shape[-1]
    return (x[..., :d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])


def _join(a, b, half):
    return torch.cat([a, b], dim=-1) if half else torch.stack([a, b], dim=-1).flatten(-2)


def _plain_rotary(s):
    ang = _angles(s)
    cos, sin = ang.cos().float(), ang.sin().float()
    out = []
    for name in ("q", "k"):
        x = s[name].float()
        r = torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) if s["l2"] else None
        if not s["back"]:
            a, b = _pairs(x * r if s["l2"] else x, s["half"])
            y = _join(a * cos - b * sin, a * sin + b * cos, s["half"]).to(s[name].dtype)
        else:
            a, b = _pairs(s["d" + name].float(), s["half"])
            y = _join(a * cos + b * sin, b * cos - a * sin, s["half"])
            if s["l2"]:
                y = r * (y - x * r * r * (x * y).sum(-1, keepdim=True))
            y = y.to(s[name].dtype)
        out.append(y)
    return tuple(out)


# ------------------------------------------------------------------ gated norm, plain form
def _plain_norm(s):
    B, H, T, d = s["B"], s["H"], s["T"], s["d"]
    o, dt = s["o"].float(), s["o"].dtype
    w = s["weight"].view(H, 1, d) if s["per_head"] else s["weight"]
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-5)
    if s["gate"]:
        g = s["gate_t"].float()
        sig = 1 / (1 + torch.exp(-g))
    if not s["back"]:
        y = o * r * w
        if s["gate"]:
            y = y * (g * sig)
        return y.transpose(1, 2).reshape(B, T, H * d).to(dt)
    dy = s["dy"].float().view(B, T, H, d).transpose(1, 2)
    n = o * r
    dgate = None
    dn = dy
    if s["gate"]:
        dgate = (dy * n * w * (sig * (1 + g * (1 - sig)))).to(dt)
        dn = dy * (g * sig)
    dw = (dn * n).sum((0, 2) if s["per_head"] else (0, 1, 2))
    dn = dn * w
    do = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    return do.to(dt), dgate, dw


# ------------------------------------------------------------------ the recurrence's gradients, plain form
#   H_t = a_t (I - b_t k_t k_t^T) H_{t-1} + b_t k_t v_t^T,   o_t = H_t^T q_t
# in chunks of C tokens: with G the running sum of log a in a chunk, D_ij = exp(G_i - G_j), X = strict lower of
# D_ij k_i.k_j and N = (I + X diag(b))^-1 X,
#   R = V - diag(exp G) K H0,  W = R - N diag(b) R,  U = diag(b) W,  H1 = exp(G_C) H0 + K^T diag(e) U
#   dU = P^T dO + diag(e) K dH1,  Z = dU - N^T diag(b) dU,  Y = diag(b) Z,
#   dH0 = exp(G_C) dH1 + Q^T diag(exp G) dO - K^T diag(exp G) Y
def _plain_gdn(s):
    B, H, T, dk, dv = s["B"], s["H"], s["T"], s["d"], s["dv"]
    nc = -(-T // C)
    dirs = 2 if s["bidi"] else 1
    n = B * H

    def chunks(x, fill=0.0):                                      # [B,H,T,...] -> [dirs*BH, nc, C, ...]
        x = x.float().reshape(n, T, *x.shape[3:])
        x = torch.cat([x, x.flip(1)]) if dirs == 2 else x
        pad = x.new_full((x.shape[0], nc * C - T, *x.shape[2:]), fill)
        return torch.cat([x, pad], 1).reshape(x.shape[0], nc, C, *x.shape[2:])

    q, k, v, do = (chunks(s[x]) for x in ("q", "k", "v", "do"))
    b, a = chunks(s["beta"]), chunks(s["decay"], 1.0)
    G = a.double().log().cumsum(-1)                               # 64 bits: the differences below lose nothing
    tri = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    D = torch.where(tri, (G[..., :, None] - G[..., None, :]).clamp(max=0.0), torch.zeros((), device=q.device, dtype=torch.float64))
    D = torch.where(tri, D.exp(), torch.zeros_like(D)).float()
    gam, e, gend = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None], G[..., -1].exp().float()
    bb = b[..., None]
    X = (D * (k @ k.mT)).tril(-1)
    P = D * (q @ k.mT)
    N = X.clone()
    Xb = X * b[..., None, :]
    for i in range(1, C):
        N[..., i:i + 1, :] -= Xb[..., i:i + 1, :i] @ N[..., :i, :]
    S = q.shape[0]
    h = q.new_zeros(S, dk, dv)
    dh = q.new_zeros(S, dk, dv)
    if s["state_in"] is not None:
        h[:n] = s["state_in"].reshape(n, dk, dv)
    if s["dstate"] is not None:
        dh[:] = s["dstate"].reshape(S, dk, dv)
    gk, ek = gam * k, e * k
    Nb, NTb = N * b[..., None, :], N.mT * b[..., None, :]
    H0, W = q.new_empty(S, nc, dk, dv), torch.empty_like(v)
    for c in range(nc):
        H0[:, c] = h
        r = v[:, c] - gk[:, c] @ h
        W[:, c] = r - Nb[:, c] @ r
        h = gend[:, c, None, None] * h + ek[:, c].mT @ (bb[:, c] * W[:, c])
    dU0 = P.mT @ do
    dH1, Z = torch.empty_like(H0), torch.empty_like(v)
    gq = gam * q
    for c in range(nc - 1, -1, -1):
        dH1[:, c] = dh
        du = dU0[:, c] + ek[:, c] @ dh
        z = du - NTb[:, c] @ du
        Z[:, c] = z
        dh = gend[:, c, None, None] * dh + gq[:, c].mT @ do[:, c] - gk[:, c].mT @ (bb[:, c] * z)
    U, Y = bb * W, bb * Z
    dP, dX = (do @ U.mT).tril(), -(Y @ U.mT).tril(-1)
    E, F = dP * D, dX * D
    hdo, hy, du1 = do @ H0.mT, Y @ H0.mT, U @ dH1.mT
    dq = gam * hdo + E @ k
    dkk = (F + F.mT) @ k + E.mT @ q - gam * hy + e * du1
    db = (Z * W).sum(-1)
    # da_t: the sum of every product that holds a_t, over a_t
    M = X.new_zeros(S, nc, C + 1, C + 1, dtype=torch.float64)
    M[..., :C, 1:] = (dX * X + dP * P).tril(-1)
    M[..., :C, 0] = (gam * (q * hdo - k * hy)).sum(-1)
    M[..., C, 1:] = (e * k * du1).sum(-1)
    M[..., C, 0] = gend * (H0 * dH1).sum((-1, -2))
    M = M.cumsum(-1).flip(-2).cumsum(-2).flip(-2)
    da = (M.diagonal(dim1=-2, dim2=-1)[..., :C] / a.double()).float()

    def whole(x, dt):                                             # [dirs*BH, nc, C, ...] -> [B,H,T,...]
        x = x.reshape(S, nc * C, *x.shape[3:])[:, :T]
        x = x[:n] + x[n:].flip(1) if dirs == 2 else x
        return x.reshape(B, H, T, *x.shape[2:]).to(dt)

    dt = s["q"].dtype
    return (whole(dq, dt), whole(dkk, dt), whole(Y, dt), whole(db, torch.float32), whole(da, torch.float32),
            dh[:n].reshape(B, H, dk, dv))


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_gdn(s)


def _exact_rotary(s):
    """y = R x / |x| with R the complex rotation exp(i angle) of each pair; its gradient by the transposed maps."""
    B, H, T, d = s["B"], s["H"], s["T"], s["d"]
    dev = s["q"].device
    if s["positions"] is not None:
        pos = s["positions"].double()
    else:
        n = torch.arange(s["start"], s["start"] + T, device=dev, dtype=torch.int64)
        row = n // s["w"]
        pos = torch.stack([row // s["h"], row % s["h"], n % s["w"]], -1).double().expand(B, T, 3)
    axis = torch.cat([torch.full((m // 2,), i, dtype=torch.int64, device=dev) for i, m in enumerate(s["axes"])])
    freq = torch.cat([torch.exp(-math.log(10000.0) * torch.arange(m // 2, device=dev, dtype=torch.float64) / (m / 2))
                      if m else torch.empty(0, device=dev, dtype=torch.float64) for m in s["axes"]])
    phase = pos[..., axis] * freq
    rot = torch.polar(torch.ones_like(phase), phase)[:, None]

    def turn(x, by):
        pair = x.unflatten(-1, (2, d // 2)).transpose(-1, -2) if s["half"] else x.unflatten(-1, (d // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by)
        return z.transpose(-1, -2).flatten(-2) if s["half"] else z.flatten(-2)

    out = []
    for name in ("q", "k"):
        x = s[name].double()
        size = ((x ** 2).sum(-1, keepdim=True) + 1e-6).sqrt() if s["l2"] else None
        if s["back"]:
            y = turn(s["d" + name].double(), rot.conj())
            if s["l2"]:
                unit = x / size
                y = (y - unit * (unit * y).sum(-1, keepdim=True)) / size
        else:
            y = turn(x / size if s["l2"] else x, rot)
        out.append(y)
    return tuple(out)


def _exact_norm(s):
    B, H, T, d = s["B"], s["H"], s["T"], s["d"]
    o = s["o"].double().transpose(1, 2)
    w = s["weight"].double()
    size = ((o ** 2).sum(-1, keepdim=True) / d + 1e-5).sqrt()
    unit = o / size
    act = torch.ones((), device=o.device, dtype=torch.float64)
    if s["gate"]:
        g = s["gate_t"].double().transpose(1, 2)
        act = g * torch.sigmoid(g)
    if not s["back"]:
        return (unit * w * act).reshape(B, T, H * d)
    dy = s["dy"].double().reshape(B, T, H, d)
    dgate = None
    if s["gate"]:
        p = torch.sigmoid(g)
        dgate = (dy * unit * w * (p + g * p * (1 - p))).transpose(1, 2)
    dw = (dy * act * unit).sum((0, 1) if s["per_head"] else (0, 1, 2))
    du = dy * act * w
    do = (du - unit * (du * unit).sum(-1, keepdim=True) / d) / size
    return do.transpose(1, 2), dgate, dw


def _exact_gdn(s):
    """Token by token: the states forward (kept at every `step`-th token and recomputed from there), then each
    token's gradients backward."""
    B, H, T, dk, dv = s["B"], s["H"], s["T"], s["d"], s["dv"]
    if T > 40000:
        return None
    n, two = B * H, s["bidi"]

    def rows(x):                                                   # [T, S, ...], the reverse scan's tokens in its order
        x = x.double().reshape(n, T, *x.shape[3:])
        return (torch.cat([x, x.flip(1)]) if two else x).transpose(0, 1).contiguous()

    q, k, v, do = (rows(s[x]).unsqueeze(-1) for x in ("q", "k", "v", "do"))
    b, a = rows(s["beta"])[..., None, None], rows(s["decay"])[..., None, None]
    S = q.shape[1]
    h = q.new_zeros(S, dk, dv)
    if s["state_in"] is not None:
        h[:n] = s["state_in"].double().reshape(n, dk, dv)
    g = q.new_zeros(S, dk, dv)
    if s["dstate"] is not None:
        g[:] = s["dstate"].double().reshape(S, dk, dv)
    vt, dot = v.mT.contiguous(), do.mT.contiguous()

    def forward(h, t):                                             # w = v - a H^T k;  H <- a H + k (b w)^T
        w = vt[t] - k[t].mT @ (a[t] * h)
        return torch.baddbmm(a[t] * h, k[t], b[t] * w), w

    step = max(1, math.isqrt(T))
    kept = []
    for t in range(T):
        if t % step == 0:
            kept.append(h)
        h, _ = forward(h, t)
    dq, dkk, dvv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    db, da = q.new_zeros(T, S), q.new_zeros(T, S)
    for block in range(len(kept) - 1, -1, -1):
        first, last = block * step, min(T, block * step + step)
        hs, ws = [kept[block]], []
        for t in range(first, last):
            h, w = forward(hs[-1], t)
            hs.append(h)
            ws.append(w)
        for t in range(last - 1, first - 1, -1):
            old, new, w = hs[t - first], hs[t - first + 1], ws[t - first]
            dq[t] = new @ do[t]
            g = torch.baddbmm(g, q[t], dot[t])                     # dH_t
            du = k[t].mT @ g                                       # u = b w
            db[t] = (du * w).sum((-1, -2))
            dw = b[t] * du
            dvv[t] = dw.mT
            m = old @ dw.mT                                        # through w = v - a H^T k
            dkk[t] = g @ (b[t] * w).mT - a[t] * m
            da[t] = (g * old).sum((-1, -2)) - (m * k[t]).sum((-1, -2))
            g = a[t] * (g - k[t] @ dw)
    def whole(x):
        x = x.transpose(0, 1)
        x = x[:n] + x[n:].flip(1) if two else x
        return x.reshape(B, H, T, *x.shape[2:])

    return (whole(dq[..., 0]), whole(dkk[..., 0]), whole(dvv[..., 0]), whole(db), whole(da), g[:n].reshape(B, H, dk, dv))
