"""The gated linear recurrence and the per-head q/k norm with rotation, measured.

The recurrence keeps a Dk x Dv state per head, S_t = alpha_t S_{t-1} + k_t^T v_t, and
reads o_t = q_t S_t; it is measured forward, backward and one token at a time.  The
q/k operator normalises every head's query and key row, rotates it by its position and
lays (B, T, H, D) slices of a fused projection out as the (B, H, T, D) the recurrence
takes; it is measured forward and backward.

``run`` computes the plain forms in float32 (decays and angles in float64) where ``own``
is false and calls the library where it is true.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = {"rms": 1e-6, "l2": 1e-12}


def listed():
    return [
        # the prefill size of this repository's benchmark
        _rec("fwd prefill", "rec_fwd", 4, 16, 4096, 128, 128, "bf16"),
        # the largest: the forgetting benchmark's size
        _rec("fwd large batch", "rec_fwd", 8, 16, 8192, 128, 128, "bf16"),
        # one long document over few heads
        _rec("fwd long", "rec_fwd", 1, 8, 65536, 128, 128, "bf16", state=True),
        # odd sizes, unequal widths, continued from a cached state
        _rec("fwd ragged", "rec_fwd", 3, 5, 1000, 64, 128, "bf16", state=True),
        # the tiny float32 configuration
        _rec("fwd tiny f32", "rec_fwd", 1, 2, 256, 64, 64, "f32"),
        # a training step of the prefill size
        _rec("bwd train", "rec_bwd", 4, 16, 4096, 128, 128, "bf16"),
        # float32 training at odd sizes, through the state
        _rec("bwd ragged f32", "rec_bwd", 2, 3, 777, 128, 64, "f32", state=True),
        # batched decode of this repository's benchmark, and a single sequence
        dict(name="step batch", op="step", B=256, H=32, Dk=128, Dv=128, dtype="bf16"),
        dict(name="step single", op="step", B=1, H=16, Dk=128, Dv=128, dtype="bf16"),
        # the layer's q and k ahead of the recurrence: prefill, one decoded token, training
        _qk("qk fwd prefill", "qk_fwd", 4, 4096, 16, 16, 128, 128, "rms", "bf16"),
        _qk("qk fwd token", "qk_fwd", 64, 1, 32, 32, 128, 64, "l2", "bf16", silu=True, far=True),
        _qk("qk bwd train", "qk_bwd", 4, 4096, 16, 16, 128, 128, "rms", "bf16"),
    ]


def _rec(name, op, B, H, T, Dk, Dv, dtype, gated=True, state=False):
    return dict(name=name, op=op, B=B, H=H, T=T, Dk=Dk, Dv=Dv, dtype=dtype, gated=gated, state=state)


def _qk(name, op, B, T, Hq, Hk, D, rot, norm, dtype, silu=False, interleaved=False, far=False):
    return dict(name=name, op=op, B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, norm=norm, dtype=dtype, silu=silu,
                interleaved=interleaved, far=far)


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["rec_fwd", "rec_fwd", "rec_bwd", "rec_bwd", "step", "qk_fwd", "qk_bwd"])
    f32 = rng.random() < 0.25
    if op == "step":
        return dict(op=op, B=_log(rng, 1, 256), H=rng.randint(1, 32), Dk=rng.choice([64, 128]),
                    Dv=rng.choice([64, 128]), dtype="f32" if f32 else "bf16")
    B, H = _log(rng, 1, 8), rng.randint(1, 32)
    if op.startswith("rec"):
        rows = 8192 if f32 else 1048576 if op == "rec_fwd" else 262144
        T = _log(rng, 1, max(1, min(65536, rows // (B * H))))
        return dict(op=op, B=B, H=H, T=T, Dk=rng.choice([64, 128]), Dv=rng.choice([64, 128]),
                    dtype="f32" if f32 else "bf16", gated=rng.random() < 0.8, state=rng.random() < 0.5)
    Hk = rng.randint(1, 32)
    D = rng.choice([64, 128])
    return dict(op=op, B=B, T=_log(rng, 1, max(1, min(65536, 524288 // (B * (H + Hk))))), Hq=H, Hk=Hk, D=D,
                rot=rng.choice([0, 16, 32, D]), norm=rng.choice(["rms", "l2"]), dtype="f32" if f32 else "bf16",
                silu=rng.random() < 0.4, interleaved=rng.random() < 0.4, far=rng.random() < 0.3)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dt = case, DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case)
    if c["op"].startswith("qk"):
        B, T, Hq, Hk, D = c["B"], c["T"], c["Hq"], c["Hk"], c["D"]
        # one fused projection holds q, k and a value part of one key width
        fused = normal(B, T, (Hq + 2 * Hk) * D).to(dt)
        s["q"] = fused[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = fused[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        s["wq"], s["wk"] = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        start = torch.randint(0, 1 << 20 if c["far"] else 2048, (B, 1), generator=g, device="cuda")
        s["pos"] = start + torch.arange(T, device="cuda")
        half = c["rot"] // 2
        s["freq"] = (10000.0 ** (-torch.arange(half, device="cuda") / half)).float() if half else None
        if c["op"] == "qk_bwd":
            s["dq"], s["dk"] = normal(B, Hq, T, D).to(dt), normal(B, Hk, T, D).to(dt)
        return s
    B, H, Dk, Dv = c["B"], c["H"], c["Dk"], c["Dv"]
    lead = (B, H) if c["op"] == "step" else (B, H, c["T"])
    s["q"] = normal(*lead, Dk).to(dt)
    k = normal(*lead, Dk)
    s["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).to(dt)
    s["v"] = normal(*lead, Dv).to(dt)
    s["alpha"] = s["S0"] = None
    if c.get("gated", True):
        # every head has its own memory, from about one token to a few thousand
        rate = 2.0 ** (-12.0 * torch.rand(H, generator=g, device="cuda"))
        rate = rate.view(1, H, *[1] * (len(lead) - 2))
        s["alpha"] = torch.exp(-rate * torch.log1p(torch.exp(normal(*lead))))
    if c["op"] == "step" or c["state"]:
        s["S0"] = normal(B, H, Dk, Dv)
    if c["op"] == "rec_bwd":
        s["dO"] = normal(*lead, Dv).to(dt)
        s["dST"] = normal(B, H, Dk, Dv) if c["state"] else None
    return s


def run(s):
    op = s["op"]
    if own:
        import deltanet_sequence_mixing_b200 as dn

        if op == "rec_fwd":
            return dn.gated_linear_attn_fwd(s["q"], s["k"], s["v"], s["alpha"], s["S0"])
        if op == "rec_bwd":
            return dn.gated_linear_attn_bwd(s["q"], s["k"], s["v"], s["dO"], s["alpha"], s["S0"], s["dST"])
        if op == "step":
            return dn.gated_linear_attn_decode_step(s["q"], s["k"], s["v"], s["S0"], s["alpha"]), s["S0"]
        how = dict(positions=s["pos"], inv_freq=s["freq"], norm=s["norm"], eps=EPS[s["norm"]], silu=s["silu"],
                   interleaved=s["interleaved"])
        if op == "qk_fwd":
            return dn.qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], **how)
        return dn.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], **how)
    if op == "rec_fwd":
        return _plain_fwd(s)
    if op == "rec_bwd":
        return _plain_bwd(s)
    if op == "step":
        return _plain_step(s)
    return _plain_qk_fwd(s) if op == "qk_fwd" else _plain_qk_bwd(s)


# ---------------------------------------------------------------- plain: recurrence --
CHUNK = 64


def _chunks(x, nc):
    """(B, H, T, ...) as (B*H, chunks, CHUNK, ...) in float32, zeros behind the end."""
    x = x.float().flatten(0, 1)
    pad = nc * CHUNK - x.shape[1]
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    return x.unflatten(1, (nc, CHUNK))


def _decays(s, N, nc):
    """Decays between tokens of a chunk (D), from its start (into) and to its end (out), and
    between chunks (enter[c, c'] from the end of c' to the start of c, first[c] from the start)."""
    T, dev = s["q"].shape[2], s["q"].device
    la = torch.zeros(N, nc * CHUNK, dtype=torch.float64, device=dev)
    if s["alpha"] is not None:
        la[:, :T] = s["alpha"].double().clamp_min(1e-300).log().flatten(0, 1)
    la = la.view(N, nc, CHUNK)
    g = la.cumsum(-1)
    gc = g[..., -1].cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    D = ((g[..., :, None] - g[..., None, :]).masked_fill(~low, -math.inf)).exp().float()
    before = gc - g[..., -1]
    lowc = torch.ones(nc, nc, dtype=torch.bool, device=dev).tril(-1)
    enter = (before[:, :, None] - gc[:, None, :]).masked_fill(~lowc, -math.inf).exp().float()
    return D, g.exp().float(), (g[..., -1:] - g).exp().float(), enter, before.exp().float(), gc


def _states(s, k, v, out, enter, first):
    """States entering every chunk, (N, chunks, Dk, Dv)."""
    dS = (k * out[..., None]).transpose(-1, -2) @ v
    S = (enter @ dS.flatten(2)).view_as(dS)
    if s["S0"] is not None:
        S = S + first[..., None, None] * s["S0"].flatten(0, 1)[:, None]
    return S, dS


def _plain_fwd(s):
    B, H, T, Dk = s["q"].shape
    N, nc = B * H, -(-T // CHUNK)
    q, k, v = (_chunks(s[n], nc) for n in "qkv")
    D, into, out, enter, first, gc = _decays(s, N, nc)
    S, dS = _states(s, k, v, out, enter, first)
    o = ((q @ k.transpose(-1, -2)) * D) @ v + into[..., None] * (q @ S)
    o = o.flatten(1, 2)[:, :T].reshape(B, H, T, -1).to(s["q"].dtype)
    last = S[:, -1] * into[:, -1, -1, None, None] + dS[:, -1]
    return o, last.view(B, H, Dk, -1)


def _plain_bwd(s):
    B, H, T, Dk = s["q"].shape
    N, nc = B * H, -(-T // CHUNK)
    q, k, v, dO = (_chunks(s[n], nc) for n in ("q", "k", "v", "dO"))
    D, into, out, enter, first, gc = _decays(s, N, nc)
    S, _ = _states(s, k, v, out, enter, first)
    dR = (q * into[..., None]).transpose(-1, -2) @ dO
    R = (enter.transpose(-1, -2) @ dR.flatten(2)).view_as(dR)  # adjoint of the state leaving each chunk
    if s["dST"] is not None:
        R = R + (gc[:, -1:] - gc).exp().float()[..., None, None] * s["dST"].flatten(0, 1)[:, None]
    qk, ov = q @ k.transpose(-1, -2), dO @ v.transpose(-1, -2)
    a, b = qk * D, ov * D
    dq_in = into[..., None] * (dO @ S.transpose(-1, -2))
    dk_out = out[..., None] * (v @ R.transpose(-1, -2))
    dq = b @ k + dq_in
    dk = b.transpose(-1, -2) @ q + dk_out
    dv = a.transpose(-1, -2) @ dO + out[..., None] * (k @ R)
    got = {}
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        got[n] = x.flatten(1, 2)[:, :T].reshape(B, H, T, -1).to(s["q"].dtype)
    got["dS0"] = (R[:, 0] * into[:, 0, -1, None, None] + dR[:, 0]).view(B, H, Dk, -1)
    got["dlog_alpha"] = None
    if s["alpha"] is not None:
        m = (qk * b).double().tril(-1)
        r, e = (q * dq_in).double().sum(-1), (k * dk_out).double().sum(-1)
        x = m.sum(-1) - m.sum(-2) + r
        through = into[..., -1].double() * (S.double() * R.double()).sum((-1, -2))
        dla = x.flip(-1).cumsum(-1).flip(-1) + e.cumsum(-1) - e + through[..., None]
        got["dlog_alpha"] = dla.flatten(1, 2)[:, :T].reshape(B, H, T).float()
    return got


def _plain_step(s):
    S = s["S0"]
    S.copy_(S * s["alpha"][..., None, None] + s["k"].float()[..., :, None] * s["v"].float()[..., None, :])
    o = (s["q"].float()[..., None, :] @ S)[..., 0, :]
    return o.to(s["q"].dtype), S


# ---------------------------------------------------------------------- plain: q and k --
def _turn(x, s, way):
    """Rotates the first `rot` columns of (B, T, H, D) by the rows' positions (way -1: back)."""
    half = s["rot"] // 2
    if not half:
        return x
    a = s["pos"].double()[..., None] * s["freq"].double()
    cos, sin = a.cos().float()[:, :, None], way * a.sin().float()[:, :, None]
    if s["interleaved"]:
        x0, x1 = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    else:
        x0, x1 = x[..., :half], x[..., half:2 * half]
        y = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _scale(x, s):
    """One over each row's norm."""
    if s["norm"] == "rms":
        return 1 / (x.square().mean(-1, keepdim=True) + EPS["rms"]).sqrt()
    return 1 / x.square().sum(-1, keepdim=True).sqrt().clamp_min(EPS["l2"])


def _plain_qk_fwd(s):
    got = []
    for n in "qk":
        x = s[n].float()
        if s["silu"]:
            x = x / (1 + (-x).exp())
        y = _turn(x * _scale(x, s) * s["w" + n], s, 1)
        got.append(y.to(s[n].dtype).transpose(1, 2).contiguous())
    return tuple(got)


def _plain_qk_bwd(s):
    got = {}
    for n in "qk":
        raw = s[n].float()
        sig = 1 / (1 + (-raw).exp())
        x = raw * sig if s["silu"] else raw
        r = _scale(x, s)
        d = _turn(s["d" + n].float().transpose(1, 2), s, -1)
        got["d%s_weight" % n] = (d * x * r).double().sum((0, 1, 2)).float()
        d = d * s["w" + n]
        width = x.shape[-1] if s["norm"] == "rms" else 1
        dx = r * (d - x * r * ((d * x * r).sum(-1, keepdim=True) / width))
        if s["silu"]:
            dx = dx * sig * (1 + raw * (1 - sig))
        got["d" + n] = dx.to(s[n].dtype)
    return got


# --------------------------------------------------------------------------- exact --
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rec_fwd":
        return _exact_fwd(s)
    if case["op"] == "rec_bwd":
        return _exact_bwd(s)
    if case["op"] == "step":
        o, S = _exact_fwd({**s, **{n: s[n][:, :, None] for n in ("q", "k", "v", "alpha")}})
        return o[:, :, 0], S
    return _exact_qk(s)


def _time_major(s, names):
    return [None if s[n] is None else s[n].double().flatten(0, 1).transpose(0, 1).contiguous() for n in names]


def _exact_fwd(s):
    """Token by token, from the definition."""
    B, H, T, Dk = s["q"].shape
    q, k, v, al = _time_major(s, ("q", "k", "v", "alpha"))
    S = q.new_zeros(B * H, Dk, v.shape[-1])
    if s["S0"] is not None:
        S += s["S0"].flatten(0, 1)
    o = torch.empty_like(v)
    for t in range(T):
        if al is not None:
            S *= al[t][:, None, None]
        S.baddbmm_(k[t][:, :, None], v[t][:, None, :])
        torch.bmm(q[t][:, None, :], S, out=o[t][:, None, :])
    return o.transpose(0, 1).reshape(B, H, T, -1), S.view(B, H, Dk, -1)


def _exact_bwd(s):
    """The reverse sweep token by token, states recomputed in stretches of 64."""
    B, H, T, Dk = s["q"].shape
    N = B * H
    q, k, v, dO, al = _time_major(s, ("q", "k", "v", "dO", "alpha"))
    Dv = v.shape[-1]

    def forward(S, t):
        S = S if al is None else S * al[t][:, None, None]
        return torch.baddbmm(S, k[t][:, :, None], v[t][:, None, :])

    S = q.new_zeros(N, Dk, Dv)
    if s["S0"] is not None:
        S += s["S0"].flatten(0, 1)
    marks = []
    for t in range(T):
        if t % 64 == 0:
            marks.append(S)
        S = forward(S, t)
    R = q.new_zeros(N, Dk, Dv)
    if s["dST"] is not None:
        R += s["dST"].flatten(0, 1)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dla = None if al is None else torch.empty_like(al)
    for m in reversed(range(len(marks))):
        stretch = [marks[m]]
        for t in range(64 * m, min(T, 64 * m + 64)):
            stretch.append(forward(stretch[-1], t))
        for t in reversed(range(64 * m, min(T, 64 * m + 64))):
            before, after = stretch[t - 64 * m], stretch[t - 64 * m + 1]
            dq[t] = torch.bmm(after, dO[t][:, :, None])[..., 0]
            R = torch.baddbmm(R, q[t][:, :, None], dO[t][:, None, :])
            dk[t] = torch.bmm(R, v[t][:, :, None])[..., 0]
            dv[t] = torch.bmm(k[t][:, None, :], R)[:, 0]
            if al is not None:
                R = R * al[t][:, None, None]
                dla[t] = (R * before).sum((1, 2))

    def back(x):
        return None if x is None else x.transpose(0, 1).reshape(B, H, T, *x.shape[2:])

    return {"dq": back(dq), "dk": back(dk), "dv": back(dv), "dlog_alpha": back(dla), "dS0": R.view(B, H, Dk, Dv)}


def _exact_qk(s):
    """Pairs as complex numbers; the gradients by differentiating the definition."""
    got, grads, half = [], {}, s["rot"] // 2
    for n in "qk":
        x = s[n].double().clone().requires_grad_()
        w = s["w" + n].double().clone().requires_grad_()
        y = x * torch.sigmoid(x) if s["silu"] else x
        if s["norm"] == "rms":
            y = y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + EPS["rms"]) * w
        else:
            y = y / y.pow(2).sum(-1, keepdim=True).sqrt().clamp_min(EPS["l2"]) * w
        if half:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                               s["pos"].double()[:, :, None, None] * s["freq"].double())
            p = y[..., :2 * half]
            p = p.unflatten(-1, (half, 2)) if s["interleaved"] else p.unflatten(-1, (2, half)).transpose(-1, -2)
            p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * turn)
            p = p.flatten(-2) if s["interleaved"] else p.transpose(-1, -2).flatten(-2)
            y = torch.cat([p, y[..., 2 * half:]], -1)
        y = y.transpose(1, 2)
        if s["op"] == "qk_fwd":
            got.append(y.detach())
        else:
            grads["d" + n], grads["d%s_weight" % n] = torch.autograd.grad(y, [x, w], s["d" + n].double())
    return tuple(got) if s["op"] == "qk_fwd" else grads


# ---------------------------------------------------------------------------- work --
def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"].startswith("qk"):
        rows = c["B"] * c["T"] * (c["Hq"] + c["Hk"])
        side = 8 * c["B"] * c["T"] + 2 * c["rot"] + 8 * c["D"]
        if c["op"] == "qk_fwd":
            return {"bytes": 2 * rows * c["D"] * e + side, "flops": 8 * rows * c["D"]}
        return {"bytes": 3 * rows * c["D"] * e + side + 8 * c["D"], "flops": 20 * rows * c["D"]}
    Dk, Dv, heads = c["Dk"], c["Dv"], c["B"] * c["H"]
    state = heads * Dk * Dv * 4
    if c["op"] == "step":
        return {"bytes": 2 * state + heads * ((2 * Dk + 2 * Dv) * e + 4), "flops": 5 * heads * Dk * Dv}
    n = heads * c["T"]
    gate = 4 * n if c["gated"] else 0
    if c["op"] == "rec_fwd":  # the recurrence itself: one write and one read of the state for each token
        return {"bytes": n * (2 * Dk + 2 * Dv) * e + gate + (2 if c["state"] else 1) * state,
                "flops": 4 * n * Dk * Dv}
    return {"bytes": n * (4 * Dk + 3 * Dv) * e + 2 * gate + (3 if c["state"] else 1) * state,
            "flops": 10 * n * Dk * Dv}
