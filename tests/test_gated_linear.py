"""The gated linear recurrence: forward, gradient and single-token step against
the recurrence written out token by token in float64.

Tolerances (2-norm of the difference over the 2-norm of the result, per output):
* float32 outputs of float32 inputs: each value is a chain of at most 128 + 32
  fused multiply-adds per chunk and one decay per chunk, each within 2^-24; the
  errors of a chain of 160 + 10 steps sum to at most 170 * 2^-24 = 1.0e-5 of the
  sum of magnitudes, which random signs keep within about twice the result: 2e-5.
* float32 states and gate gradients of bfloat16 inputs: an operand that carries
  a decay, or a state that enters a product, is split into two bfloat16 values,
  which leaves at most 2^-8 * 2^-8 = 2^-16 = 1.5e-5 of it behind, and about a
  third of that in the 2-norm; with the float32 sums above: 2e-5.
* bfloat16 outputs: the result's own rounding, and one rounding each of the
  decayed scores and of the state they are added to; three roundings of at most
  2^-8, in the 2-norm of many values at most sqrt(3) * 2^-8 = 6.8e-3.
"""
import ctypes

import pytest
import torch

TOL = {torch.float32: 2e-5, torch.bfloat16: 6.8e-3}


def rel(x, ref):
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert x.shape == ref.shape
    return float((x - ref).norm() / ref.norm().clamp_min(1e-300))


def plain(q, k, v, alpha=None, S0=None):
    """The recurrence token by token, in float64 (differentiable)."""
    q, k, v = q.double(), k.double(), v.double()
    S = q.new_zeros(*q.shape[:2], q.shape[-1], v.shape[-1]) if S0 is None else S0.double()
    o = []
    for t in range(q.shape[2]):
        if alpha is not None:
            S = S * alpha[:, :, t, None, None].double()
        S = S + k[:, :, t, :, None] * v[:, :, t, None, :]
        o.append((q[:, :, t, :, None] * S).sum(-2))
    return torch.stack(o, 2) if o else torch.zeros_like(v), S


def plain_grads(q, k, v, dO, alpha=None, S0=None, dS_T=None):
    leaves = {"dq": q, "dk": k, "dv": v}
    if alpha is not None:
        leaves["dlog_alpha"] = alpha
    leaves["dS0"] = S0 if S0 is not None else q.new_zeros(*q.shape[:2], q.shape[-1], v.shape[-1])
    x = {n: t.double().clone().requires_grad_() for n, t in leaves.items()}
    o, S = plain(x["dq"], x["dk"], x["dv"], x.get("dlog_alpha"), x["dS0"])
    loss = (o * dO.double()).sum()
    if dS_T is not None:
        loss = loss + (S * dS_T.double()).sum()
    got = dict(zip(x, torch.autograd.grad(loss, list(x.values()))))
    if alpha is not None:
        got["dlog_alpha"] = got["dlog_alpha"] * alpha.double()
    return got


def case(B, H, T, Dk, Dv, dtype, gate="mixed", state=True, seed=0, device="cuda"):
    """Inputs; gate: None, "mixed" (memories of one token to thousands, by head),
    "wipes" (runs of exact ones with exact zeros in between)."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    k = n(B, H, T, Dk)
    x = dict(q=n(B, H, T, Dk).to(dtype), k=(k / k.norm(dim=-1, keepdim=True)).to(dtype), v=n(B, H, T, Dv).to(dtype))
    alpha = None
    if gate:
        rate = 2.0 ** (-12 * torch.rand(1, H, 1, generator=g))
        alpha = torch.exp(-rate * torch.nn.functional.softplus(n(B, H, T)))
    if gate == "wipes":
        u = torch.rand(B, H, T, generator=g)
        alpha = torch.where(u < 0.5, torch.ones(()), alpha)
        alpha = torch.where(u > 0.96, torch.zeros(()), alpha)
    x["alpha"] = alpha
    x["S0"] = n(B, H, Dk, Dv) if state else None
    x["dO"] = n(B, H, T, Dv).to(dtype)
    x["dS_T"] = n(B, H, Dk, Dv) if state else None
    return {m: None if t is None else t.to(device) for m, t in x.items()}


FWD = ("q", "k", "v", "alpha", "S0")
BWD = ("q", "k", "v", "dO", "alpha", "S0", "dS_T")
pick = lambda x, names: [x[n] for n in names]


def check_fwd(dn, x, dtype):
    o, S = dn.gated_linear_attn_fwd(*pick(x, FWD))
    assert o.dtype == dtype and S.dtype == torch.float32
    ro, rS = plain(*pick(x, FWD))
    assert rel(o, ro) <= TOL[dtype]
    assert rel(S, rS) <= TOL[torch.float32]
    return o, S


def check_bwd(dn, x, dtype):
    got, want = dn.gated_linear_attn_bwd(*pick(x, BWD)), plain_grads(*pick(x, BWD))
    assert (got["dlog_alpha"] is None) == (x["alpha"] is None)
    errs = {n: (rel(got[n], want[n]), TOL[got[n].dtype]) for n in want}
    for n in ("dq", "dk", "dv"):
        assert got[n].dtype == dtype
    assert all(e <= t for e, t in errs.values()), errs
    return got


@pytest.fixture(scope="module")
def dn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deltanet_sequence_mixing_b200 as m

    m.lib()
    return m


# ----------------------------------------------------------------- on the CPU --
def test_plain_gradients_against_differences():
    """The reference's own gradients, against central differences in float64."""
    x = case(1, 2, 9, 3, 4, torch.float64, "mixed", True, 1, "cpu")
    x["alpha"] = x["alpha"].double().clamp(0.2, 0.9)
    want = plain_grads(*pick(x, BWD))

    def loss(**new):
        o, S = plain(*pick({**x, **new}, FWD))
        return float((o * x["dO"]).sum() + (S * x["dS_T"].double()).sum())

    g = torch.Generator().manual_seed(2)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("alpha", "dlog_alpha"), ("S0", "dS0")):
        u = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        h = 1e-6
        step = x["alpha"] * u if n == "alpha" else u  # the gradient by log alpha
        diff = (loss(**{n: x[n] + h * step}) - loss(**{n: x[n] - h * step})) / (2 * h)
        assert abs(diff - float((want[d] * u).sum())) <= 1e-7 * max(1.0, abs(diff)), n


A, MB = 1 << 32, 1 << 20  # device addresses that nothing reads: the calls are refused on the host
vp = lambda x: None if x is None else ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def L():
    from deltanet_sequence_mixing_b200 import _lib
    from deltanet_sequence_mixing_b200.build import build

    build()
    return _lib.lib()


def test_fwd_refusals(L):
    from deltanet_sequence_mixing_b200 import _lib as E

    def call(q=A, k=A + 64 * MB, v=A + 128 * MB, alpha=A + 192 * MB, S0=None, o=A + 256 * MB, S_out=A + 320 * MB,
             B=2, H=2, T=100, Dk=64, Dv=64, dt=1, ws=A + 400 * MB, nb=1 << 20):
        return L.gated_linear_attn_fwd(vp(q), vp(k), vp(v), vp(alpha), vp(S0), vp(o), vp(S_out), B, H, T, Dk, Dv, dt,
                                       vp(ws), nb, None)

    for n in ("q", "k", "v", "o"):
        assert call(**{n: None}) == E.DN_ERR_INVALID_ARG
    for n in ("B", "H", "T"):
        assert call(**{n: -1}) == E.DN_ERR_INVALID_ARG
    for n in ("Dk", "Dv"):
        assert call(**{n: 96}) == E.DN_ERR_UNSUPPORTED
    assert call(dt=5) == E.DN_ERR_UNSUPPORTED
    assert call(B=1 << 16, H=1 << 16) == E.DN_ERR_UNSUPPORTED
    assert call(ws=None) == E.DN_ERR_WORKSPACE
    assert call(nb=16) == E.DN_ERR_WORKSPACE
    for n, at in (("q", A + 8), ("o", A + 256 * MB + 2), ("S0", A + 500 * MB + 4), ("alpha", A + 192 * MB + 2),
                  ("ws", A + 400 * MB + 8)):
        assert call(**{n: at}) == E.DN_ERR_ALIGNMENT
    assert call(o=A + 64) == E.DN_ERR_INVALID_ARG  # o inside q
    assert call(S_out=A + 256 * MB) == E.DN_ERR_INVALID_ARG  # S_out on o
    assert call(S0=A + 320 * MB + 64) == E.DN_ERR_INVALID_ARG  # S_out partly on S0
    assert call(ws=A + 128 * MB) == E.DN_ERR_INVALID_ARG  # workspace on v


def test_bwd_refusals(L):
    from deltanet_sequence_mixing_b200 import _lib as E

    def call(q=A, k=A + 32 * MB, v=A + 64 * MB, alpha=A + 96 * MB, S0=None, dO=A + 128 * MB, dS_T=None,
             dq=A + 160 * MB, dk=A + 192 * MB, dv=A + 224 * MB, dla=A + 256 * MB, dS0=A + 288 * MB, B=2, H=2, T=100,
             Dk=64, Dv=64, dt=1, ws=A + 512 * MB, nb=None):
        if nb is None:
            nb = max(256, L.gated_linear_attn_bwd_workspace_bytes(2, 2, 100, 64, 64, 1))
        return L.gated_linear_attn_bwd(vp(q), vp(k), vp(v), vp(alpha), vp(S0), vp(dO), vp(dS_T), vp(dq), vp(dk),
                                       vp(dv), vp(dla), vp(dS0), B, H, T, Dk, Dv, dt, vp(ws), nb, None)

    for n in ("q", "k", "v", "dO", "dq", "dk", "dv"):
        assert call(**{n: None}) == E.DN_ERR_INVALID_ARG
    assert call(alpha=None) == E.DN_ERR_INVALID_ARG  # a gate gradient without a gate
    assert call(T=-1) == E.DN_ERR_INVALID_ARG
    assert call(Dk=32) == E.DN_ERR_UNSUPPORTED
    assert call(dt=2) == E.DN_ERR_UNSUPPORTED
    assert call(ws=None) == E.DN_ERR_WORKSPACE
    assert call(nb=1024) == E.DN_ERR_WORKSPACE
    assert call(dq=A + 160 * MB + 8) == E.DN_ERR_ALIGNMENT
    assert call(dla=A + 256 * MB + 2) == E.DN_ERR_ALIGNMENT
    assert call(dk=A + 160 * MB) == E.DN_ERR_INVALID_ARG  # dk on dq
    assert call(dv=A + 128 * MB) == E.DN_ERR_INVALID_ARG  # dv on dO
    assert call(dS0=A + 288 * MB, dS_T=A + 288 * MB) == E.DN_ERR_INVALID_ARG


def test_step_refusals(L):
    from deltanet_sequence_mixing_b200 import _lib as E

    def call(q=A, k=A + MB, v=A + 2 * MB, alpha=A + 3 * MB, S=A + 8 * MB, o=A + 4 * MB, B=2, H=2, Dk=64, Dv=64, dt=1):
        return L.gated_linear_attn_decode_step(vp(q), vp(k), vp(v), vp(alpha), vp(S), vp(o), B, H, Dk, Dv, dt, None)

    for n in ("q", "k", "v", "S", "o"):
        assert call(**{n: None}) == E.DN_ERR_INVALID_ARG
    assert call(B=-1) == E.DN_ERR_INVALID_ARG
    assert call(Dv=48) == E.DN_ERR_UNSUPPORTED
    assert call(dt=3) == E.DN_ERR_UNSUPPORTED
    assert call(S=A + 8 * MB + 4) == E.DN_ERR_ALIGNMENT
    assert call(o=A + 8 * MB) == E.DN_ERR_INVALID_ARG  # o on S
    assert call(S=A) == E.DN_ERR_INVALID_ARG  # S on q
    assert call(B=0, q=None, k=None, v=None, S=None, o=None) == E.DN_OK


def test_workspace_sizes(L):
    for fn in (L.gated_linear_attn_workspace_bytes, L.gated_linear_attn_bwd_workspace_bytes):
        for dt in (0, 1):
            assert fn(2, 3, 100, 64, 128, dt) >= 256
            assert fn(0, 3, 0, 64, 128, dt) >= 256
        assert fn(2, 3, 100, 96, 128, 1) == 0
        assert fn(2, 3, 100, 64, 128, 9) == 0
        assert fn(2, -3, 100, 64, 128, 1) == 0


def test_binding_refuses_host_tensors():
    import deltanet_sequence_mixing_b200 as m

    x = case(1, 1, 4, 64, 64, torch.float32, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        m.gated_linear_attn_fwd(*pick(x, FWD))
    with pytest.raises(ValueError, match="CUDA"):
        m.gated_linear_attn_bwd(*pick(x, BWD))


# ----------------------------------------------------------------- on the GPU --
gpu = pytest.mark.gpu
DIMS = [(64, 64), (128, 128), (128, 64), (64, 128)]
LENGTHS = [1, 2, 31, 33, 64, 127, 128, 129, 300]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("T", LENGTHS)
def test_forward(dn, dtype, Dk, Dv, T):
    check_fwd(dn, case(2, 3, T, Dk, Dv, dtype, "mixed", T % 2 == 0, T + Dk + Dv), dtype)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [None, "wipes"])
@pytest.mark.parametrize("state", [False, True])
def test_forward_gates(dn, dtype, gate, state):
    check_fwd(dn, case(2, 4, 290, 128, 128, dtype, gate, state, 5), dtype)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("T", LENGTHS)
def test_backward(dn, dtype, Dk, Dv, T):
    check_bwd(dn, case(2, 3, T, Dk, Dv, dtype, "mixed", T % 2 == 1, T + Dk + Dv + 1), dtype)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", [None, "wipes"])
@pytest.mark.parametrize("state", [False, True])
def test_backward_gates(dn, dtype, gate, state):
    got = check_bwd(dn, case(2, 4, 290, 128, 128, dtype, gate, state, 6), dtype)
    if gate:
        assert bool((got["dlog_alpha"] == got["dlog_alpha"]).all())


@gpu
def test_gradient_against_differences(dn):
    """The kernel's gradient along random directions against central
    differences of the float64 recurrence."""
    x = case(1, 2, 140, 64, 64, torch.float32, "mixed", True, 7)
    got = dn.gated_linear_attn_bwd(*pick(x, BWD))
    x = {n: t.double() for n, t in x.items()}

    def loss(**new):
        o, S = plain(*pick({**x, **new}, FWD))
        return float((o * x["dO"]).sum() + (S * x["dS_T"]).sum())

    g = torch.Generator(device="cuda").manual_seed(8)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("alpha", "dlog_alpha"), ("S0", "dS0")):
        u = torch.randn(x[n].shape, generator=g, dtype=torch.float64, device="cuda")
        h = 1e-5
        step = x["alpha"] * u if n == "alpha" else u
        diff = (loss(**{n: x[n] + h * step}) - loss(**{n: x[n] - h * step})) / (2 * h)
        # the projection of an error of 2e-5 of the gradient's norm on a random direction, three deviations
        assert abs(diff - float((got[d].double() * u).sum())) <= 3 * 2e-5 * float(got[d].double().norm()) + 1e-6


@gpu
@pytest.mark.parametrize("B,H,T", [(1, 1, 5000), (1, 3, 2049), (2, 1, 8192)])
def test_long_sequences(dn, B, H, T):
    """Few heads, long sequences: the segments run side by side and meet."""
    x = case(B, H, T, 128, 128, torch.bfloat16, "mixed", True, T)
    check_fwd(dn, x, torch.bfloat16)
    check_bwd(dn, x, torch.bfloat16)


@gpu
@pytest.mark.parametrize("gate", [None, "wipes"])
@pytest.mark.parametrize("B,H,T,Dk,Dv", [(1, 1, 4100, 64, 128), (1, 2, 1500, 128, 64), (3, 3, 6000, 64, 64)])
def test_segments_enter_in_place(dn, gate, B, H, T, Dk, Dv):
    """Long sequences over few heads, whose parts start from the states of the
    parts before them, with S_out on S0."""
    x = case(B, H, T, Dk, Dv, torch.bfloat16, gate, seed=T)
    o, S = check_fwd(dn, x, torch.bfloat16)
    check_bwd(dn, x, torch.bfloat16)
    S0 = x["S0"].clone()
    o2, S2 = dn.gated_linear_attn_fwd(*pick(x, FWD[:4]), S0, S_out=S0)
    assert S2 is S0 and torch.equal(o, o2) and torch.equal(S, S2)


@gpu
def test_many_heads(dn):
    x = case(8, 40, 150, 64, 64, torch.bfloat16, "mixed", True, 9)
    check_fwd(dn, x, torch.bfloat16)
    check_bwd(dn, x, torch.bfloat16)


@gpu
@pytest.mark.parametrize("Dk,Dv", DIMS)
def test_many_heads_float32(dn, Dk, Dv):
    """Heads that fill the GPU several times: each walks its chunks, S_out on S0."""
    x = case(8, 40, 77, Dk, Dv, torch.float32, "wipes", True, 10)
    o, S = check_fwd(dn, x, torch.float32)
    S0 = x["S0"].clone()
    o2, S2 = dn.gated_linear_attn_fwd(*pick(x, FWD[:4]), S0, S_out=S0)
    assert torch.equal(o, o2) and torch.equal(S, S2)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("Dk,Dv", DIMS)
@pytest.mark.parametrize("B,H,gated", [(1, 1, True), (3, 5, False), (16, 33, True)])
def test_step(dn, dtype, Dk, Dv, B, H, gated):
    x = case(B, H, 1, Dk, Dv, dtype, "mixed" if gated else None, True, B + H)
    S = x["S0"].clone()
    al = x["alpha"][:, :, 0].contiguous() if gated else None
    o = dn.gated_linear_attn_decode_step(*(x[n][:, :, 0].contiguous() for n in "qkv"), S, al)
    ro, rS = plain(*pick(x, FWD))
    # o of the step reads the float32 state: one rounding
    assert rel(o, ro[:, :, 0]) <= (2.0 ** -8 if dtype == torch.bfloat16 else TOL[dtype])
    assert rel(S, rS) <= 3 * 2.0 ** -24


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_then_steps_and_continued_prefill(dn, dtype):
    """A prompt, then tokens one at a time, then a second prompt into the same
    state, against one run over all of it."""
    x = case(2, 3, 200, 128, 64, dtype, "wipes", True, 10)
    ro, rS = plain(*pick(x, FWD))
    part = lambda a, b: [x[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "alpha")]
    S = x["S0"].clone()
    o1, _ = dn.gated_linear_attn_fwd(*part(0, 77), S, S_out=S)  # in place
    outs = [o1]
    for t in range(77, 82):
        q, k, v, al = (y[:, :, 0].contiguous() for y in part(t, t + 1))
        outs.append(dn.gated_linear_attn_decode_step(q, k, v, S, al)[:, :, None])
    o3, S3 = dn.gated_linear_attn_fwd(*part(82, 200), S)
    assert rel(torch.cat(outs + [o3], 2), ro) <= TOL[dtype]
    assert rel(S3, rS) <= TOL[torch.float32]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padding_leaves_the_state(dn, dtype):
    """Right-padded batches: k = 0 and alpha = 1 behind the end."""
    x = case(2, 2, 150, 64, 64, dtype, "mixed", True, 11)
    n = 93
    x["k"][1, :, n:] = 0
    x["alpha"][1, :, n:] = 1
    _, S = dn.gated_linear_attn_fwd(*pick(x, FWD))
    _, rS = plain(*[t[1:, :, :n] for t in pick(x, FWD[:4])], x["S0"][1:])
    assert rel(S[1:], rS) <= TOL[torch.float32]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_documents_do_not_mix(dn, dtype):
    """alpha = 0 at a document's first token forgets everything before, exactly,
    in outputs and gradients, whatever stood there."""
    x = case(1, 2, 260, 64, 64, dtype, "mixed", True, 12)
    x["alpha"][:, :, 150] = 0
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "dO"):
        y[n][:, :, :150] *= -3
    y["S0"] += 5
    a, b = (dn.gated_linear_attn_fwd(*pick(z, FWD)) for z in (x, y))
    assert torch.equal(a[0][:, :, 150:], b[0][:, :, 150:]) and torch.equal(a[1], b[1])
    ga, gb = (dn.gated_linear_attn_bwd(*pick(z, BWD)) for z in (x, y))
    for n in ("dq", "dk", "dv"):
        assert torch.equal(ga[n][:, :, 150:], gb[n][:, :, 150:]), n
    assert bool((ga["dlog_alpha"][:, :, 150] == 0).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_tokens_and_no_heads(dn, dtype):
    S0 = torch.randn(2, 3, 64, 128, device="cuda")
    e = torch.empty(2, 3, 0, 64, dtype=dtype, device="cuda")
    ev = torch.empty(2, 3, 0, 128, dtype=dtype, device="cuda")
    al = torch.empty(2, 3, 0, device="cuda")
    o, S = dn.gated_linear_attn_fwd(e, e, ev, al, S0)
    assert o.shape == ev.shape and torch.equal(S, S0)
    assert not dn.gated_linear_attn_fwd(e, e, ev)[1].any()
    g = dn.gated_linear_attn_bwd(e, e, ev, ev, al, S0, S0)
    assert torch.equal(g["dS0"], S0) and g["dq"].shape == e.shape
    assert not dn.gated_linear_attn_bwd(e, e, ev, ev)["dS0"].any()
    z = torch.empty(0, 3, 5, 64, dtype=dtype, device="cuda")
    assert dn.gated_linear_attn_fwd(z, z, z)[0].shape == z.shape
    assert dn.gated_linear_attn_bwd(z, z, z, z)["dv"].shape == z.shape
    zs = torch.empty(0, 3, 64, dtype=dtype, device="cuda")
    assert dn.gated_linear_attn_decode_step(zs, zs, zs, torch.empty(0, 3, 64, 64, device="cuda")).shape == zs.shape


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_same_bits_twice_and_nothing_outside(dn, dtype):
    """Two runs agree bit for bit; guards around the outputs stay."""
    x = case(2, 3, 201, 128, 128, dtype, "mixed", True, 13)
    n = x["v"].numel()
    buf = torch.full((n + 256,), 7.0, dtype=dtype, device="cuda")
    o = buf[128:128 + n].view(x["v"].shape)
    a = dn.gated_linear_attn_fwd(*pick(x, FWD), o=o)
    b = dn.gated_linear_attn_fwd(*pick(x, FWD))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool((buf[:128] == 7).all() and (buf[128 + n:] == 7).all())
    a, b = (dn.gated_linear_attn_bwd(*pick(x, BWD)) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


@gpu
@pytest.mark.parametrize("T", [5, 300])
def test_sixteen_byte_alignment(dn, T):
    """Every buffer at an odd multiple of 16 bytes."""
    x = case(2, 2, T, 64, 128, torch.bfloat16, "mixed", True, T)

    def shifted(t):
        n = 16 // t.element_size()
        buf = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
        buf[n:].copy_(t.reshape(-1))
        assert buf[n:].data_ptr() % 32 == 16
        return buf[n:].view(t.shape)

    want = dn.gated_linear_attn_fwd(*pick(x, FWD)), dn.gated_linear_attn_bwd(*pick(x, BWD))
    y = {n: shifted(t) for n, t in x.items()}
    o, S = shifted(x["v"]), shifted(x["S0"])
    dn.gated_linear_attn_fwd(*pick(y, FWD), o=o, S_out=S)
    assert torch.equal(o, want[0][0]) and torch.equal(S, want[0][1])
    got = dn.gated_linear_attn_bwd(*pick(y, BWD))
    assert all(torch.equal(got[n], want[1][n]) for n in got)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_stays_in_its_head_and_behind_its_chunk(dn, dtype):
    x = case(1, 3, 400, 64, 64, dtype, "mixed", False, 14)
    want = plain(*pick(x, FWD))
    x["v"][0, 1, 300, 5] = float("nan")
    o, S = dn.gated_linear_attn_fwd(*pick(x, FWD))
    for h in (0, 2):
        assert rel(o[:, h], want[0][:, h]) <= TOL[dtype] and rel(S[:, h], want[1][:, h]) <= TOL[torch.float32]
    assert rel(o[:, 1, :256], want[0][:, 1, :256]) <= TOL[dtype]  # whole chunks of 128 before it
    assert bool(o[0, 1, 300:, 5].isnan().all()) and bool(S[0, 1, :, 5].isnan().all())


@gpu
@pytest.mark.parametrize("T", [300, 5000])
def test_streams_and_graphs(dn, T):
    """On another stream, two at once, and captured: two graphs with workspaces
    of their own, replayed on new inputs in the same buffers."""
    xs = [case(1, 2, T, 128, 128, torch.bfloat16, "mixed", True, 20 + i) for i in range(2)]
    want = [(dn.gated_linear_attn_fwd(*pick(x, FWD)), dn.gated_linear_attn_bwd(*pick(x, BWD))) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append([(dn.gated_linear_attn_fwd(*pick(x, FWD)), dn.gated_linear_attn_bwd(*pick(x, BWD)))
                        for _ in range(3)][-1])
    torch.cuda.synchronize()

    def same(a, b):
        return (torch.equal(a[0][0], b[0][0]) and torch.equal(a[0][1], b[0][1])
                and all(torch.equal(a[1][n], b[1][n]) for n in a[1]))

    assert all(same(a, b) for a, b in zip(got, want))
    graphs, outs, ins = [], [], [{n: t.clone() for n, t in xs[0].items()} for _ in range(2)]
    for x in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((dn.gated_linear_attn_fwd(*pick(x, FWD)), dn.gated_linear_attn_bwd(*pick(x, BWD))))
        graphs.append(g)
    for i in range(2):
        for n, t in xs[i].items():
            ins[i][n].copy_(t)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(outs, want))


@gpu
def test_threads_on_one_stream(dn):
    """Threads that share a stream share its scratch too: a call's launches stay together."""
    import threading

    xs = [case(1, 2, 3000, 64, 64, torch.bfloat16, seed=s) for s in range(4)]
    run = lambda x: (*dn.gated_linear_attn_fwd(*pick(x, FWD)), *dn.gated_linear_attn_bwd(*pick(x, BWD)).values())
    want = [run(x) for x in xs]
    bad = []

    def work(i):
        for _ in range(30):
            if not all(torch.equal(a, b) for a, b in zip(run(xs[i]), want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@gpu
def test_status_after_a_stream_is_gone(dn):
    import gc

    x = case(1, 2, 3000, 64, 64, torch.bfloat16, seed=1)
    want = dn.gated_linear_attn_fwd(*pick(x, FWD))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = dn.gated_linear_attn_fwd(*pick(x, FWD))
    del s
    gc.collect()
    assert dn.deltanet_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_binding_refusals(dn):
    x = case(1, 2, 8, 64, 64, torch.bfloat16)
    bad = [dict(k=x["k"][:, :, :4].contiguous()), dict(v=x["v"].float()), dict(alpha=x["alpha"][:, :1].contiguous()),
           dict(alpha=x["alpha"].double()), dict(S0=x["S0"][..., :32].contiguous()),
           dict(q=x["q"].transpose(1, 2)), dict(q=x["q"].half(), k=x["k"].half(), v=x["v"].half()),
           dict(q=x["q"][0]), dict(k=None)]
    for new in bad:
        with pytest.raises((ValueError, TypeError)):
            dn.gated_linear_attn_fwd(*pick({**x, **new}, FWD))
        with pytest.raises((ValueError, TypeError)):
            dn.gated_linear_attn_bwd(*pick({**x, **new}, BWD))
    with pytest.raises(dn.DeltaNetError):
        y = torch.zeros(1, 1, 4, 96, dtype=torch.bfloat16, device="cuda")
        dn.gated_linear_attn_fwd(y, y, y)
    with pytest.raises(dn.DeltaNetError):
        dn.gated_linear_attn_fwd(*pick(x, FWD), o=x["q"])
    assert dn.deltanet_get_device_status("cuda") == 0
