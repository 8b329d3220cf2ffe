"""Per-head norm and rotation of queries and keys: forward, gradient and their
run together with the mixing calls, against float64.

Tolerances (2-norm of the difference over the 2-norm of the result):
* float32: about ten float32 operations per value and sums of at most 128
  squares, and the fast reciprocal, root and exponential with relative errors
  up to 2^-21: 32 * 2^-24 = 2e-6.
* bfloat16: one rounding, at most 2^-8.
* weight gradients: float32 sums of B*T*H products in a tree of at most 64
  terms a level: 1e-5 of the result where it is not smaller than its terms' root
  sum of squares.
"""
import ctypes

import pytest
import torch

TOL = {torch.float32: 2e-6, torch.bfloat16: 2.0 ** -8}
EPS = {"rms": 1e-6, "l2": 1e-12}


def rel(x, ref):
    x, ref = x.detach().double(), ref.detach().double()
    assert x.shape == ref.shape
    return float((x - ref).norm() / ref.norm().clamp_min(1e-300))


def plain(x, w, pos, freq, norm="rms", eps=None, silu=False, interleaved=False):
    """(B,T,H,D) -> (B,H,T,D), the definition in float64."""
    eps = EPS[norm] if eps is None else eps
    x = x.double()
    if silu:
        x = x * torch.sigmoid(x)
    if norm == "rms":
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    else:
        # max(||x||, eps), written so that its derivative exists at x = 0
        y = x / x.square().sum(-1, keepdim=True).clamp_min(eps * eps).sqrt()
    if w is not None:
        y = y * w.double()
    if freq is not None and len(freq):
        B, T = x.shape[:2]
        if pos is None:
            pos = torch.arange(T, device=x.device)
        a = (pos.expand(B, T).double()[..., None] * freq.double())[:, :, None]
        n = len(freq)
        i = torch.arange(n, device=x.device)
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        u, v = y[..., lo], y[..., hi]
        y = y.clone()
        y[..., lo], y[..., hi] = u * a.cos() - v * a.sin(), v * a.cos() + u * a.sin()
    return y.transpose(1, 2)


def freqs(rot, device="cuda"):
    return (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float().to(device) if rot else None


def case(B, T, Hq, Hk, D, dtype, rot, seed=0, far=False):
    """q and k as slices of a fused projection with a value part behind."""
    g = torch.Generator().manual_seed(seed)
    fused = torch.randn(B, T, (Hq + 2 * Hk) * D, generator=g).to(dtype).cuda()
    q = fused[..., :Hq * D].unflatten(-1, (Hq, D))
    k = fused[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    w = [(1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    pos = torch.randint(0, 1 << 28 if far else 4096, (B, T), generator=g).cuda()
    grads = [torch.randn(B, H, T, D, generator=g).to(dtype).cuda() for H in (Hq, Hk)]
    return q, k, *w, pos, freqs(rot), grads


@pytest.fixture(scope="module")
def dn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deltanet_sequence_mixing_b200 as m

    m.lib()
    return m


def check(dn, q, k, wq, wk, pos, freq, grads, **how):
    dtype = q.dtype
    got = dn.qk_norm_rope_fwd(q, k, wq, wk, pos, freq, **how)
    back = dn.qk_norm_rope_bwd(q, k, *grads, wq, wk, pos, freq, **how)
    for n, x, w, y, d in (("q", q, wq, got[0], grads[0]), ("k", k, wk, got[1], grads[1])):
        x = x.double().clone().requires_grad_()
        w64 = None if w is None else w.double().clone().requires_grad_()
        want = plain(x, w64, pos, freq, **how)
        assert y.is_contiguous() and y.dtype == dtype
        assert rel(y, want) <= TOL[dtype], (n, rel(y, want))
        g = torch.autograd.grad(want, [x] + ([] if w is None else [w64]), d.double())
        assert back["d" + n].dtype == dtype
        # the gradient's projection off the row costs float32 one more digit where it cancels
        assert rel(back["d" + n], g[0]) <= max(TOL[dtype], 1e-5), (n, rel(back["d" + n], g[0]))
        if w is None:
            assert back[f"d{n}_weight"] is None
        else:
            assert rel(back[f"d{n}_weight"], g[1]) <= 1e-5, (n, rel(back[f"d{n}_weight"], g[1]))


# ----------------------------------------------------------------- on the CPU --
A, MB = 1 << 32, 1 << 20
vp = lambda x: None if x is None else ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def L():
    from deltanet_sequence_mixing_b200 import _lib
    from deltanet_sequence_mixing_b200.build import build

    build()
    return _lib.lib()


def _fwd(L, q=A, k=A + 16 * MB, wq=A + 32 * MB, wk=A + 33 * MB, pos=A + 34 * MB, freq=A + 36 * MB, qo=A + 64 * MB,
         ko=A + 96 * MB, B=2, T=10, Hq=2, Hk=2, D=64, rot=64, s=None, ps=10, eps=1e-6, opts=0, dt=1):
    s = s or [10 * 128, 128, 64] * 2
    return L.qk_norm_rope_fwd(vp(q), vp(k), vp(wq), vp(wk), vp(pos), vp(freq), vp(qo), vp(ko), B, T, Hq, Hk, D, rot,
                              *s, ps, eps, opts, dt, None)


def test_fwd_refusals(L):
    from deltanet_sequence_mixing_b200 import _lib as E

    for n in ("q", "k", "freq", "qo", "ko"):
        assert _fwd(L, **{n: None}) == E.DN_ERR_INVALID_ARG
    for n in ("B", "T", "Hq", "Hk", "ps"):
        assert _fwd(L, **{n: -1}) == E.DN_ERR_INVALID_ARG
    assert _fwd(L, D=96) == E.DN_ERR_UNSUPPORTED
    for rot in (-16, 8, 24, 80):
        assert _fwd(L, rot=rot) == E.DN_ERR_UNSUPPORTED
    assert _fwd(L, dt=4) == E.DN_ERR_UNSUPPORTED
    assert _fwd(L, B=1 << 16, T=1 << 16) == E.DN_ERR_UNSUPPORTED
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _fwd(L, eps=eps) == E.DN_ERR_INVALID_ARG
    assert _fwd(L, opts=8) == E.DN_ERR_INVALID_ARG
    assert _fwd(L, s=[1280, 128, -64, 1280, 128, 64]) == E.DN_ERR_INVALID_ARG
    assert _fwd(L, s=[1280, 128, 66, 1280, 128, 64]) == E.DN_ERR_ALIGNMENT
    assert _fwd(L, q=A + 8) == E.DN_ERR_ALIGNMENT
    assert _fwd(L, ko=A + 96 * MB + 8) == E.DN_ERR_ALIGNMENT
    assert _fwd(L, pos=A + 34 * MB + 4) == E.DN_ERR_ALIGNMENT
    assert _fwd(L, qo=A) == E.DN_ERR_INVALID_ARG  # in place: the layouts differ
    assert _fwd(L, ko=A + 64 * MB) == E.DN_ERR_INVALID_ARG
    assert _fwd(L, T=0, q=None, k=None, qo=None, ko=None) == E.DN_OK


def test_bwd_refusals(L):
    from deltanet_sequence_mixing_b200 import _lib as E

    s = [1280, 128, 64] * 2

    def call(q=A, dq=A + 64 * MB, dk=A + 80 * MB, gq=A + 96 * MB, gk=A + 112 * MB, dwq=A + 128 * MB,
             dwk=A + 129 * MB, wk=A + 33 * MB, ds=s, dt=1, gdt=1, ws=A + 200 * MB, nb=1 << 20):
        return L.qk_norm_rope_bwd(vp(q), vp(A + 16 * MB), vp(gq), vp(gk), vp(A + 32 * MB), vp(wk), vp(A + 34 * MB),
                                  vp(A + 36 * MB), vp(dq), vp(dk), vp(dwq), vp(dwk), 2, 10, 2, 2, 64, 64, *s, *ds, 10,
                                  1e-6, 0, dt, gdt, vp(ws), nb, None)

    for n in ("q", "dq", "dk", "gq", "gk", "wk"):
        assert call(**{n: None}) == E.DN_ERR_INVALID_ARG
    assert call(dt=0, gdt=1) == E.DN_ERR_UNSUPPORTED
    assert call(gdt=3) == E.DN_ERR_UNSUPPORTED
    assert call(ws=None) == E.DN_ERR_WORKSPACE
    assert call(nb=16) == E.DN_ERR_WORKSPACE
    assert call(ws=A + 200 * MB + 4) == E.DN_ERR_ALIGNMENT
    assert call(ds=[1280, 128, 60, 1280, 128, 64]) == E.DN_ERR_ALIGNMENT
    assert call(ds=[1280, 128, 0, 1280, 128, 64]) == E.DN_ERR_INVALID_ARG  # heads on one another
    assert call(ds=[1280, 64, 64, 1280, 128, 64]) == E.DN_ERR_INVALID_ARG  # tokens on one another
    assert call(ds=[0, 128, 64, 1280, 128, 64]) == E.DN_ERR_INVALID_ARG
    assert call(dq=A) == E.DN_ERR_INVALID_ARG  # dq on q
    assert call(dwq=A + 200 * MB) == E.DN_ERR_INVALID_ARG  # a weight's gradient in the workspace


def test_bwd_refuses_dq_and_dk_on_one_another(L):
    from deltanet_sequence_mixing_b200 import _lib as E

    def call(delta, s, B=2, T=10, Hq=2, Hk=2, sk=None):
        in_s = [T * Hq * 64, Hq * 64, 64, T * Hk * 64, Hk * 64, 64]
        return L.qk_norm_rope_bwd(vp(A), vp(A + 16 * MB), vp(A + 96 * MB), vp(A + 112 * MB), None, None, None,
                                  vp(A + 36 * MB), vp(A + 64 * MB), vp(A + 64 * MB + 2 * delta), None, None, B, T,
                                  Hq, Hk, 64, 64, *in_s, *s, *(sk or s), 0, 1e-6, 0, 1, 1, None, 0, None)

    bad = E.DN_ERR_INVALID_ARG
    assert call(0, [1280, 128, 64]) == bad  # one tensor
    assert call(256, [1280, 128, 64]) == bad  # two tokens on
    assert call(-1280, [1280, 128, 64]) == bad  # one sequence back
    assert call(64, [5120, 512, 64]) == bad  # k's first head on q's second
    assert call(128, [5120, 512, 64], Hq=3) == bad
    assert call(512 + 64, [5120, 512, 64]) == bad  # the same in the next token
    assert call(32, [2560, 256, 64], Hq=1, Hk=1) == bad  # half a row
    assert call(128, [2560, 256, 64], sk=[2560, 128, 64]) == bad  # strides of their own in one range
    assert call(640 + 64, [2560, 64, 640]) == bad  # heads outside tokens


def test_binding_refuses_host_tensors():
    import deltanet_sequence_mixing_b200 as m

    x = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.qk_norm_rope_fwd(x, x)


# ----------------------------------------------------------------- on the GPU --
gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (64, 16), (128, 112), (64, 0)])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes(dn, dtype, D, rot, norm, interleaved):
    check(dn, *case(2, 37, 3, 2, D, dtype, rot, D + rot), norm=norm, interleaved=interleaved)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (5, 1, 32, 4), (1, 700, 1, 1), (3, 129, 16, 16), (1, 3, 150, 7)])
def test_sizes_with_silu(dn, dtype, norm, B, T, Hq, Hk):
    check(dn, *case(B, T, Hq, Hk, 128, dtype, 64, B + T), norm=norm, silu=True)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_weights_and_positions(dn, dtype):
    q, k, wq, wk, pos, freq, grads = case(2, 50, 4, 2, 64, dtype, 64, 3)
    check(dn, q, k, None, None, None, freq, grads)
    check(dn, q, k, wq, None, pos[0].contiguous(), freq, grads)  # one row of positions for all
    check(dn, q, k, None, wk, pos, None, grads, norm="l2")


@gpu
def test_far_positions(dn):
    """Angles of positions up to 2^28, to float32."""
    check(dn, *case(2, 40, 2, 2, 128, torch.float32, 128, 4, far=True))
    q, k, wq, wk, pos, freq, grads = case(2, 40, 2, 2, 128, torch.float32, 128, 5)
    check(dn, q, k, wq, wk, -pos, freq, grads)


@gpu
def test_strides_and_slices_of_one_gradient(dn):
    """Inputs and gradients in other orders; what lies between rows stays."""
    q, k, wq, wk, pos, freq, grads = case(2, 20, 3, 3, 64, torch.bfloat16, 64, 6)
    qt = q.permute(2, 1, 0, 3).contiguous().permute(2, 1, 0, 3)
    kt = k.transpose(1, 2).contiguous().transpose(1, 2)
    for a, b in zip(dn.qk_norm_rope_fwd(q, k, wq, wk, pos, freq), dn.qk_norm_rope_fwd(qt, kt, wq, wk, pos, freq)):
        assert torch.equal(a, b)
    want = dn.qk_norm_rope_bwd(q, k, *grads, wq, wk, pos, freq)
    fused = torch.full((2, 20, 9 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk = (fused[..., i * 192:(i + 1) * 192].unflatten(-1, (3, 64)) for i in range(2))
    got = dn.qk_norm_rope_bwd(qt, kt, *grads, wq, wk, pos, freq, dq=dq, dk=dk)
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert bool((fused[..., 384:] == 7).all())
    # one row of q and k for every head (a broadcast input): each head's gradient apart
    one = q[:, :, :1].expand(2, 20, 3, 64)
    check(dn, one, k, wq, wk, pos, freq, grads)


@gpu
@pytest.mark.parametrize("B,T,Hq,Hk", [(2, 20, 3, 3), (2, 20, 1, 4), (1, 20, 4, 1), (3, 1, 2, 5)])
@pytest.mark.parametrize("axis", [1, 2, 3, 4])
def test_gradients_side_by_side(dn, B, T, Hq, Hk, axis):
    """dq and dk in one buffer: q's heads in front of k's, heads inside or outside
    the tokens (axis 2, 1); with as many of both, in pairs (3) or k's in front (4)."""
    if axis >= 3 and Hq != Hk:
        Hk = Hq
    q, k, wq, wk, pos, freq, grads = case(B, T, Hq, Hk, 64, torch.bfloat16, 64, 21)
    if axis == 1:
        buf = torch.full((B, Hq + Hk + 1, T, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    else:
        buf = torch.full((B, T, Hq + Hk + 1, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk = buf[:, :, 1:1 + Hq], buf[:, :, 1 + Hq:]
    if axis == 3:
        dq, dk = buf[:, :, 1::2], buf[:, :, 2::2]
    if axis == 4:
        dq, dk = buf[:, :, 1 + Hq:], buf[:, :, 1:1 + Hq]
    want = dn.qk_norm_rope_bwd(q, k, *grads, wq, wk, pos, freq)
    got = dn.qk_norm_rope_bwd(q, k, *grads, wq, wk, pos, freq, dq=dq, dk=dk)
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert bool((buf[:, :, 0] == 7).all())


@gpu
def test_float32_gradients_into_bfloat16(dn):
    q, k, wq, wk, pos, freq, grads = case(2, 20, 3, 2, 128, torch.bfloat16, 128, 7)
    check(dn, q, k, wq, wk, pos, freq, [g.float() + 1e-3 for g in grads])


@gpu
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_rows_of_zeros_and_of_nan(dn, norm):
    """Zero rows give zeros; below the floor the l2 map is linear; a NaN stays in its row."""
    q, k, wq, wk, pos, freq, grads = case(1, 6, 2, 2, 64, torch.float32, 64, 8)
    q, k = q.clone(), k.clone()
    q[0, 2, 1] = 0
    k[0, 3, 0] *= 1e-15
    check(dn, q, k, wq, wk, pos, freq, grads, norm=norm)
    clean = dn.qk_norm_rope_fwd(q, k, wq, wk, pos, freq, norm=norm)[0]
    q[0, 4, 0, 3] = float("nan")
    got = dn.qk_norm_rope_fwd(q, k, wq, wk, pos, freq, norm=norm)[0]
    assert bool(got[0, 0, 4].isnan().all())
    got[0, 0, 4] = clean[0, 0, 4]
    assert torch.equal(got, clean)


@gpu
def test_no_tokens_and_no_heads(dn):
    e = torch.empty(2, 0, 3, 64, device="cuda")
    w, freq = torch.ones(64, device="cuda"), freqs(64)
    assert dn.qk_norm_rope_fwd(e, e, w, w, None, freq)[0].shape == (2, 3, 0, 64)
    g = torch.empty(2, 3, 0, 64, device="cuda")
    got = dn.qk_norm_rope_bwd(e, e, g, g, w, w, None, freq)
    assert not got["dq_weight"].any() and got["dk"].shape == e.shape
    q, k0 = torch.randn(2, 5, 3, 64, device="cuda"), torch.empty(2, 5, 0, 64, device="cuda")
    assert rel(dn.qk_norm_rope_fwd(q, k0, w, w, None, freq)[0], plain(q, w, None, freq)) <= TOL[torch.float32]
    got = dn.qk_norm_rope_bwd(q, k0, torch.randn(2, 3, 5, 64, device="cuda"),
                              torch.empty(2, 0, 5, 64, device="cuda"), w, w, None, freq)
    assert not got["dk_weight"].any() and got["dq_weight"].any()


@gpu
def test_same_bits_twice_other_stream_and_graph(dn):
    args = case(4, 300, 5, 3, 128, torch.bfloat16, 128, 9)
    call = lambda: (dn.qk_norm_rope_fwd(*args[:6]), dn.qk_norm_rope_bwd(*args[:2], *args[6], *args[2:6]))
    want = call()
    torch.cuda.synchronize()
    same = lambda a, b: (all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
                         and all(torch.equal(a[1][n], b[1][n]) for n in a[1]))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call()
    torch.cuda.synchronize()
    assert same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for t in (*got[0], *got[1].values()):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert same(got, want)


@gpu
def test_is_the_map_of_the_prestep(dn):
    """silu and l2 without weights or rotation, then the plain delta rule: the
    call with the pre-step inside.  Its own maps use the hardware tanh (2^-11)
    and round q and k to bfloat16 once, as here: a few roundings of 2^-8 apart."""
    B, T, H, D = 2, 200, 2, 64
    g = torch.Generator().manual_seed(10)
    x = torch.randn(B, T, 3 * H * D, generator=g).bfloat16().cuda()
    q, k, v = (x[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    logit = torch.randn(B, H, T, generator=g).cuda()
    v = v.transpose(1, 2).contiguous()
    qn, kn = dn.qk_norm_rope_fwd(q, k, norm="l2", silu=True)
    o, S = dn.deltanet_chunk_fwd(qn, kn, v, torch.sigmoid(logit))
    ro, rS = dn.deltanet_chunk_fwd(q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous(), v, logit,
                                   prestep=True)
    assert rel(o, ro) <= 2e-2 and rel(S, rS) <= 2e-2


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_forward_backward_and_token(dn, dtype):
    """The calls as a layer runs them: fused projection -> norm and rotation ->
    gated recurrence; its gradient back to the projection; and the same sequence
    as a prompt with single tokens behind it."""
    B, T, H, D = 2, 150, 3, 64
    g = torch.Generator().manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=g)
    x = n(B, T, 3 * H * D).to(dtype).cuda()
    alpha = torch.exp(-0.05 * torch.rand(B, H, T, generator=g)).cuda()
    w = [(1 + 0.1 * n(D)).cuda() for _ in range(2)]
    freq, dO = freqs(D), n(B, H, T, D).to(dtype).cuda()
    pos = torch.arange(T).expand(B, T).contiguous().cuda() + 1000
    parts = lambda y: [y[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3)]
    from test_gated_linear import plain as recurrence

    def run(y):
        q, k, v = parts(y)
        q, k = dn.qk_norm_rope_fwd(q, k, *w, pos, freq, norm="l2")
        return q, k, v.transpose(1, 2).contiguous()

    q, k, v = run(x)
    o, S = dn.gated_linear_attn_fwd(q, k, v, alpha)
    d = dn.gated_linear_attn_bwd(q, k, v, dO, alpha)
    dx = torch.empty_like(x)
    dq, dk, dv = parts(dx)
    gw = dn.qk_norm_rope_bwd(*parts(x)[:2], d["dq"], d["dk"], *w, pos, freq, norm="l2", dq=dq, dk=dk)
    dv.copy_(d["dv"].transpose(1, 2))

    x64, al64 = x.double().requires_grad_(), alpha.double().requires_grad_()
    w64 = [t.double().requires_grad_() for t in w]
    q64, k64, v64 = parts(x64)
    ro, rS = recurrence(plain(q64, w64[0], pos, freq, "l2"), plain(k64, w64[1], pos, freq, "l2"),
                        v64.transpose(1, 2), al64)
    rx, ral, *rw = torch.autograd.grad((ro * dO.double()).sum(), [x64, al64, *w64])
    # q and k are rounded between the calls, and so are their gradients: two
    # roundings more on each side of the recurrence's three, sqrt(7) * 2^-8 in the 2-norm
    tol = 2e-5 if dtype == torch.float32 else 7 ** 0.5 * 2.0 ** -8
    assert rel(o, ro) <= tol and rel(S, rS) <= tol and rel(dx, rx) <= tol
    assert rel(d["dlog_alpha"], ral * al64) <= tol
    assert rel(gw["dq_weight"], rw[0]) <= tol and rel(gw["dk_weight"], rw[1]) <= tol

    cut = 140
    y = x[:, :cut]
    a = lambda i, j: alpha[:, :, i:j].contiguous()
    qp, kp = dn.qk_norm_rope_fwd(*parts(y)[:2], *w, pos[:, :cut].contiguous(), freq, norm="l2")
    op, S = dn.gated_linear_attn_fwd(qp, kp, parts(y)[2].transpose(1, 2).contiguous(), a(0, cut))
    outs = [op]
    for t in range(cut, T):
        q1, k1, v1 = parts(x[:, t:t + 1])
        q1, k1 = dn.qk_norm_rope_fwd(q1, k1, *w, pos[:, t:t + 1].contiguous(), freq, norm="l2")
        o1 = dn.gated_linear_attn_decode_step(q1[:, :, 0], k1[:, :, 0], v1[:, 0].contiguous(), S,
                                              alpha[:, :, t].contiguous())
        outs.append(o1[:, :, None])
    assert rel(torch.cat(outs, 2), ro) <= tol


@gpu
def test_binding_refusals(dn):
    q, k, wq, wk, pos, freq, grads = case(2, 8, 2, 2, 64, torch.bfloat16, 64, 12)
    ok = dict(q=q, k=k, q_weight=wq, k_weight=wk, positions=pos, inv_freq=freq)
    bad = [dict(q=q.half()), dict(k=k.float()), dict(k=k[:, :4]), dict(q_weight=wq.bfloat16()),
           dict(k_weight=wk[:32].contiguous()), dict(positions=pos.int()), dict(positions=pos[:1].contiguous()),
           dict(inv_freq=freq.double()), dict(inv_freq=freq[:, None]), dict(norm="layer"), dict(q=q.transpose(2, 3)),
           dict(q=q[0])]
    for new in bad:
        with pytest.raises((ValueError, TypeError)):
            dn.qk_norm_rope_fwd(**{**ok, **new})
    for new in (dict(inv_freq=freq[:5].contiguous()), dict(eps=0.0), dict(q=q[..., :48], k=k[..., :48],
                q_weight=None, k_weight=None)):
        with pytest.raises(dn.DeltaNetError):
            dn.qk_norm_rope_fwd(**{**ok, **new})
    with pytest.raises((ValueError, TypeError)):
        dn.qk_norm_rope_bwd(q, k, grads[0], grads[1].float(), wq, wk, pos, freq)
    with pytest.raises(dn.DeltaNetError):  # rows of dq on one another
        dn.qk_norm_rope_bwd(q, k, *grads, wq, wk, pos, freq, dq=torch.empty_like(q[:, :, :1]).expand(2, 8, 2, 64))
