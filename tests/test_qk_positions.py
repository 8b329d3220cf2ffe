"""Rotation at positions of any size, against angles reduced in exact arithmetic.

Tolerance: that of float32 values in test_qk_norm_rope.py (32 * 2^-24 = 2e-6 of
the 2-norm, 1e-5 in the gradient); an angle that is off by e turns a row by e of
its norm.
"""
from fractions import Fraction

import pytest
import torch


def two_pi(bits=320):
    """2 pi in units of 2^-bits: Machin's 16 atan(1/5) - 4 atan(1/239), doubled."""
    one = 1 << (bits + 16)

    def atan(n):
        total, power, k, sign = 0, one // n, 1, 1
        while power:
            total += sign * (power // k)
            power //= n * n
            k, sign = k + 2, -sign
        return total

    return 2 * (16 * atan(5) - 4 * atan(239)) >> 16


def turned_part(pos, freq, bits=320):
    """pos * freq / (2 pi) without its whole part, in [-1/2, 1/2]."""
    x = Fraction(pos) * Fraction(freq) * (1 << bits) / two_pi(bits)
    return float(x - round(x))


def test_the_reference_reduces_angles():
    assert abs(two_pi(60) / (1 << 60) - 6.283185307179586) < 1e-15
    for pos, freq in ((1, 1.0), (12345, 0.25), (-77, 0.125)):
        x = pos * freq / 6.283185307179586
        assert abs(turned_part(pos, freq) - (x - round(x))) < 1e-12
    # far out: the parts of a sum of positions add up
    a, b = turned_part((1 << 62) + 3, 0.75), turned_part(1 << 62, 0.75)
    assert abs((a - b - turned_part(3, 0.75) + 0.5) % 1 - 0.5) < 1e-12


POSITIONS = [0, 1, 4095, 1 << 24, (1 << 24) + 1, (1 << 28) + 1, (1 << 32) - 1, 1 << 34, (1 << 40) + 12345, (1 << 50) + 1, (1 << 53) + 1,
             (1 << 54) + 2047, (1 << 62) + 987654321, (1 << 63) - 1]


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_any_position(interleaved):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deltanet_sequence_mixing_b200 as dn

    D, n = 64, 32
    freq = (10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)).float()
    pos = POSITIONS + [-p for p in POSITIONS] + [-(1 << 63)]
    turns = torch.tensor([[turned_part(p, f) for f in freq.tolist()] for p in pos], dtype=torch.float64)
    c, s = (t.cuda()[None, :, None] for t in ((turns * 2 * torch.pi).cos(), (turns * 2 * torch.pi).sin()))
    g = torch.Generator().manual_seed(31)
    q, k, dq, dk = (torch.randn(1, len(pos), 2, D, generator=g).cuda() for _ in range(4))
    dq, dk = dq.transpose(1, 2).contiguous(), dk.transpose(1, 2).contiguous()
    at = torch.arange(n)
    lo, hi = (2 * at, 2 * at + 1) if interleaved else (at, at + n)
    args = dict(positions=torch.tensor(pos, device="cuda"), inv_freq=freq.cuda(), interleaved=interleaved)
    got = dn.qk_norm_rope_fwd(q, k, **args)
    back = dn.qk_norm_rope_bwd(q, k, dq, dk, **args)
    rel = lambda a, b: float((a.double() - b.detach()).norm() / b.detach().norm())
    for x, y, d, dx in ((q, got[0], dq, back["dq"]), (k, got[1], dk, back["dk"])):
        x = x.double().requires_grad_()
        z = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        u, v = z[..., lo], z[..., hi]
        want = z.clone()
        want[..., lo], want[..., hi] = u * c - v * s, v * c + u * s
        want = want.transpose(1, 2)
        for t, p in enumerate(pos):
            assert rel(y[:, :, t], want[:, :, t]) <= 2e-6, p
        (grad,) = torch.autograd.grad(want, x, d.double())
        assert rel(dx, grad) <= 1e-5
