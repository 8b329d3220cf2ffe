"""Sizes at which the kernels take the ways of large calls: the q/k forward with
both tensors in one CTA, the q/k gradient and the recurrence's gradient with
several rounds of tiles or chunks to a CTA, all of them with a ragged last one.
References and tolerances are those of the small tests, whose derivations do not
depend on the sizes met here (a thread's sums of a weight's gradient have up to
25 terms more).
"""
import pytest
import torch

import test_gated_linear as rec
import test_qk_norm_rope as qk

gpu = pytest.mark.gpu
SMS = 148


@pytest.fixture(scope="module")
def dn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deltanet_sequence_mixing_b200 as m

    m.lib()
    return m


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm,silu", [("rms", False), ("l2", True)])
@pytest.mark.parametrize("B,T,Hq,Hk,D,rot", [(1, 10007, 16, 16, 128, 128), (3, 3343, 16, 4, 64, 32),
                                             (2, 3701, 3, 20, 128, 64), (1, 9533, 1, 1, 64, 64)])
def test_qk(dn, dtype, norm, silu, B, T, Hq, Hk, D, rot):
    tile = min(256 // max(Hq, Hk), 16)
    assert B * T >= 4 * SMS * tile and B * T % tile
    qk.check(dn, *qk.case(B, T, Hq, Hk, D, dtype, rot, T), norm=norm, silu=silu)


@gpu
@pytest.mark.parametrize("Dk,Dv", rec.DIMS)
@pytest.mark.parametrize("gate", ["mixed", "wipes", None])
def test_gradient_of_many_chunks(dn, Dk, Dv, gate):
    B, H, T = 3, 33, 389
    assert B * H * -(-T // 128) > 2 * SMS
    rec.check_bwd(dn, rec.case(B, H, T, Dk, Dv, torch.bfloat16, gate, True, Dk + Dv), torch.bfloat16)


@gpu
def test_gradient_of_many_chunks_in_segments(dn):
    B, H, T = 1, 2, 19001
    assert B * H * -(-T // 128) > 2 * SMS
    x = rec.case(B, H, T, 128, 128, torch.bfloat16, "wipes", True, 3)
    rec.check_fwd(dn, x, torch.bfloat16)
    rec.check_bwd(dn, x, torch.bfloat16)


@gpu
@pytest.mark.parametrize("Dk,Dv", rec.DIMS)
@pytest.mark.parametrize("gate", ["wipes", None])
def test_forward_of_many_heads(dn, Dk, Dv, gate):
    """More CTAs than run at once, chunks beyond the first reuse of every stage."""
    B, H, T = 5, 31, 1003
    assert B * H * (Dv // 64) > SMS
    x = rec.case(B, H, T, Dk, Dv, torch.bfloat16, gate, True, Dk)
    rec.check_fwd(dn, x, torch.bfloat16)
