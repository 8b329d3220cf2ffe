"""Sizes at which the recurrence's index arithmetic ends: refused on the host."""
import ctypes

import pytest

INT_MAX = 2 ** 31 - 1
vp = lambda x: None if x is None else ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def L():
    from deltanet_sequence_mixing_b200 import _lib
    from deltanet_sequence_mixing_b200.build import build

    build()
    return _lib.lib()


@pytest.mark.parametrize("dt", [0, 1])
def test_lengths_at_the_end_of_an_int(L, dt):
    """Chunks are counted and tokens addressed past T, up to two chunks of 128."""
    from deltanet_sequence_mixing_b200 import _lib as E

    for fn in (L.gated_linear_attn_workspace_bytes, L.gated_linear_attn_bwd_workspace_bytes):
        for T in (INT_MAX, INT_MAX - 31, INT_MAX - 127, INT_MAX - 255):
            assert fn(1, 1, T, 64, 64, dt) == 0
        assert 256 <= fn(1, 1, INT_MAX - 256, 64, 64, dt) < 1 << 43
    A = 1 << 44
    at = [vp(A * (i + 1)) for i in range(12)]
    assert L.gated_linear_attn_fwd(*at[:7], 1, 1, INT_MAX, 64, 64, dt, at[7], 1 << 43, None) == E.DN_ERR_UNSUPPORTED
    assert L.gated_linear_attn_bwd(*at, 1, 1, INT_MAX, 64, 64, dt, vp(A * 13), 1 << 43, None) == E.DN_ERR_UNSUPPORTED
