"""States written over a tensor that other threads still read are refused before
anything is enqueued.  Needs no GPU."""
import ctypes

import pytest

import linear_attention_feature_gb300 as la
from linear_attention_feature_gb300 import build as labuild

INVALID = 1
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def refused(lib, status):
    return status == INVALID and "aliases" in lib.la_last_error().decode()


@pytest.mark.parametrize("which", [0, 1, 2])
def test_last_state_over_the_sequence(lib, which):
    x, z, out = P[:3]
    assert refused(lib, lib.la_forward_recurrence(x, z, None, out, P[which], None, 1, 5, 8, 0, 0,
                                                  0, 0, None, 0, None))


@pytest.mark.parametrize("which", range(6))
def test_first_states_gradient_over_the_sequence(lib, which):
    dout, z, out, x, dx, dz = P[:6]
    assert refused(lib, lib.la_backward_recurrence(dout, z, out, x, None, None, dx, dz, P[which],
                                                   None, 1, 5, 8, 0, 1, 0, 0, None, 0, None))


@pytest.mark.parametrize("dtype, gdtype, strides, which", [
    (1, 1, None, 0), (1, 1, None, 1), (1, 0, None, 0),  # 16-bit values under an fp32 state
    (0, 0, (9, 8, 8), 0), (0, 0, (8, 9, 8), 1), (1, 0, (8, 16, 8), 1)])
def test_new_state_over_an_input(lib, dtype, gdtype, strides, which):
    st = (ctypes.c_longlong * 3)(*strides) if strides else None
    x, z, h, out = P[:4]
    assert refused(lib, lib.la_decode_step_recurrence(h, P[which], x, z, out, st, 2, 8, 0, 0,
                                                      dtype, gdtype, None))
