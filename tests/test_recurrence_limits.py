"""The largest channel counts of the per-channel recurrence: refused before
anything is enqueued, in both directions.  Needs no GPU."""
import ctypes

import pytest

import linear_attention_feature_gb300 as la
from linear_attention_feature_gb300 import build as labuild

UNSUPPORTED = 2
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(6)]  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("C", [(1 << 29) + 1024, (1 << 31) - 32, (1 << 31) - 31, (1 << 31) - 1])
def test_too_many_channels(lib, C, dtype):
    # C + 31 passes 2^31 from 2^31 - 31 on
    assert lib.la_forward_recurrence(P[0], P[1], None, P[2], None, None, 1, 3, C, 0, 0, dtype, 0,
                                     None, 0, None) == UNSUPPORTED
    assert "too large" in lib.la_last_error().decode()
    assert lib.la_backward_recurrence(P[0], P[1], P[2], None, None, None, P[3], P[4], None, None,
                                      1, 3, C, 0, 0, dtype, 0, None, 0, None) == UNSUPPORTED
    assert "too large" in lib.la_last_error().decode()
