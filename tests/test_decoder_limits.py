"""Sizes that the kernels' 32-bit counts do not hold are refused, and the largest that they
hold are not.  Every call returns during validation, so none needs a GPU."""
import ctypes

import pytest

import linear_attention_feature_gb300 as la
from linear_attention_feature_gb300 import build as labuild

UNSUPPORTED, INVALID = 2, 1
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]  # never dereferenced
MOST = (1 << 31) - 256  # tokens: tiles and rows of a last tile are counted past them


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("N, M", [(MOST + 1, 7), (7, MOST + 1), ((1 << 31) - 1, 7), (7, (1 << 31) - 1)])
def test_tokens_beyond_a_count(lib, N, M, dtype):
    ws = (P[8], 1 << 40, None)
    assert lib.la_forward_cross(*P[:6], None, None, 1, 1, 1, N, M, 1, None, dtype, *ws) == UNSUPPORTED
    assert "too large" in lib.la_last_error().decode()
    assert lib.la_backward_cross(*P[:6], None, *P[6:8], P[9], None, 1, 1, 1, N, M, 1, None, dtype,
                                 P[10], 1 << 40, None) == UNSUPPORTED
    assert "too large" in lib.la_last_error().decode()
    if N > M:
        assert lib.la_decode_step_cross(*P[:4], None, 1, 1, 1, N, 1, None, dtype, None) == UNSUPPORTED
        assert "too large" in lib.la_last_error().decode()


def test_the_most_tokens_are_not_refused(lib):
    # (they get as far as the missing tensor)
    assert lib.la_forward_cross(None, *P[1:6], None, None, 1, 1, 1, MOST, MOST, 1, None, 1, P[8],
                                1 << 40, None) == INVALID
    assert "null tensor" in lib.la_last_error().decode()


@pytest.mark.parametrize("dtype, N", [(0, 2), (0, 24), (1, 4)])
def test_more_tokens_of_one_state_than_a_count(lib, dtype, N):
    Hq = (1 << 31) // N + 1
    assert lib.la_decode_step_cross(*P[:4], None, 1, Hq, 1, N, 1, None, dtype, None) == UNSUPPORTED


def test_more_tiles_of_queries_than_a_count(lib):
    class Cache(ctypes.Structure):
        _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_longlong * 3),
                    ("vs", ctypes.c_longlong * 3), ("table", ctypes.c_void_p),
                    ("table_stride", ctypes.c_longlong), ("lengths", ctypes.c_void_p),
                    ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int)]

    Hk, T = 1 << 11, 1 << 20
    c = Cache(P[0], P[1], (Hk, 1, 1), (Hk, 1, 1), P[2], 1, P[3], 1, 1, 1)
    # 2^24 queries of each of 2048 heads, 16 a tile: 2^31 tiles of a sequence
    assert lib.la_decode_step_paged(P[4], P[5], ctypes.byref(c), None, 1.0, 0, 1, 16 * Hk, Hk, T, 1, 1,
                                    P[8], 1 << 40, None) == UNSUPPORTED
    assert "too many" in lib.la_last_error().decode()


@pytest.mark.parametrize("Hq, Hk", [((1 << 31) - 1, 1), (0, 1 << 30), ((1 << 31) - 4096, 0)])
def test_more_heads_than_a_count(lib, Hq, Hk):
    # (a thread takes its token's heads in strides, and stops behind the last of them)
    class Cache(ctypes.Structure):
        _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_longlong * 3),
                    ("vs", ctypes.c_longlong * 3), ("table", ctypes.c_void_p),
                    ("table_stride", ctypes.c_longlong), ("lengths", ctypes.c_void_p),
                    ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int)]

    c = Cache(P[0], P[1], (Hk, 1, 1), (Hk, 1, 1), P[2], 1, P[3], 1, 1, 1)
    assert lib.la_append_cache(P[4], P[5], P[6], P[7], ctypes.byref(c), None, None, None, 1, Hq, Hk, 1,
                               1, 1, None) == UNSUPPORTED
    assert "too many heads" in lib.la_last_error().decode()
