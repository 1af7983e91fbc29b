"""Argument checks of the query/key norm and rotation and of the per-channel
recurrence.  Every call here returns during validation, so none needs a GPU."""
import array
import ctypes

import pytest

import linear_attention_feature_gb300 as la
from linear_attention_feature_gb300 import build as labuild

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]  # never dereferenced
ODD = ctypes.c_void_p(0x10001)
BAD_FREQ = {"nan": float("nan"), "inf": float("inf"), "big": 2e9}


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def strides(*v):
    return (ctypes.c_longlong * len(v))(*v)


class Rope(ctypes.Structure):
    _fields_ = [("frequencies", ctypes.c_void_p), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("positions", ctypes.c_void_p),
                ("position_bytes", ctypes.c_int),
                ("position_stride_b", ctypes.c_longlong),
                ("position_stride_n", ctypes.c_longlong), ("offset", ctypes.c_longlong)]


def rope(n=32, rotary=None, interleaved=0, positions=None, nbytes=8, sb=0, sn=0, freq=None,
         values=None):
    f = array.array("d", values if values is not None else [0.5] * n)
    r = Rope(f.buffer_info()[0] if freq is None else freq, 2 * n if rotary is None else rotary,
             interleaved, positions, nbytes, sb, sn, 0)
    r.keep = f
    return r


def qk(lib, q=P[0], k=P[1], qo=P[2], ko=P[3], st=None, wq=None, wk=None, norm=1, eps=1e-6,
       rp="default", B=1, Hq=2, Hk=2, N=3, d=64, dtype=1, wdtype=0):
    rp = rope() if rp == "default" else rp
    return lib.la_qk_norm_rope(q, k, qo, ko, st, wq, wk, norm, eps,
                               ctypes.byref(rp) if rp is not None else None, B, Hq, Hk, N, d,
                               dtype, wdtype, None)


CONT = (2 * 3 * 64, 3 * 64, 64)


@pytest.mark.parametrize("kw, code, msg", [
    (dict(q=None), INVALID, "null"),
    (dict(ko=None), INVALID, "null"),
    (dict(B=-1), INVALID, "negative"),
    (dict(Hk=-1), INVALID, "negative"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=257), INVALID, "d must"),
    (dict(dtype=2), INVALID, "dtype"),
    (dict(wq=P[4], wdtype=5), INVALID, "weight dtype"),
    (dict(norm=2), INVALID, "norm"),
    (dict(eps=0.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(eps=float("inf")), INVALID, "eps"),
    (dict(norm=0, wq=P[4]), INVALID, "weights need norm"),
    (dict(q=ODD), INVALID, "unaligned"),
    (dict(ko=ODD), INVALID, "unaligned"),
    (dict(wq=ctypes.c_void_p(0x10002)), INVALID, "unaligned"),
    (dict(qo=P[1]), INVALID, "aliases"),
    (dict(ko=P[0]), INVALID, "aliases"),
    (dict(qo=P[3]), INVALID, "aliases"),
    (dict(qo=P[0], st=strides(*(128, 64, 128), *CONT, *CONT, *CONT)), INVALID, "in place"),
    (dict(st=strides(*CONT, *CONT, *(384, 192, 32), *CONT)), INVALID, "overlap"),
    (dict(st=strides(*CONT, *CONT, *(0, 0, 64), *CONT)), INVALID, "overlap"),
    (dict(st=strides(*(384, -192, 64), *CONT, *CONT, *CONT)), INVALID, "negative stride"),
    (dict(rp=rope(n=32, rotary=66)), INVALID, "rotary_dim"),
    (dict(rp=rope(n=32, rotary=63)), INVALID, "rotary_dim"),
    (dict(rp=rope(n=32, rotary=-2)), INVALID, "rotary_dim"),
    (dict(rp=rope(interleaved=2)), INVALID, "interleaved"),
    (dict(rp=rope(freq=0)), INVALID, "null frequencies"),
    (dict(rp=rope(positions=0x1000, nbytes=2)), INVALID, "position_bytes"),
    (dict(rp=rope(positions=0x1004, nbytes=8)), INVALID, "unaligned"),
    (dict(rp=rope(positions=0x1000, sn=-1)), INVALID, "position stride"),
    (dict(rp=rope(values=[0.1] * 31 + [BAD_FREQ["nan"]])), INVALID, "frequencies"),
    (dict(rp=rope(values=[0.1] * 31 + [BAD_FREQ["inf"]])), INVALID, "frequencies"),
    (dict(rp=rope(values=[0.1] * 31 + [BAD_FREQ["big"]])), INVALID, "frequencies"),
])
def test_qk_norm_rope_refuses(lib, kw, code, msg):
    assert qk(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def test_qk_norm_rope_empty_problems(lib):
    nothing = dict(q=None, k=None, qo=None, ko=None)
    assert qk(lib, B=0, **nothing) == OK
    assert qk(lib, N=0, **nothing) == OK
    assert qk(lib, Hq=0, Hk=0, **nothing) == OK


def back(lib, gq=P[0], gk=P[1], q=P[2], k=P[3], dq=P[4], dk=P[5], dwq=None, dwk=None, st=None,
         norm=1, B=1, Hq=2, Hk=2, N=3, d=64, ws=None, ws_bytes=0):
    return lib.la_backward_qk_norm_rope(gq, gk, q, k, dq, dk, dwq, dwk, st, None, None, norm, 1e-6,
                                        None, B, Hq, Hk, N, d, 1, 0, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, msg", [
    (dict(gq=None), "null"),
    (dict(q=None), "null"),
    (dict(dk=None), "null"),
    (dict(gq=ODD), "unaligned"),
    (dict(dk=ODD), "unaligned"),
    (dict(dwq=ctypes.c_void_p(0x10002)), "unaligned"),
    (dict(dq=P[2]), "aliases"),
    (dict(dk=P[2]), "aliases"),
    (dict(dq=P[1]), "aliases"),
    (dict(dq=P[5]), "aliases"),
    (dict(dwq=P[6], dwk=P[6]), "one buffer"),
    (dict(norm=0, dwq=P[6]), "need norm"),
    (dict(dq=P[0], st=strides(*(128, 64, 128), *(CONT * 5))), "in place"),
    (dict(st=strides(*(CONT * 4), *(0, 0, 0), *CONT)), "overlap"),
])
def test_backward_qk_norm_rope_refuses(lib, kw, msg):
    assert back(lib, **kw) == INVALID
    assert msg in lib.la_last_error().decode()


def test_backward_qk_norm_rope_without_rows_or_gradients(lib):
    assert back(lib, B=0, gq=None, gk=None, q=None, k=None, dq=None, dk=None) == OK


def rec(lib, x=P[0], z=P[1], h0=None, out=P[2], hl=None, st=None, B=2, N=3, C=8, gate=0, comp=0,
        dtype=1, gdtype=0):
    return lib.la_forward_recurrence(x, z, h0, out, hl, st, B, N, C, gate, comp, dtype, gdtype,
                                     None, 0, None)


@pytest.mark.parametrize("kw, code, msg", [
    (dict(x=None), INVALID, "null"),
    (dict(z=None), INVALID, "null"),
    (dict(out=None), INVALID, "null"),
    (dict(B=-1), INVALID, "negative"),
    (dict(C=-1), INVALID, "negative"),
    (dict(gate=3), INVALID, "gate"),
    (dict(gate=-1), INVALID, "gate"),
    (dict(comp=2), INVALID, "complement"),
    (dict(dtype=9), INVALID, "dtype"),
    (dict(dtype=0, gdtype=1), INVALID, "gate_dtype"),
    (dict(gdtype=4), INVALID, "gate_dtype"),
    (dict(x=ODD), INVALID, "unaligned"),
    (dict(z=ctypes.c_void_p(0x10002)), INVALID, "unaligned"),
    (dict(h0=ctypes.c_void_p(0x10002)), INVALID, "unaligned"),
    (dict(out=P[1]), INVALID, "aliases"),
    (dict(out=P[0], st=strides(48, 16, 24, 8, 24, 8)), INVALID, "in place"),
    (dict(st=strides(24, 8, 24, 8, 24, 7)), INVALID, "overlap"),
    (dict(st=strides(24, 8, 24, 8, 23, 8)), INVALID, "overlap"),
    (dict(st=strides(24, 8, 24, 8, 0, 8)), INVALID, "overlap"),
    (dict(st=strides(24, -8, 24, 8, 24, 8)), INVALID, "negative stride"),
    (dict(B=1 << 30, C=1 << 10), UNSUPPORTED, "too large"),
])
def test_forward_recurrence_refuses(lib, kw, code, msg):
    assert rec(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def test_recurrence_empty_problems(lib):
    assert rec(lib, B=0, x=None, z=None, out=None) == OK
    assert rec(lib, C=0, x=None, z=None, out=None) == OK
    assert rec(lib, N=0, x=None, z=None, out=None) == OK  # no h_last to fill


def rec_back(lib, dout=P[0], z=P[1], out=P[2], x=P[3], dx=P[4], dz=P[5], st=None, comp=1, N=3,
             gdtype=1):
    return lib.la_backward_recurrence(dout, z, out, x, None, None, dx, dz, None, st, 2, N, 8, 0,
                                      comp, 1, gdtype, None, 0, None)


@pytest.mark.parametrize("kw, msg", [
    (dict(dout=None), "null"),
    (dict(out=None), "null"),
    (dict(x=None), "null"),
    (dict(dz=None), "null"),
    (dict(dout=ODD), "unaligned"),
    (dict(dz=ODD), "unaligned"),
    (dict(dx=P[1]), "aliases"),
    (dict(dx=P[2]), "aliases"),
    (dict(dx=P[3]), "aliases"),
    (dict(dx=P[5]), "aliases"),
    (dict(dz=P[0]), "aliases"),
    (dict(dz=P[1]), "aliases"),
    (dict(dz=P[2]), "aliases"),
    (dict(dz=P[3]), "aliases"),
    (dict(dx=P[0], st=strides(48, 16, *((24, 8) * 5))), "in place"),
    (dict(st=strides(*((24, 8) * 5), 24, 0)), "overlap"),
    (dict(gdtype=7), "gate_dtype"),
])
def test_backward_recurrence_refuses(lib, kw, msg):
    assert rec_back(lib, **kw) == INVALID
    assert msg in lib.la_last_error().decode()


def test_backward_recurrence_empty(lib):
    assert rec_back(lib, N=0) == OK


def step(lib, h=P[0], ho=P[1], x=P[2], z=P[3], out=P[4], st=None, B=2, C=8, gate=0, comp=0):
    return lib.la_decode_step_recurrence(h, ho, x, z, out, st, B, C, gate, comp, 1, 1, None)


@pytest.mark.parametrize("kw, msg", [
    (dict(h=None), "null"),
    (dict(ho=None), "null"),
    (dict(out=None), "null"),
    (dict(h=ctypes.c_void_p(0x10002)), "unaligned"),
    (dict(x=ODD), "unaligned"),
    (dict(B=-2), "negative"),
    (dict(gate=5), "gate"),
    (dict(comp=-1), "complement"),
    (dict(out=P[0]), "aliases"),
    (dict(out=P[1]), "aliases"),
    (dict(out=P[3]), "aliases"),
    (dict(out=P[2], st=strides(16, 8, 8)), "in place"),
    (dict(st=strides(8, 8, 7)), "overlap"),
    (dict(st=strides(-8, 8, 8)), "negative stride"),
])
def test_decode_step_recurrence_refuses(lib, kw, msg):
    assert step(lib, **kw) == INVALID
    assert msg in lib.la_last_error().decode()


def test_the_packed_rotation_is_the_struct():
    assert la._ROPE.size == ctypes.sizeof(Rope)
    packed = la._ROPE.pack(1, 2, True, 3, 4, 5, 6, 7)
    assert packed == bytes(Rope(1, 2, 1, 3, 4, 5, 6, 7))


def test_workspace_query(lib):
    f = lib.la_backward_qk_norm_rope_workspace_bytes
    assert f(0) == 0 and f(257) == 0
    assert f(128) == 2 * f(64) > 0
    g = lib.la_recurrence_workspace_bytes
    assert g(0, 8, 1) == g(8, 0, 1) == g(1, 8, 7) == 0
    assert g(1, 64, 1) > 0 and g(1, 64, 0) > 0
    assert g(256, 4096, 1) == 0  # enough channels: nothing is cut into pieces
    # what the binding goes by: none above 1024 channels, and bytes by feature
    assert g(1, 1025, 1) == g(1, 1025, 0) == g(205, 5, 1) == g(205, 5, 0) == 0
    assert all(f(d) == d * f(1) for d in (1, 7, 64, 256))


def test_rope_frequencies():
    f = la.rope_frequencies(8, base=100.0)
    assert list(f) == [100.0 ** (-i / 4) for i in range(4)]
    assert len(la.rope_frequencies(0)) == 0
    with pytest.raises(ValueError, match="even"):
        la.rope_frequencies(7)


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        la.qk_norm_rope(q, q)
    with pytest.raises(ValueError, match="CUDA"):
        la.backward_qk_norm_rope(q, q, q, q)
    with pytest.raises(ValueError, match="number of heads"):
        la.qk_norm_rope(q, q[:, :, :2])
    with pytest.raises(ValueError, match="one token"):
        la.qk_norm_rope(q[0, 0], q[0, 0])
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        la.forward_recurrence(x, x)
    with pytest.raises(ValueError, match="share one shape"):
        la.forward_recurrence(x, x[:1])
    with pytest.raises(ValueError, match="gate must be"):
        la.forward_recurrence(x, x, gate="sigmoid")
    with pytest.raises(ValueError, match="x is needed"):
        la.backward_recurrence(x, x, x, complement=True)
    with pytest.raises(ValueError, match="CUDA"):
        la.decode_step_recurrence(x[:, 0], x[:, 0], x[:, 0])
