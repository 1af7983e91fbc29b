"""Argument checks of the paged cache, its attention and linear cross attention.
Every call here returns during validation, so none needs a GPU."""
import array
import ctypes

import pytest

import linear_attention_feature_gb300 as la
from linear_attention_feature_gb300 import build as labuild

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]  # never dereferenced
ODD, HALF = ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def strides(*v):
    return (ctypes.c_longlong * len(v))(*v)


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_longlong * 3),
                ("vs", ctypes.c_longlong * 3), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_longlong), ("lengths", ctypes.c_void_p),
                ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int)]


def cache(k=P[0], v=P[1], ks=(2 * 16 * 64, 16 * 64, 64), vs=(2 * 16 * 64, 16 * 64, 64), table=P[2],
          table_stride=4, lengths=P[3], pages=9, page_size=16, max_pages=4):
    return Cache(k, v, ks, vs, table, table_stride, lengths, pages, page_size, max_pages)


def rope(values=(0.5,) * 8, rotary=None, interleaved=0, positions=0):
    f = array.array("d", values)
    r = la._ROPE.pack(f.buffer_info()[0], 2 * len(f) if rotary is None else rotary, interleaved,
                      positions, 8, 0, 0, 0)
    return r, f


BAD_CACHE = [
    (dict(k=None), INVALID, "null cache pointer"),
    (dict(v=None), INVALID, "null cache pointer"),
    (dict(k=ODD), INVALID, "unaligned cache"),
    (dict(v=P[0]), INVALID, "one buffer"),
    (dict(table=None), INVALID, "null table"),
    (dict(lengths=None), INVALID, "null table or lengths"),
    (dict(table=HALF), INVALID, "unaligned table"),
    (dict(lengths=HALF), INVALID, "unaligned table or lengths"),
    (dict(table_stride=-1), INVALID, "negative stride"),
    (dict(ks=(1024, -64, 64)), INVALID, "negative stride"),
    (dict(pages=-1), INVALID, "negative pages"),
    (dict(max_pages=-1), INVALID, "negative pages"),
    (dict(page_size=0), INVALID, "page_size"),
    (dict(page_size=-4), INVALID, "page_size"),
    (dict(page_size=1 << 20, max_pages=1 << 11), UNSUPPORTED, "2^30"),
]


def append(lib, q=P[4], k=P[5], v=P[6], qo=P[7], c="default", counts=None, st=None, rp=None, B=2,
           Hq=4, Hk=2, T=3, d=64, dtype=1):
    c = cache() if c == "default" else c
    return lib.la_append_cache(q, k, v, qo, ctypes.byref(c) if c is not None else None, counts, st,
                               rp[0] if rp is not None else None, B, Hq, Hk, T, d, dtype, None)


CONT_Q, CONT_K = (4 * 3 * 64, 3 * 64, 64), (2 * 3 * 64, 3 * 64, 64)


@pytest.mark.parametrize("kw, code, msg", [
    (dict(q=None), INVALID, "null tensor"),
    (dict(k=None), INVALID, "null tensor"),
    (dict(v=None), INVALID, "null tensor"),
    (dict(qo=None), INVALID, "null tensor"),
    (dict(c=None), INVALID, "null cache"),
    (dict(k=ODD), INVALID, "unaligned tensor"),
    (dict(qo=ODD), INVALID, "unaligned tensor"),
    (dict(counts=HALF), INVALID, "unaligned counts"),
    (dict(B=-1), INVALID, "negative"),
    (dict(Hq=-1), INVALID, "negative"),
    (dict(Hk=-1), INVALID, "negative"),
    (dict(T=-1), INVALID, "negative"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=257), INVALID, "d must"),
    (dict(dtype=2), INVALID, "dtype"),
    (dict(qo=P[5]), INVALID, "aliases"),
    (dict(qo=P[0]), INVALID, "aliases"),
    (dict(k=P[0]), INVALID, "the cache aliases"),
    (dict(q=P[1]), INVALID, "the cache aliases"),
    (dict(qo=P[4], st=strides(*CONT_Q, *CONT_K, *CONT_K, 768, 64, 256)), INVALID, "in place"),
    (dict(st=strides(*CONT_Q, *CONT_K, *CONT_K, 768, 192, 32)), INVALID, "overlap"),
    (dict(st=strides(*CONT_Q, 384, -1, 64, *CONT_K, *CONT_Q)), INVALID, "negative stride"),
    (dict(c=cache(ks=(0, 1024, 64))), INVALID, "cache rows overlap"),
    (dict(c=cache(vs=(2048, 1024, 32))), INVALID, "cache rows overlap"),
    (dict(rp=rope(rotary=66)), INVALID, "rotary_dim"),
    (dict(rp=rope(rotary=15)), INVALID, "rotary_dim"),
    (dict(rp=rope(rotary=-2)), INVALID, "rotary_dim"),
    (dict(rp=rope(interleaved=2)), INVALID, "interleaved"),
    (dict(rp=rope(positions=0x1000)), INVALID, "positions are those"),
    (dict(rp=rope(values=(0.5, float("nan")))), INVALID, "frequencies"),
    (dict(rp=rope(values=(0.5, 2e9))), INVALID, "frequencies"),
    *[(dict(c=cache(**kw)), code, msg) for kw, code, msg in BAD_CACHE],
])
def test_append_cache_refuses(lib, kw, code, msg):
    assert append(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def test_append_cache_empty(lib):
    nothing = dict(q=None, k=None, v=None, qo=None)
    assert append(lib, B=0, c=cache(lengths=None, table=None), **nothing) == OK
    assert append(lib, T=0, **nothing) == OK
    assert append(lib, Hq=0, Hk=0, **nothing) == OK


def attend(lib, q=P[4], out=P[5], c="default", st=None, scale=0.125, window=0, B=2, Hq=4, Hk=2,
           T=3, d=64, dtype=1, ws=P[8], ws_bytes=1 << 30):
    c = cache() if c == "default" else c
    return lib.la_decode_step_paged(q, out, ctypes.byref(c) if c is not None else None, st, scale,
                                    window, B, Hq, Hk, T, d, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, code, msg", [
    (dict(q=None), INVALID, "null tensor"),
    (dict(out=None), INVALID, "null tensor"),
    (dict(c=None), INVALID, "null cache"),
    (dict(q=ODD), INVALID, "unaligned tensor"),
    (dict(out=ODD), INVALID, "unaligned tensor"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(window=-1), INVALID, "window"),
    (dict(B=-1), INVALID, "negative"),
    (dict(T=-1), INVALID, "negative"),
    (dict(Hq=3), INVALID, "multiple"),
    (dict(Hk=0), INVALID, "multiple"),
    (dict(d=300), INVALID, "d must"),
    (dict(dtype=5), INVALID, "dtype"),
    (dict(out=P[4]), INVALID, "aliases"),
    (dict(out=P[1]), INVALID, "aliases"),
    (dict(st=strides(*CONT_Q, 0, 192, 64)), INVALID, "overlap"),
    (dict(st=strides(768, -192, 64, *CONT_Q)), INVALID, "negative stride"),
    (dict(T=(1 << 20) + 1), UNSUPPORTED, "too many"),
    *[(dict(c=cache(**kw)), code, msg) for kw, code, msg in BAD_CACHE],
])
def test_decode_step_paged_refuses(lib, kw, code, msg):
    assert attend(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def test_decode_step_paged_empty(lib):
    assert attend(lib, B=0, q=None, out=None) == OK
    assert attend(lib, T=0, q=None, out=None) == OK
    assert attend(lib, Hq=0, q=None, out=None) == OK


CQ, CK = (4 * 5 * 64, 5 * 64, 64), (2 * 7 * 64, 7 * 64, 64)


def fwd(lib, q=P[0], k=P[1], v=P[2], out=P[3], S=P[4], z=P[5], lengths=None, st=None, B=2, Hq=4,
        Hk=2, N=5, M=7, d=64, var=None, dtype=1, ws=P[8], ws_bytes=1 << 30):
    return lib.la_forward_cross(q, k, v, out, S, z, lengths, st, B, Hq, Hk, N, M, d, var, dtype,
                                ws, ws_bytes, None)


BAD_SHAPE = [
    (dict(B=-1), INVALID, "negative"),
    (dict(Hq=-4), INVALID, "negative"),
    (dict(N=-1), INVALID, "negative"),
    (dict(Hq=3), INVALID, "multiple"),
    (dict(Hk=0), INVALID, "multiple"),
    (dict(d=0), INVALID, "d must"),
    (dict(d=257), INVALID, "d must"),
    (dict(dtype=3), INVALID, "dtype"),
    (dict(var=ctypes.byref(la._Variant(2, 1))), INVALID, "variant"),
    (dict(var=ctypes.byref(la._Variant(0, 2))), INVALID, "variant"),
    (dict(S=None), INVALID, "null state"),
    (dict(z=None), INVALID, "null state"),
    (dict(S=HALF), INVALID, "unaligned state"),
    (dict(B=1 << 20, Hq=1 << 12, Hk=1 << 12), UNSUPPORTED, "too large"),
]


@pytest.mark.parametrize("kw, code, msg", BAD_SHAPE + [
    (dict(M=-1), INVALID, "negative"),
    (dict(q=None), INVALID, "null tensor"),
    (dict(k=None), INVALID, "null tensor"),
    (dict(v=ODD), INVALID, "unaligned tensor"),
    (dict(out=None), INVALID, "null tensor"),
    (dict(lengths=HALF), INVALID, "unaligned lengths"),
    (dict(out=P[0]), INVALID, "aliases"),
    (dict(out=P[2]), INVALID, "aliases"),
    (dict(S=P[1]), INVALID, "aliases"),
    (dict(S=P[5]), INVALID, "aliases"),
    (dict(st=strides(*CQ, *CK, *CK, *CQ[:2], 32)), INVALID, "overlap"),
    (dict(st=strides(*CQ, -1, *CK[1:], *CK, *CQ)), INVALID, "negative stride"),
    (dict(M=1 << 20, ws_bytes=16), INVALID, "workspace"),
    (dict(M=1 << 20, ws=ctypes.c_void_p(0x80008)), INVALID, "workspace"),
])
def test_forward_cross_refuses(lib, kw, code, msg):
    if "ws_bytes" in kw or "ws" in kw:  # the check comes after the device's SM count
        torch = pytest.importorskip("torch")
        if not torch.cuda.is_available():
            pytest.skip("needs a device")
    assert fwd(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def test_forward_cross_empty(lib):
    assert fwd(lib, B=0, q=None, k=None, v=None, out=None, S=None, z=None) == OK
    assert fwd(lib, Hq=0, Hk=0, q=None, k=None, v=None, out=None, S=None, z=None) == OK


def back(lib, dout=P[0], q=P[1], k=P[2], v=P[3], S=P[4], z=P[5], lengths=None, dq=P[6], dk=P[7],
         dv=P[9], st=None, B=2, Hq=4, Hk=2, N=5, M=7, d=64, var=None, dtype=1):
    return lib.la_backward_cross(dout, q, k, v, S, z, lengths, dq, dk, dv, st, B, Hq, Hk, N, M, d,
                                 var, dtype, P[10], 1 << 30, None)


@pytest.mark.parametrize("kw, code, msg", BAD_SHAPE + [
    (dict(dout=None), INVALID, "null tensor"),
    (dict(dv=None), INVALID, "null tensor"),
    (dict(q=ODD), INVALID, "unaligned tensor"),
    (dict(dq=P[0]), INVALID, "aliases"),
    (dict(dq=P[1]), INVALID, "aliases"),
    (dict(dk=P[9]), INVALID, "aliases"),
    (dict(dv=P[5]), INVALID, "aliases"),
    (dict(st=strides(*CQ, *CQ, *CK, *CK, *CQ, *CK, 0, 0, 64)), INVALID, "overlap"),
    (dict(st=strides(*CQ, *CQ, *CK, *CK, *CQ, *CK, 896, 448, -64)), INVALID, "negative stride"),
])
def test_backward_cross_refuses(lib, kw, code, msg):
    assert back(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def step(lib, S=P[0], z=P[1], q=P[2], out=P[3], st=None, B=2, Hq=4, Hk=2, N=1, d=64, var=None,
         dtype=1):
    return lib.la_decode_step_cross(S, z, q, out, st, B, Hq, Hk, N, d, var, dtype, None)


@pytest.mark.parametrize("kw, code, msg", BAD_SHAPE + [
    (dict(q=None), INVALID, "null tensor"),
    (dict(out=ODD), INVALID, "unaligned tensor"),
    (dict(out=P[0]), INVALID, "aliases"),
    (dict(out=P[2]), INVALID, "aliases"),
    (dict(st=strides(256, 64, 64, 256, 32, 64)), INVALID, "overlap"),
])
def test_decode_step_cross_refuses(lib, kw, code, msg):
    assert step(lib, **kw) == code
    assert msg in lib.la_last_error().decode()


def test_decode_step_cross_empty(lib):
    assert step(lib, N=0, q=None, out=None) == OK
    assert step(lib, Hq=0, q=None, out=None) == OK


def test_workspace_queries(lib):
    f = lib.la_decode_step_paged_workspace_bytes
    assert f(32, 8, 1, 128, 1) > 0 and f(32, 8, 4, 128, 1) > f(32, 8, 1, 128, 1)
    assert f(32, 0, 1, 128, 1) == f(30, 8, 1, 128, 1) == f(32, 8, 1, 300, 1) == 0
    assert f(32, 8, 1, 128, 7) == 0
    g = lib.la_cross_workspace_bytes
    assert g(1, 4, 2, 100, 100000, 64, 1, 0) > 0 and g(1, 4, 2, 100, 100, 64, 1, 1) > 0
    assert g(0, 4, 2, 5, 7, 64, 1, 0) == g(1, 3, 2, 5, 7, 64, 1, 0) == g(1, 4, 2, 5, 7, 0, 1, 1) == 0


def test_workspaces_stay_bounded(lib):
    # the parts of many states over long sequences: 256 MB and the states themselves
    g = lib.la_cross_workspace_bytes
    states = 1024 * (256 * 256 + 256) * 4
    assert g(64, 16, 16, 1, 1 << 20, 256, 0, 0) <= (1 << 28) + 2 * states
    assert g(64, 16, 16, 1 << 16, 1, 256, 0, 1) <= (1 << 28) + 3 * states + 8 * 1024 * (1 << 16)
    f = lib.la_decode_step_paged_workspace_bytes
    assert f(128, 1, 1 << 20, 256, 1) == f(16, 1, 1, 256, 1)  # whatever the queries are


def test_the_packed_cache_is_the_struct():
    assert la._CACHE.size <= ctypes.sizeof(Cache)  # the struct is padded behind its last member
    packed = la._CACHE.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14)
    whole = bytes(Cache(1, 2, (3, 4, 5), (6, 7, 8), 9, 10, 11, 12, 13, 14))
    assert packed == whole[:la._CACHE.size] and not any(whole[la._CACHE.size:])


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    k, pool = torch.zeros(1, 2, 3, 4), torch.zeros(5, 2, 8, 4)
    table, lengths = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        la.append_cache(k, k, pool, pool, table, lengths)
    with pytest.raises(ValueError, match="share one shape"):
        la.append_cache(k, k[..., :2], pool, pool, table, lengths)
    with pytest.raises(ValueError, match="number of heads"):
        la.append_cache(k, k, pool, pool, table, lengths, q=k[:, :, :2])
    with pytest.raises(ValueError, match="without q"):
        la.append_cache(k, k, pool, pool, table, lengths, q_out=k)
    with pytest.raises(ValueError, match="CUDA"):
        la.decode_step_paged(k, pool, pool, table, lengths)
    with pytest.raises(ValueError, match="one token"):
        la.decode_step_paged(k[0, 0], pool, pool, table, lengths)
    with pytest.raises(ValueError, match="page_size"):
        la.decode_step_paged(k, pool[0], pool[0], table, lengths)
    for window in (-1, 1 << 31, 1 << 32):
        with pytest.raises(ValueError, match="window"):
            la.decode_step_paged(k, pool, pool, table, lengths, window=window)
    with pytest.raises(ValueError, match="CUDA"):
        la.forward_cross(k, k, k)
    with pytest.raises(ValueError, match="heads and tokens"):
        la.forward_cross(k, k[..., :2], k[..., :2])
    with pytest.raises(ValueError, match="must be"):
        la.forward_cross(k[0], k, k)
    S, z = torch.zeros(1, 2, 4, 4), torch.zeros(1, 2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        la.backward_cross(k, k, k, k, S, z)
    with pytest.raises(ValueError, match="shape"):
        la.backward_cross(k[:, :1], k, k, k, S, z)
    with pytest.raises(ValueError, match="CUDA"):
        la.decode_step_cross(S, z, k)
    with pytest.raises(ValueError, match="S must be"):
        la.decode_step_cross(S[0], z, k)


def test_binding_checks_the_small_tensors():
    # what the calls check of tables, lengths and caches, here on the CPU (device -1)
    torch = pytest.importorskip("torch")
    pool = torch.zeros(5, 2, 8, 4)
    table, lengths = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    packed = la._cache(pool, pool, table, lengths, 3, 2, 4, torch.float32, -1)
    assert len(packed) == la._CACHE.size
    for bad, err, msg in [
        (dict(k_cache=pool[:, :1]), ValueError, "pages, Hk"),
        (dict(v_cache=pool[..., :2]), ValueError, "pages, Hk"),
        (dict(v_cache=pool.bfloat16()), TypeError, "dtype"),
        (dict(k_cache=pool.transpose(2, 3).contiguous().transpose(2, 3)), ValueError, "contiguous"),
        (dict(page_table=table.long()), TypeError, "page_table must be int32"),
        (dict(page_table=table[:2]), ValueError, "page_table must have"),
        (dict(page_table=table.t().contiguous().t()), ValueError, "contiguous"),
        (dict(lengths=lengths[:2]), ValueError, "lengths must have"),
        (dict(lengths=lengths.float()), TypeError, "lengths must be int32"),
        (dict(lengths=torch.zeros(6, dtype=torch.int32)[::2]), ValueError, "contiguous"),
    ]:
        kw = dict(k_cache=pool, v_cache=pool, page_table=table, lengths=lengths, B=3, Hk=2, d=4,
                  dtype=torch.float32, index=-1)
        kw.update(bad)
        with pytest.raises(err, match=msg):
            la._cache(**kw)
