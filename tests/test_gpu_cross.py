"""Linear cross attention, forward, backward and single tokens, against the
definition in 64 bits and its automatic differentiation."""
import math

import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def phi(x, fmap):
    return x if fmap == "identity" else torch.where(x > 0, x + 1, torch.exp(torch.clamp(x, max=0)))


def slope(x, fmap):
    return torch.ones_like(x) if fmap == "identity" else torch.exp(torch.clamp(x, max=0))


def case(dtype, B, Hq, Hk, N, M, d, lengths, layout="tokens", seed=1, mean=0.3):
    """q, k, v, dout as 64-bit copies and as the library gets them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = DT[dtype]

    def rows(H, L, shift=0.0):
        if layout == "tokens":
            x = torch.randn(B, L, H * d, generator=g, device="cuda").add_(shift).mul_(0.7).to(t)
            return x.view(B, L, H, d).transpose(1, 2)
        if layout == "heads":
            return torch.randn(B, H, L, d, generator=g, device="cuda").add_(shift).mul_(0.7).to(t)
        x = torch.randn(B, H, L, d + 5, generator=g, device="cuda").add_(shift).mul_(0.7).to(t)
        return x[..., 1:d + 1]  # no alignment

    q, dout, k, v = rows(Hq, N), rows(Hq, N), rows(Hk, M), rows(Hk, M, mean)
    if lengths is not None:  # the padding is not finite
        for b, n in enumerate(lengths):
            k[b, :, max(n, 0):] = math.nan
            v[b, :, max(n, 0):] = -math.inf
    return q, k, v, dout


def plain(q, k, v, dout, lengths, fmap, norm):
    """The results and what the bounds go by: the same sums of absolute values."""
    B, Hq, N, d = q.shape
    Hk, M = k.shape[1], k.shape[2]
    G = Hq // Hk
    q, k, v, dy = (x.double() for x in (q, k, v, dout))
    keep = torch.ones(B, 1, M, 1, dtype=torch.float64, device="cuda")
    if lengths is not None:
        keep = (torch.arange(M, device="cuda") < ints(lengths)[:, None])[:, None, :, None].double()
        k = torch.where(keep > 0, k, torch.zeros_like(k))
        v = torch.where(keep > 0, v, torch.zeros_like(v))
    f, g = phi(q, fmap).reshape(B, Hk, G * N, d), phi(k, fmap) * keep
    dy = dy.reshape(B, Hk, G * N, d)
    r = {}

    def both(name, a, b, kind):
        """einsum of a, b; of their absolute values."""
        r[name] = torch.einsum(kind, a[0], b[0]), torch.einsum(kind, a[1], b[1])
        return r[name]

    A = lambda x: (x, x.abs())  # noqa: E731
    S = both("S", A(g), A(v), "bhma,bhmc->bhac")
    r["z"] = z = (g.sum(2), g.abs().sum(2))
    den = (f @ z[0][..., None])
    den1 = torch.where(den == 0, torch.ones_like(den), den)
    inv = torch.where(den == 0, torch.zeros_like(den), 1 / den1) if norm else torch.ones_like(den)
    num = both("num", A(f), S, "bhna,bhac->bhnc")
    r["out"] = num[0] * inv, num[1] * inv.abs()
    G_ = both("G", A(dy), S, "bhnc,bhac->bhna")
    zero = torch.zeros_like(den)
    t = ((f * G_[0]).sum(-1, keepdim=True) * inv, (f.abs() * G_[1]).sum(-1, keepdim=True) * inv.abs()) \
        if norm else (zero, zero)
    zz = z[0][:, :, None], z[1][:, :, None]
    s = slope(q, fmap).reshape(f.shape)
    r["dq"] = (G_[0] - t[0] * zz[0]) * inv * s, (G_[1] + t[1] * zz[1]) * inv.abs() * s
    psi = f * inv
    dS = both("dS", A(psi), A(dy), "bhna,bhnc->bhac")
    dz = -(psi * t[0]).sum(2), (psi.abs() * t[1]).sum(2)
    dg = torch.einsum("bhac,bhmc->bhma", dS[0], v) + dz[0][:, :, None], \
        torch.einsum("bhac,bhmc->bhma", dS[1], v.abs()) + dz[1][:, :, None]
    s = slope(k, fmap) * keep
    r["dk"] = dg[0] * s, dg[1] * s
    r["dv"] = torch.einsum("bhac,bhma->bhmc", dS[0], g), torch.einsum("bhac,bhma->bhmc", dS[1], g.abs())
    shape = (B, Hq, N, d)
    return {n: (x.reshape(shape), y.reshape(shape)) if n in ("out", "dq") else (x, y)
            for n, (x, y) in r.items()}


def check(name, got, ref, dtype, terms):
    """A product of sums is off by the number of its additions in one chain (`terms`: at
    most 1024 tokens and 64 parts, 256 features, and the same again where two sums
    follow) times u of the sums of absolute values; 4 u more per exponential.  The
    tensor cores may cut where they add (2 u).  With bf16: 2^-16 for a factor that is
    kept as two bf16 numbers (S), 2^-8 for one kept as one (phi(q) and S in out; r
    phi(q), phi(k) and dS in the gradients: two of them at a time, and the result)."""
    x, size = ref
    rel = 2 * terms * U
    if dtype == "bf16":
        rel += 2.0 ** -16 if name in ("S", "z") else 3 * 2.0 ** -8
    bound = rel * size + (2.0 ** -8 if dtype == "bf16" and name not in ("S", "z") else U) * x.abs()
    off = (got.double() - x).abs()
    assert bool((off <= bound + 1e-30).all()), (name, float((off / (bound + 1e-30)).max()))


CASES = [
    ("f32", 1, 1, 1, 1, 1, 1, None, "heads"),
    ("f32", 2, 4, 2, 5, 7, 8, [7, 3], "tokens"),
    ("f32", 2, 6, 2, 100, 333, 80, [333, 1], "tokens"),
    ("f32", 3, 2, 2, 65, 1500, 64, [0, 1500, 900], "heads"),
    ("f32", 1, 3, 1, 33, 129, 36, None, "apart"),
    ("f32", 1, 2, 1, 70, 200, 256, [131], "heads"),
    ("f32", 2, 1, 1, 300, 31, 61, None, "apart"),
    ("f32", 1, 1, 1, 3, 5000, 128, None, "tokens"),
    ("bf16", 1, 2, 2, 1, 1, 64, None, "heads"),
    ("bf16", 2, 4, 2, 129, 300, 64, [300, 127], "tokens"),
    ("bf16", 2, 4, 4, 448, 1500, 64, [1500, 750], "tokens"),
    ("bf16", 3, 8, 2, 130, 257, 128, [257, 0, 128], "tokens"),
    ("bf16", 1, 2, 1, 1000, 4096, 128, None, "heads"),
    ("bf16", 1, 16, 2, 64, 128, 128, [-3], "heads"),
    ("bf16", 2, 3, 1, 77, 99, 80, [50, 99], "tokens"),
    ("bf16", 2, 2, 2, 50, 140, 64, [140, 100], "apart"),
    ("bf16", 1, 2, 1, 40, 61, 37, None, "apart"),
    ("bf16", 1, 1, 1, 40, 300, 256, [299], "heads"),
    ("bf16", 2, 2, 1, 50, 70, 8, [70, 33], "tokens"),
    ("bf16", 1, 4, 2, 140, 130, 72, None, "tokens"),
    ("bf16", 2, 2, 2, 300, 700, 120, [64, 700], "heads"),
    ("f32", 1, 2, 1, 260, 300, 200, [290], "tokens"),
]


@pytest.mark.parametrize("fmap, norm", [("elu1", True), ("identity", False), ("elu1", False)])
@pytest.mark.parametrize("dtype, B, Hq, Hk, N, M, d, lengths, layout", CASES)
def test_forward_and_backward(dtype, B, Hq, Hk, N, M, d, lengths, layout, fmap, norm):
    q, k, v, dout = case(dtype, B, Hq, Hk, N, M, d, lengths, layout)
    ref = plain(q, k, v, dout, lengths, fmap, norm)
    form = {"feature_map": fmap, "normalise": norm}
    lens = None if lengths is None else ints(lengths)
    out, S, z = la.forward_cross(q, k, v, lens, **form)
    la.check_device_status()
    assert out.shape == q.shape and out.dtype == q.dtype and S.dtype == z.dtype == torch.float32
    check("S", S, ref["S"], dtype, 1100)
    check("z", z, ref["z"], dtype, 1100)
    check("out", out, ref["out"], dtype, 1100 + 600)
    dq, dk, dv = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    la.check_device_status()
    # S is itself off, then a sum over features, and for dk and dv over the queries
    check("dq", dq, ref["dq"], dtype, 1100 + 600)
    check("dk", dk, ref["dk"], dtype, 2 * 1100 + 900)
    check("dv", dv, ref["dv"], dtype, 2 * 1100 + 900)
    for b, n in enumerate(lengths or []):
        assert not bool(dk[b, :, max(n, 0):].any()) and not bool(dv[b, :, max(n, 0):].any())
        if n <= 0 and norm:
            assert not bool(out[b].any()) and not bool(dq[b].any())
    # the same bits again, on another stream, into strided tensors
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    to = [torch.zeros(x.shape[0], x.shape[2], x.shape[1], x.shape[3] + 1, dtype=x.dtype,
                      device="cuda")[..., 1:].transpose(1, 2) for x in (q, q, k, k)]
    torch.cuda.synchronize()
    out2, S2, z2 = la.forward_cross(q, k, v, lens, to[0], stream=s, **form)
    back = la.backward_cross(dout, q, k, v, S, z, lens, dq=to[1], dk=to[2], dv=to[3], stream=s,
                             **form)
    s.synchronize()
    aligned = layout != "apart" and d % 8 == 0 and d <= 128 and dtype == "bf16"
    if not aligned:  # one kernel whatever the outputs' strides are
        assert torch.equal(out2, out) and torch.equal(S2, S) and torch.equal(z2, z)
        assert all(torch.equal(a, b) for a, b in zip(back, (dq, dk, dv)))
    else:
        check("out", out2, ref["out"], dtype, 1700)
        for name, x in zip(("dq", "dk", "dv"), back):
            check(name, x, ref[name], dtype, 3100)
    again = la.forward_cross(q, k, v, lens, **form)
    assert all(torch.equal(a, b) for a, b in zip(again, (out, S, z)))
    again = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dv)))


@pytest.mark.parametrize("B, Hq, Hk, N, M, d, lengths, layout", [
    (1, 2, 1, 3000, 5000, 256, None, "tokens"), (2, 8, 1, 129, 257, 200, [257, 31], "tokens"),
    (2, 6, 3, 31, 1100, 129, [1100, 1], "apart"), (1, 2, 2, 128, 33, 3, None, "heads"),
    (2, 2, 1, 200, 700, 65, [700, 640], "tokens"), (1, 3, 1, 127, 300, 254, None, "heads"),
    (1, 4, 2, 300, 513, 128, [512], "apart"), (3, 2, 2, 40, 64, 66, [64, 0, 63], "tokens"),
])
def test_bf16_of_any_size(B, Hq, Hk, N, M, d, lengths, layout):
    # widths of 64, 128 and 256 columns, rows by 8 bytes, by words and by single values
    test_forward_and_backward("bf16", B, Hq, Hk, N, M, d, lengths, layout, "elu1", True)
    test_forward_and_backward("bf16", B, Hq, Hk, N, M, d, lengths, layout, "identity", False)


@pytest.mark.parametrize("d, bad", [(256, float("nan")), (61, float("inf")), (130, float("nan"))])
def test_padding_of_bf16_rows_of_any_size(d, bad):
    # what lies behind a sequence's length, and beside a row, reaches nothing
    lengths, N, M = [70, 5], 33, 100
    q, k, v, dout = case("bf16", 2, 2, 1, N, M, d, lengths, layout="apart")
    lens = ints(lengths)
    clean = la.forward_cross(q, k, v, lens)
    grads = la.backward_cross(dout, q, k, v, clean[1], clean[2], lens)
    for x in (k, v):
        for b, n in enumerate(lengths):
            x[b, :, n:] = bad
    for x in (q, k, v, dout):  # the rows' neighbours in memory
        whole = torch.as_strided(x, x.shape[:3] + (d + 5,), x.stride(), x.storage_offset() - 1)
        whole[..., 0] = bad
        whole[..., d + 1:] = bad
    got = la.forward_cross(q, k, v, lens)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    got = la.backward_cross(dout, q, k, v, clean[1], clean[2], lens)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("d", [61, 66, 132, 250])
def test_outputs_of_any_size_inside_larger_tensors(d):
    B, H, N, M = 2, 2, 130, 90
    q, k, v, dout = case("bf16", B, H, H, N, M, d, [90, 40])
    lens = ints([90, 40])
    want = la.forward_cross(q, k, v, lens)
    grads = la.backward_cross(dout, q, k, v, want[1], want[2], lens)

    def inside(L):
        whole = torch.full((B, L + 3, H, d + 6), 7.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[:, 1:L + 1, :, 3:d + 3].transpose(1, 2)

    whole, views = zip(*(inside(L) for L in (N, N, M, M)))
    la.forward_cross(q, k, v, lens, views[0])
    la.backward_cross(dout, q, k, v, want[1], want[2], lens, dq=views[1], dk=views[2], dv=views[3])
    for got, ref, w in zip(views, (want[0], *grads), whole):
        assert torch.equal(got, ref)
        got.fill_(7.0)
        assert bool((w == 7.0).all())


@pytest.mark.parametrize("d", [8, 64, 72, 128])
def test_outputs_inside_larger_tensors(d):
    # token-major outputs with other features beside them: the tiles' columns and rows
    # beyond the tensor leave those as they were
    B, H, N, M, pad = 2, 2, 130, 200, 16
    q, k, v, dout = case("bf16", B, H, H, N, M, d, [200, 90])
    lens = ints([200, 90])
    want = la.forward_cross(q, k, v, lens)
    grads = la.backward_cross(dout, q, k, v, want[1], want[2], lens)

    def inside(L):
        whole = torch.full((B, L + 3, H, d + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[:, 1:L + 1, :, 8:d + 8].transpose(1, 2)

    whole, views = zip(*(inside(L) for L in (N, N, M, M)))
    la.forward_cross(q, k, v, lens, views[0])
    la.backward_cross(dout, q, k, v, want[1], want[2], lens, dq=views[1], dk=views[2], dv=views[3])
    la.check_device_status()
    for got, ref, w in zip(views, (want[0], *grads), whole):
        assert torch.equal(got, ref)
        got.fill_(7.0)
        assert bool((w == 7.0).all())


@pytest.mark.parametrize("dtype, d", [("bf16", 64), ("bf16", 128), ("f32", 40)])
def test_empty_sides(dtype, d):
    q, k, v, dout = case(dtype, 2, 4, 2, 30, 50, d, None)
    none = k[:, :, :0]
    out, S, z = la.forward_cross(q, none, none)
    assert not bool(out.any()) and not bool(S.any()) and not bool(z.any())
    dq, dk, dv = la.backward_cross(dout, q, none, none, S, z)
    assert not bool(dq.any()) and dk.shape == none.shape
    out, S, z = la.forward_cross(q[:, :, :0], k, v)
    assert out.shape[2] == 0
    whole = la.forward_cross(q, k, v)
    assert torch.equal(S, whole[1]) and torch.equal(z, whole[2])
    dq, dk, dv = la.backward_cross(dout[:, :, :0], q[:, :, :0], k, v, S, z)
    assert not bool(dk.any()) and not bool(dv.any())


def test_gradients_are_automatic_differentiation_s_and_differences():
    q, k, v, dout = case("f32", 2, 4, 2, 9, 13, 12, [13, 6])
    lens = ints([13, 6])
    leaves = [torch.nan_to_num(x.double(), 0.0, posinf=0.0, neginf=0.0).requires_grad_()
              for x in (q, k, v)]
    keep = (torch.arange(13, device="cuda") < lens[:, None])[:, None, :, None]

    def loss(q, k, v):
        f = torch.where(q > 0, q + 1, torch.exp(q)).unflatten(1, (2, 2))
        g = torch.where(k > 0, k + 1, torch.exp(k)) * keep
        w = torch.einsum("bhgna,bhma->bhgnm", f, g)
        y = torch.einsum("bhgnm,bhmc->bhgnc", w / w.sum(-1, keepdim=True), v).flatten(1, 2)
        return (y * dout.double()).sum()

    loss(*leaves).backward()
    _, S, z = la.forward_cross(q, k, v, lens)
    got = la.backward_cross(dout, q, k, v, S, z, lens)
    for x, leaf in zip(got, leaves):  # sums of some ten terms
        assert float((x.double() - leaf.grad).abs().max()) <= 200 * U * (1 + float(leaf.grad.abs().max()))
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    with torch.no_grad():
        for i in range(3):  # along a random direction, central differences in 64 bits
            way = torch.randn(leaves[i].shape, generator=g, device="cuda", dtype=torch.float64)
            args = [x.detach() for x in leaves]
            h = 1e-5
            up, down = (loss(*[a + e * way if j == i else a for j, a in enumerate(args)])
                        for e in (h, -h))
            along = float((got[i].double() * way).sum())
            # a kink at 0 is passed by none of these values; h^2 of third derivatives
            assert abs(float(up - down) / (2 * h) - along) <= 1e-4 * (1 + abs(along))


def test_a_mean_far_from_zero_does_not_cost_the_gradient():
    # values around 8: df and dg are small differences of large sums, of which S as one
    # bf16 number would leave little
    q, k, v, dout = case("bf16", 1, 2, 1, 256, 2048, 64, None, mean=11.0)
    ref = plain(q, k, v, dout, None, "elu1", True)
    _, S, z = la.forward_cross(q, k, v)
    got = dict(zip(("dq", "dk", "dv"), la.backward_cross(dout, q, k, v, S, z)))
    for name, x in got.items():
        rel = float((x.double() - ref[name][0]).norm() / ref[name][0].norm())
        # S in two bf16 numbers: 2^-16 of sums that are 8 sqrt(2048) times what is left
        # of them; r phi(q), phi(k) and dS in one or two, and the result's rounding
        assert rel <= 2.0 ** -16 * 8 * 2048 ** 0.5 / 1.4 + 3 * 2.0 ** -8, (name, rel)


@pytest.mark.parametrize("dtype, d", [("bf16", 64), ("bf16", 256), ("f32", 40)])
def test_keys_without_queries(dtype, d):
    # no heads of queries, or no tokens of them: states all the same, gradients of 0
    for Hq, N in ((0, 5), (2, 0)):
        q, k, v, dout = case(dtype, 2, Hq, 2, N, 70, d, None, layout="heads")
        out, S, z = la.forward_cross(q, k, v)
        ref = plain(q.new_zeros(2, 2, 1, d), k, v, k.new_zeros(2, 2, 1, d), None, "elu1", True)
        check("S", S, ref["S"], dtype, 600)
        check("z", z, ref["z"], dtype, 600)
        assert out.shape == q.shape
        dq, dk, dv = la.backward_cross(dout, q, k, v, S, z)
        assert dq.shape == q.shape and not dk.any() and not dv.any()


# ---------------------------------------------------------------- single tokens

@pytest.mark.parametrize("fmap, norm", [("elu1", True), ("identity", False)])
@pytest.mark.parametrize("dtype, B, Hq, Hk, N, d, shift", [
    ("bf16", 2, 8, 8, 1, 128, 0), ("bf16", 1, 32, 8, 1, 128, 0), ("bf16", 3, 4, 2, 3, 64, 0),
    ("bf16", 2, 24, 2, 1, 80, 0), ("bf16", 1, 4, 1, 100, 64, 0), ("bf16", 2, 4, 1, 200, 128, 0),
    ("f32", 2, 2, 2, 1, 61, 0), ("f32", 1, 7, 7, 1, 256, 0), ("f32", 2, 3, 1, 5, 8, 0),
    ("f32", 1, 2, 1, 40, 33, 0), ("f32", 1, 4, 4, 1, 64, 1), ("bf16", 1, 1, 1, 1, 1, 0),
])
def test_decode_step(dtype, B, Hq, Hk, N, d, shift, fmap, norm):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    k, v = (torch.randn(B, Hk, 50, d, generator=g, device="cuda").double() for _ in range(2))
    f = phi(k, fmap)
    S = torch.empty(B * Hk * d * d + shift, device="cuda")[shift:].view(B, Hk, d, d)
    S.copy_(torch.einsum("bhma,bhmc->bhac", f, v))
    z = f.sum(2).float()
    q = torch.randn(B, N, Hq * d, generator=g, device="cuda").to(DT[dtype])
    q = q.view(B, N, Hq, d).transpose(1, 2)
    q = q[:, :, 0] if N == 1 else q
    got = la.decode_step_cross(S, z, q, feature_map=fmap, normalise=norm)
    x = phi((q if q.dim() == 4 else q[:, :, None]).double(), fmap).reshape(B, Hk, -1, d)
    num, size = x @ S.double(), x.abs() @ S.double().abs()
    if norm:
        den = x @ z.double()[..., None]
        num, size = num / den, size / den
    name = "out"
    check(name, got.reshape(num.shape), (num, size), dtype, 600)


@pytest.mark.parametrize("dtype, rows", [("bf16", 4), ("bf16", 5), ("bf16", 9), ("bf16", 17),
                                         ("f32", 24), ("f32", 25), ("f32", 65)])
@pytest.mark.parametrize("d", [64, 128, 100])
def test_steps_of_several_queries(dtype, rows, d):
    # either side of the sizes where queries go as tiles, shared heads and tokens alike
    for Hq, N in ((rows, 1), (1, rows)):
        q, k, v, _ = case(dtype, 2, Hq, 1, N, 90, d, [90, 0])
        _, S, z = la.forward_cross(q, k, v, ints([90, 0]))
        ref = plain(q, k, v, q, [90, 0], "elu1", True)
        got = la.decode_step_cross(S, z, q)
        check("out", got, ref["out"], dtype, 600)
        assert not got[1].any()


def test_decode_step_continues_the_forward():
    q, k, v, _ = case("bf16", 2, 4, 2, 60, 300, 128, [300, 99])
    out, S, z = la.forward_cross(q, k, v, ints([300, 99]))
    for i in (0, 17, 59):
        y = la.decode_step_cross(S, z, q[:, :, i])
        # phi(q) and S rounded to bf16 in the forward, neither in the step
        size = plain(q, k, v, q, [300, 99], "elu1", True)["out"][1][:, :, i]
        assert bool(((y.double() - out[:, :, i].double()).abs() <= 5 * 2.0 ** -8 * size).all())
    some = la.decode_step_cross(S, z, q)
    assert some.shape == q.shape


def test_captured_training_step():
    # forward and backward in one graph, replayed on new inputs, while eager calls go on
    q, k, v, dout = case("bf16", 2, 4, 2, 200, 300, 64, [300, 120], "heads")
    lens = ints([300, 120])

    def both():
        out, S, z = la.forward_cross(q, k, v, lens)
        return (out, S, z, *la.backward_cross(dout, q, k, v, S, z, lens))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = both()
    for seed in (5, 6):
        for x, y in zip((q, k, v, dout), case("bf16", 2, 4, 2, 200, 300, 64, [300, 120], "heads",
                                              seed)):
            x.copy_(y)
        graph.replay()
        mine = [x.clone() for x in res]
        assert all(torch.equal(a, b) for a, b in zip(mine, both()))


def test_a_workspace_that_cannot_be_had():
    lib = la.load_library()
    q, k, v, dout = case("f32", 1, 1, 1, 4, 5000, 32, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    lib.la_debug_fail_next_allocs(1)
    try:
        with pytest.raises(la.LinAttnError) as e:
            la.forward_cross(q, k, v, stream=s)
        assert e.value.status == 4
    finally:
        lib.la_debug_fail_next_allocs(0)
    out, S, z = la.forward_cross(q, k, v, stream=s)
    lib.la_debug_fail_next_allocs(1)
    try:
        with pytest.raises(la.LinAttnError):
            la.backward_cross(dout, q, k, v, S, z, stream=s)
    finally:
        lib.la_debug_fail_next_allocs(0)
    s.synchronize()
