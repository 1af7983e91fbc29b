"""qk_norm_rope and its gradient against a plain implementation in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32) and half = half a step of the
output's type, relative:
- forward: r = 1/sqrt(mean + eps) carries the rounding of a sum of at most 128
  pairs as a binary tree (9 u, halved by the root), the mean and the root (4 u);
  w n adds 2 u; cos and sin are off by at most 4 u for fp32 rows (the angle's
  conversion to fp32 is 1.6 u, the function 2 u) and 12 u for bf16 ones (2^-21.2
  of the special function unit); the products and their sum 3 u.  That is below
  40 u (|u1| + |u2|), plus half |y|.
- dx: the turned-back gradient is off by 16 u (|dy1| + |dy2|) =: 16 u G; dx is
  r (w g - n m) with m = mean(n w g) off by at most 38 u mean(|n| |w| G), n by
  10 u and r by 9 u, so 64 u r (|w| G + |n| mean(|n| |w| G)), plus half |dx|.
- dw: a sum over rows whose longest chain of additions is the rows of one
  thread, the threads of a block and the blocks, below 1500 at these sizes:
  (1500 + 64) u sum(G |n|)."""
import math

import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def half(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


# ---- the plain implementation, in 64 bits on the CPU; rows [B, H, N, d]

def pairs_of(d, R, interleaved):
    i = torch.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def turn(u, pos, freq, interleaved, sign=1.0):
    R = 2 * len(freq)
    if R == 0:
        return u.clone()
    a, b = pairs_of(u.shape[-1], R, interleaved)
    t = pos.double()[..., None] * torch.tensor(list(freq), dtype=torch.float64)
    t = t[:, None]                                   # [B, 1, N, R/2]
    c, s = torch.cos(t), torch.sin(t) * sign
    y = u.clone()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., b] * c + u[..., a] * s
    return y


def plain(x, w, pos, freq, interleaved, norm=True, eps=EPS):
    v = x.double()
    if norm:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        if w is not None:
            v = v * w.double()
    return turn(v, pos, freq, interleaved)


def pair_sum(m, freq, interleaved):
    """|m1| + |m2| at both features of each pair, |m| elsewhere."""
    R = 2 * len(freq)
    m = m.abs()
    if R == 0:
        return m
    a, b = pairs_of(m.shape[-1], R, interleaved)
    y = m.clone()
    y[..., a] = y[..., b] = m[..., a] + m[..., b]
    return y


def check_forward(y, x, w, pos, freq, interleaved, norm=True, eps=EPS):
    ref = plain(x.cpu(), None if w is None else w.cpu(), pos.cpu(), freq, interleaved, norm, eps)
    mag = pair_sum(turn(ref, pos.cpu(), freq, interleaved, -1.0), freq, interleaved)
    tol = 40 * U * mag + half(y.dtype) * ref.abs() * (1 + 1e-3) + 1e-37
    err = (y.cpu().double() - ref).abs()
    assert torch.all(err <= tol), float((err / tol).max())


def plain_back(dy, x, w, pos, freq, interleaved, norm=True):
    g = turn(dy.double(), pos, freq, interleaved, -1.0)
    if not norm:
        return g, None
    v = x.double()
    d = v.shape[-1]
    size = torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    n = v / size
    dw = (g * n).sum((0, 1, 2))
    g = g * (w.double() if w is not None else 1.0)
    return (g - n * (g * n).sum(-1, keepdim=True) / d) / size, dw


def check_backward(dx, dw, dy, x, w, pos, freq, interleaved, norm=True):
    dy, x, pos = dy.cpu(), x.cpu(), pos.cpu()
    w = None if w is None else w.cpu()
    ref, ref_w = plain_back(dy, x, w, pos, freq, interleaved, norm)
    G = pair_sum(dy.double(), freq, interleaved)
    if norm:
        v = x.double()
        size = torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
        n = (v / size).abs()
        wa = w.double().abs() if w is not None else torch.ones(x.shape[-1], dtype=torch.float64)
        mag = (wa * G + n * (n * wa * G).mean(-1, keepdim=True)) / size
    else:
        mag = G
    tol = 64 * U * mag + half(dx.dtype) * ref.abs() * (1 + 1e-3) + 1e-37
    err = (dx.cpu().double() - ref).abs()
    assert torch.all(err <= tol), float((err / tol).max())
    if dw is not None:
        tol = 1564 * U * (G * n).sum((0, 1, 2)) + 1e-37
        err = (dw.cpu().double() - ref_w).abs()
        assert torch.all(err <= tol), float((err / tol).max())


def rows(B, H, N, d, dtype, seed, layout="token"):
    """[B, H, N, d] values: a slice of a token-major projection, or contiguous."""
    g = torch.Generator().manual_seed(seed)
    if layout == "token":
        buf = torch.randn(B, N, (H + 1) * d, generator=g).to(DT[dtype]).cuda()
        return buf[..., :H * d].view(B, N, H, d).transpose(1, 2)
    return torch.randn(B, H, N, d, generator=g).to(DT[dtype]).cuda()


def weights(d, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda(),
            (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda())


def token_positions(B, N, offset=0):
    return (offset + torch.arange(N)).expand(B, N)


SHAPES = [  # B, Hq, Hk, N, d, R
    (1, 1, 1, 1, 1, 0),
    (1, 1, 1, 1, 2, 2),
    (2, 3, 1, 5, 4, 4),
    (1, 2, 2, 7, 37, 10),
    (2, 6, 2, 33, 80, 40),
    (3, 4, 4, 65, 64, 64),
    (2, 5, 3, 129, 128, 128),
    (1, 2, 2, 31, 96, 32),
    (1, 3, 3, 17, 100, 100),
    (2, 2, 1, 9, 256, 256),
    (1, 2, 2, 6, 255, 254),
    (1, 1, 2, 1000, 48, 16),
    (4, 16, 16, 70, 72, 24),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, interleaved, dtype):
    B, Hq, Hk, N, d, R = shape
    q = rows(B, Hq, N, d, dtype, 1)
    k = rows(B, Hk, N, d, dtype, 2, "head")
    wq, wk = weights(d, 3)
    freq = la.rope_frequencies(R)
    pos = token_positions(B, N, 12345)
    yq, yk = la.qk_norm_rope(q, k, wq, wk, freq, offset=12345, interleaved=interleaved)
    assert yq.is_contiguous() and yk.is_contiguous()
    check_forward(yq, q, wq, pos, freq, interleaved)
    check_forward(yk, k, wk, pos, freq, interleaved)
    gq = rows(B, Hq, N, d, dtype, 4, "head")
    gk = rows(B, Hk, N, d, dtype, 5)
    dq, dk, dwq, dwk = la.backward_qk_norm_rope(gq, gk, q, k, wq, wk, freq, offset=12345,
                                                interleaved=interleaved)
    check_backward(dq, dwq, gq, q, wq, pos, freq, interleaved)
    check_backward(dk, dwk, gk, k, wk, pos, freq, interleaved)


@pytest.mark.parametrize("dtype, wdtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_options(dtype, wdtype, norm, weighted):
    if weighted and not norm:
        pytest.skip("weights need norm")
    B, Hq, Hk, N, d = 2, 4, 2, 21, 64
    q, k = rows(B, Hq, N, d, dtype, 11), rows(B, Hk, N, d, dtype, 12)
    wq, wk = weights(d, 13, DT[wdtype]) if weighted else (None, None)
    freq = la.rope_frequencies(32, 500000.0)
    pos = token_positions(B, N)
    yq, yk = la.qk_norm_rope(q, k, wq, wk, freq, norm=norm)
    check_forward(yq, q, wq, pos, freq, False, norm)
    check_forward(yk, k, wk, pos, freq, False, norm)
    gq, gk = rows(B, Hq, N, d, dtype, 14, "head"), rows(B, Hk, N, d, dtype, 15, "head")
    dq, dk, dwq, dwk = la.backward_qk_norm_rope(gq, gk, q, k, wq, wk, freq, norm=norm)
    assert (dwq is None) == (not weighted) and (dwk is None) == (not weighted)
    check_backward(dq, dwq, gq, q, wq, pos, freq, False, norm)
    check_backward(dk, dwk, gk, k, wk, pos, freq, False, norm)


def test_norm_alone_and_one_side_weighted():
    q, k = rows(2, 3, 10, 64, "bf16", 21), rows(2, 3, 10, 64, "bf16", 22)
    wq, _ = weights(64, 23)
    pos = token_positions(2, 10)
    yq, yk = la.qk_norm_rope(q, k, wq, None)
    check_forward(yq, q, wq, pos, [], False)
    check_forward(yk, k, None, pos, [], False)
    dq, dk, dwq, dwk = la.backward_qk_norm_rope(yq, yk, q, k, wq, None)
    assert dwk is None
    check_backward(dq, dwq, yq, q, wq, pos, [], False)
    check_backward(dk, None, yk, k, None, pos, [], False)


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("form", ["batch", "shared", "strided"])
def test_positions(itype, form):
    # packed documents restart at 0; some positions lie far out or below zero
    B, N, d = 2, 40, 64
    q, k = rows(B, 2, N, d, "f32", 31), rows(B, 2, N, d, "f32", 32)
    freq = la.rope_frequencies(d)
    g = torch.Generator().manual_seed(33)
    pos = torch.randint(-5000, 1 << 30, (B, N), generator=g)
    pos[:, 10:20] = torch.arange(10)
    pos[1, 3] = (1 << 31) - 1
    if form == "shared":
        pos = pos[:1].expand(B, N)
        given = pos[0].to(itype).cuda()
    elif form == "strided":
        given = pos.to(itype).t().contiguous().cuda().t()
    else:
        given = pos.to(itype).cuda()
    yq, yk = la.qk_norm_rope(q, k, None, None, freq, given)
    # the 64-bit reference itself is off by |t| 2^-53 < 2^-21 radians here:
    # compare with the angle reduced exactly, in rationals
    check_exact_angles(yq, q, pos, freq)
    check_exact_angles(yk, k, pos, freq)


def check_exact_angles(y, x, pos, freq):
    from fractions import Fraction
    two_pi = Fraction(6283185307179586476925286766559005768394, 10 ** 39)
    v = x.cpu().double()
    n = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    R, h = 2 * len(freq), len(freq)
    f = [Fraction(t) for t in freq]
    for b, i in ((0, 0), (1, 3), (0, 12), (1, 39), (0, 25)):
        if i >= x.shape[2]:
            continue
        t = torch.tensor([float(int(pos[b, i]) * w % two_pi) for w in f], dtype=torch.float64)
        u1, u2 = n[b, :, i, :h], n[b, :, i, h:R]
        ref = torch.cat((u1 * t.cos() - u2 * t.sin(), u2 * t.cos() + u1 * t.sin()), -1)
        mag = torch.cat((u1.abs() + u2.abs(),) * 2, -1)
        assert torch.all((y[b, :, i].cpu().double() - ref).abs() <= 40 * U * mag)


@pytest.mark.parametrize("freq", [[1.0, -0.3, 1e-4, -1e-4], [6.5, 1e-9, 12345.678, -3.0],
                                  [0.0, -0.0, 1e9, -1e9]])
def test_any_frequencies(freq):
    # any sign and size; far positions (a frequency is off by at most some
    # 2^-64 turns per position beyond its own last bit)
    q, k = rows(2, 2, 40, 8, "f32", 35), rows(2, 2, 40, 8, "f32", 36)
    pos = torch.arange(40).expand(2, 40) + (1 << 33)
    yq, yk = la.qk_norm_rope(q, k, None, None, freq, offset=1 << 33)
    check_exact_angles(yq, q, pos, freq)
    check_exact_angles(yk, k, pos, freq)


def test_far_offset_keeps_relative_positions():
    # <y_q(p), y_k(p')> depends on p - p' alone, however far out p is
    d = 64
    q, k = rows(1, 1, 8, d, "f32", 41, "head"), rows(1, 1, 8, d, "f32", 42, "head")
    freq = la.rope_frequencies(d)
    near = la.qk_norm_rope(q, k, None, None, freq)
    far = la.qk_norm_rope(q, k, None, None, freq, offset=(1 << 40) + 12345)
    s = [torch.einsum("bhid,bhjd->bhij", a.double(), b.double()) for a, b in (near, far)]
    # |y| = sqrt(d): each of the d products is off by 80 u |u1 u2|-like terms
    assert float((s[0] - s[1]).abs().max()) <= 4 * 80 * U * d


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B, H, d", [(1, 32, 128), (256, 8, 64), (3, 2, 40), (7, 5, 37)])
def test_single_tokens(B, H, d, dtype):
    q = rows(B, H, 1, d, dtype, 51)[:, :, 0]
    k = rows(B, H, 1, d, dtype, 52)[:, :, 0]
    wq, wk = weights(d, 53)
    freq = la.rope_frequencies(d // 2 * 2)
    pos = torch.randint(0, 1 << 20, (B,), generator=torch.Generator().manual_seed(54))
    yq, yk = la.qk_norm_rope(q, k, wq, wk, freq, pos.cuda())
    assert yq.shape == (B, H, d)
    check_forward(yq[:, :, None], q[:, :, None], wq, pos[:, None], freq, False)
    check_forward(yk[:, :, None], k[:, :, None], wk, pos[:, None], freq, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_equals_sequence(dtype):
    # a token alone gives the bits that it gives inside a sequence
    q, k = rows(2, 4, 50, 128, dtype, 61), rows(2, 4, 50, 128, dtype, 62)
    wq, wk = weights(128, 63)
    freq = la.rope_frequencies(128)
    yq, yk = la.qk_norm_rope(q, k, wq, wk, freq, offset=7)
    for n in (0, 13, 49):
        p = torch.full((2,), n + 7, device="cuda")
        sq, sk = la.qk_norm_rope(q[:, :, n], k[:, :, n], wq, wk, freq, p)
        assert torch.equal(sq, yq[:, :, n]) and torch.equal(sk, yk[:, :, n])


@pytest.mark.parametrize("d, R", [(64, 64), (80, 40), (37, 36), (128, 100)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_any_strides_and_alignment(d, R, dtype):
    # rows that start at odd elements, outputs into slices of a buffer whose
    # other values stay as they are, and in place: all give the same bits
    B, H, N = 2, 3, 11
    g = torch.Generator().manual_seed(71)
    buf = torch.randn(B, N, H * d + 5, generator=g).to(DT[dtype]).cuda()
    q = buf[..., 3:3 + H * d].view(B, N, H, d).transpose(1, 2)
    kbuf = torch.randn(H, N, B, d + 1, generator=g).to(DT[dtype]).cuda()
    k = kbuf[..., 1:].permute(2, 0, 1, 3)
    wq, wk = weights(d, 72)
    freq = la.rope_frequencies(R)
    ref = la.qk_norm_rope(q.contiguous(), k.contiguous(), wq, wk, freq)
    got = la.qk_norm_rope(q, k, wq, wk, freq)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    room = torch.full((B, N, H * d + 7), 9.0, dtype=DT[dtype], device="cuda")
    qo = room[..., 5:5 + H * d].view(B, N, H, d).transpose(1, 2)
    la.qk_norm_rope(q, k, wq, wk, freq, q_out=qo)
    assert torch.equal(qo, ref[0])
    assert torch.all(room[..., :5] == 9.0) and torch.all(room[..., 5 + H * d:] == 9.0)
    gq, gk = rows(B, H, N, d, dtype, 73, "head"), rows(B, H, N, d, dtype, 74, "head")
    back = la.backward_qk_norm_rope(gq, gk, q.contiguous(), k.contiguous(), wq, wk, freq)
    odd = torch.empty(B, H, N, d + 1, dtype=DT[dtype], device="cuda")[..., 1:]
    odd.copy_(gq)
    got = la.backward_qk_norm_rope(odd, gk, q, k, wq, wk, freq, dq=qo)
    for a, b in zip(got[:2], back[:2]):
        assert torch.equal(a, b)
    assert torch.all(room[..., :5] == 9.0) and torch.all(room[..., 5 + H * d:] == 9.0)
    # in place
    gq2, gk2 = gq.clone(), gk.clone()
    got = la.backward_qk_norm_rope(gq2, gk2, q, k, wq, wk, freq, dq=gq2, dk=gk2)
    assert torch.equal(gq2, back[0]) and torch.equal(gk2, back[1])
    la.qk_norm_rope(q, k, wq, wk, freq, q_out=q, k_out=k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])


def test_broadcast_inputs_get_whole_gradients():
    # one key head shared by all queries' positions: an expanded input
    base = rows(1, 1, 6, 64, "f32", 81, "head")
    q = base.expand(3, 4, 6, 64)
    gq = rows(3, 4, 6, 64, "f32", 82, "head")
    freq = la.rope_frequencies(64)
    pos = token_positions(3, 6)
    dq, dk, _, _ = la.backward_qk_norm_rope(gq, gq, q, q.contiguous(), None, None, freq)
    check_backward(dq, None, gq, q, None, pos, freq, False)
    assert torch.equal(dq, dk)


def test_rows_of_zeros_and_non_finite_values_stay_apart():
    q = rows(1, 4, 6, 64, "bf16", 91, "head")
    q[0, 1, 2] = 0.0
    q[0, 2, 3, 5] = float("inf")
    q[0, 3, 4, 7] = float("nan")
    freq = la.rope_frequencies(64)
    y, _ = la.qk_norm_rope(q, q, None, None, freq)
    assert torch.all(y[0, 1, 2] == 0)
    assert torch.isnan(y[0, 3, 4]).all()
    good = torch.ones(4, 6, dtype=torch.bool)
    good[2, 3] = good[3, 4] = False
    assert torch.isfinite(y[0].cpu()[good]).all()
    pos = token_positions(1, 6)
    clean = q.clone()
    clean[0, 2, 3] = clean[0, 3, 4] = 1.0
    ref, _ = la.qk_norm_rope(clean, clean, None, None, freq)
    assert torch.equal(y[0].cpu()[good], ref[0].cpu()[good])


def test_gradient_against_differences():
    # the 64-bit plain forward's central differences (step 1e-6: off by
    # about 1e-9 of the loss's magnitude) along single values
    B, H, N, d = 1, 2, 5, 16
    q, k = rows(B, H, N, d, "f32", 101, "head"), rows(B, H, N, d, "f32", 102, "head")
    wq, wk = weights(d, 103)
    freq = la.rope_frequencies(8)
    pos = token_positions(B, N, 3)
    gq, gk = rows(B, H, N, d, "f32", 104, "head"), rows(B, H, N, d, "f32", 105, "head")
    dq, dk, dwq, dwk = la.backward_qk_norm_rope(gq, gk, q, k, wq, wk, freq, offset=3)

    def loss(x, w, gy):
        return float((plain(x, w, pos, freq, False) * gy.cpu().double()).sum())

    for x, w, gy, dx, dw in ((q, wq, gq, dq, dwq), (k, wk, gk, dk, dwk)):
        x, w = x.cpu().double(), w.cpu().double()
        for i in range(0, x.numel(), 23):
            e = torch.zeros_like(x).view(-1)
            e[i] = 1e-6
            e = e.view_as(x)
            num = (loss(x + e, w, gy) - loss(x - e, w, gy)) / 2e-6
            assert abs(num - float(dx.flatten()[i])) <= 1e-5
        for i in range(d):
            e = torch.zeros(d, dtype=torch.float64)
            e[i] = 1e-6
            num = (loss(x, w + e, gy) - loss(x, w - e, gy)) / 2e-6
            assert abs(num - float(dw[i])) <= 2e-5


def test_weight_gradient_over_many_rows_repeats_its_bits():
    q, k = rows(2, 8, 3000, 64, "bf16", 111), rows(2, 8, 3000, 64, "bf16", 112)
    wq, wk = weights(64, 113)
    freq = la.rope_frequencies(64)
    gq, gk = rows(2, 8, 3000, 64, "bf16", 114, "head"), rows(2, 8, 3000, 64, "bf16", 115, "head")
    a = la.backward_qk_norm_rope(gq, gk, q, k, wq, wk, freq)
    b = la.backward_qk_norm_rope(gq, gk, q, k, wq, wk, freq)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    pos = token_positions(2, 3000)
    check_backward(a[0], a[2], gq, q, wq, pos, freq, False)
    check_backward(a[1], a[3], gk, k, wk, pos, freq, False)


def test_empty_sides_and_batches():
    q = rows(2, 3, 4, 64, "f32", 121, "head")
    none = torch.empty(2, 0, 4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, z = la.qk_norm_rope(q, none)
    check_forward(y, q, None, token_positions(2, 4), [], False)
    assert z.shape == (2, 0, 4, 64)
    dq, dk, dwq, dwk = la.backward_qk_norm_rope(q, none, q, none, w, w)
    assert torch.all(dwk == 0) and torch.any(dwq != 0)
    e = torch.empty(2, 3, 0, 64, device="cuda")
    dwq = la.backward_qk_norm_rope(e, e, e, e, w, w)[2]
    assert torch.all(dwq == 0)
    assert la.qk_norm_rope(e, e)[0].shape == e.shape


def test_other_stream_and_captured_graph():
    q, k = rows(2, 4, 100, 128, "bf16", 131), rows(2, 4, 100, 128, "bf16", 132)
    wq, wk = weights(128, 133)
    freq = la.rope_frequencies(128)
    pos = torch.arange(100, device="cuda").expand(2, 100).contiguous()
    args = (q, k, wq, wk, freq, pos)
    ref = la.qk_norm_rope(*args)
    gq, gk = rows(2, 4, 100, 128, "bf16", 134, "head"), rows(2, 4, 100, 128, "bf16", 135, "head")
    ref_b = la.backward_qk_norm_rope(gq, gk, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = la.qk_norm_rope(*args)
    s.synchronize()
    assert torch.equal(y[0], ref[0]) and torch.equal(y[1], ref[1])
    y = la.qk_norm_rope(*args, stream=s)
    s.synchronize()
    assert torch.equal(y[0], ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = la.qk_norm_rope(*args)
        b = la.backward_qk_norm_rope(gq, gk, *args)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], ref[0]) and torch.equal(y[1], ref[1])
    for a, r in zip(b, ref_b):
        assert torch.equal(a, r)
    # positions are read when the graph runs
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    check_forward(y[0], q, wq, pos, freq, False)


def test_workspaces():
    # the binding brings one on the current stream; on a stream given by the
    # caller the library allocates, and reports a failure
    q = rows(1, 2, 9, 64, "f32", 141, "head")
    w = torch.ones(64, device="cuda")
    lib = la.load_library()
    here = torch.cuda.current_stream()
    ref = la.backward_qk_norm_rope(q, q, q, q.clone(), w, w)
    got = la.backward_qk_norm_rope(q, q, q, q.clone(), w, w, stream=here)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    assert lib.la_debug_fail_next_allocs(1) == 0
    try:
        la.backward_qk_norm_rope(q, q, q, q.clone(), w, w)  # allocates nothing
        with pytest.raises(la.LinAttnError) as e:
            la.backward_qk_norm_rope(q, q, q, q.clone(), w, w, stream=here)
        assert e.value.status == 4
    finally:
        lib.la_debug_fail_next_allocs(0)


def test_offsets_past_32_bits():
    # heads 2^31 elements apart: the last row's address needs 64 bits
    d, gap = 64, 1 << 31
    room = torch.empty(gap + 4 * d, dtype=torch.bfloat16, device="cuda")
    q = room.as_strided((1, 2, 2, d), (0, gap, d, 1))
    src = rows(1, 2, 2, d, "bf16", 151, "head")
    q.copy_(src)
    k = rows(1, 2, 2, d, "bf16", 152, "head")
    freq = la.rope_frequencies(d)
    ref = la.qk_norm_rope(src, k, None, None, freq)[0]
    y = la.qk_norm_rope(q, k, None, None, freq)[0]
    assert torch.equal(y, ref)
    la.qk_norm_rope(q, k, None, None, freq, q_out=q)
    assert torch.equal(q, ref)
