"""Features that the rotation leaves alone (those from its dimension on, or all of
them) pass as they are: a value that is not finite stays with its own feature, and
with its pair where it is rotated.  Forward and backward; no tolerance, since
without norm such a feature's result is its input."""
import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BAD = [float("inf"), -float("inf"), float("nan")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def partner(i, R, interleaved):
    if i >= R:
        return i
    if interleaved:
        return i ^ 1
    return (i + R // 2) % R


def rows(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(1, 3, d + 2, d, generator=g).to(DT[dtype])
    for n in range(d):  # token n has a bad value at feature n
        x[0, 0, n, n] = BAD[n % 3]
    x[0, 1, :, 0] = -0.0
    return x.cuda()


def same(a, b):
    """Equal values, zeros with their sign, NaN for NaN."""
    both = torch.isnan(a) & torch.isnan(b)
    return both | ((a == b) & (torch.signbit(a) == torch.signbit(b)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d, R", [(64, 0), (64, 16), (128, 32), (80, 40), (66, 2), (37, 10),
                                  (256, 254), (128, 128)])
def test_without_norm(d, R, interleaved, dtype):
    x = rows(d, dtype, d + R)
    freq = la.rope_frequencies(R)
    y, _ = la.qk_norm_rope(x, x[:, :1], None, None, freq, offset=3, norm=False,
                           interleaved=interleaved)
    dx = la.backward_qk_norm_rope(x, x[:, :1], x, x[:, :1], None, None, freq, offset=3,
                                  norm=False, interleaved=interleaved)[0]
    for got in (y, dx):
        assert same(got[..., R:], x[..., R:]).all()
        bad = ~torch.isfinite(got.cpu())
        want = torch.zeros_like(bad)
        for n in range(d):
            want[0, 0, n, n] = want[0, 0, n, partner(n, R, interleaved)] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d, R", [(64, 0), (128, 32), (37, 10)])
def test_infinite_value_under_the_norm(d, R, dtype):
    # an infinite square makes the norm's factor 0: the row's other values become 0,
    # the value itself (and its pair, where rotated) has none
    x = torch.ones(1, 1, d, d, dtype=DT[dtype], device="cuda")
    x[0, 0].fill_diagonal_(float("inf"))
    y, _ = la.qk_norm_rope(x, x, None, None, la.rope_frequencies(R), offset=3)
    want = torch.zeros(d, d, dtype=torch.bool)
    for n in range(d):
        want[n, n] = want[n, partner(n, R, False)] = True
    assert torch.equal(torch.isnan(y[0, 0].cpu()), want)
    assert torch.all(y[0, 0].cpu()[~want] == 0)


def test_weight_gradient_of_an_unrotated_feature():
    x = torch.randn(1, 2, 40, 64, generator=torch.Generator().manual_seed(5)).cuda()
    dy = torch.ones_like(x)
    dy[0, 1, 7, 50] = float("inf")
    w = torch.ones(64, device="cuda")
    dw = la.backward_qk_norm_rope(dy, dy, x, x, w, w, la.rope_frequencies(16))[2]
    want = torch.zeros(64, dtype=torch.bool)
    want[50] = True
    assert torch.equal(~torch.isfinite(dw.cpu()), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d, R", [(64, 64), (128, 32), (37, 10), (66, 66)])
def test_backward_without_norm_is_the_rotation_back(d, R, interleaved, dtype):
    # into a strided gradient and in place: the same bits; and the forward with the
    # opposite frequencies, whose turns differ by 2^-64 of a turn per position, gives
    # them but for a step of 2^-32 turns (2^-29 radians) of the angle and the roundings
    g = torch.Generator().manual_seed(d)
    dy = torch.randn(2, 5, 33, d, generator=g).to(DT[dtype]).cuda()
    freq = la.rope_frequencies(R)
    back = [-f for f in freq]
    kw = dict(norm=False, interleaved=interleaved)
    pos = torch.randint(0, 1 << 20, (2, 33), generator=g).cuda()
    want, wk = la.qk_norm_rope(dy, dy[:, :2], None, None, back, pos, **kw)
    dq, dk, dwq, dwk = la.backward_qk_norm_rope(dy, dy[:, :2], dy, dy[:, :2], None, None, freq,
                                                pos, **kw)
    assert dwq is None and dwk is None
    # two values of up to |dy| by sines and cosines that a step of the angle, its
    # rounding (8 u at most for bf16) and the functions move, then the result's rounding
    tol = 2 * (2.0 ** -29 + (16 if dtype == "bf16" else 4) * 2.0 ** -24) * 2
    tol += 2 * torch.finfo(DT[dtype]).eps
    for a, b in ((dq, want), (dk, wk)):
        assert float((a.double() - b.double()).abs().max()) <= tol * float(dy.double().abs().max())
    room = torch.full((2, 33, 5 * d + 3), 9.0, dtype=DT[dtype], device="cuda")
    out = room[..., 1:1 + 5 * d].view(2, 33, 5, d).transpose(1, 2)
    la.backward_qk_norm_rope(dy, dy[:, :0], dy, dy[:, :0], None, None, freq, pos, dq=out, **kw)
    assert torch.equal(out, dq)
    assert torch.all(room[..., 0] == 9.0) and torch.all(room[..., 1 + 5 * d:] == 9.0)
    inp = dy.clone()
    got = la.backward_qk_norm_rope(inp, dk, inp, dk, None, None, freq, pos, dq=inp, **kw)
    assert got[0].data_ptr() == inp.data_ptr() and torch.equal(inp, dq)
