"""Linear cross attention where values are not finite: what the formula makes of them in
the results that they reach, zeros where zeros are promised, and the other results
bit for bit as without them, on each set of kernels."""
import math

import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
INF, NAN = math.inf, math.nan

# bf16 by tiles, with a head that fills them and one that does not; bf16 of any size and
# stride; fp32
PATHS = [("bf16", 64, 0), ("bf16", 80, 0), ("bf16", 128, 0), ("bf16", 256, 0), ("bf16", 61, 0),
         ("bf16", 64, 5), ("f32", 64, 0), ("f32", 100, 0)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


LENGTHS, N, M = [70, 200, 0], 150, 200


def inputs(dtype, d, pad, shift=0.0):
    """q, dout [3, 4, N, d] and k, v [3, 2, M, d], rows d + pad apart."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rows(H, L):
        x = torch.randn(3, H, L, d + pad, generator=g, device="cuda").mul_(0.7).add_(shift).to(t)
        return x[..., 1:d + 1] if pad else x

    return rows(4, N), rows(4, N), rows(2, M), rows(2, M)


def same(a, b):
    """Bit for bit, every NaN being like any other."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(torch.nan_to_num(a, 9.0, INF, -INF),
                                                             torch.nan_to_num(b, 9.0, INF, -INF))


def but(x, *at):
    """x without what lies at `at`."""
    x = x.clone()
    x[at] = 0
    return x


def padding_is_zero(*xs):
    for x in xs:
        for b, n in enumerate(LENGTHS):
            assert not bool(x[b, :, n:].ne(0).any()), b  # (a NaN is not 0)


@pytest.mark.parametrize("dtype, d, pad", PATHS)
def test_an_infinite_query(dtype, d, pad):
    # one feature's phi and the denominator are infinite: inf / inf in all of the row
    q, dout, k, v = inputs(dtype, d, pad)
    lens, at = ints(LENGTHS), (0, 3, 77)
    want = la.forward_cross(q, k, v, lens)
    grads = la.backward_cross(dout, q, k, v, *want[1:], lens)
    q[(*at, d // 2)] = INF
    out, S, z = la.forward_cross(q, k, v, lens)
    assert bool(out[at].isnan().all()) and torch.equal(but(out, *at), but(want[0], *at))
    assert torch.equal(S, want[1]) and torch.equal(z, want[2])
    # tokens of a head by ones and by many: the same row of NaN
    for n in (1, 3, 9, 40):
        some = la.decode_step_cross(S, z, q[:, :, 77 - n // 2:77 - n // 2 + n])
        assert bool(some[0, 3, n // 2].isnan().all())
        some[0, 3, n // 2] = 0
        assert bool(some.isfinite().all())
    # the head's state is the one that heads 2 and 3 share: its dk and dv are NaN
    dq, dk, dv = la.backward_cross(dout, q, k, v, S, z, lens)
    assert bool(dq[at].isnan().all()) and torch.equal(but(dq, *at), but(grads[0], *at))
    for x, y in ((dk, grads[1]), (dv, grads[2])):
        assert bool(x[0, 1, :70].isnan().all())
        assert torch.equal(but(x, 0, 1, slice(70)), but(y, 0, 1, slice(70)))
    padding_is_zero(dk, dv)
    la.check_device_status()


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype, d, pad", PATHS)
def test_a_gradient_that_is_not_finite(dtype, d, pad, bad):
    q, dout, k, v = inputs(dtype, d, pad)
    lens, at, c = ints(LENGTHS), (0, 1, 100), d // 3
    _, S, z = la.forward_cross(q, k, v, lens)
    want = la.backward_cross(dout, q, k, v, S, z, lens)
    dout[(*at, c)] = bad
    dq, dk, dv = la.backward_cross(dout, q, k, v, S, z, lens)
    assert not bool(dq[at].isfinite().any()) and torch.equal(but(dq, *at), but(want[0], *at))
    # the state of heads 0 and 1: its dS is not finite in one column, its dz in all rows
    # (with bf16 NaN may stand for an infinity: a low part of 0 times it)
    assert not bool(dk[0, 0, :70].isfinite().any())
    assert torch.equal(but(dk, 0, 0, slice(70)), but(want[1], 0, 0, slice(70)))
    column = (0, 0, slice(70), c)
    assert not bool(dv[column].isfinite().any())
    assert torch.equal(but(dv, *column), but(want[2], *column))
    padding_is_zero(dk, dv)
    la.check_device_status()


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype, d, pad", PATHS)
def test_a_key_that_is_not_finite(dtype, d, pad, bad):
    # with the identity, whose phi takes both signs
    q, dout, k, v = inputs(dtype, d, pad)
    lens, a, form = ints(LENGTHS), d // 2, {"feature_map": "identity", "normalise": False}
    want = la.forward_cross(q, k, v, lens, **form)
    k[1, 1, 150, a] = bad
    out, S, z = la.forward_cross(q, k, v, lens, **form)
    row = (1, 1, a)
    assert same(S[row], bad * v[1, 1, 150].float())  # (no value is 0)
    assert same(z[row], torch.full_like(z[row], bad))
    assert torch.equal(but(S, *row), but(want[1], *row)) and torch.equal(but(z, *row), but(want[2], *row))
    # the heads 2 and 3 of the second sequence: that row of S times q's feature
    f = q[1, 2:, :, a].float()
    ref = f[..., None] * (bad * v[1, 1, 150].float())
    assert same(out[1, 2:].float(), ref)
    assert torch.equal(but(out, 1, slice(2, 4)), but(want[0], 1, slice(2, 4)))
    dq, dk, dv = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    assert not bool(dq[1, 2:, :, a].isfinite().any())
    assert bool(but(dq, 1, slice(2, 4), slice(None), a).isfinite().all())
    assert bool(dk.isfinite().all())  # dS v, without the key itself
    assert not bool(dv[1, 1, 150].isfinite().any())
    assert bool(but(dv, 1, 1, 150).isfinite().all())
    padding_is_zero(dk, dv)
    la.check_device_status()


@pytest.mark.parametrize("dtype, d, pad", PATHS)
def test_an_infinite_key_with_the_normaliser(dtype, d, pad):
    q, dout, k, v = inputs(dtype, d, pad)
    lens, a = ints(LENGTHS), d // 2
    want = la.forward_cross(q, k, v, lens)
    k[1, 1, 150, a] = INF
    out, S, z = la.forward_cross(q, k, v, lens)
    row = (1, 1, a)
    assert same(S[row], INF * v[1, 1, 150].float()) and float(z[row]) == INF
    assert torch.equal(but(S, *row), but(want[1], *row)) and torch.equal(but(z, *row), but(want[2], *row))
    assert bool(out[1, 2:].isnan().all())  # inf / inf
    assert torch.equal(but(out, 1, slice(2, 4)), but(want[0], 1, slice(2, 4)))


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("dtype, d, pad", PATHS)
def test_a_denominator_of_zero_gives_zeros_whatever_the_rest_is(dtype, d, pad, bad):
    # a query of zeros has phi = 0 with the identity, and a sequence without keys has z = 0
    q, dout, k, v = inputs(dtype, d, pad, shift=0.5)
    lens, at, form = ints(LENGTHS), (1, 2, 33), {"feature_map": "identity", "normalise": True}
    q[at] = 0
    dout[at] = 0
    out, S, z = la.forward_cross(q, k, v, lens, **form)
    assert not bool(out[at].any()) and not bool(out[2].any())
    want = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    dout[at] = bad
    dout[2, :, 5] = bad
    got = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert not bool(got[0][at].any()) and not bool(got[0][2].any())
    # the state not finite: the row's outputs and gradients are still zeros
    v[1, 1, 40, 3] = bad
    out, S, z = la.forward_cross(q, k, v, lens, **form)
    assert not bool(S[1, 1, :, 3].isfinite().any())
    assert not bool(out[at].ne(0).any())
    for n in (1, 9, 40):
        some = la.decode_step_cross(S, z, q[:, :, 33 - n // 2:33 - n // 2 + n], **form)
        assert not bool(some[1, 2, n // 2].ne(0).any())
    dq, dk, dv = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    assert not bool(dq[at].ne(0).any())
    padding_is_zero(dk, dv)
    la.check_device_status()


@pytest.mark.parametrize("fmap", ["identity", "elu1"])
@pytest.mark.parametrize("dtype, d, pad", PATHS)
def test_without_the_normaliser_z_is_not_used(dtype, d, pad, fmap):
    # its sum may overflow where that of the products does not
    q, dout, k, v = inputs(dtype, d, pad)
    lens, form = ints(LENGTHS), {"feature_map": fmap, "normalise": False}
    _, S, z = la.forward_cross(q, k, v, lens, **form)
    want = la.backward_cross(dout, q, k, v, S, z, lens, **form)
    steps = [la.decode_step_cross(S, z, q[:, :, :n], **form) for n in (1, 9, 40)]
    for bad in (INF, NAN):
        z.fill_(bad)
        assert all(torch.equal(a, b) for a, b in
                   zip(la.backward_cross(dout, q, k, v, S, z, lens, **form), want))
        assert all(torch.equal(a, la.decode_step_cross(S, z, q[:, :, :n], **form))
                   for a, n in zip(steps, (1, 9, 40)))
    la.check_device_status()
