"""Roundings of the bf16 cross attention that the sizes of its terms do not hide: sums
that nearly cancel, on each set of kernels, and single tokens, which round nothing but
their results."""
import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def phi(x):
    return torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))


def rows(g, H, L, d, pad, scale=1.0, shift=0.0):
    x = torch.randn(1, H, L, d + pad, generator=g, device="cuda").mul_(scale).add_(shift)
    return x.bfloat16()[..., pad:]


def gradients(q, k, v, dout, S, z):
    """By the formulas in 64 bits, from the states that the backward is given."""
    B, Hk, M, d = k.shape
    q64, dy = (x.double().reshape(B, Hk, -1, d) for x in (q, dout))
    k, v, S, z = k.double(), v.double(), S.double(), z.double()
    f = phi(q64)
    r = 1 / (f @ z[..., None])
    G = dy @ S.transpose(2, 3)
    t = (f * G).sum(-1, keepdim=True) * r
    dq = r * (G - t * z[:, :, None]) * torch.exp(q64.clamp(max=0))
    psi = r * f
    dS, dz = psi.transpose(2, 3) @ dy, -(psi * t).sum(2)
    dk = (v @ dS.transpose(2, 3) + dz[:, :, None]) * torch.exp(k.clamp(max=0))
    return dq.reshape(q.shape), dk, phi(k) @ dS


def off(x, ref):
    return float((x.double() - ref).norm() / ref.norm())


# by tiles; of any size, by 8 bytes and one by one
SHAPES = [(64, 0), (128, 0), (80, 0), (256, 0), (200, 0), (129, 0), (64, 5), (128, 3)]


@pytest.mark.parametrize("d, pad", SHAPES)
def test_queries_gradient_where_values_have_a_mean(d, pad):
    """M values of deviation s around c: S dy and t z are c sqrt(M) / s times what is left of
    them.  S and m as two bf16 numbers lose 2^-16 of that, S centred by m nothing that
    matters; r phi, phi' and the result are fp32 and one rounding."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    M, c = 2048, 8.0
    q, k = rows(g, 2, 200, d, pad, 0.7), rows(g, 1, M, d, pad, 0.7)
    v, dout = rows(g, 1, M, d, pad, shift=c), rows(g, 2, 200, d, pad)
    _, S, z = la.forward_cross(q, k, v)
    dq, _, _ = la.backward_cross(dout, q, k, v, S, z)
    assert off(dq, gradients(q, k, v, dout, S, z)[0]) <= 2.0 ** -16 * c * M ** 0.5 + 3 * 2.0 ** -8
    la.check_device_status()


@pytest.mark.parametrize("d, pad", SHAPES)
def test_keys_gradient_where_values_have_a_mean(d, pad):
    """dS v and dz are c / s times what is left of them, where all dout have a mean.  dS, t
    and m are two bf16 numbers each, dS, t and z sums of fp32: six times 2^-16 of the
    terms at most, next to psi, dy (v - y) and the result rounded to bf16 once each."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    c = 64.0
    q, k = rows(g, 2, 256, d, pad, 0.7), rows(g, 1, 64, d, pad, 0.7)
    v, dout = rows(g, 1, 64, d, pad, shift=c), rows(g, 2, 256, d, pad, 0.5, 1.0)
    _, S, z = la.forward_cross(q, k, v)
    _, dk, dv = la.backward_cross(dout, q, k, v, S, z)
    ref = gradients(q, k, v, dout, S, z)
    assert off(dk, ref[1]) <= 6 * 2.0 ** -16 * c + 3 * 2.0 ** -8
    assert off(dv, ref[2]) <= 3 * 2.0 ** -8
    la.check_device_status()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("d, Hq, Hk, N", [(64, 4, 2, 1), (128, 8, 8, 1), (61, 2, 1, 1), (256, 4, 1, 1),
                                          (128, 2, 2, 4), (80, 16, 2, 3), (37, 2, 2, 4)])
def test_single_tokens_round_their_results_alone(d, Hq, Hk, N, norm):
    """With the identity and signs of either kind, so that results are small against their
    terms: d products and sums in fp32, as many of the denominator, and half a step."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    B = 3
    S, z = (torch.randn(*s, generator=g, device="cuda") for s in ((B, Hk, d, d), (B, Hk, d)))
    q = torch.randn(B, Hq, N, d, generator=g, device="cuda").bfloat16()
    got = la.decode_step_cross(S, z, q, feature_map="identity", normalise=norm)
    x, S, z = q.double().reshape(B, Hk, -1, d), S.double(), z.double()
    ref, size = x @ S, x.abs() @ S.abs()
    rel = (d + 4) * U
    if norm:
        den, of = x @ z[..., None], x.abs() @ z.abs()[..., None]
        ref, size = ref / den, size / den.abs()
        bound = rel * size + rel * of / den.abs() * ref.abs() * 2
    else:
        bound = rel * size
    bound = bound + 2.0 ** -8 * ref.abs()
    keep = 1.0  # the denominators' own loss is small against them
    if norm:
        keep = (rel * of / den.abs() <= 0.25).double()
    assert bool((((got.double().reshape(ref.shape) - ref).abs() <= bound) | (keep == 0)).all())
