"""The gradients of cross attention where a state's sums over the queries are long: what the
tensor cores cut off at each addition must not pile up over them."""
import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def phi(x):
    return torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))


@pytest.mark.parametrize("B, Hk, G, N, d, early", [
    (20, 8, 8, 1 << 17, 8, True),    # a million queries of each state, a state per SM
    (20, 8, 8, 1 << 17, 8, False),
    (20, 8, 4, 1 << 14, 64, True),
    (20, 8, 2, 1 << 14, 128, True),
    (1, 3, 4, 1 << 15, 72, True),    # states in several blocks
    (160, 2, 2, 1500, 72, True),     # and several in a block
])
def test_sums_of_many_queries(B, Hk, G, N, d, early):
    """Values around 64 make dk a small difference of dS v and dz.  With `early`, half of
    the columns get their sums from the first tokens and the others from the last, so
    that losses which grow with the additions behind do not cancel."""
    g = torch.Generator(device="cuda")
    g.manual_seed(N + d)
    M, half = 64, d // 2
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q = torch.empty(B, Hk * G, N, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(0.7)
    dout = torch.empty_like(q).normal_(generator=g)
    if early:
        dout.mul_(2.0 ** -6)
        dout[:, :, :N // 16, :half] += 1
        dout[:, :, -(N // 16):, half:] += 1
    else:
        dout.mul_(0.5).add_(1)
    k, v = (0.7 * randn(B, Hk, M, d)).bfloat16(), (randn(B, Hk, M, d) + 64).bfloat16()
    _, S, z = la.forward_cross(q[:, :, :1], k, v)
    dq, dk, dv = la.backward_cross(dout, q, k, v, S, z)
    la.check_device_status()
    for b, h in {(0, 0), (B // 2, Hk // 2), (B - 1, Hk - 1)}:
        f = phi(q[b, h * G:(h + 1) * G].double()).reshape(-1, d)
        dy = dout[b, h * G:(h + 1) * G].double().reshape(-1, d)
        K, V, s, zz = (x[b, h].double() for x in (k, v, S, z))
        r = 1 / (f @ zz)
        t = ((f @ s) * dy).sum(1) * r
        psi = f * r[:, None]
        dS, dz = psi.T @ dy, -(psi * t[:, None]).sum(0)
        slope = torch.exp(K.clamp(max=0))
        ref = (V @ dS.T + dz) * slope
        terms = (V.abs() @ dS.abs().T + dz.abs()) * slope
        # dS and t as two bf16 numbers, 2^-16 each; a chain of 2048 tokens, 128 products that are
        # cut (2^-23 each); fp32 sums of the chains, rounded to nearest, whose errors grow by the
        # root; the result and the queries' rounded factors, which average out
        rel = 2 * 2.0 ** -16 + 128 * 2.0 ** -23 + (G * N / 2048) ** 0.5 * 2.0 ** -24
        off = float((dk[b, h].double() - ref).norm())
        assert off <= rel * float(terms.norm()) + 2 * 2.0 ** -8 * float(ref.norm()), (b, h, off / float(
            ref.norm()), float(terms.norm() / ref.norm()))
        # dv: the bias of its sums shows beside its own rounding, which has none
        x, y = dv[b, h].double(), phi(K) @ dS
        assert float((x - y).norm()) <= 3 * 2.0 ** -8 * float(y.norm())
    # the same bits again
    assert all(torch.equal(a, b) for a, b in zip(la.backward_cross(dout, q, k, v, S, z), (dq, dk, dv)))
