"""The weight gradients of backward_qk_norm_rope over many rows.

All rows are the same row (inputs expanded with stride 0, one position), so every
term of the sum is the same number t, and the gradient of a call of one row is t
rounded to fp32.  What is left is the sum itself, which may be off by 19 u of the
terms' magnitudes, u = 2^-24, whatever their number: chains of 16 rows 8.5 u
(1 + 2 + ... + 16 = 136 u t in 16 t), 5 u for the sums over a warp's lanes, and one u
each for a chain's residue and the rounding of a thread's sum, a block's, the last
one and the product.
Adding equal terms in one chain of n rounds off the same part of a step for a
whole binade, so it is off by about n u / 8 and cannot pass; a row left out or
taken twice is an error of 1 / n."""
import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B, Hq, Hk, N, d, R, dtype", [
    (1, 1, 1, 9, 64, 64, "f32"),
    (2, 8, 2, 3000, 64, 64, "bf16"),
    (2, 8, 2, 3001, 37, 10, "bf16"),
    (2, 8, 2, 3001, 66, 66, "bf16"),
    (3, 6, 2, 1001, 80, 40, "f32"),
    (2, 8, 2, 5000, 250, 100, "f32"),
    (4, 8, 8, 16384, 128, 128, "bf16"),
    (8, 32, 1, 32768, 64, 64, "f32"),
])
def test_many_equal_rows(B, Hq, Hk, N, d, R, dtype, interleaved):
    g = torch.Generator().manual_seed(7 + d)
    x, dy = (torch.randn(1, 1, 1, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    freq = la.rope_frequencies(R)
    pos = torch.full((1,), 77, device="cuda")

    def gradients(B, Hq, Hk, N):
        q, k = x.expand(B, Hq, N, d), x.expand(B, Hk, N, d)
        gq, gk = dy.expand(B, Hq, N, d), dy.expand(B, Hk, N, d)
        dq, dk, dwq, dwk = la.backward_qk_norm_rope(gq, gk, q, k, w, w, freq, pos.expand(N),
                                                    interleaved=interleaved)
        return dwq.double(), dwk.double()

    one = gradients(1, 1, 1, 1)
    assert torch.equal(one[0], one[1]) and torch.all(one[0] != 0)
    for got, H in zip(gradients(B, Hq, Hk, N), (Hq, Hk)):
        n = B * H * N
        off = ((got - n * one[0]).abs() / (n * one[0].abs())).max()
        assert float(off) <= 19 * U, float(off) / U


def test_an_infinite_gradient_gives_an_infinite_sum():
    q = torch.randn(1, 2, 3000, 64, generator=torch.Generator().manual_seed(3)).cuda()
    dy = torch.ones(1, 2, 3000, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    dy[0, 1, 100, 5] = float("inf")
    dwq = la.backward_qk_norm_rope(dy, dy[:, :1], q, q[:, :1], w, w)[2]
    assert float(dwq[5]) == float("inf") * float(q[0, 1, 100, 5].sign())
    assert torch.isfinite(dwq[:5]).all() and torch.isfinite(dwq[6:37]).all()
