"""cos and sin of the rotation's angles, seen through rows that leave nothing else.

Without norm the row (1, 0) becomes (cos t, sin t) with no further rounding.  In the
backward, a row of values +-1/2 with eps 3/4 has a norm of exactly 1 (1/4 + 3/4), so
the weight gradient of the output gradient (1, 0) is (cos t, -sin t) / 2 for values of
1/2, again exactly.  Bound, u = 2^-24: the position times the frequency in 2^-64 turns
is cut to 2^-32 turns (0.03 u), its rest beyond whole quarter turns rounded to fp32
(0.39 u: at most 16 steps of 2^-32 turns), the polynomials off by 0.2 u with
coefficients rounded (0.2 u), the result rounded (0.5 u): 1.4 u with the roundings
inside."""
import math

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


def angles(pos, freq):
    """In 64 bits: off by 2^-33 at most below 2^21 radians, where u is 2^-24."""
    return pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64)


@pytest.mark.parametrize("freq", [[0.7390851332151607, 1e-6], [math.pi / 7, -1.0], [1.9, 2e-3]])
def test_forward(freq):
    n = 1 << 20
    x = torch.zeros(1, 1, n, 4, device="cuda")
    x[..., :2] = 1
    y, _ = la.qk_norm_rope(x, x[:, :0], None, None, freq, norm=False)
    t = angles(torch.arange(n), freq)
    want = torch.cat((t.cos(), t.sin()), -1)
    assert float((y[0, 0].cpu().double() - want).abs().max()) <= 1.4 * U


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weight_gradient(dtype):
    d = 64
    freq = list(la.rope_frequencies(d))
    x = torch.full((1, 1, 1, d), 0.5, dtype=DT[dtype], device="cuda")
    dy = torch.zeros(1, 1, 1, d, dtype=DT[dtype], device="cuda")
    dy[..., :d // 2] = 1
    w = torch.ones(d, device="cuda")
    plain, _ = la.qk_norm_rope(x, x, w, w, eps=0.75)
    assert torch.equal(plain, x)  # the norm is 1
    g = torch.Generator().manual_seed(9)
    pos = torch.randint(0, 1 << 20, (150,), generator=g)
    t = angles(pos, freq)
    want = torch.cat((t.cos(), -t.sin()), -1) / 2
    for i, p in enumerate(pos.tolist()):
        dw = la.backward_qk_norm_rope(dy, dy, x, x, w, w, freq, offset=p, eps=0.75)[2]
        assert float((dw.cpu().double() - want[i]).abs().max()) <= 0.7 * U, p
