"""The attention over the paged cache: keys that some queries of a call look at and
others do not, where they are not finite, however the cache's rows are fetched; and
lengths beyond what a table can hold."""
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


@pytest.mark.parametrize("dtype, T", [("bf16", 1), ("bf16", 3), ("f32", 1), ("f32", 3)])
def test_windows_of_lengths_beyond_the_table(dtype, T):
    """Queries past all that a table can hold (2^30 tokens) look at the keys that their
    windows reach, counted from where the queries are."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    t, d, n = DT[dtype], 64, 96
    kc, vc = (torch.randn(6, 1, 16, d, generator=g, device="cuda").to(t) for _ in range(2))
    table = torch.arange(6, dtype=torch.int32, device="cuda").expand(7, 6)
    top, window = (1 << 31) - 1, (1 << 30) + 40
    before = [top, (1 << 30) + 50, (1 << 30) + 39, (1 << 30) + 135, 1 << 30, (1 << 30) - 1, n - T]
    q = torch.randn(7, 2, T, d, generator=g, device="cuda").to(t)
    got = la.decode_step_paged(q, kc, vc, table, ints(before), window=window)
    k, v = (x[:, 0].reshape(n, d).double() for x in (kc, vc))
    for b, p0 in enumerate(before):
        for i in range(T):
            lo = max(0, p0 + i + 1 - window)
            hi = min(n, p0 + i + 1)
            if lo >= hi:
                assert not bool(got[b, :, i].any()), (b, i)
                continue
            s = q[b, :, i].double() @ k[lo:hi].T / d ** 0.5
            w = torch.softmax(s, -1)
            ref, mean = w @ v[lo:hi], w @ v[lo:hi].abs()
            size = (q[b, :, i].double().abs() @ k[lo:hi].abs().T).amax(-1, keepdim=True) / d ** 0.5
            rel = 2 * ((d + 4) * 2 * U * size + 2.0 ** -22) + 2 * 96 * 2 * U
            rel = rel + (2 * 2.0 ** -8 if dtype == "bf16" else 0)
            bound = rel * mean + (2.0 ** -8 if dtype == "bf16" else U) * ref.abs()
            assert bool(((got[b, :, i].double() - ref).abs() <= bound).all()), (b, i)
    # the largest window there is, which ends behind the first key for the last position only
    got = la.decode_step_paged(q[:1], kc, vc, table[:1], ints([top]), window=top)
    every = la.decode_step_paged(q[:1], kc, vc, table[:1], ints([top]))
    assert bool(every.any()) and not torch.equal(got, every)
