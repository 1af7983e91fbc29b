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


# tiles, and rows by 16 bytes, by words and one by one, of each width; fp32 likewise
FETCHES = [("bf16", 64, 16, 0), ("bf16", 128, 32, 0), ("bf16", 192, 16, 0), ("bf16", 256, 16, 0),
           ("bf16", 72, 16, 0), ("bf16", 64, 7, 0), ("bf16", 128, 5, 0), ("bf16", 256, 24, 0),
           ("bf16", 200, 3, 0), ("bf16", 66, 16, 0), ("bf16", 130, 9, 0), ("bf16", 250, 16, 0),
           ("bf16", 64, 16, 1), ("bf16", 33, 16, 0), ("bf16", 255, 6, 0), ("bf16", 129, 16, 0),
           ("f32", 64, 16, 0), ("f32", 128, 7, 0), ("f32", 200, 16, 0), ("f32", 61, 5, 0),
           ("f32", 128, 16, 1)]


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype, d, page, pad", FETCHES)
def test_a_key_that_other_queries_look_at(dtype, d, page, pad, value):
    """Five tokens of 90, 6 heads on 2: the key of the third is not finite.  The first two
    do not look at it, and neither do any with a window that begins behind it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    t, T, n = DT[dtype], 5, 90
    pages = -(-n // page) + 1
    kc, vc = (torch.randn(pages, 2, page, d + pad, generator=g, device="cuda").to(t)[..., pad:]
              for _ in range(2))
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    q = torch.randn(1, 6, T, d, generator=g, device="cuda").to(t)
    before, bad = ints([n - T]), n - T + 2
    at = (int(table[0, bad // page]), slice(None), bad % page)
    k = torch.stack([kc[int(table[0, p // page]), :, p % page] for p in range(n)], 1).double()
    v = torch.stack([vc[int(table[0, p // page]), :, p % page] for p in range(n)], 1).double()
    # a value that is not finite, in some columns, behind a weight that is; and the key's own
    # score not finite either
    for which in ("value", "both"):
        vc[at][..., ::3] = value
        if which == "both":
            kc[at][..., 1::2] = value
        for window in (0, 1, 2, 40):
            got = la.decode_step_paged(q, kc, vc, table, before, window=window)
            for i in range(T):
                p = n - T + i
                lo = max(0, p + 1 - window) if window else 0
                if lo <= bad <= p:
                    if which == "value":  # a weight above 0 reaches just those columns
                        assert not bool(got[0, :, i, ::3].isfinite().any()), (window, i)
                    continue
                s = torch.einsum("hgd,hnd->hgn", q[0, :, i].double().unflatten(0, (2, 3)),
                                 k[:, lo:p + 1]) / d ** 0.5
                size = torch.einsum("hgd,hnd->hgn", q[0, :, i].double().abs().unflatten(0, (2, 3)),
                                    k[:, lo:p + 1].abs()).amax(-1) / d ** 0.5
                w = torch.softmax(s, -1)
                ref = torch.einsum("hgn,hnd->hgd", w, v[:, lo:p + 1]).flatten(0, 1)
                mean = torch.einsum("hgn,hnd->hgd", w, v[:, lo:p + 1].abs()).flatten(0, 1)
                # scores good to d + 4 roundings of their terms (2 u where they are cut), which
                # move a weight and the weights' sum; sums of 90 terms; bf16 weights, 2^-8 each
                # of themselves, and the result's own rounding
                rel = 2 * ((d + 4) * 2 * U * size.flatten()[:, None] + 2.0 ** -22) + 2 * 90 * 2 * U
                rel = rel + (2 * 2.0 ** -8 if dtype == "bf16" else 0)
                bound = rel * mean + (2.0 ** -8 if dtype == "bf16" else U) * ref.abs()
                off = (got[0, :, i].double() - ref).abs()
                assert bool((off <= bound).all()), (which, window, i)
    la.check_device_status()


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
