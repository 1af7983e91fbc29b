"""The paged cache: appending tokens with the rotation on the way, and the softmax
attention of new tokens over it, against plain implementations in 64 bits.

Everything of the pool that belongs to no sequence holds NaN, so that a read out
of place shows."""
import math

import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}  # half a step of the type, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def pool_of(layout, pages, Hk, page, d, t):
    """[pages, Hk, page, d] with several orders in memory, all NaN."""
    if layout == "heads":
        return torch.full((pages, Hk, page, d), math.nan, dtype=t, device="cuda")
    if layout == "tokens":  # a slot's heads side by side
        return torch.full((pages, page, Hk, d), math.nan, dtype=t, device="cuda").transpose(1, 2)
    if layout == "apart":   # rows that are not whole 16-byte units apart
        return torch.full((pages, Hk, page, d + 3), math.nan, dtype=t, device="cuda")[..., 1:d + 1]
    return torch.full((pages, 2, Hk, page, d), math.nan, dtype=t, device="cuda")[:, 1]


def table_of(lengths, page, g, spare=2):
    need = [-(-max(n, 0) // page) for n in lengths]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lengths), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rotated(x, pos, freq, interleaved):
    """x [B, H, T, d] at positions [B, T], in 64 bits, and the pairs' sizes |x1| + |x2|."""
    x = x.double()
    R = 2 * len(freq)
    a = (pos.double()[..., None] * torch.tensor(list(freq), dtype=torch.float64, device="cuda"))[:, None]
    i = torch.arange(R // 2, device="cuda")
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i0] = x[..., i0] * a.cos() - x[..., i1] * a.sin()
    y[..., i1] = x[..., i1] * a.cos() + x[..., i0] * a.sin()
    size[..., i0] = size[..., i1] = x[..., i0].abs() + x[..., i1].abs()
    return y, size


@pytest.mark.parametrize("dtype, B, Hq, Hk, T, d, page, R, inter, layout, qdim", [
    ("bf16", 3, 8, 2, 1, 128, 16, 128, False, "heads", 3),
    ("bf16", 2, 4, 4, 77, 64, 16, 32, True, "tokens", 4),
    ("bf16", 1, 32, 8, 1, 128, 64, 64, False, "heads", 4),
    ("bf16", 5, 3, 3, 9, 66, 5, 66, False, "apart", 4),
    ("bf16", 2, 0, 2, 6, 7, 3, 6, True, "apart", 4),
    ("bf16", 300, 2, 1, 8, 96, 32, 0, False, "half", 4),
    ("f32", 2, 6, 2, 33, 80, 24, 80, False, "tokens", 4),
    ("f32", 4, 2, 1, 3, 36, 1, 20, True, "heads", 4),
    ("f32", 1, 1, 1, 5, 255, 7, 254, False, "apart", 4),
    ("f32", 2, 16, 16, 1, 256, 128, 256, True, "half", 3),
    ("bf16", 2, 2, 2, 700, 256, 48, 128, False, "heads", 4),
])
def test_append(dtype, B, Hq, Hk, T, d, page, R, inter, layout, qdim):
    g, t = gen(B * 1000 + T), DT[dtype]
    before = [int(x) for x in torch.randint(0, 3 * page + 5, (B,), generator=g, device="cuda")]
    counts = [int(x) for x in torch.randint(0, T + 1, (B,), generator=g, device="cuda")]
    counts[0] = T
    if B > 2:
        before[1] = -1  # a place that is not in use
    table, pages = table_of([n + T for n in before], page, g)
    kc, vc = (pool_of(layout, pages, Hk, page, d, t) for _ in range(2))
    proj = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=g, device="cuda").to(t)
    q, k, v = (proj[..., lo * d:(lo + H) * d].unflatten(-1, (H, d)).transpose(1, 2) if H else None
               for lo, H in ((0, Hq), (Hq, Hk), (Hq + Hk, Hk)))
    freq, offset = la.rope_frequencies(R), 1 << 20
    pos = ints(before).long()[:, None] + torch.arange(T, device="cuda")
    k_ref, k_size = rotated(k, pos + offset, freq, inter)
    cut = (lambda x: x[:, :, 0]) if qdim == 3 else (lambda x: x)
    qo = la.append_cache(cut(k), cut(v), kc, vc, table, ints(before), freq,
                         q=None if q is None else cut(q), counts=ints(counts), offset=offset,
                         interleaved=inter)
    # angles are good to 1.4 u in fp32, to 2^-21 in bf16; two products and a sum on top
    trig = 6 * U if dtype == "f32" else 2.0 ** -20
    if q is not None:
        q_ref, q_size = rotated(q, pos + offset, freq, inter)
        bound = trig * q_size + HALF[dtype] * q_ref.abs()
        assert bool(((qo.view(q.shape).double() - q_ref).abs() <= bound).all())
    else:
        assert qo is None
    want_k, want_v = torch.full(kc.shape, math.nan, device="cuda", dtype=torch.float64), \
        torch.full(kc.shape, math.nan, device="cuda", dtype=torch.float64)
    bound = torch.zeros_like(want_k)
    for b in range(B):
        for i in range(counts[b] if before[b] >= 0 else 0):
            p = before[b] + i
            at = (int(table[b, p // page]), slice(None), p % page)
            want_k[at], want_v[at] = k_ref[b, :, i], v[b, :, i].double()
            bound[at] = trig * k_size[b, :, i] + HALF[dtype] * k_ref[b, :, i].abs()
    assert bool((want_k.isnan() == kc.isnan()).all()) and bool((want_v.isnan() == vc.isnan()).all())
    assert bool(((kc.double() - want_k).abs() <= bound).logical_or(want_k.isnan()).all())
    assert torch.equal(torch.nan_to_num(vc.double(), 9.0), torch.nan_to_num(want_v, 9.0))


def test_append_leaves_tokens_without_a_page_out():
    g = gen(3)
    table = ints([[0, -1, 2], [3, 9, 1]])  # -1 and 9 are no pages of five
    kc, vc = (pool_of("heads", 5, 2, 4, 8, torch.float32) for _ in range(2))
    k, v = (torch.randn(2, 2, 9, 8, generator=g, device="cuda") for _ in range(2))
    la.append_cache(k, v, kc, vc, table, ints([2, 5]))
    # sequence 0: positions 2..10; sequence 1: 5..13, of which 12 and 13 are past the table
    want = torch.full_like(vc, math.nan)
    for b, i, page, slot in ([(0, i, 0, 2 + i) for i in range(2)]
                             + [(0, 6 + i, 2, i) for i in range(3)]
                             + [(1, 3 + i, 1, i) for i in range(4)]):
        want[page, :, slot] = v[b, :, i]
    assert torch.equal(torch.nan_to_num(vc, 9.0), torch.nan_to_num(want, 9.0))
    assert torch.equal(kc.isnan(), want.isnan())


def test_append_in_place_and_features_that_pass():
    g = gen(4)
    kc, vc = (pool_of("heads", 3, 1, 4, 16, torch.bfloat16) for _ in range(2))
    q = torch.randn(1, 2, 3, 16, generator=g, device="cuda").bfloat16()
    k = torch.randn(1, 1, 3, 16, generator=g, device="cuda").bfloat16()
    k[..., 8:] = math.nan
    k[0, 0, 1, 12] = math.inf
    q0 = q.clone()
    freq = la.rope_frequencies(8)
    apart = la.append_cache(k, k, kc, vc, ints([[2]]), ints([0]), freq, q=q)
    assert la.append_cache(k, k, kc, vc, ints([[2]]), ints([0]), freq, q=q, q_out=q) is q
    assert torch.equal(q, apart) and not torch.equal(q[..., :8], q0[..., :8])
    assert torch.equal(q[..., 8:], q0[..., 8:])
    assert torch.equal(kc[2, 0, :3].view(torch.int16)[:, 8:], k[0, 0].view(torch.int16)[:, 8:])
    assert torch.equal(vc[2, 0, :3].view(torch.int16), k[0, 0].view(torch.int16))


# ---------------------------------------------------------------- attention

def plain_attention(q, kc, vc, table, before, scale, window):
    """[B, Hq, T, d] in 64 bits; and the weighted mean of |v| and the largest sum of
    |scale q k| of each row, for the bounds."""
    B, Hq, T, d = q.shape
    P, Hk, page, _ = kc.shape
    out, mean, size = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    for b in range(B):
        n = before[b] + T if before[b] >= 0 else 0
        pos = [p for p in range(n) if p // page < table.shape[1]]
        pages = [int(x) for x in table[b].cpu()]
        pos = [p for p in pos if 0 <= pages[p // page] < P]
        if not pos:
            continue
        at = torch.tensor(pos, device="cuda")
        pg = torch.tensor([pages[p // page] for p in pos], device="cuda")
        k, v = (c[pg, :, at % page].transpose(0, 1).double() for c in (kc, vc))  # [Hk, n, d]
        for t in range(T):
            see = at <= before[b] + t
            if window:
                see &= at > before[b] + t - window
            if not bool(see.any()):
                continue
            kk, vv = k[:, see], v[:, see]
            qq = q[b, :, t].double().unflatten(0, (Hk, Hq // Hk))
            s = torch.einsum("hgd,hnd->hgn", qq, kk) * scale
            w = torch.softmax(s, -1)
            out[b, :, t] = torch.einsum("hgn,hnd->hgd", w, vv).flatten(0, 1)
            mean[b, :, t] = torch.einsum("hgn,hnd->hgd", w, vv.abs()).flatten(0, 1)
            size[b, :, t] = (torch.einsum("hgd,hnd->hgn", qq.abs(), kk.abs()) * abs(scale)).amax(-1).flatten(0, 1)[:, None]
    return out, mean, size


def bound_of(dtype, ref, mean, size, d, n):
    """A score is off by (d + 2) u of its terms, 2 u more for the exponent's product, and
    its weight relative to the others by twice that and 2^-22 for the exponential; sums
    of n terms, cut in at least four, add n / 4 u each (numerator and sum; the tensor
    cores may cut instead of round: 2 u).  With bf16 a weight is rounded by 2^-8 of
    itself, which moves a mean of values by at most twice that of the mean of |v|."""
    rel = 2 * ((d + 4) * 2 * U * size + 2.0 ** -22) + 2 * (n / 4 + 64) * 2 * U
    if dtype == "bf16":
        rel = rel + 2 * 2.0 ** -8
    return rel * mean + HALF[dtype] * ref.abs() + 1e-30


def fill(lengths, table, page, kc, vc, g):
    """Random keys and values at all positions below each length."""
    P, Hk, _, d = kc.shape
    for b, n in enumerate(lengths):
        for c in range(-(-max(n, 0) // page)):
            pg, m = int(table[b, c]), min(page, n - c * page)
            for x in (kc, vc):
                x[pg, :, :m] = torch.randn(Hk, m, d, generator=g, device="cuda").to(x.dtype)


@pytest.mark.parametrize("dtype, lengths, Hq, Hk, T, d, page, window, layout", [
    ("bf16", [1], 1, 1, 1, 64, 16, 0, "heads"),                    # the first token
    ("bf16", [1, 2, 63, 64, 65, 129], 8, 2, 1, 128, 16, 0, "heads"),
    ("bf16", [5000], 4, 1, 1, 128, 64, 0, "tokens"),               # one long sequence
    ("bf16", [700, 3, 1500, 64], 32, 2, 1, 64, 32, 0, "tokens"),   # 16 queries a head
    ("bf16", [300, 40], 12, 1, 3, 96, 24, 0, "heads"),             # 36 of them: three tiles
    ("bf16", [400, 5, 90], 4, 4, 4, 64, 16, 0, "half"),            # drafted tokens
    ("bf16", [1000, 17], 4, 2, 1, 128, 16, 100, "heads"),          # a window
    ("bf16", [1000, 17, 260], 4, 2, 5, 64, 8, 33, "heads"),        # both
    ("bf16", [130, 70], 2, 1, 1, 80, 7, 0, "heads"),               # odd pages
    ("bf16", [130, 70], 2, 1, 2, 66, 5, 0, "apart"),               # no alignment
    ("bf16", [200, 33], 3, 3, 1, 37, 1, 0, "tokens"),              # odd head size, pages of one
    ("bf16", [300, 301], 8, 1, 1, 256, 64, 0, "heads"),
    ("bf16", [90], 6, 2, 7, 192, 16, 20, "half"),
    ("f32", [1, 2, 31, 33, 64, 200], 2, 2, 1, 64, 16, 0, "heads"),
    ("f32", [3000, 10], 6, 2, 1, 80, 24, 0, "tokens"),
    ("f32", [700], 8, 1, 2, 128, 64, 0, "heads"),
    ("f32", [600, 400], 3, 1, 3, 36, 5, 50, "half"),
    ("f32", [130, 4], 4, 2, 1, 256, 16, 0, "heads"),
    ("f32", [130, 65], 5, 1, 1, 61, 3, 0, "apart"),
])
def test_attention(dtype, lengths, Hq, Hk, T, d, page, window, layout):
    g, t = gen(len(lengths) * 100 + d), DT[dtype]
    lengths = [max(n, T) for n in lengths]
    table, pages = table_of(lengths, page, g)
    kc, vc = (pool_of(layout, pages, Hk, page, d, t) for _ in range(2))
    fill(lengths, table, page, kc, vc, g)
    q = (1.5 * torch.randn(len(lengths), T, Hq * d, generator=g, device="cuda")).to(t)
    q = q.view(len(lengths), T, Hq, d).transpose(1, 2)
    before = [n - T for n in lengths]
    if window:  # pages before all windows may be gone
        for b, n in enumerate(before):
            table[b, :max(0, n + 1 - window) // page] = -1
    got = la.decode_step_paged(q, kc, vc, table, ints(before), window=window)
    ref, mean, size = plain_attention(q, kc, vc, table, before, d ** -0.5, window)
    bound = bound_of(dtype, ref, mean, size, d, max(lengths))
    assert got.shape == q.shape and got.dtype == t
    assert bool(((got.double() - ref).abs() <= bound).all()), \
        float(((got.double() - ref).abs() / bound).max())
    # again the same bits, on another stream and into strided rows
    s, out = torch.cuda.Stream(), torch.empty_like(q)
    s.wait_stream(torch.cuda.current_stream())
    la.decode_step_paged(q, kc, vc, table, ints(before), out, window=window, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, got)


@pytest.mark.parametrize("dtype, Hq, Hk, T, d, page, scale", [
    ("bf16", 6, 2, 40, 64, 48, -0.2),   # a short prompt: many tiles of queries
    ("bf16", 2, 1, 33, 200, 16, 0.05),
    ("bf16", 8, 8, 5, 128, 112, 0.0),   # all keys alike
    ("f32", 6, 2, 40, 64, 48, -0.2),
])
def test_more_queries_and_other_scales(dtype, Hq, Hk, T, d, page, scale):
    g, t = gen(T), DT[dtype]
    lengths = [T + 250, T, T + 17]
    table, pages = table_of(lengths, page, g)
    kc, vc = (pool_of("tokens", pages, Hk, page, d, t) for _ in range(2))
    fill(lengths, table, page, kc, vc, g)
    q = torch.randn(3, Hq, T, d, generator=g, device="cuda").to(t)
    before = [n - T for n in lengths]
    got = la.decode_step_paged(q, kc, vc, table, ints(before), scale=scale)
    ref, mean, size = plain_attention(q, kc, vc, table, before, scale, 0)
    bound = bound_of(dtype, ref, mean, size, d, max(lengths))
    assert bool(((got.double() - ref).abs() <= bound).all())
    la.check_device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_batch_with_unused_places_and_missing_pages(dtype):
    g, t = gen(8), DT[dtype]
    lengths = [-1, 40, -7, 100, 0]
    table, pages = table_of(lengths, 16, g)
    kc, vc = (pool_of("heads", pages, 2, 16, 64, t) for _ in range(2))
    fill(lengths, table, 16, kc, vc, g)
    table[3, 2] = pages + 4   # no page: its 16 keys are left out
    table[1, :] = -1          # none at all: nothing to look at
    before = [-1, 39, -7, 99, 5]  # the last one's table holds no page
    q = torch.randn(5, 4, 64, generator=g, device="cuda").to(t)
    got = la.decode_step_paged(q, kc, vc, table, ints(before), scale=0.3)
    ref, mean, size = plain_attention(q[:, :, None], kc, vc, table, before, 0.3, 0)
    bound = bound_of(dtype, ref, mean, size, 64, 100)[:, :, 0]
    assert bool(((got.double() - ref[:, :, 0]).abs() <= bound).all())
    for b in (0, 1, 2, 4):
        assert not bool(got[b].any())
    assert bool(got[3].any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_a_query_does_not_look_at_does_not_reach_it(dtype):
    # the second of two drafted tokens is not finite, and so are keys before a window
    g, t = gen(9), DT[dtype]
    table, pages = table_of([70], 16, g)
    kc, vc = (pool_of("heads", pages, 1, 16, 64, t) for _ in range(2))
    fill([70], table, 16, kc, vc, g)
    q = torch.randn(1, 2, 2, 64, generator=g, device="cuda").to(t)
    clean = la.decode_step_paged(q, kc, vc, table, ints([68]))
    for value in (math.inf, math.nan):
        for x in (kc, vc):
            x[int(table[0, 4]), :, 5, ::3] = value  # position 69
        got = la.decode_step_paged(q, kc, vc, table, ints([68]))
        assert torch.equal(got[:, :, 0], clean[:, :, 0]) or float(
            (got[:, :, 0].double() - clean[:, :, 0].double()).abs().max()) <= 2.0 ** -7
        assert not bool(got[:, :, 1].isfinite().all())
        # a window of one key per token: 68 sees itself, 69 not finite
        got = la.decode_step_paged(q, kc, vc, table, ints([68]), window=1)
        assert torch.equal(got[0, 0, 0], vc[int(table[0, 4]), 0, 4])


def test_extreme_scores():
    g = gen(10)
    table, pages = table_of([200], 16, g)
    kc, vc = (pool_of("heads", pages, 1, 16, 64, torch.bfloat16) for _ in range(2))
    fill([200], table, 16, kc, vc, g)
    q = torch.zeros(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 1e18
    kc[..., 0] = torch.where(kc[..., 0].isnan(), kc[..., 0], torch.full_like(kc[..., 0], -1e18))
    at = int(table[0, 7])
    kc[at, 0, 3, 0] = 1e18  # one key far above the others: its value comes back
    got = la.decode_step_paged(q, kc, vc, table, ints([199]), scale=1.0)
    assert torch.equal(got[0, 0], vc[at, 0, 3])
    # equal scores, as low as they get: the mean of the values
    kc[at, 0, 3, 0] = -1e18
    got = la.decode_step_paged(q, kc, vc, table, ints([199]), scale=1.0)
    mean = torch.cat([vc[int(table[0, c]), 0, :min(16, 200 - 16 * c)] for c in range(13)]).double().mean(0)
    assert float((got[0, 0].double() - mean).abs().max()) <= 2.0 ** -8 * 3


def test_offsets_beyond_32_bits():
    # a pool of more than 2^31 elements: the sequence's pages lie at its end
    pages = (1 << 31) // (64 * 128) + 40
    kc = torch.zeros(pages, 1, 64, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = gen(11)
    table = ints([[pages - 1, 0, pages - 30, pages - 7]])
    k, v = (torch.randn(1, 1, 250, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    la.append_cache(k, v, kc, vc, table, ints([0]))
    assert torch.equal(vc[pages - 7, 0, :58], v[0, 0, 192:])
    q = torch.randn(1, 4, 128, generator=g, device="cuda").bfloat16()
    got = la.decode_step_paged(q, kc, vc, table, ints([249]))
    ref, mean, size = plain_attention(q[:, :, None], kc, vc, table, [249], 128 ** -0.5, 0)
    assert bool(((got[:, :, None].double() - ref).abs() <=
                 bound_of("bf16", ref, mean, size, 128, 250)).all())


@pytest.mark.parametrize("dtype, d, page", [("bf16", 64, 16), ("bf16", 80, 7), ("bf16", 33, 16),
                                            ("bf16", 256, 32), ("f32", 48, 16)])
def test_many_sequences_and_one_list(dtype, d, page):
    # more sequences than threads of a block, of all lengths: the pieces' borders fall
    # anywhere, and a block has many stretches
    g = gen(12)
    lengths = [int(x) for x in torch.randint(1, 300, (700,), generator=g, device="cuda")]
    table, pages = table_of(lengths, page, g)
    kc, vc = (pool_of("heads", pages, 2, page, d, DT[dtype]) for _ in range(2))
    for x in (kc, vc):
        x.normal_(generator=g)
    q = torch.randn(700, 4, d, generator=g, device="cuda").to(DT[dtype])
    got = la.decode_step_paged(q, kc, vc, table, ints([n - 1 for n in lengths]))
    some = list(range(0, 700, 41))
    ref, mean, size = plain_attention(q[some][:, :, None], kc, vc, table[some],
                                      [lengths[b] - 1 for b in some], d ** -0.5, 0)
    assert bool(((got[some][:, :, None].double() - ref).abs() <=
                 bound_of(dtype, ref, mean, size, d, 300)).all())
    # each sequence alone: other pieces, the same within rounding
    for b in some[:4]:
        one = la.decode_step_paged(q[b:b + 1], kc, vc, table[b:b + 1], ints([lengths[b] - 1]))
        assert float((one.double() - got[b:b + 1].double()).abs().max()) <= 2.0 ** -6


def test_a_captured_step_follows_the_lengths():
    # one graph of append and attention, replayed while lengths and table grow
    g = gen(13)
    Hq, Hk, d, page = 4, 2, 64, 16
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6)
    kc, vc = (pool_of("heads", 6, Hk, page, d, torch.bfloat16) for _ in range(2))
    q, k, v = (torch.randn(90, 1, H, d, generator=g, device="cuda").bfloat16() for H in (Hq, Hk, Hk))
    freq, lengths = la.rope_frequencies(d), ints([0])
    qi, ki, vi = q[0].clone(), k[0].clone(), v[0].clone()
    kc2, vc2 = kc.clone(), vc.clone()

    def step(kc, vc, lengths):
        r = la.append_cache(ki, vi, kc, vc, table, lengths, freq, q=qi)
        return la.decode_step_paged(r, kc, vc, table, lengths)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(kc2, vc2, lengths)
    torch.cuda.current_stream().wait_stream(s)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(kc, vc, lengths)
        lengths += 1
    with torch.cuda.graph(other):  # a second graph between: no workspace in common
        out2 = step(kc2, vc2, lengths)
    lengths.zero_()
    kc.fill_(math.nan)
    vc.fill_(math.nan)
    eager, len2 = [], ints([0])
    for t in range(90):
        qi.copy_(q[t]), ki.copy_(k[t]), vi.copy_(v[t])
        graph.replay()
        mine = out.clone()
        len2.fill_(t)
        lengths.fill_(t)
        other.replay()
        assert torch.equal(out2, mine), t
        assert torch.equal(step(kc2, vc2, len2), mine), t
        lengths.fill_(t + 1)
    assert torch.equal(kc, kc2) or bool((kc.isnan() == kc2.isnan()).all())


def test_a_workspace_that_cannot_be_had():
    lib = la.load_library()
    kc = torch.zeros(4, 1, 16, 64, device="cuda")
    q, table, s = torch.zeros(1, 1, 64, device="cuda"), ints([[0, 1, 2, 3]]), torch.cuda.Stream()
    args = (q, kc, kc.clone(), table, ints([50]))
    torch.cuda.synchronize()
    lib.la_debug_fail_next_allocs(1)
    try:
        with pytest.raises(la.LinAttnError) as e:
            la.decode_step_paged(*args, stream=s)
        assert e.value.status == 4
    finally:
        lib.la_debug_fail_next_allocs(0)
    assert not bool(la.decode_step_paged(*args, stream=s).any())
    torch.cuda.synchronize()
