"""A decoder layer of a hybrid encoder-decoder, as the operators are used together:
a prompt goes into the paged cache, then token after token is normed, rotated and
appended, attends to the cache, and looks at the encoder's states."""
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


def test_prompt_then_tokens_equal_the_whole():
    B, Hq, Hk, d, page, M, prompt, total = 3, 4, 2, 64, 16, 90, [20, 1, 33], 45
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    proj = normal(B, total, (Hq + 2 * Hk) * d)
    cq = normal(B, total, Hq * d).view(B, total, Hq, d).transpose(1, 2)
    ek, ev = normal(B, Hk, M, d), normal(B, Hk, M, d)
    frames = torch.tensor([90, 30, 61], dtype=torch.int32, device="cuda")
    heads = lambda x, lo, H: x[..., lo * d:(lo + H) * d].unflatten(-1, (H, d)).transpose(1, 2)  # noqa: E731
    q, k, v = heads(proj, 0, Hq), heads(proj, Hq, Hk), heads(proj, Hq + Hk, Hk)
    wq, wk, freq = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d), la.rope_frequencies(d)

    # the whole in 64 bits
    t = torch.arange(total, device="cuda").double()[:, None] * torch.tensor(
        list(freq), dtype=torch.float64, device="cuda")

    def rows(x, w):
        x = x.double()
        u = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        a, b = u[..., :d // 2], u[..., d // 2:]
        return torch.cat((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()), -1)

    Q = rows(q, wq).unflatten(1, (Hk, Hq // Hk))
    score = torch.einsum("bhgnd,bhmd->bhgnm", Q, rows(k, wk)) / d ** 0.5
    score = score.masked_fill(~torch.ones(total, total, dtype=torch.bool, device="cuda").tril(), -1e300)
    own = torch.einsum("bhgnm,bhmd->bhgnd", score.softmax(-1), v.double()).flatten(1, 2)
    f = lambda x: torch.where(x > 0, x + 1, torch.exp(x))  # noqa: E731
    keep = (torch.arange(M, device="cuda") < frames[:, None])[:, None, :, None]
    w = torch.einsum("bhgna,bhma->bhgnm", f(cq.double()).unflatten(1, (Hk, Hq // Hk)),
                     f(ek.double()) * keep)
    other = torch.einsum("bhgnm,bhmd->bhgnd", w / w.sum(-1, keepdim=True), ev.double()).flatten(1, 2)

    # the library: the cache, and the encoder's states once
    table = torch.randperm(B * 4, generator=g, device="cuda").int()[:B * 3].view(B, 3)
    kc = torch.full((B * 4, page, Hk, d), float("nan"), device="cuda").transpose(1, 2)
    vc = kc.clone()
    counts = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    longest = max(prompt)
    cross, S, z = la.forward_cross(cq[:, :, :longest], ek, ev, frames)
    qn, kn = la.qk_norm_rope(q[:, :, :longest], k[:, :, :longest], wq, wk)
    qr = la.append_cache(kn, v[:, :, :longest], kc, vc, table, lengths, freq, q=qn, counts=counts)
    y = la.decode_step_paged(qr, kc, vc, table, lengths)
    # scores of some units good to d u, sums of 45 and 90 terms, three stages
    tol = 2.0 ** 10 * 2.0 ** -24
    for b, n in enumerate(prompt):
        assert float((y[b, :, :n] - own[b, :, :n]).abs().max()) <= tol * 4
        assert float((cross[b, :, :n] - other[b, :, :n]).abs().max()) <= tol * 4
    lengths += counts
    for _ in range(total - longest):
        at = lengths.long()
        pick = lambda x: torch.stack([x[b, :, int(at[b])] for b in range(B)])  # noqa: E731
        qn, kn = la.qk_norm_rope(pick(q), pick(k), wq, wk)
        qr = la.append_cache(kn, pick(v), kc, vc, table, lengths, freq, q=qn)
        y = la.decode_step_paged(qr, kc, vc, table, lengths)
        c = la.decode_step_cross(S, z, pick(cq))
        assert float((y - pick(own)).abs().max()) <= tol * 4
        assert float((c - pick(other)).abs().max()) <= tol * 4
        lengths += 1
    la.check_device_status()
