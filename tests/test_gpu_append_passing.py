"""Features that the rotation of an append passes, bit for bit: next to rotated ones
in one access, and with values that no arithmetic keeps."""
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


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype, d, rotary", [
    ("bf16", 16, 2), ("bf16", 16, 6), ("bf16", 16, 8), ("bf16", 64, 20), ("bf16", 64, 40),
    ("bf16", 18, 4), ("bf16", 17, 6), ("bf16", 128, 0), ("bf16", 24, 24),
    ("f32", 16, 2), ("f32", 16, 4), ("f32", 16, 6), ("f32", 36, 10), ("f32", 33, 12),
])
def test_features_that_pass(dtype, d, rotary, interleaved):
    g = torch.Generator(device="cuda")
    g.manual_seed(d + rotary)
    t, words = (torch.bfloat16, torch.int16) if dtype == "bf16" else (torch.float32, torch.int32)
    top = torch.iinfo(words).max
    # any bits: NaN of either sign and with any payload among them, numbers too small to be normal
    q, k, v = (torch.randint(-top - 1, top, (2, H, 5, d), generator=g, device="cuda",
                             dtype=words) for H in (3, 2, 2))
    for x in (q, k):  # what is rotated is finite
        x.view(t)[..., :rotary] = torch.randn(*x.shape[:3], rotary, generator=g, device="cuda").to(t)
    nan = 0x7FC0 if dtype == "bf16" else 0x7FC00000
    for x in (q, k, v):
        x[..., -1] = nan + 5                   # a payload
        if d - rotary > 1 or x is v:
            x[..., -2] = nan + 3 - top - 1     # the other sign
    if rotary == d:
        q.view(t).copy_(torch.randn(q.shape, generator=g, device="cuda").to(t))
        k.view(t).copy_(torch.randn(k.shape, generator=g, device="cuda").to(t))
    kc, vc = (torch.zeros(3, 2, 4, d, dtype=t, device="cuda") for _ in range(2))
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    freq = la.rope_frequencies(rotary) if rotary else None
    out = la.append_cache(k.view(t), v.view(t), kc, vc, table, lengths, freq, q=q.view(t),
                          interleaved=interleaved)
    assert torch.equal(out.view(words)[..., rotary:], q[..., rotary:])
    for b, at in ((0, [(2, 1), (2, 2), (2, 3), (0, 0), (0, 1)]), (1, [(1, i) for i in range(4)])):
        for i, (page, slot) in enumerate(at):
            assert torch.equal(kc.view(words)[page, :, slot, rotary:], k[b, :, i, rotary:])
            assert torch.equal(vc.view(words)[page, :, slot], v[b, :, i])
    assert bool(out[..., :rotary].isfinite().all())
    if rotary:  # (the second token of the second sequence is at position 1)
        assert not torch.equal(out[1, :, 1, :rotary], q.view(t)[1, :, 1, :rotary])
