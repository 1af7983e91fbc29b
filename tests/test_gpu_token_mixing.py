"""The operators in a row, as a recurrent linear-attention layer uses them:
the gated recurrence mixes the token stream per channel, a projection makes q,
k and v out of it, q and k are normed and rotated, causal linear attention
reads them; then the same sequences are continued token by token.  And the
training direction of the same front end, against 64-bit automatic
differentiation."""
import math

import pytest

import oracle
import linear_attention_feature_gb300 as la
from linear_attention_feature_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
B, H, N, D = 2, 3, 150, 64
C = H * D


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def layer(dtype, seed, tokens=N):
    g = torch.Generator().manual_seed(seed)
    t = wl.torch_dtype(dtype)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return {"x": r(B, tokens, C).to(t), "z": (r(B, tokens, C) + 2).to(t),
            "W": (r(C, 3 * C) / math.sqrt(C)).to(t), "wq": 1 + 0.1 * r(D), "wk": 1 + 0.1 * r(D)}


def heads(p, i):
    """Third i of a projection [B, N, 3 C] as a [B, H, N, D] view."""
    return p[..., i * C:(i + 1) * C].unflatten(-1, (H, D)).transpose(1, 2)


def test_prefill_then_decode_equals_the_whole():
    p = {k: v.cuda() for k, v in layer("f32", 5).items()}
    freq = la.rope_frequencies(D)
    # whole sequences
    mixed, h_end = la.forward_recurrence(p["x"], p["z"], gate="logit", complement=True)
    proj = (mixed.double() @ p["W"].double()).float()
    q, k = la.qk_norm_rope(heads(proj, 0), heads(proj, 1), p["wq"], p["wk"], freq)
    v = heads(proj, 2).contiguous()
    whole, S_end, z_end = la.forward_causal_state(q, k, v)
    la.check_device_status()
    ref = oracle.causal(q.cpu(), k.cpu(), v.cpu())
    assert wl.max_row_rel_err(whole.cpu(), ref) <= wl.TOL["f32"]
    # a prefill of 130 tokens, then single tokens
    n0 = 130
    mixed, h = la.forward_recurrence(p["x"][:, :n0], p["z"][:, :n0], gate="logit", complement=True)
    proj0 = (mixed.double() @ p["W"].double()).float()
    q, k = la.qk_norm_rope(heads(proj0, 0), heads(proj0, 1), p["wq"], p["wk"], freq)
    y, S, z = la.forward_causal_state(q, k, heads(proj0, 2).contiguous())
    assert wl.max_row_rel_err(y.cpu(), ref[:, :, :n0]) <= wl.TOL["f32"]
    for t in range(n0, N):
        m = la.decode_step_recurrence(h, p["x"][:, t], p["z"][:, t], gate="logit", complement=True)
        pt = (m.double() @ p["W"].double()).float()[:, None]
        pos = torch.full((B,), t, device="cuda")
        q, k = la.qk_norm_rope(heads(pt, 0)[:, :, 0], heads(pt, 1)[:, :, 0], p["wq"], p["wk"],
                               freq, pos)
        y = la.decode_step(S, z, q, k, heads(pt, 2)[:, :, 0].contiguous())
        assert wl.max_row_rel_err(y.cpu(), ref[:, :, t]) <= wl.TOL["f32"], t
    la.check_device_status()
    for got, want in ((h, h_end), (S, S_end), (z, z_end)):
        assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())


def test_rotated_retention_on_the_tensor_cores():
    # bf16: normed and rotated q and k into retention (identity map, no
    # normaliser, decay), which then sees relative positions only
    p = {k: v.cuda() for k, v in layer("bf16", 6, 500).items()}
    freq = la.rope_frequencies(D)
    mixed, _ = la.forward_recurrence(p["x"], p["z"], gate="logit", complement=True)
    proj = mixed @ p["W"]
    v = heads(proj, 2).contiguous()
    dec = [0.96875, 0.984375, 0.9921875]
    scale = D ** -0.25
    ys = []
    for offset in (0, 1 << 20):
        q, k = la.qk_norm_rope(heads(proj, 0), heads(proj, 1), p["wq"] * scale, p["wk"] * scale,
                               freq, offset=offset)
        ys.append(la.forward_variant(q, k, v, decay=dec, feature_map="identity", normalise=False))
        la.check_device_status()
        ref = oracle.causal(q.float().cpu(), k.float().cpu(), v.float().cpu(), dec,
                            fmap=oracle.FMAP_IDENTITY, normalise=False)
        assert wl.max_row_rel_err(ys[-1].cpu(), ref) <= wl.TOL["bf16"]
    # q and k are rounded to bf16 at other angles: each of the products'
    # factors is off by 2^-8, and a row sums some dozens of them
    norm = ys[0].float().norm()
    assert float((ys[1].float() - ys[0].float()).norm() / norm) <= 2 * 2.0 ** -8 + 2 * wl.TOL["bf16"]


def test_gradients_of_the_front_end():
    p = layer("f32", 7)
    freq = la.rope_frequencies(D)
    g = torch.Generator().manual_seed(8)
    gq, gk = torch.randn(B, H, N, D, generator=g), torch.randn(B, H, N, D, generator=g)
    # 64-bit automatic differentiation of the formulas
    x, z, W, wq, wk = (p[n].double().requires_grad_() for n in ("x", "z", "W", "wq", "wk"))
    a = torch.sigmoid(z)
    h, hs = torch.zeros(B, C, dtype=torch.float64), []
    for t in range(N):
        h = a[:, t] * h + (1 - a[:, t]) * x[:, t]
        hs.append(h)
    proj = torch.stack(hs, 1) @ W
    angle = torch.arange(N).double()[:, None] * torch.tensor(list(freq), dtype=torch.float64)
    loss = 0.0
    for i, w, gy in ((0, wq, gq), (1, wk, gk)):
        r = heads(proj, i)
        u = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-6) * w
        u1, u2 = u[..., :D // 2], u[..., D // 2:]
        y = torch.cat((u1 * angle.cos() - u2 * angle.sin(), u2 * angle.cos() + u1 * angle.sin()), -1)
        loss = loss + (y * gy.double()).sum()
    loss.backward()
    # the library
    d = {n: t.cuda() for n, t in p.items()}
    mixed, _ = la.forward_recurrence(d["x"], d["z"], gate="logit", complement=True)
    pr = (mixed.double() @ d["W"].double()).float()
    dpr = torch.zeros_like(pr)
    _, _, dwq, dwk = la.backward_qk_norm_rope(gq.cuda(), gk.cuda(), heads(pr, 0), heads(pr, 1),
                                              d["wq"], d["wk"], freq, dq=heads(dpr, 0),
                                              dk=heads(dpr, 1))
    dmixed = (dpr.double() @ d["W"].double().T).float()
    dx, dz, _ = la.backward_recurrence(dmixed, d["z"], mixed, d["x"], gate="logit",
                                       complement=True)
    dW = torch.einsum("bnc,bnk->ck", mixed.double(), dpr.double())
    # each stage is good to some tens of u = 2^-24 of its terms' size; the
    # sums over 150 tokens and 192 channels are far shorter than 2^10 terms
    for got, leaf in ((dx, x), (dz, z), (dW, W), (dwq, wq), (dwk, wk)):
        err = (got.cpu().double() - leaf.grad).abs().max()
        assert float(err) <= 2.0 ** 10 * 2.0 ** -24 * float(leaf.grad.abs().max())
