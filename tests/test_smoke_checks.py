"""The smoke run's check of the token-mixing operators has to refuse wrong results:
a plain implementation passes it, and each of its mistakes, planted here on the CPU
one at a time, does not.  Needs no GPU."""
import types

import pytest

import __graft_entry__ as entry
import linear_attention_feature_gb300 as la

torch = pytest.importorskip("torch")


def turned(u, freq, sign):
    t = torch.arange(u.shape[2]).double()[:, None] * torch.tensor(list(freq), dtype=torch.float64)
    c, s = t.cos(), sign * t.sin()
    u1, u2 = u.chunk(2, -1)
    return torch.cat((u1 * c - u2 * s, u2 * c + u1 * s), -1)


def norm_back(dy, v, w, freq, wrong):
    dy, v = dy.double(), v.double()
    size = (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    n = v / size
    g = turned(dy, freq, 1.0 if wrong == "turned on" else -1.0)
    dw = (g * n).sum((0, 1, 2) if wrong != "one head's dw" else (0, 2))
    if wrong == "one head's dw":
        dw = dw[0]
    g = g * w.double()
    mean = 0.0 if wrong == "no mean" else (g * n).mean(-1, keepdim=True)
    dx = (g - n * mean) / size
    return (torch.zeros_like(dx) if wrong == "zeros" else dx).float(), dw.float()


def library(wrong=None):
    def qk(q, k, wq, wk, freq):
        out = []
        for v, w in ((q, wq), (k, wk)):
            v = v.double()
            n = v / (v.square().mean(-1, keepdim=True) + (0.1 if wrong == "eps" else 1e-6)).sqrt()
            out.append(turned(n * w, freq, 1.0).float())
        return tuple(out)

    def qk_back(dq, dk, q, k, wq, wk, freq):
        a, b = norm_back(dq, q, wq, freq, wrong), norm_back(dk, k, wk, freq, wrong)
        return (a[0], a[0] if wrong == "dk is dq" else b[0], a[1], b[1])

    def gates(z):
        a = torch.sigmoid(z.double())
        return a, 1 - a

    def rec(x, z, h0, gate, complement):
        a, rest = gates(z)
        h, hs = h0.double(), []
        if wrong == "no h0":
            h = torch.zeros_like(h)
        for i in range(x.shape[1]):
            h = a[:, i] * h + rest[:, i] * x[:, i].double()
            hs.append(h)
        return torch.stack(hs, 1).float(), h.float()

    def rec_back(dout, z, out, x, h0, dh, gate, complement):
        a, rest = gates(z)
        g, gs = dh.double(), []
        if wrong == "no dh_last":
            g = torch.zeros_like(g)
        for i in range(x.shape[1] - 1, -1, -1):
            if wrong == "nothing carried" and i + 1 < x.shape[1]:
                g = torch.zeros_like(g)
            g = dout[:, i].double() + g
            gs.append(g)
            g = a[:, i] * g
        gs = torch.stack(gs[::-1], 1)
        before = torch.cat((h0[:, None], out[:, :-1]), 1).double()
        if wrong != "dgates without x":
            before = before - x.double()
        dx = gs if wrong == "dx without 1 - a" else gs * rest
        return dx.float(), (a * rest * gs * before).float(), (gs[:, 0] if wrong == "dh0" else g).float()

    return types.SimpleNamespace(rope_frequencies=la.rope_frequencies, qk_norm_rope=qk,
                                 backward_qk_norm_rope=qk_back, forward_recurrence=rec,
                                 backward_recurrence=rec_back, check_device_status=lambda: None)


def test_the_plain_implementation_passes():
    entry.check_token_mixing(library(), "cpu")


@pytest.mark.parametrize("wrong, name", [
    ("eps", "q"), ("zeros", "dq"), ("turned on", "dq"), ("no mean", "dq"), ("dk is dq", "dk"),
    ("one head's dw", "dq_weight"), ("no h0", "out"), ("nothing carried", "dx"),
    ("no dh_last", "dx"), ("dgates without x", "dgates"), ("dx without 1 - a", "dx"),
    ("dh0", "dh0")])
def test_each_mistake_is_refused(wrong, name):
    with pytest.raises(RuntimeError, match=f"{name} off by"):
        entry.check_token_mixing(library(wrong), "cpu")
