"""The smoke run's check of the paged cache and the cross attention has to refuse wrong
results: a plain implementation passes it, and each of its mistakes, planted here on the
CPU one at a time, does not.  Needs no GPU."""
import types

import pytest

import __graft_entry__ as entry

torch = pytest.importorskip("torch")


def phi(x):
    return torch.where(x > 0, x + 1, torch.exp(x))


def groups(x, S):
    return x.double().unflatten(1, (S.shape[1], -1))


def library(wrong=None):
    def append(k, v, kc, vc, table, before):
        for b in range(k.shape[0]):
            for t in range(k.shape[2]):
                p = int(before[b]) + t + (wrong == "a slot late")
                at = int(table[b, p // 16 % table.shape[1]])
                kc[at, :, p % 16], vc[at, :, p % 16] = k[b, :, t], v[b, :, t]

    def paged(q, kc, vc, table, before):
        B, Hq, T, d = q.shape
        k, v = (torch.stack([c[table[b].long()].transpose(0, 1).flatten(1, 2)[:, :T]
                             for b in range(B)]).double() for c in (kc, vc))
        s = torch.einsum("bhgnd,bhmd->bhgnm", groups(q, k), k) * (1 if wrong == "scale" else d ** -0.5)
        if wrong != "no mask":
            s = s.masked_fill(~torch.ones(T, T, dtype=torch.bool).tril(), -1e300)
        y = torch.einsum("bhgnm,bhmd->bhgnd", s.softmax(-1), v)
        if wrong == "heads the other way round":
            y = y.flip(2)
        return y.flatten(1, 2).float()

    def read(S, z, q):
        f = phi(groups(q if q.dim() == 4 else q[:, :, None], S))
        y = f @ S[:, :, None] / (f @ z[:, :, None, :, None])
        y = y.flatten(1, 2)
        return (y if q.dim() == 4 else y[:, :, 0]).float()

    def cross(q, k, v, lengths):
        g = phi(k.double())
        if wrong != "padding":
            g = g * (torch.arange(k.shape[2]) < lengths[:, None])[:, None, :, None]
        S, z = g.transpose(2, 3) @ v.double(), g.sum(2)
        return read(S, z, q), S, z

    def back(dout, q, k, v, S, z, lengths):
        Q, dy = groups(q, S), groups(dout, S)
        f = phi(Q)
        r = 1 / (f @ z[:, :, None, :, None])
        G = dy @ S[:, :, None].transpose(-1, -2)
        t = (f * G).sum(-1, keepdim=True) * r
        if wrong == "no mean":
            t = 0 * t
        dq = (G - t * z[:, :, None, None]) * r * torch.exp(Q.clamp(max=0))
        w = f * r
        dS = torch.einsum("bhgna,bhgnc->bhac", w, dy)
        if wrong == "one head's dS":
            dS = w[:, :, 0].transpose(2, 3) @ dy[:, :, 0]
        dz = -(w * t).sum((2, 3))
        keep = (torch.arange(k.shape[2]) < lengths[:, None])[:, None, :, None]
        k, v = k.double(), v.double()
        dk = (v @ dS.transpose(2, 3) + dz[:, :, None]) * keep
        if wrong != "no slope":
            dk = dk * torch.exp(k.clamp(max=0))
        dv = phi(k) * keep @ dS
        if wrong == "dv is dk":
            dv = dk
        return dq.flatten(1, 2).float(), dk.float(), dv.float()

    step = (lambda S, z, q: read(S, torch.ones_like(z), q)) if wrong == "a step without z" else read
    return types.SimpleNamespace(append_cache=append, decode_step_paged=paged, forward_cross=cross,
                                 backward_cross=back, decode_step_cross=step,
                                 check_device_status=lambda: None)


def test_a_right_library_passes():
    entry.check_decoder(library(), torch.device("cpu"))


@pytest.mark.parametrize("wrong", ["a slot late", "scale", "no mask", "heads the other way round",
                                   "padding", "no mean", "one head's dS", "no slope", "dv is dk",
                                   "a step without z"])
def test_a_mistake_is_refused(wrong):
    with pytest.raises(RuntimeError, match="smoke: decoder"):
        entry.check_decoder(library(wrong), torch.device("cpu"))
