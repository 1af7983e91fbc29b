"""Workloads of the operators around a cache and an encoder: new keys and values
appended to a paged cache with the rotation on the way, the softmax attention of
new tokens over that cache, and linear cross attention to an encoder's tokens
(forward, backward and single tokens), in plain torch and through the library."""
import math
import random
from array import array

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one new token of a single stream: what counts is the call itself
        append("append b1", 1, 32, 8, 1, 128, 64, 30000, 128, "bf16"),
        # prompts of unequal length go into the cache, out of the fused projection
        append("append prompts b8 t8192", 8, 32, 8, 8192, 128, 64, 0, 128, "bf16"),
        # a long conversation of a single stream: the length has to give the parallelism
        attend("attend b1 n131072", 1, 32, 8, 1, 128, 64, 131072, "bf16"),
        # a full serving batch, every sequence at a length of its own
        attend("attend b256 n4096", 256, 32, 8, 1, 128, 64, 4096, "bf16"),
        # four drafted tokens of each stream are looked at in one call, head size 64
        attend("attend drafts b32 n8192 d64", 32, 16, 16, 4, 64, 16, 8192, "bf16"),
        # full precision: an odd head size, odd pages, a window
        attend("attend f32 d80 window", 7, 6, 2, 1, 80, 24, 5000, "f32", window=1000),
        # a decoder's prompt looks at audio frames, batch padded to the longest
        cross("cross b16 h16 n448 m1500 d64", "cross", 16, 16, 16, 448, 1500, 64, "bf16", True),
        # long documents on the encoder's side, shared heads
        cross("cross b4 h32 n4096 m16384 d128", "cross", 4, 32, 8, 4096, 16384, 128, "bf16", True),
        # training, sequences of unequal length on the two sides
        cross("cross back b4 h8 n4096 m16384 d128", "cross_back", 4, 8, 8, 4096, 16384, 128,
              "bf16", True),
        # training in full precision: an odd head size, shared heads, odd lengths
        cross("cross back f32 d80", "cross_back", 3, 6, 2, 333, 1001, 80, "f32", True),
        # one decoder token of a full serving batch reads the encoder's states
        cross("cross step b256 h32 d128", "cross_step", 256, 32, 32, 1, 0, 128, "bf16", False),
        # the same of a single stream with shared heads
        cross("cross step b1 h32", "cross_step", 1, 32, 8, 1, 0, 128, "bf16", False),
    ]


def append(name, B, Hq, Hk, T, d, page, before, rotary, dtype, interleaved=False, mix=1):
    """T new tokens (fewer in some sequences) behind up to `before` old ones."""
    c = {"op": "append", "B": B, "Hq": Hq, "Hk": Hk, "T": T, "d": d, "page": page,
         "before": before, "rotary": rotary, "dtype": dtype, "interleaved": interleaved,
         "mix": mix}
    return dict(c, name=name) if name else c


def attend(name, B, Hq, Hk, T, d, page, longest, dtype, window=0, mix=1):
    c = {"op": "attend", "B": B, "Hq": Hq, "Hk": Hk, "T": T, "d": d, "page": page,
         "longest": longest, "dtype": dtype, "window": window, "mix": mix}
    return dict(c, name=name) if name else c


def cross(name, op, B, Hq, Hk, N, M, d, dtype, ragged, feature_map="elu1", normalise=True, mix=1):
    c = {"op": op, "B": B, "Hq": Hq, "Hk": Hk, "N": N, "M": M, "d": d, "dtype": dtype,
         "ragged": ragged, "feature_map": feature_map, "normalise": normalise, "mix": mix}
    return dict(c, name=name) if name else c


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend", "cross", "cross_back", "cross_step"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 64, 128, 256, 80, 96, rng.randint(8, 200)])
    Hk = spread(1, 16)
    Hq = Hk * rng.choice([1, 1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 64, 128, 256, rng.randint(1, 100)])
    mix = rng.randint(0, 1 << 20)
    if op == "append":
        d += d % 2
        rotary = d if rng.random() < 0.6 else 2 * rng.randint(0, d // 2)
        B = spread(1, 256)
        T = 1 if rng.random() < 0.5 else spread(1, max(2, min(8192, (1 << 23) // (B * Hq * d) * 8)))
        before = 0 if rng.random() < 0.3 else spread(1, max(2, min(65536, (1 << 28) // (B * Hk * d))))
        return append(None, B, Hq, Hk, T, d, page, before, rotary, dtype,
                      rng.random() < 0.3, mix)
    if op == "attend":
        B = spread(1, 256)
        T = rng.choice([1, 1, 1, 2, 4, 7])
        longest = spread(T, max(T + 1, min(131072, (1 << 29) // (B * Hk * d))))
        window = 0 if rng.random() < 0.7 else spread(1, longest)
        return attend(None, B, Hq, Hk, T, d, page, longest, dtype, window, mix)
    feature_map, normalise = ("elu1", True) if rng.random() < 0.75 else ("identity", False)
    if op == "cross_step":
        B = spread(1, max(2, min(256, (1 << 27) // (Hk * d * d))))
        return cross(None, op, B, Hq, Hk, 1, 0, d, dtype, False, feature_map, normalise, mix)
    B, most = spread(1, 16), 1 << (26 if dtype == "bf16" else 24)
    N = spread(1, max(2, min(16384, most // (B * Hq * d))))
    M = spread(1, max(2, min(32768, most // (B * Hk * d))))
    return cross(None, op, B, Hq, Hk, N, M, d, dtype, rng.random() < 0.7, feature_map,
                 normalise, mix)


# Lengths belong to the case: a program's scheduler holds them on the host, too.

def _counts(c):
    """(tokens before the call, new tokens) of each sequence of an append."""
    r = random.Random(c["mix"])
    return [(r.randint(c["before"] // 2, c["before"]),
             c["T"] if c["T"] == 1 else r.randint((c["T"] + 1) // 2, c["T"]))
            for _ in range(c["B"])]


def _lengths(c):
    """Tokens in the cache of each sequence, the call's own among them; the
    first is the longest."""
    r = random.Random(c["mix"])
    low = max(c["T"], c["longest"] // 8)
    return [c["longest"]] + [r.randint(low, c["longest"]) for _ in range(c["B"] - 1)]


def _frames(c):
    """Tokens of each sequence on the encoder's side; the first is the longest."""
    r = random.Random(c["mix"])
    if not c["ragged"]:
        return [c["M"]] * c["B"]
    return [c["M"]] + [r.randint((c["M"] + 1) // 2, c["M"]) for _ in range(c["B"] - 1)]


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def integers(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    s = dict(case)
    B, Hq, Hk, d, t = case["B"], case["Hq"], case["Hk"], case["d"], DT[case["dtype"]]

    def cache(lengths):
        """Pages in any order, as a pool that has been in use for a while gives them."""
        page = case["page"]
        need = [-(-n // page) for n in lengths]
        s["pages"] = sum(need) + 3
        order = torch.randperm(s["pages"], generator=gen, device="cuda").int()
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table
        for name in ("k_cache", "v_cache"):
            s[name] = torch.empty(s["pages"], Hk, page, d, dtype=t, device="cuda").normal_(
                generator=gen)

    if case["op"] == "append":
        T, R = case["T"], case["rotary"]
        qkv = normal(B, T, (Hq + 2 * Hk) * d).to(t)
        for name, lo, H in (("q", 0, Hq), ("k", Hq, Hk), ("v", Hq + Hk, Hk)):
            s[name] = qkv[..., lo * d:(lo + H) * d].view(B, T, H, d).transpose(1, 2)
        s["freq"] = array("d", [10000.0 ** (-2.0 * i / R) for i in range(R // 2)])
        s["f"] = torch.tensor(list(s["freq"]), dtype=torch.float64, device="cuda")
        both = _counts(case)
        cache([before + new for before, new in both])
        s["before"] = integers([before for before, _ in both])
        s["counts"] = integers([new for _, new in both])
        # the new tokens one after the other: what the scheduler knows of them
        s["seq"] = torch.cat([torch.full((new,), b) for b, (_, new) in enumerate(both)]).cuda()
        s["tok"] = torch.cat([torch.arange(new) for _, new in both]).cuda()
        return s
    if case["op"] == "attend":
        cache(_lengths(case))
        q = normal(B, case["T"], Hq * d).mul_(1.5).to(t)
        s["q"] = q.view(B, case["T"], Hq, d).transpose(1, 2)
        s["before"] = integers([n - case["T"] for n in _lengths(case)])
        return s
    if case["op"] == "cross_step":
        # the states of some hundred encoder tokens
        k = _plain_phi(s, normal(B, Hk, 200, d).mul_(0.7))
        v = normal(B, Hk, 200, d) + 0.3
        s["S"], s["z"] = k.transpose(2, 3) @ v, k.sum(2)
        s["q"] = normal(B, Hq * d).mul_(0.7).to(t).view(B, Hq, d)
        return s
    N, M = case["N"], case["M"]
    q, kv = normal(B, N, Hq * d).mul_(0.7).to(t), normal(B, M, 2 * Hk * d)
    kv[..., :Hk * d] *= 0.7
    kv[..., Hk * d:] += 0.3
    kv = kv.to(t)
    s["q"] = q.view(B, N, Hq, d).transpose(1, 2)
    s["k"] = kv[..., :Hk * d].view(B, M, Hk, d).transpose(1, 2)
    s["v"] = kv[..., Hk * d:].view(B, M, Hk, d).transpose(1, 2)
    s["lengths"] = integers(_frames(case)) if case["ragged"] else None
    if case["op"] == "cross_back":
        s["S"], s["z"] = _plain_state(s)
        s["dout"] = normal(B, N, Hq * d).to(t).view(B, N, Hq, d).transpose(1, 2)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        import linear_attention_feature_gb300 as la
        form = {"feature_map": s.get("feature_map"), "normalise": s.get("normalise")}
        if op == "append":
            q = la.append_cache(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                                s["before"], s["freq"], q=s["q"], counts=s["counts"],
                                interleaved=s["interleaved"])
            return q, s["k_cache"], s["v_cache"]
        if op == "attend":
            return la.decode_step_paged(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                        s["before"], window=s["window"])
        if op == "cross":
            return la.forward_cross(s["q"], s["k"], s["v"], s["lengths"], **form)
        if op == "cross_back":
            return la.backward_cross(s["dout"], s["q"], s["k"], s["v"], s["S"], s["z"],
                                     s["lengths"], **form)
        return la.decode_step_cross(s["S"], s["z"], s["q"], **form)
    if op == "append":
        return _plain_append(s)
    if op == "attend":
        return _plain_attend(s)
    if op == "cross":
        S, z = _plain_state(s)
        return _plain_read(s, s["q"], S, z), S, z
    if op == "cross_back":
        return _plain_cross_back(s)
    return _plain_read(s, s["q"].unsqueeze(2), s["S"], s["z"]).squeeze(2)


def _plain_append(s):
    T, R = s["T"], s["rotary"]
    p = s["before"].double()[:, None] + torch.arange(T, device="cuda")
    angle = (p[..., None] * s["f"])[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def rotate(x):
        u = x.float()
        if s["interleaved"]:
            u1, u2 = u[..., 0:R:2], u[..., 1:R:2]
            y = torch.stack((u1 * cos - u2 * sin, u2 * cos + u1 * sin), dim=-1).flatten(-2)
        else:
            u1, u2 = u[..., :R // 2], u[..., R // 2:R]
            y = torch.cat((u1 * cos - u2 * sin, u2 * cos + u1 * sin), dim=-1)
        return torch.cat((y, u[..., R:]), dim=-1).to(x.dtype)

    seq, tok = s["seq"], s["tok"]
    at = s["before"][seq].long() + tok
    page, slot = s["table"][seq, at // s["page"]].long(), at % s["page"]
    s["k_cache"][page, :, slot] = rotate(s["k"])[seq, :, tok]
    s["v_cache"][page, :, slot] = s["v"][seq, :, tok]
    return rotate(s["q"]), s["k_cache"], s["v_cache"]


def _plain_attend(s):
    B, Hq, Hk, T, d = s["B"], s["Hq"], s["Hk"], s["T"], s["d"]
    table = s["table"].clamp(min=0).long()
    L = table.shape[1] * s["page"]

    def rows(c):
        return c[table].transpose(1, 2).float().reshape(B, Hk, L, d)

    q = s["q"].float().reshape(B, Hk, Hq // Hk * T, d)
    score = (q @ rows(s["k_cache"]).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    at = s["before"][:, None] + torch.arange(T, device="cuda")
    key = torch.arange(L, device="cuda")
    seen = key <= at[..., None]
    if s["window"]:
        seen = seen & (key > at[..., None] - s["window"])
    score = score.view(B, Hk, -1, T, L).masked_fill(~seen[:, None, None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True)).view(B, Hk, -1, L)
    y = (w @ rows(s["v_cache"])) / w.sum(-1, keepdim=True)
    return y.view(B, Hq, T, d).to(s["q"].dtype)


def _plain_phi(s, x):
    if s["feature_map"] == "identity":
        return x.float()
    v = x.float()
    return torch.where(v > 0, v + 1.0, torch.exp(v))


def _plain_valid(s, x):
    """1 for the encoder's tokens, 0 for the padding behind them."""
    key = torch.arange(x.shape[2], device=x.device)
    return (key < s["lengths"][:, None]).float()[:, None, :, None]


def _plain_state(s):
    k, v = _plain_phi(s, s["k"]), s["v"].float()
    if s["lengths"] is not None:
        k = k * _plain_valid(s, k)
    return k.transpose(2, 3) @ v, k.sum(2)


def _plain_groups(s, x, H):
    """[B, Hq, N, d] as [B, Hk, Hq / Hk * N, d]."""
    return x.reshape(x.shape[0], H, -1, x.shape[-1])


def _plain_read(s, q, S, z):
    y = _plain_groups(s, _plain_phi(s, q), S.shape[1])
    num = y @ S
    if s["normalise"]:
        num = num / (y @ z[..., None])
    return num.view(q.shape).to(q.dtype)


def _plain_cross_back(s):
    S, z, shape = s["S"], s["z"], s["q"].shape
    q = _plain_groups(s, s["q"].float(), S.shape[1])
    dy = _plain_groups(s, s["dout"].float(), S.shape[1])
    k, v = s["k"].float(), s["v"].float()
    fq, fk = _plain_phi(s, q), _plain_phi(s, k)
    if s["lengths"] is not None:
        fk = fk * _plain_valid(s, fk)
    dfq = dy @ S.transpose(2, 3)
    if s["normalise"]:
        r = 1.0 / (fq @ z[..., None])
        t = (fq * dfq).sum(-1, keepdim=True) * r
        dfq = (dfq - t * z[:, :, None]) * r
        fq = fq * r
        dz = -(fq * t).sum(2)
    else:
        dz = torch.zeros_like(z)
    dS = fq.transpose(2, 3) @ dy
    dfk = v @ dS.transpose(2, 3) + dz[:, :, None]
    dv = fk @ dS
    if s["feature_map"] != "identity":
        dfq = dfq * torch.where(q > 0, torch.ones_like(q), torch.exp(q))
        dfk = dfk * torch.where(k > 0, torch.ones_like(k), torch.exp(k))
    if s["lengths"] is not None:
        dfk = dfk * _plain_valid(s, dfk)
    t = s["q"].dtype
    return dfq.view(shape).to(t), dfk.to(t), dv.to(t)


# ---------------------------------------------------------------- the floor

def work(case):
    B, Hq, Hk, d, size = case["B"], case["Hq"], case["Hk"], case["d"], SIZE[case["dtype"]]
    if case["op"] == "append":
        both = _counts(case)
        new, pages = sum(n for _, n in both), sum(-(-n // case["page"]) for _, n in both)
        values = B * case["T"] * Hq * d + 2 * new * Hk * d
        return {"bytes": 2 * values * size + 4 * pages + 8 * B, "flops": 4 * values}
    if case["op"] == "attend":
        keys = 0
        for n in _lengths(case):
            keys += min(n, case["window"] + case["T"] - 1) if case["window"] else n
        return {"bytes": 2 * keys * Hk * d * size + 2 * B * Hq * case["T"] * d * size
                + 4 * keys // case["page"] + 4 * B,
                "flops": 4 * keys * Hq * case["T"] * d}
    states = 4 * B * Hk * (d * d + d)
    q = B * case["N"] * Hq * d
    if case["op"] == "cross_step":
        return {"bytes": states + 2 * q * size, "flops": 2 * q * (d + 1)}
    k = sum(_frames(case)) * Hk * d
    padded = B * case["M"] * Hk * d
    if case["op"] == "cross":
        return {"bytes": (2 * q + 2 * k) * size + states, "flops": 2 * (q + k) * (d + 1)}
    return {"bytes": (3 * q + 2 * k + 2 * padded) * size + states,
            "flops": 4 * (q + k) * (d + 1)}


# -------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["feature_map"] == "elu1":
        def phi(x):
            x = x.double()
            return 1 + torch.clamp(x, min=0) + torch.expm1(torch.clamp(x, max=0))
    else:
        def phi(x):
            return x.double()
    G = case["Hq"] // case["Hk"]
    if case["op"] == "cross_step":
        f = phi(s["q"]).unflatten(1, (-1, G))
        y = torch.einsum("bhga,bhac->bhgc", f, s["S"].double())
        if case["normalise"]:
            y = y / torch.einsum("bhga,bha->bhg", f, s["z"].double())[..., None]
        return y.flatten(1, 2)
    if case["op"] == "cross":
        out = torch.empty(case["B"], case["Hq"], case["N"], case["d"], dtype=torch.float64,
                          device="cuda")
        S = torch.empty(case["B"], case["Hk"], case["d"], case["d"], dtype=torch.float64,
                        device="cuda")
        z = torch.empty_like(S[..., 0])
        for b, M in enumerate(_frames(case)):
            fk = phi(s["k"][b, :, :M])
            S[b] = torch.einsum("hma,hmc->hac", fk, s["v"][b, :, :M].double())
            z[b] = fk.sum(1)
            f = phi(s["q"][b]).unflatten(0, (-1, G))
            y = torch.einsum("hgna,hac->hgnc", f, S[b])
            if case["normalise"]:
                y = y / torch.einsum("hgna,ha->hgn", f, z[b])[..., None]
            out[b] = y.flatten(0, 1)
        return out, S, z
    return _exact_back(case, s, phi, G)


def _exact_append(case, s):
    R = case["rotary"]
    f = torch.tensor([10000.0 ** (-2.0 * i / R) for i in range(R // 2)], dtype=torch.float64,
                     device="cuda")

    def turned(x, at):  # x [H, T, d]
        x = x.double()
        angle = torch.outer(at.double(), f)
        turn = torch.polar(torch.ones_like(angle), angle)
        head = x[..., :R]
        pairs = head.unflatten(-1, (-1, 2)) if case["interleaved"] else \
            torch.stack(head.chunk(2, -1), -1)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn) if R else pairs
        y = y.flatten(-2) if case["interleaved"] else torch.cat(y.unbind(-1), -1)
        return torch.cat((y, x[..., R:]), -1)

    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    table = s["table"].tolist()
    for b, (before, new) in enumerate(_counts(case)):
        at = before + torch.arange(case["T"], device="cuda")
        q[b] = turned(s["q"][b], at)
        k = turned(s["k"][b], at)
        done = 0
        while done < new:
            slot = (before + done) % case["page"]
            n = min(new - done, case["page"] - slot)
            page = table[b][(before + done) // case["page"]]
            kc[page, :, slot:slot + n] = k[:, done:done + n]
            vc[page, :, slot:slot + n] = s["v"][b, :, done:done + n].double()
            done += n
    return q, kc, vc


def _exact_attend(case, s):
    B, Hq, T, d = case["B"], case["Hq"], case["T"], case["d"]
    G = Hq // case["Hk"]
    out = torch.empty(B, Hq, T, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        pages = s["table"][b, :-(-n // case["page"])].long()
        k, v = (torch.cat(s[c][pages].unbind(0), 1)[:, :n].double() for c in ("k_cache", "v_cache"))
        for t in range(T):
            hi = n - T + t + 1
            lo = max(0, hi - case["window"]) if case["window"] else 0
            q = s["q"][b, :, t].double().unflatten(0, (-1, G)) / d ** 0.5
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k[:, lo:hi]), -1)
            out[b, :, t] = torch.einsum("hgn,hnd->hgd", w, v[:, lo:hi]).flatten(0, 1)
    return out


def _exact_back(case, s, phi, G):
    """From the gradient of a weighted mean: with w_ij = phi(q_i) . phi(k_j) / den_i,
    the key's term is w_ij dy_i . (v_j - y_i)."""
    dq = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    dk = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    curved = case["feature_map"] == "elu1"
    for b, M in enumerate(_frames(case)):
        q, k, v = s["q"][b].double(), s["k"][b, :, :M].double(), s["v"][b, :, :M].double()
        f, g = phi(q).unflatten(0, (-1, G)), phi(k)
        dy = s["dout"][b].double().unflatten(0, (-1, G))
        S, z = s["S"][b].double(), s["z"][b].double()
        df = torch.einsum("hgnc,hac->hgna", dy, S)
        t = 0.0 * f[..., 0]
        if case["normalise"]:
            den = torch.einsum("hgna,ha->hgn", f, z)
            y = torch.einsum("hgna,hac->hgnc", f, S) / den[..., None]
            t = (y * dy).sum(-1)
            df = (df - t[..., None] * z[:, None, None]) / den[..., None]
            f = f / den[..., None]
        dS = torch.einsum("hgna,hgnc->hac", f, dy)
        dg = torch.einsum("hac,hmc->hma", dS, v) - torch.einsum("hgna,hgn->ha", f, t)[:, None]
        dv[b, :, :M] = torch.einsum("hac,hma->hmc", dS, g)
        if curved:
            df = df * torch.exp(torch.clamp(q, max=0)).unflatten(0, (-1, G))
            dg = dg * torch.exp(torch.clamp(k, max=0))
        dq[b], dk[b, :, :M] = df.flatten(0, 1), dg
    return dq, dk, dv
