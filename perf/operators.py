"""Workloads of the operators around the linear-attention kernels: the norm and
rotation of queries and keys, and the per-channel gated linear recurrence, each
forward, backward and for single tokens, in plain torch and through the
library."""
import math
from array import array

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a single stream: what counts is the call itself
        qk("qk step b1", "qk_step", 1, 32, 32, 1, 128, 128, "bf16"),
        # one decode step of a full serving batch, each sequence at a place of its own
        qk("qk step b256", "qk_step", 256, 32, 32, 1, 128, 128, "bf16"),
        # prefill of a mid-size batch out of the fused projection, head size 64
        qk("qk b4 h16 n4096 d64", "qk", 4, 16, 16, 4096, 64, 64, "bf16"),
        # prefill of long contexts, head size 128
        qk("qk b2 h16 n32768 d128", "qk", 2, 16, 16, 32768, 128, 128, "bf16"),
        # training, long sequences
        qk("qk back b4 h8 n16384 d128", "qk_back", 4, 8, 8, 16384, 128, 128, "bf16"),
        # training in full precision: an odd head size, shared keys, part of the head rotated, neighbours as pairs
        qk("qk back f32 d80 part", "qk_back", 3, 6, 2, 1001, 80, 40, "f32", interleaved=True),
        # one decode step of the recurrent layer for a full serving batch
        rec("rec step b256", "rec_step", 256, 1, 4096, "bf16", "bf16", "logit", True),
        # prefill of long contexts, gate and input mixed as in gated recurrent units
        rec("rec b2 n32768 c2048", "rec", 2, 32768, 2048, "bf16", "bf16", "logit", True),
        # one very long sequence with few channels: the length has to give the parallelism
        rec("rec long n262144 c256", "rec", 1, 262144, 256, "f32", "f32", "log", False),
        # packed documents, gates of exactly zero between them, odd sizes
        rec("rec f32 odd packed", "rec", 3, 1001, 201, "f32", "f32", "value", False),
        # training, the mid-size batch, gates kept in 32 bits beside bf16 values
        rec("rec back b4 n4096 c1024", "rec_back", 4, 4096, 1024, "bf16", "f32", "log", False),
        # training, long sequences
        rec("rec back b4 n16384 c1024", "rec_back", 4, 16384, 1024, "bf16", "bf16", "logit", True),
    ]


def qk(name, op, B, Hq, Hk, N, d, rotary, dtype, interleaved=False):
    c = {"op": op, "B": B, "Hq": Hq, "Hk": Hk, "N": N, "d": d, "rotary": rotary,
         "dtype": dtype, "interleaved": interleaved}
    return dict(c, name=name) if name else c


def rec(name, op, B, N, C, dtype, gate_dtype, gate, complement):
    c = {"op": op, "B": B, "N": N, "C": C, "dtype": dtype, "gate_dtype": gate_dtype,
         "gate": gate, "complement": complement}
    return dict(c, name=name) if name else c


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["qk", "qk_back", "qk_step", "rec", "rec_back", "rec_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("qk"):
        d = rng.choice([64, 128, 128, 256, 80, 96, 36, 2 * rng.randint(4, 100)])
        rotary = d if rng.random() < 0.6 else 2 * rng.randint(0, d // 2)
        Hq = spread(1, 32)
        Hk = Hq if rng.random() < 0.7 else rng.randint(1, Hq)
        B = spread(1, 256) if op == "qk_step" else spread(1, 4)
        N = 1 if op == "qk_step" else spread(1, max(2, min(32768, (1 << 26) // (B * Hq * d))))
        return qk(None, op, B, Hq, Hk, N, d, rotary, dtype, rng.random() < 0.3)
    gate_dtype = "f32" if dtype == "f32" or rng.random() < 0.4 else "bf16"
    gate = rng.choice(["value", "log", "logit"])
    C = spread(64, 4096) // rng.choice([1, 1, 8]) * rng.choice([1, 1, 8]) or 8
    B = spread(1, 256) if op == "rec_step" else spread(1, 8)
    N = 1 if op == "rec_step" else spread(1, min(262144, (1 << 26) // (B * C)))
    return rec(None, op, B, N, C, dtype, gate_dtype, gate, rng.random() < 0.5)


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = dict(case)
    B, N, t = case["B"], case["N"], DT[case["dtype"]]
    if case["op"].startswith("qk"):
        Hq, Hk, d, R = case["Hq"], case["Hk"], case["d"], case["rotary"]
        # q and k are slices of the fused projection's output, token after token
        qkv = normal(B, N, (Hq + 2 * Hk) * d).mul_(0.7).to(t)
        q = qkv[..., :Hq * d].view(B, N, Hq, d).transpose(1, 2)
        k = qkv[..., Hq * d:(Hq + Hk) * d].view(B, N, Hk, d).transpose(1, 2)
        s["freq"] = array("d", [10000.0 ** (-2.0 * i / R) for i in range(R // 2)])
        s["f"] = torch.tensor(list(s["freq"]), dtype=torch.float64, device="cuda")
        s["wq"], s["wk"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        if case["op"] == "qk_step":
            q, k = q[:, :, 0], k[:, :, 0]
            s["positions"] = torch.randint(0, 1 << 20, (B,), generator=gen, device="cuda")
            s["offset"] = 0
        else:
            s["positions"] = None
            s["offset"] = int(torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda"))
        if case["op"] == "qk_back":
            s["dq_out"], s["dk_out"] = normal(B, Hq, N, d).to(t), normal(B, Hk, N, d).to(t)
        s["q"], s["k"] = q, k
        return s
    C, tg = case["C"], DT[case["gate_dtype"]]
    z = normal(B, N, C)
    if case["gate"] == "log":
        z = -torch.exp(z - 4.0)          # decays of a few tokens to some thousands
    elif case["gate"] == "logit":
        z = z * 1.5 + 3.0
    else:
        z = torch.sigmoid(z + 4.0)
        if N > 300:
            z[:, 300::300] = 0.0         # a document ends: nothing passes
    s["gates"] = z.to(tg)
    s["x"] = normal(B, N, C).to(t)
    s["h0"] = normal(B, C)
    if case["op"] == "rec_step":
        s["x"], s["gates"] = s["x"][:, 0], s["gates"][:, 0]
        s["h_out"] = torch.empty_like(s["h0"])
    if case["op"] == "rec_back":
        s["out"] = _plain_recurrence(s)[0]
        s["dout"] = normal(B, N, C).to(t)
        s["dh"] = normal(B, C)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if own:
        import linear_attention_feature_gb300 as la
        if op in ("qk", "qk_step"):
            return la.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["freq"], s["positions"],
                                   offset=s["offset"], interleaved=s["interleaved"])
        if op == "qk_back":
            return la.backward_qk_norm_rope(s["dq_out"], s["dk_out"], s["q"], s["k"], s["wq"],
                                            s["wk"], s["freq"], s["positions"],
                                            offset=s["offset"], interleaved=s["interleaved"])
        if op == "rec":
            return la.forward_recurrence(s["x"], s["gates"], s["h0"], gate=s["gate"],
                                         complement=s["complement"])
        if op == "rec_back":
            return la.backward_recurrence(s["dout"], s["gates"], s["out"], s["x"], s["h0"],
                                          s["dh"], gate=s["gate"], complement=s["complement"])
        y = la.decode_step_recurrence(s["h0"], s["x"], s["gates"], h_out=s["h_out"],
                                      gate=s["gate"], complement=s["complement"])
        return y, s["h_out"]
    if op in ("qk", "qk_step"):
        return (_plain_norm_rope(s, s["q"], s["wq"]), _plain_norm_rope(s, s["k"], s["wk"]))
    if op == "qk_back":
        dq, dwq = _plain_norm_rope_back(s, s["dq_out"], s["q"], s["wq"])
        dk, dwk = _plain_norm_rope_back(s, s["dk_out"], s["k"], s["wk"])
        return dq, dk, dwq, dwk
    if op == "rec":
        return _plain_recurrence(s)
    if op == "rec_back":
        return _plain_recurrence_back(s)
    a, c = _plain_gate(s)
    h = a * s["h0"] + c * s["x"].float()
    return h.to(s["x"].dtype), h


EPS = 1e-6


def _plain_angles(s, x):
    """cos and sin of the tokens' angles, [1 or B, 1, N or nothing, rotary / 2]."""
    f = s["f"]
    if s["positions"] is None:
        p = s["offset"] + torch.arange(x.shape[2], device=x.device)
        angle = (p.double()[:, None] * f)[None, None]
    else:
        angle = (s["positions"].double()[:, None] * f)[:, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _plain_rotate(s, u, sign):
    R = s["rotary"]
    cos, sin = _plain_angles(s, u)
    sin = sin * sign
    if s["interleaved"]:
        u1, u2 = u[..., 0:R:2], u[..., 1:R:2]
        y = torch.stack((u1 * cos - u2 * sin, u2 * cos + u1 * sin), dim=-1).flatten(-2)
    else:
        u1, u2 = u[..., :R // 2], u[..., R // 2:R]
        y = torch.cat((u1 * cos - u2 * sin, u2 * cos + u1 * sin), dim=-1)
    return torch.cat((y, u[..., R:]), dim=-1)


def _plain_norm_rope(s, x, w):
    v = x.float()
    n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    return _plain_rotate(s, n * w, 1.0).to(x.dtype)


def _plain_norm_rope_back(s, dy, x, w):
    v = x.float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    n = v * r
    g = _plain_rotate(s, dy.float(), -1.0)
    dw = (g * n).double().sum((0, 1, 2)).float()
    g = g * w
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _plain_gate(s):
    """The gate a and the input's factor."""
    z = s["gates"].float()
    if s["gate"] == "value":
        a, b = z, 1.0 - z
    elif s["gate"] == "log":
        a, b = torch.exp(z), -torch.expm1(z)
    else:
        a, b = torch.sigmoid(z), torch.sigmoid(-z)
    return a, (b if s["complement"] else torch.ones_like(b))


def _plain_scan(a, b):
    """h_t = a_t h_{t-1} + b_t over dimension 1, by doubling the reach."""
    reach = 1
    while reach < b.shape[1]:
        b = torch.cat((b[:, :reach], b[:, reach:] + a[:, reach:] * b[:, :-reach]), 1)
        a = torch.cat((a[:, :reach], a[:, reach:] * a[:, :-reach]), 1)
        reach *= 2
    return b


def _plain_recurrence(s):
    a, c = _plain_gate(s)
    b = c * s["x"].float()
    b[:, 0] += a[:, 0] * s["h0"]
    h = _plain_scan(a, b)
    return h.to(s["x"].dtype), h[:, -1].clone()


def _plain_recurrence_back(s):
    a, c = _plain_gate(s)
    dy = s["dout"].float()
    dy[:, -1] += s["dh"]
    after = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    g = _plain_scan(after.flip(1), dy.flip(1)).flip(1)
    before = torch.cat((s["h0"][:, None], s["out"][:, :-1].float()), 1)
    if s["complement"]:
        before = before - s["x"].float()
    if s["gate"] == "value":
        slope = 1.0
    elif s["gate"] == "log":
        slope = a
    else:
        slope = a * torch.sigmoid(-s["gates"].float())
    dz = slope * g * before
    return (c * g).to(s["x"].dtype), dz.to(s["gates"].dtype), a[:, 0] * g[:, 0]


# ---------------------------------------------------------------- the floor

def work(case):
    B, N = case["B"], case["N"]
    size = {"bf16": 2, "f32": 4}
    if case["op"].startswith("qk"):
        values = B * N * (case["Hq"] + case["Hk"]) * case["d"]
        back = case["op"] == "qk_back"
        extra = 8 * case["d"] * (2 if back else 1) + (8 * B if case["op"] == "qk_step" else 0)
        return {"bytes": values * size[case["dtype"]] * (3 if back else 2) + extra,
                "flops": values * (20 if back else 10)}
    values, sx, sg = B * N * case["C"], size[case["dtype"]], size[case["gate_dtype"]]
    states = 8 * B * case["C"]
    if case["op"] == "rec_back":
        arrays = 3 * sx + 2 * sg + (sx if case["complement"] else 0)
        return {"bytes": values * arrays + 12 * B * case["C"], "flops": values * 12}
    return {"bytes": values * (2 * sx + sg) + states, "flops": values * 6}


# -------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("qk"):
        back = case["op"] == "qk_back"
        got = [_exact_rows(case, s, s["d%s_out" % n] if back else None, s[n], s["w" + n])
               for n in ("q", "k")]
        return (got[0][0], got[1][0], got[0][1], got[1][1]) if back else (got[0], got[1])
    z, x, h = s["gates"].double(), s["x"].double(), s["h0"].double()
    a = {"value": lambda: z, "log": lambda: z.exp(), "logit": lambda: 1 / (1 + (-z).exp())}[case["gate"]]()
    rest = {"value": lambda: 1 - z, "log": lambda: -torch.expm1(z),
            "logit": lambda: 1 / (1 + z.exp())}[case["gate"]]()
    if case["op"] == "rec_step":
        h = a * h + (rest * x if case["complement"] else x)
        return h, h
    N = case["N"]
    if case["op"] == "rec":
        into = rest * x if case["complement"] else x
        for t in range(N):
            h = torch.addcmul(into[:, t], a[:, t], h, out=into[:, t])
        return into, h.clone()
    g, dx, dz = s["dh"].double(), torch.empty_like(x), torch.empty_like(z)
    dy, out = s["dout"], s["out"]
    G = torch.empty_like(x)
    for t in range(N - 1, -1, -1):
        g = torch.add(g, dy[:, t], out=G[:, t])
        g = a[:, t] * g
    h = torch.cat((h[:, None], out[:, :-1].double()), 1)
    dx = G * rest if case["complement"] else G
    slope = {"value": 1.0, "log": a, "logit": a * rest}[case["gate"]]
    dz = G * slope * ((h - x) if case["complement"] else h)
    return dx, dz, g


def _exact_rows(case, s, dy, x, w):
    """The rotation as a product of complex numbers, the norm's gradient as its Jacobian's product."""
    R, d = case["rotary"], case["d"]
    x, w = x.double(), w.double()
    f = torch.tensor(list(s["freq"]), dtype=torch.float64, device=x.device)
    p = s["positions"] if s["positions"] is not None else s["offset"] + torch.arange(case["N"], device=x.device)
    angle = p.double().unsqueeze(-1) * f
    angle = angle.unsqueeze(1) if s["positions"] is not None else angle
    turn = torch.complex(angle.cos(), angle.sin())

    def rotate(u, by):
        head = u[..., :R]
        pairs = head.unflatten(-1, (R // 2, 2)) if case["interleaved"] else head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
        v = torch.view_as_real(torch.view_as_complex(pairs.clone(memory_format=torch.contiguous_format)) * by)
        v = v if case["interleaved"] else v.transpose(-1, -2)
        return torch.cat((v.flatten(-2), u[..., R:]), -1)

    size = ((x ** 2).sum(-1, keepdim=True) / d + EPS) ** 0.5
    if dy is None:
        return rotate(x / size * w, turn)
    g = rotate(dy.double(), turn.conj())
    dw = (g * x / size).sum((0, 1, 2))
    dn = g * w
    dx = dn / size - x * (dn * x).sum(-1, keepdim=True) / (d * size ** 3)
    return dx, dw
