"""The gated linear recurrence with a gate per channel, forward, backward and
single tokens, against plain loops in 64 bits.

Tolerances, with u = 2^-24 and half = half a step of the output's type: let
M_t = a_t M_{t-1} + |c_t x_t| (M_0 = |h0|) bound every partial sum.  A step
injects at most K u M_t of error: the gate (exp 2 u, the logistic function 6 u,
its complement 6 u), its products over a piece of the sequence and their use
(one rounding per token each), the input's product and the sum; K = 16 covers
them.  Errors decay with the state: E_t = a_t E_{t-1} + M_t, so
|h_t - exact| <= 16 u E_t + half |h_t|.  Backwards the same holds for g with
|dout|; dx adds 16 u |c g| and dgates 16 u |s g| (|h| + |x|)."""
import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


def half(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def gates_of(z, gate):
    z = z.double()
    if gate == "value":
        return z, 1 - z
    if gate == "log":
        return z.exp(), -torch.expm1(z)
    return torch.sigmoid(z), torch.sigmoid(-z)


def scan(a, y, h):
    out = torch.empty_like(y)
    for t in range(y.shape[1]):
        h = a[:, t] * h + y[:, t]
        out[:, t] = h
    return out


def plain(x, z, h0, gate, complement):
    a, rest = gates_of(z, gate)
    y = x.double() * (rest if complement else 1.0)
    return scan(a, y, h0.double())


def bound(x, z, h0, gate, complement):
    a, rest = gates_of(z, gate)
    m = scan(a.abs(), (x.double() * (rest if complement else 1.0)).abs(), h0.double().abs())
    return scan(a.abs(), m, torch.zeros_like(m[:, 0]))


def close(got, ref, tol):
    err = (got.cpu().double() - ref).abs()
    tol = tol + half(got.dtype) * ref.abs() * (1 + 1e-3) + 1e-37
    assert torch.all(err <= tol), float((err / tol).max())


def inputs(B, N, C, types, gate, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, C, generator=g)
    z = torch.randn(B, N, C, generator=g)
    if gate == "value":
        z = torch.sigmoid(z + 3)
        z[:, ::37] = 0.0
        z[:, 5::41] = 1.0
    elif gate == "log":
        z = -torch.exp(z - 3)
        z[:, 3::37] = -float("inf")
        z[:, 5::41] = 0.0
    else:
        z = 2 * z + 3
        z[:, 3::37] = -float("inf")
        z[:, 5::41] = float("inf")
    h0 = torch.randn(B, C, generator=g)
    return x.to(DT[types[0]]), z.to(DT[types[1]]), h0


def check_forward(x, z, h0, gate, complement, out, h_last):
    ref = plain(x, z, h0, gate, complement)
    tol = 16 * U * bound(x, z, h0, gate, complement)
    close(out, ref, tol)
    close(h_last, ref[:, -1], tol[:, -1])


def plain_back(dout, z, out, x, h0, dh, gate, complement):
    """(dx, dgates, dh0) and the magnitudes that bound their errors."""
    a, rest = gates_of(z, gate)
    N = z.shape[1]
    g = torch.empty_like(a)
    m, e = torch.empty_like(a), torch.empty_like(a)
    s, sm, se = dh.double(), dh.double().abs(), torch.zeros_like(a[:, 0])
    for t in range(N - 1, -1, -1):
        g[:, t] = dout[:, t].double() + s
        m[:, t] = dout[:, t].double().abs() + sm
        e[:, t] = se + m[:, t]
        s, sm, se = a[:, t] * g[:, t], a[:, t].abs() * m[:, t], a[:, t].abs() * e[:, t]
    before = torch.cat((h0.double()[:, None], out[:, :-1].double()), 1)
    size = before.abs()
    if complement:
        before = before - x.double()
        size = size + x.double().abs()
    slope = {"value": torch.ones_like(a), "log": a, "logit": a * rest}[gate]
    c = rest if complement else torch.ones_like(a)
    dx, dz = c * g, slope * g * before
    return (dx, 32 * U * c.abs() * e), (dz, 32 * U * slope.abs() * e * size), (s, 32 * U * se)


SHAPES = [(1, 1, 1), (2, 2, 3), (3, 17, 5), (1, 130, 64), (2, 129, 66), (3, 257, 201),
          (1, 1000, 40), (2, 2049, 32), (1, 5000, 7), (5, 64, 512)]


@pytest.mark.parametrize("gate", ["value", "log", "logit"])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, types, complement, gate):
    B, N, C = shape
    x, z, h0 = inputs(B, N, C, types, gate, 7 + N)
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), gate=gate,
                                    complement=complement)
    check_forward(x, z, h0, gate, complement, out, hl)
    g = torch.Generator().manual_seed(8 + N)
    dout = torch.randn(B, N, C, generator=g).to(x.dtype)
    dh = torch.randn(B, C, generator=g)
    got = la.backward_recurrence(dout.cuda(), z.cuda(), out, x.cuda(), h0.cuda(), dh.cuda(),
                                 gate=gate, complement=complement)
    want = plain_back(dout, z, out.cpu(), x, h0, dh, gate, complement)
    assert got[1].dtype == z.dtype
    for a, (ref, tol) in zip(got, want):
        close(a, ref, tol)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("B, N, C", [(200, 90, 60), (90, 200, 130), (170, 300, 33), (70, 515, 201)])
def test_more_strips_than_run_at_once(B, N, C, types):
    # a block takes several strips one after the other, each of one, two, three
    # or more rounds, so that its two groups of warps pass from one to the next
    x, z, h0 = inputs(B, N, C, types, "logit", 11 + N)
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), gate="logit", complement=True)
    check_forward(x, z, h0, "logit", True, out, hl)
    g = torch.Generator().manual_seed(12)
    dout, dh = torch.randn(B, N, C, generator=g).to(x.dtype), torch.randn(B, C, generator=g)
    got = la.backward_recurrence(dout.cuda(), z.cuda(), out, x.cuda(), h0.cuda(), dh.cuda(),
                                 gate="logit", complement=True)
    for a, (ref, tol) in zip(got, plain_back(dout, z, out.cpu(), x, h0, dh, "logit", True)):
        close(a, ref, tol)


@pytest.mark.parametrize("B, N, C", [(1, 200000, 64), (1, 30000, 64), (1, 3000, 512),
                                     (3, 700, 1000), (1, 50, 40)])
def test_state_in_place(B, N, C):
    # h_last over h0, dh0 over dh_last, whatever the sequence is cut into:
    # pieces, clusters, single blocks
    x, z, h0 = (t.cuda() for t in inputs(B, N, C, ("bf16", "bf16"), "logit", 13 + N))
    dh = torch.randn(B, C, generator=torch.Generator().manual_seed(14)).cuda()
    out, hl = la.forward_recurrence(x, z, h0, gate="logit")
    back = la.backward_recurrence(x, z, out, None, h0, dh, gate="logit")
    for _ in range(5):
        h, d = h0.clone(), dh.clone()
        o, _ = la.forward_recurrence(x, z, h, h_last=h, gate="logit")
        assert torch.equal(o, out) and torch.equal(h, hl)
        got = la.backward_recurrence(x, z, out, None, h0, d, dh0=d, gate="logit")
        for a, b in zip(got, back):
            assert torch.equal(a, b)


@pytest.mark.parametrize("N, launches", [(4000, 1), (40000, 2), (200000, 2)])
def test_workspaces(N, launches):
    # few channels: from some length on a sequence is cut into pieces (their
    # maps, then the walk).  The binding brings a workspace on the current
    # stream, the library allocates on one given by the caller
    x, z, h0 = (t.cuda() for t in inputs(1, N, 40, ("f32", "f32"), "log", 15))
    n0 = la.kernel_launch_count()
    ref = la.forward_recurrence(x, z, h0, gate="log")
    assert la.kernel_launch_count() == n0 + launches
    here = torch.cuda.current_stream()
    got = la.forward_recurrence(x, z, h0, gate="log", stream=here)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    if launches == 1:
        return
    lib = la.load_library()
    assert lib.la_debug_fail_next_allocs(1) == 0
    try:
        la.forward_recurrence(x, z, h0, gate="log")
        with pytest.raises(la.LinAttnError) as e:
            la.forward_recurrence(x, z, h0, gate="log", stream=here)
        assert e.value.status == 4
    finally:
        lib.la_debug_fail_next_allocs(0)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    st = lib.la_forward_recurrence(x.data_ptr(), z.data_ptr(), None, ref[0].data_ptr(), None, None,
                                   1, N, 40, 1, 0, 0, 0, small.data_ptr(), 64, None)
    assert st == 1 and "workspace too small" in lib.la_last_error().decode()


@pytest.mark.parametrize("types, C, complement", [(("f32", "f32"), 40, False),
                                                  (("bf16", "bf16"), 64, True),
                                                  (("bf16", "f32"), 7, False)])
def test_sequences_in_pieces(types, C, complement):
    N = 120007
    g = torch.Generator().manual_seed(17)
    x = torch.randn(1, N, C, generator=g).to(DT[types[0]])
    z = (2 * torch.randn(1, N, C, generator=g) + 5).to(DT[types[1]])
    h0, dh = torch.randn(1, C, generator=g), torch.randn(1, C, generator=g)
    n0 = la.kernel_launch_count()
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), gate="logit",
                                    complement=complement)
    assert la.kernel_launch_count() == n0 + 2
    check_forward(x, z, h0, "logit", complement, out, hl)
    got = la.backward_recurrence(x.cuda(), z.cuda(), out, x.cuda(), h0.cuda(), dh.cuda(),
                                 gate="logit", complement=complement)
    for a, (ref, tol) in zip(got, plain_back(x, z, out.cpu(), x, h0, dh, "logit", complement)):
        close(a, ref, tol)


def test_without_states():
    x, z, _ = inputs(2, 300, 65, ("f32", "f32"), "log", 21)
    zero = torch.zeros(2, 65)
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), gate="log")
    check_forward(x, z, zero, "log", False, out, hl)
    got = la.backward_recurrence(x.cuda(), z.cuda(), out, gate="log")
    for a, (ref, tol) in zip(got, plain_back(x, z, out.cpu(), x, zero, zero, "log", False)):
        close(a, ref, tol)


@pytest.mark.parametrize("types, C", [(("f32", "f32"), 96), (("bf16", "bf16"), 256),
                                      (("bf16", "f32"), 33)])
def test_long_sequences(types, C):
    # gates near 1 keep a state over thousands of tokens
    N = 20011
    g = torch.Generator().manual_seed(31)
    x = torch.randn(1, N, C, generator=g).to(DT[types[0]])
    z = (-torch.exp(torch.randn(1, N, C, generator=g) - 7)).to(DT[types[1]])
    h0 = torch.randn(1, C, generator=g)
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), gate="log")
    check_forward(x, z, h0, "log", False, out, hl)
    dh = torch.randn(1, C, generator=g)
    got = la.backward_recurrence(x.cuda(), z.cuda(), out, None, h0.cuda(), dh.cuda(), gate="log")
    for a, (ref, tol) in zip(got, plain_back(x, z, out.cpu(), x, h0, dh, "log", False)):
        close(a, ref, tol)


@pytest.mark.parametrize("types", TYPES)
def test_strides_alignment_and_in_place(types):
    # slices of fused projections, odd starts, outputs into a buffer whose
    # other values stay; all give the contiguous call's bits
    B, N, C = 2, 200, 70
    x, z, h0 = inputs(B, N, C, types, "logit", 41)
    xd, zd, hd = x.cuda(), z.cuda(), h0.cuda()
    ref, rl = la.forward_recurrence(xd, zd, hd, gate="logit", complement=True)
    for off, pad in ((0, 2), (1, 1), (3, 8)):
        xs = torch.zeros(B, N, C + off + pad, dtype=x.dtype, device="cuda")[..., off:off + C]
        zs = torch.zeros(N, B, C + off + pad, dtype=z.dtype, device="cuda")
        zs = zs[..., off:off + C].transpose(0, 1)
        xs.copy_(xd)
        zs.copy_(zd)
        room = torch.full((B, N, C + 9), 7.0, dtype=x.dtype, device="cuda")
        out, hl = la.forward_recurrence(xs, zs, hd, out=room[..., 5:5 + C], gate="logit",
                                        complement=True)
        assert torch.equal(out, ref) and torch.equal(hl, rl)
        assert torch.all(room[..., :5] == 7.0) and torch.all(room[..., 5 + C:] == 7.0)
        want = la.backward_recurrence(xd, zd, ref, xd, hd, hd, gate="logit", complement=True)
        got = la.backward_recurrence(xs, zs, out, xs, hd, hd, dx=room[..., 5:5 + C].clone(),
                                     gate="logit", complement=True)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        got = la.backward_recurrence(xs, zs, ref, xd, hd, hd, dx=xs, gate="logit",
                                     complement=True)
        assert torch.equal(xs, want[0]) and torch.equal(got[1], want[1])
    h = hd.clone()
    out, hl = la.forward_recurrence(xd, zd, h, out=xd, h_last=h, gate="logit", complement=True)
    assert out.data_ptr() == xd.data_ptr() and torch.equal(out, ref) and torch.equal(h, rl)
    dh = hd.clone()
    want = la.backward_recurrence(ref, zd, ref, None, hd, hd, gate="logit")
    got = la.backward_recurrence(ref, zd, ref, None, hd, dh, dh0=dh, gate="logit")
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_broadcast_gates():
    # one gate for all channels' sequences: stride 0 over batch and tokens
    x, _, h0 = inputs(3, 100, 64, ("f32", "f32"), "value", 51)
    z = torch.full((1, 1, 64), 0.9)
    zz = z.cuda().expand(3, 100, 64)
    out, hl = la.forward_recurrence(x.cuda(), zz, h0.cuda())
    check_forward(x, z.expand(3, 100, 64), h0, "value", False, out, hl)
    got = la.backward_recurrence(x.cuda(), zz, out, None, h0.cuda(), None)
    want = plain_back(x, z.expand(3, 100, 64), out.cpu(), x, h0, torch.zeros(3, 64), "value", False)
    for a, (ref, tol) in zip(got, want):
        close(a, ref, tol)


@pytest.mark.parametrize("gate", ["value", "log", "logit"])
@pytest.mark.parametrize("types", TYPES)
def test_decode_continues_the_forward(types, gate):
    B, N, C, more = 3, 150, 129, 12
    x, z, h0 = inputs(B, N + more, C, types, gate, 61)
    ref = plain(x, z, h0, gate, True)
    tol = 16 * U * bound(x, z, h0, gate, True)
    xd, zd = x.cuda(), z.cuda()
    _, h = la.forward_recurrence(xd[:, :N], zd[:, :N], h0.cuda(), gate=gate, complement=True)
    for t in range(N, N + more):
        y = la.decode_step_recurrence(h, xd[:, t], zd[:, t], gate=gate, complement=True)
        close(y, ref[:, t], tol[:, t])
    close(h, ref[:, -1], tol[:, -1])


@pytest.mark.parametrize("B, C", [(1, 1), (1, 4096), (256, 128), (7, 37)])
@pytest.mark.parametrize("types", TYPES)
def test_decode_step(B, C, types):
    x, z, h0 = inputs(B, 1, C, types, "logit", 71)
    z[:] = torch.randn(z.shape, generator=torch.Generator().manual_seed(72)).to(z.dtype)
    h, h_out = h0.cuda(), torch.empty(B, C, device="cuda")
    keep = h.clone()
    y = la.decode_step_recurrence(h, x.cuda()[:, 0], z.cuda()[:, 0], h_out=h_out, gate="logit")
    assert torch.equal(h, keep)
    ref = plain(x, z, h0, "logit", False)[:, 0]
    tol = 16 * U * bound(x, z, h0, "logit", False)[:, 0]
    close(y, ref, tol)
    close(h_out, ref, tol)


def test_pieces_of_a_sequence_equal_the_whole():
    # a prefill in two calls; the state passes unrounded between them
    x, z, h0 = inputs(2, 777, 64, ("bf16", "bf16"), "logit", 81)
    xd, zd = x.cuda(), z.cuda()
    _, h = la.forward_recurrence(xd[:, :300], zd[:, :300], h0.cuda(), gate="logit")
    out, hl = la.forward_recurrence(xd[:, 300:], zd[:, 300:], h, gate="logit")
    ref = plain(x, z, h0, "logit", False)
    tol = 16 * U * bound(x, z, h0, "logit", False)
    close(out, ref[:, 300:], tol[:, 300:])
    close(hl, ref[:, -1], tol[:, -1])


def test_padding_keeps_and_zero_gates_reset():
    # right padding: gate 1 and x = 0 keep the state; a document's first
    # token has gate 0, so what came before does not matter
    x, z, h0 = inputs(2, 400, 64, ("f32", "f32"), "value", 91)
    z[:, 250:] = 1.0
    x[:, 250:] = 0.0
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda())
    assert torch.equal(hl, out[:, -1])
    # the state is kept up to rounding: out[249] and each later state are the
    # same exact number, reached by pieces joined differently, each within 16 u E
    E = bound(x, z, h0, "value", False)
    for t in (250, 300, 399):
        err = (out[:, t] - out[:, 249]).abs().cpu().double()
        assert torch.all(err <= 16 * U * (E[:, t] + E[:, 249]))
    z[:, 100] = 0.0
    a, _ = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda())
    b, _ = la.forward_recurrence(x.cuda(), z.cuda(), 5 + h0.cuda())
    assert torch.equal(a[:, 100:], b[:, 100:])


@pytest.mark.parametrize("types", TYPES)
def test_non_finite_values_stay_in_their_channel(types):
    x, z, h0 = inputs(2, 300, 66, types, "value", 101)
    clean, _ = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda())
    x[0, 140, 9] = float("nan")
    x[1, 20, 64] = float("inf")
    z[1, 260:, 10] = float("nan")
    out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda())
    assert torch.isnan(out[0, 140:, 9]).all() and torch.isnan(hl[0, 9])
    assert not torch.isfinite(out[1, 20:, 64]).any()
    assert torch.isnan(out[1, 260:, 10]).all()
    same = torch.ones(2, 300, 66, dtype=torch.bool)
    same[0, 140:, 9] = same[1, 20:, 64] = same[1, 260:, 10] = False
    assert torch.equal(out.cpu()[same], clean.cpu()[same])


def test_gradient_against_differences():
    # h is affine in x, in h0 and in each single gate: central differences of
    # the library's own forward are exact but for its rounding, 16 u E on
    # either side; dgates reads the states that the forward rounded (16 u E)
    B, N, C = 2, 70, 6
    x, z, h0 = inputs(B, N, C, ("f32", "f32"), "value", 111)
    g = torch.Generator().manual_seed(112)
    dout, dh = torch.randn(B, N, C, generator=g), torch.randn(B, C, generator=g)
    delta = 0.125
    for complement in (False, True):
        def loss(x, z, h0):
            out, hl = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), complement=complement)
            E = 16 * U * bound(x, z, h0, "value", complement)
            return ((out.cpu().double() * dout.double()).sum(1) + hl.cpu().double() * dh.double(),
                    (E * dout.abs().double()).sum(1) + E[:, -1] * dh.abs().double())

        def difference(hi, lo):
            (p, ep), (m, em) = loss(*hi), loss(*lo)
            return (p - m) / (2 * delta), (ep + em) / (2 * delta)

        out, _ = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), complement=complement)
        got = la.backward_recurrence(dout.cuda(), z.cuda(), out, x.cuda(), h0.cuda(), dh.cuda(),
                                     complement=complement)
        got = [t.cpu().double() for t in got]
        want = plain_back(dout, z, out.cpu(), x, h0, dh, "value", complement)
        E = 16 * U * bound(x, z, h0, "value", complement)
        E = torch.cat((torch.zeros(B, 1, C, dtype=torch.float64), E[:, :-1]), 1)
        _, rest = gates_of(z, "value")
        g_abs = plain_back(dout, z, out.cpu(), x, h0, dh, "value", False)[0][0].abs()
        for t in (0, 1, 33, 69):
            for which in (0, 1):
                hi, lo = [x.clone(), z.clone(), h0], [x.clone(), z.clone(), h0]
                hi[which][:, t] += delta
                lo[which][:, t] -= delta
                num, err = difference(hi, lo)
                err = err + want[which][1][:, t] + (E * g_abs)[:, t]
                assert torch.all((num - got[which][:, t]).abs() <= err)
        num, err = difference((x, z, h0 + delta), (x, z, h0 - delta))
        assert torch.all((num - got[2]).abs() <= err + want[2][1])


@pytest.mark.parametrize("gate", ["log", "logit"])
@pytest.mark.parametrize("complement", [False, True])
def test_gate_forms_agree_with_autograd(gate, complement):
    # the gradient by the gate as given, against 64-bit automatic
    # differentiation of the plain loop
    B, N, C = 2, 40, 5
    g = torch.Generator().manual_seed(121)
    x, h0 = torch.randn(B, N, C, generator=g), torch.randn(B, C, generator=g)
    z = torch.randn(B, N, C, generator=g)
    z = -torch.exp(z) if gate == "log" else z
    dout, dh = torch.randn(B, N, C, generator=g), torch.randn(B, C, generator=g)
    leaves = [t.double().requires_grad_() for t in (x, z, h0)]
    a, rest = gates_of(leaves[1], gate)
    y = leaves[0] * (rest if complement else 1.0)
    h, hs = leaves[2], []
    for t in range(N):
        h = a[:, t] * h + y[:, t]
        hs.append(h)
    ((torch.stack(hs, 1) * dout.double()).sum() + (h * dh.double()).sum()).backward()
    out, _ = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), gate=gate, complement=complement)
    got = la.backward_recurrence(dout.cuda(), z.cuda(), out, x.cuda(), h0.cuda(), dh.cuda(),
                                 gate=gate, complement=complement)
    # dgates reads the states that the forward rounded: 16 u E each
    want = plain_back(dout, z, out.cpu(), x, h0, dh, gate, complement)
    E = 16 * U * bound(x, z, h0, gate, complement)
    E = torch.cat((torch.zeros(B, 1, C, dtype=torch.float64), E[:, :-1]), 1)
    a, rest = (t.detach() for t in gates_of(z, gate))
    slope = a if gate == "log" else a * rest
    g_abs = plain_back(dout, z, out.cpu(), x, h0, dh, gate, False)[0][0].abs()
    for leaf, t, (ref, tol), more in zip(leaves, got, want, (0.0, slope * g_abs * E, 0.0)):
        err = (t.cpu().double() - leaf.grad).abs()
        assert torch.all(err <= tol + more + 1e-12), float(err.max())


def test_repeats_its_bits_and_other_stream_and_graph():
    x, z, h0 = (t.cuda() for t in inputs(2, 3000, 128, ("bf16", "bf16"), "logit", 131))
    ref = la.forward_recurrence(x, z, h0, gate="logit", complement=True)
    back = la.backward_recurrence(x, z, ref[0], x, h0, h0, gate="logit", complement=True)
    again = la.forward_recurrence(x, z, h0, gate="logit", complement=True)
    assert torch.equal(ref[0], again[0]) and torch.equal(ref[1], again[1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = la.forward_recurrence(x, z, h0, gate="logit", complement=True)
        b = la.backward_recurrence(x, z, ref[0], x, h0, h0, gate="logit", complement=True)
    s.synchronize()
    for p, q in zip((*y, *b), (*ref, *back)):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = la.forward_recurrence(x, z, h0, gate="logit", complement=True)
        b = la.backward_recurrence(x, z, y[0], x, h0, h0, gate="logit", complement=True)
        d = la.decode_step_recurrence(y[1], x[:, 0], z[:, 0], gate="logit", complement=True)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for p, q in zip((y[0], *b), (ref[0], *back)):
        assert torch.equal(p, q)
    h = ref[1].clone()
    assert torch.equal(d, la.decode_step_recurrence(h, x[:, 0], z[:, 0], gate="logit",
                                                    complement=True))
    assert torch.equal(h, y[1])


def test_no_tokens():
    e = torch.empty(2, 0, 8, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    out, hl = la.forward_recurrence(e, e, h0)
    assert out.shape == (2, 0, 8) and torch.equal(hl, h0)
    assert torch.all(la.forward_recurrence(e, e)[1] == 0)
    assert torch.equal(la.backward_recurrence(e, e, e, None, h0, h0)[2], h0)
    n = torch.empty(0, 5, 8, device="cuda")
    assert la.forward_recurrence(n, n)[0].shape == (0, 5, 8)


def test_offsets_past_32_bits():
    # token rows 2^30 elements apart: the last one's offset needs 64 bits
    C, gap, N = 64, 1 << 30, 4
    room = torch.empty(gap * (N - 1) + C, dtype=torch.bfloat16, device="cuda")
    xs = room.as_strided((1, N, C), (0, gap, 1))
    x, z, h0 = inputs(1, N, C, ("bf16", "bf16"), "logit", 141)
    xs.copy_(x)
    ref = la.forward_recurrence(x.cuda(), z.cuda(), h0.cuda(), gate="logit")
    got = la.forward_recurrence(xs, z.cuda(), h0.cuda(), out=xs, gate="logit")
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
