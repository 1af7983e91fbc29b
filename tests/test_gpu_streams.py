"""Calls with `stream=`: what they allocate has to be that stream's memory.  Memory
of the current stream's allocator may still be read by work enqueued there before it
was freed, and a kernel on another stream does not wait for that.  Checked by the
allocator's own record of which stream a segment belongs to."""
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


NAMES = ["forward", "forward_variant", "forward_gated", "forward_delta", "forward_causal_state",
         "decode_step", "decode_step_gated", "decode_step_delta", "qk_norm_rope",
         "backward_qk_norm_rope", "forward_recurrence", "backward_recurrence",
         "decode_step_recurrence"]


def owner(t):
    """The stream whose allocator t's memory came from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def calls():
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    q, k, v = (r(2, 3, 130, 64) for _ in range(3))
    gates = torch.rand(2, 3, 130, generator=g).cuda()
    q1, k1, v1 = (t[:, :, 0].contiguous() for t in (q, k, v))
    S, z, g1 = r(2, 3, 64, 64), r(2, 3, 64).abs(), gates[:, :, 0].contiguous()
    w = torch.ones(64, device="cuda")
    x, c, h = r(2, 100, 40), torch.rand(2, 100, 40, generator=g).cuda(), r(2, 40)
    token_major = r(2, 130, 3, 64).transpose(1, 2)
    return {
        "forward": lambda **s: la.forward(q, k, v, **s),
        "forward_variant": lambda **s: la.forward_variant(q, k, v, feature_map="identity",
                                                          normalise=False, **s),
        "forward_gated": lambda **s: la.forward_gated(q, k, v, gates, **s),
        "forward_delta": lambda **s: la.forward_delta(q, k, v, gates, **s),
        "forward_causal_state": lambda **s: la.forward_causal_state(q, k, v, **s),
        "decode_step": lambda **s: la.decode_step(S, z, q1, k1, v1, **s),
        "decode_step_gated": lambda **s: la.decode_step_gated(S, z, q1, k1, v1,
                                                              g1, **s),
        "decode_step_delta": lambda **s: la.decode_step_delta(S, q1, k1, v1, g1, **s),
        "qk_norm_rope": lambda **s: la.qk_norm_rope(q, k, w, w, **s),
        "backward_qk_norm_rope": lambda **s: la.backward_qk_norm_rope(q, k, token_major, v, w, w,
                                                                      **s),
        "forward_recurrence": lambda **s: la.forward_recurrence(x, c, h, **s),
        "backward_recurrence": lambda **s: la.backward_recurrence(x, c, x, None, h, h, **s),
        "decode_step_recurrence": lambda **s: la.decode_step_recurrence(h, x[:, 0],
                                                                        c[:, 0], **s),
    }


class Raw:
    """A stream of another library: nothing but the handle."""
    def __init__(self, s):
        self.cuda_stream = s.cuda_stream


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_results_are_the_streams_memory(name, raw):
    tensors = lambda r: [r] if torch.is_tensor(r) else list(r)  # noqa: E731
    want = tensors(calls()[name]())
    call = calls()[name]  # with states of its own
    torch.cuda.synchronize()
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    got = tensors(call(stream=Raw(side) if raw else side))
    assert torch.cuda.current_stream() == current
    side.synchronize()
    for a, b in zip(got, want):
        assert owner(a) == side.cuda_stream
        # by their bits: the delta rule on these keys ends in NaN
        assert a.stride() == b.stride() and torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_host_forward_allocates_its_workspace_there():
    q, k, v = (torch.randn(1, 2, 200, 64).pin_memory() for _ in range(3))
    want = la.forward_host(q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def held():
        return sum(s["total_size"] for s in torch.cuda.memory_snapshot()
                   if s["stream"] == side.cuda_stream)

    before = held()
    got = la.forward_host(q, k, v, stream=side)
    side.synchronize()
    assert held() > before and torch.equal(got, want)
