"""The recurrence's bounded waits, made to run out through the library's testing
hook: a round that the first block of each cluster never fetches, with a short
bound, must come back as LA_ERR_TIMEOUT from la_check_device_status, whatever
carries the rows and whichever way the sequence is cut (the block's own warps, its
other group and the cluster's other blocks all wait in vain), and the next ordinary
calls must give their usual bits."""
import pytest

import linear_attention_feature_gb300 as la

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TIMEOUT = 5
BOUND = 1 << 20  # cycles, about half a millisecond


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    return la.load_library()


# blocks alone over many strips, clusters, a sequence in pieces; rows by TMA,
# by words and by half words
SHAPES = [(200, 515, 64, 0), (2, 20000, 1024, 0), (1, 60000, 64, 0),
          (2, 5000, 510, 1), (90, 700, 65, 0)]


def calls(B, N, C, skew):
    g = torch.Generator().manual_seed(N)
    x, z = (torch.randn(B, N, C + skew, generator=g).bfloat16().cuda()[..., skew:]
            for _ in range(2))
    h0 = torch.randn(B, C, generator=g).cuda()
    out, last = la.forward_recurrence(x, z, h0, gate="logit", complement=True)
    return {"forward": lambda: la.forward_recurrence(x, z, h0, gate="logit", complement=True),
            "backward": lambda: la.backward_recurrence(x, z, out, x, h0, last, gate="logit",
                                                       complement=True)}


@pytest.mark.parametrize("hold", [0, 1])
@pytest.mark.parametrize("way", ["forward", "backward"])
@pytest.mark.parametrize("shape", SHAPES)
def test_wait_that_runs_out_is_reported(lib, shape, way, hold):
    call = calls(*shape)[way]
    want = call()
    la.check_device_status()
    assert lib.la_debug_inject_timeout(BOUND, hold) == 0
    call()
    with pytest.raises(la.LinAttnError) as e:
        la.check_device_status()
    assert e.value.status == TIMEOUT
    for _ in range(2):  # the hook is used up, the context and the kernel are sound
        for a, b in zip(call(), want):
            assert torch.equal(a, b)
        la.check_device_status()


@pytest.mark.parametrize("way", ["forward", "backward"])
@pytest.mark.parametrize("shape", SHAPES)
def test_nothing_held_back(lib, shape, way):
    call = calls(*shape)[way]
    want = call()
    assert lib.la_debug_inject_timeout(BOUND, -1) == 0
    for _ in range(2):
        for a, b in zip(call(), want):
            assert torch.equal(a, b)
        la.check_device_status()
