"""The recurrence where TMA brings the rows (starts and strides of whole 16-byte
units) and there are more strips than blocks run at once: a block passes from strip
to strip, with its stages, maps and states in the middle of their rings, after one,
two, three or more rounds, forward (128 tokens a round) and backward (64).  Against
the plain loops in 64 bits and by the tolerances of test_gpu_recurrence.py."""
import pytest

import linear_attention_feature_gb300 as la
import test_gpu_recurrence as base

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    la.build.build()
    la.load_library()


@pytest.mark.parametrize("gate, complement", [("logit", True), ("log", False)])
@pytest.mark.parametrize("types", base.TYPES)
@pytest.mark.parametrize("B, N, C", [
    (200, 60, 64),    # one round either way
    (200, 90, 64),    # one forward, two backward
    (90, 200, 128),   # two and four
    (100, 64, 72),    # a strip of which 8 channels are left, one round
    (180, 385, 72),   # the same, four and seven
    (70, 515, 256),   # five and nine
    (320, 1100, 8),   # one narrow strip each, many rounds
])
def test_more_strips_than_run_at_once(B, N, C, types, gate, complement):
    x, z, h0 = base.inputs(B, N, C, types, gate, 11 + N)
    for t in (x, z):
        assert t.stride(1) * t.element_size() % 16 == 0
    xd, zd, hd = x.cuda(), z.cuda(), h0.cuda()
    out, hl = la.forward_recurrence(xd, zd, hd, gate=gate, complement=complement)
    la.check_device_status()
    base.check_forward(x, z, h0, gate, complement, out, hl)
    g = torch.Generator().manual_seed(12)
    dout, dh = torch.randn(B, N, C, generator=g).to(x.dtype), torch.randn(B, C, generator=g)
    got = la.backward_recurrence(dout.cuda(), zd, out, xd, hd, dh.cuda(), gate=gate,
                                 complement=complement)
    la.check_device_status()
    want = base.plain_back(dout, z, out.cpu(), x, h0, dh, gate, complement)
    for a, (ref, tol) in zip(got, want):
        base.close(a, ref, tol)
