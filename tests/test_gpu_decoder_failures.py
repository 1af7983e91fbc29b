"""The bounded waits of the paged attention and of the cross attention's kernels, made to run
out through the library's testing hook: tiles that are never fetched, with a short
bound, must come back as LA_ERR_TIMEOUT from la_check_device_status, and the next
ordinary calls must give their usual bits."""
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


def paged(B, Hq, Hk, T, n, d, page):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    pages = -(-n // page)
    kc, vc = (torch.randn(B * pages, Hk, page, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    lengths = torch.randint(n // 2, n - T, (B,), generator=g, device="cuda").int()
    q = torch.randn(B, Hq, T, d, generator=g, device="cuda").bfloat16()
    return lambda: (la.decode_step_paged(q, kc, vc, table, lengths),)


def cross(B, Hq, Hk, N, M, d, ragged=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + M)
    r = lambda H, L: torch.randn(B, H, L, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, dout, k, v = r(Hq, N), r(Hq, N), r(Hk, M), r(Hk, M)
    lens = torch.randint(M // 3, M, (B,), generator=g, device="cuda").int() if ragged else None
    _, S, z = la.forward_cross(q, k, v, lens)
    return (lambda: la.forward_cross(q, k, v, lens), lambda: (la.decode_step_cross(S, z, q),),
            lambda: la.backward_cross(dout, q, k, v, S, z, lens))


# tiles of a block (or of a warp): more than its stages, so that one is awaited while others
# are under way and stages are filled again
CALLS = {
    "paged 64": lambda: paged(32, 16, 16, 4, 4096, 64, 16),
    "paged 128, one sequence": lambda: paged(1, 32, 8, 1, 65536, 128, 64),
    "paged 128, many stretches": lambda: paged(300, 8, 8, 1, 500, 128, 32),
    "paged 256": lambda: paged(32, 16, 4, 2, 2048, 256, 16),
    "states 64": lambda: cross(2, 8, 8, 10, 16384, 64)[0],
    "states 128": lambda: cross(4, 8, 8, 10, 8192, 128, True)[0],
    "steps 64": lambda: cross(4, 32, 8, 4096, 50, 64)[1],
    "steps 128": lambda: cross(4, 32, 8, 4096, 50, 128)[1],
    "queries' gradient 64": lambda: cross(4, 32, 8, 8192, 100, 64)[2],
    "queries' gradient 128": lambda: cross(4, 32, 8, 4096, 100, 128)[2],
    "keys' gradient 64": lambda: cross(4, 8, 8, 100, 16384, 64, True)[2],
    "keys' gradient 128": lambda: cross(4, 8, 8, 100, 16384, 128, True)[2],
}


@pytest.mark.parametrize("hold", [0, 1, 5])
@pytest.mark.parametrize("name", CALLS)
def test_wait_that_runs_out_is_reported(lib, name, hold):
    call = CALLS[name]()
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


@pytest.mark.parametrize("name", CALLS)
def test_nothing_held_back(lib, name):
    call = CALLS[name]()
    want = call()
    assert lib.la_debug_inject_timeout(1 << 28, -1) == 0
    for _ in range(2):
        for a, b in zip(call(), want):
            assert torch.equal(a, b)
        la.check_device_status()
