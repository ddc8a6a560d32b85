"""Calls on a stream that is not the current one, with workspaces of their own,
while the current stream takes and fills memory of the same sizes."""
import pytest
import torch

from experts_util import BF, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield g
    assert g.coda_get_device_status() == g.CODA_OK


def beside(call, sizes):
    """The call's results on another stream, which is busy when it is made, with blocks of `sizes` bytes taken and
    filled on the current one right behind it."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)  # about a millisecond
    out = call(side)
    held = [torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del held
    return out


@pytest.mark.parametrize("by_address", [False, True])
@pytest.mark.parametrize("rows, experts, top", [(3000, 64, 8), (1025, 200, 1)])
def test_router(g, by_address, rows, experts, top):
    logits = torch.randn(rows, experts, generator=gen(1)).to(BF).cuda()
    want = g.coda_route(logits, top)
    outs = {k: torch.empty_like(v) for k, v in want.items()}
    size = max(4, g.load_library().coda_route_workspace_bytes(rows, experts, top))
    got = beside(lambda s: g.coda_route(logits, top, stream=s.cuda_stream if by_address else s, **outs), [size])
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("by_address", [False, True])
def test_norm_gradient(g, by_address):
    M, N = 2000, 1024
    H, dY = (torch.randn(M, N, generator=gen(s)).to(BF).cuda() for s in (2, 3))
    gamma, r = torch.rand(N, generator=gen(4)).cuda() + 0.5, torch.rand(M, generator=gen(5)).cuda() + 0.5
    want = g.coda_add_rmsnorm_backward(dY, H, r, gamma)
    dH, dgamma = torch.empty_like(H), torch.empty_like(gamma)
    size = g.load_library().coda_add_rmsnorm_backward_workspace_bytes(M, N)
    got = beside(lambda s: g.coda_add_rmsnorm_backward(dY, H, r, gamma, dH=dH, dgamma=dgamma,
                                                       stream=s.cuda_stream if by_address else s), [size])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_dense_norm_gradient(g):
    M, N = 2000, 1024
    H, dY = (torch.randn(M, N, generator=gen(s)).to(BF).cuda() for s in (6, 7))
    gamma, r = torch.rand(N, generator=gen(8)).cuda() + 0.5, torch.rand(M, generator=gen(9)).cuda() + 0.5
    S = torch.randn(M, g.coda_partial_cols(N), generator=gen(10)).cuda()
    want = g.coda_rmsnorm_backward(dY, H, r, gamma, S)
    out = {"dH": torch.empty_like(H), "Yt": torch.empty_like(H), "dgamma": torch.empty_like(gamma)}
    size = g.load_library().coda_rmsnorm_backward_workspace_bytes(M, N)
    got = beside(lambda s: g.coda_rmsnorm_backward(dY, H, r, gamma, S, stream=s, **out), [size])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_default_stream_by_its_address(g):
    """Address 0, with another stream current."""
    logits = torch.randn(2000, 64, generator=gen(11)).to(BF).cuda()
    want = g.coda_route(logits, 4)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = g.coda_route(logits, 4, stream=0)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
