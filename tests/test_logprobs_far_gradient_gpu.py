"""The gradient of rows whose lse is so large that fp32 cannot hold log V beside
it: rows masked with the type's lowest value, and rows with a large offset."""
import pytest
import torch

import decode_util as U
from test_logprobs_gpu import BF, F32, padded
from test_logprobs_range_gpu import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield
    g.coda_get_device_status()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 300, 5001, 50257])
@pytest.mark.parametrize("far", ["lowest", "largest", 1e30, -1e30, 1e10, -1e10, 2.0 ** 25, -3e7, 2.0 ** 20, 1e6, 70000.0, -40000.0,
                                 30000.0])
def test_gradient_of_rows_with_a_large_offset(dt, V, far):
    import gemm_epilogue_fusion_gb300 as gg
    g = U.gen(V)
    M = 7
    lim = torch.finfo(dt).max
    far = {"lowest": -lim, "largest": lim}.get(far, far)
    x = (torch.full((M, V), far, dtype=U.F64) + 2 * torch.randn(M, V, generator=g)).clamp(-lim, lim).to(dt)
    x[0] = torch.tensor(far, dtype=U.F64).to(dt)                  # a uniform row
    x[1] = (2 * torch.randn(V, generator=g)).to(dt)               # ordinary rows between them
    x[3] = (2 * torch.randn(V, generator=g)).to(dt)
    x[4, ::2] = -torch.inf
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    t[5] = -1
    t[4] = 1
    dl, dh = torch.randn(M, generator=g), torch.randn(M, generator=g)
    xd = padded(x)
    f = gg.coda_logprobs(xd, t.cuda())
    got = gg.coda_logprobs_backward(xd, t.cuda(), f["lse"], f["entropy"], dl.cuda(), dh.cuda()).cpu().to(U.F64)
    assert gg.coda_get_device_status() == gg.CODA_OK
    _, ent, _, _, lp = reference(x, t)
    p, lp = torch.exp(lp), torch.where(torch.isfinite(lp), lp, torch.zeros((), dtype=U.F64))
    live = torch.where(t >= 0, dl, torch.zeros(())).to(U.F64)
    want = -p * (live[:, None] + dh.to(U.F64)[:, None] * (lp + ent[:, None]))
    rows = torch.nonzero(t >= 0)[:, 0]
    want[rows, t[rows].long()] += live[rows]
    size = p * (live.abs()[:, None] + dh.abs().to(U.F64)[:, None] * (lp.abs() + ent[:, None] + 1))
    # p within 2^-10 (half a step of fp32 where lse is just below 2^15), or the entropy's own error; one rounding
    bound = U.HALF[dt] * want.abs() + 2.0 ** -9 * size + 2.0 ** -22 * live.abs()[:, None] + 1e-36
    assert ((got - want).abs() <= bound).all(), ((got - want).abs() / bound).amax(1)
