"""e4m3 rows whose largest value is so small that its 448th part is subnormal,
or below every float: the codes stay finite and stand for the values."""
import pytest
import torch

from experts_util import BF, E4, F32, F64, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    return g


def check_rows(q, s, x):
    """The scale is the row's largest over 448, to half a step or, where that is subnormal, up to the next one; a value
    is off by half a step of its code."""
    x, s, v = x.to(F64), s.cpu().to(F64)[:, None], q.view(E4).cpu().to(F64)
    want = x.abs().amax(1, keepdim=True) / 448
    want = torch.where(want > 0, want, torch.ones_like(want))
    assert torch.isfinite(v).all() and (s > 0).all()
    assert (s >= want * (1 - 2.0 ** -24)).all() and (s <= want * (1 + 2.0 ** -24) + 2.0 ** -149).all()
    assert ((v * s - x).abs() <= x.abs() * (2.0 ** -4 + 2.0 ** -23) + s * 2.0 ** -10).all()


@pytest.mark.parametrize("N", [16, 2048, 8192])
@pytest.mark.parametrize("steps", [1, 3, 224, 447, 448, 449, 671, 672, 673, 1000, 5000, 2 ** 15, 2 ** 23, 2 ** 31, 2 ** 33])
def test_rows_of_few_steps(g, N, steps):
    """Values up to `steps` of the smallest fp32, 2^-149, zeros among them."""
    u = (torch.rand(4, N, generator=gen(N), dtype=F64) * 2 - 1) * steps
    u = u.round() if steps < 2 ** 23 else u
    u[:, 0], u[0, 1:], u[1, 1::2] = steps, 0, 0
    u[2] = -u[2]
    x = (u * 2.0 ** -149).to(F32)
    check_rows(*g.coda_quantize_rows_e4m3(x.cuda()), x)


@pytest.mark.parametrize("size", [2.0 ** -133, 2.0 ** -130, 2.0 ** -126, 2.0 ** -118, 2.0 ** -117])
def test_bf16_rows(g, size):
    x = ((torch.rand(5, 256, generator=gen(1)) * 2 - 1).double() * size * 3).to(BF)
    x[0], x[:, 7] = 0, 0
    check_rows(*g.coda_quantize_rows_e4m3(x.cuda()), x)


def test_a_norm_with_a_tiny_gamma(g):
    """y itself is tiny: h r is about 1."""
    x, gamma = torch.randn(5, 512, generator=gen(2)), torch.full((512,), 2.0 ** -146)
    x[:, 3] = 0
    got = g.coda_add_rmsnorm(x.cuda(), gamma.cuda(), 1e-5, want_q=True)
    check_rows(got["q"], got["scale"], got["y"].cpu())
