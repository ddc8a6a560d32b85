"""RMSNorm with an eps of zero, below fp32's squares, and beyond its sums, on
rows of any size, against 64 bits: one warp a row and many."""
import pytest
import torch

from experts_util import BF, E4, F32, F64, HALF, check, gen

pytestmark = pytest.mark.gpu

WIDTHS = [16, 512, 4096, 8192, 32768]


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    return g


def norm(g, x, eps):
    """The call's outputs, checked against 64 bits: r loses half of the sum's relative error (N additions), of its
    root's and of its quotient's; y a rounding for each of its products more.  gamma is 1."""
    N = x.shape[1]
    got = g.coda_add_rmsnorm(x.cuda(), torch.ones(N, device="cuda"), eps, want_q=True)
    eps = torch.tensor(eps, dtype=F32).to(F64)  # as the call takes it
    h = x.to(F64)
    r = 1 / torch.sqrt(h.square().mean(1) + eps)
    slack = (N / 2 + 8) * 2.0 ** -24
    check(got["r"], r, r * slack + 2.0 ** -149, "r")
    y = h * r[:, None]
    check(got["y"], y, y.abs() * (HALF[x.dtype] + slack * 1.01 + 2.0 ** -22) + 2.0 ** -149, "y")
    v = got["q"].view(E4).cpu().to(F64) * got["scale"].cpu().to(F64)[:, None]
    top = y.abs().amax(1, keepdim=True)
    check(v, y, y.abs() * (2.0 ** -4 + slack * 2.02 + 2.0 ** -21) + top / 448 * 2.0 ** -10 * 1.01 + 2.0 ** -149, "codes")
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("size", [2.0 ** -125, 1e-37, 1e-30, 1e-18, 1.0, 1e18, 1e30, 1e37])
def test_no_eps(g, N, dtype, size):
    x = (size * (torch.rand(5, N, generator=gen(N)) + 0.5)).to(dtype)  # no value below the smallest normal one
    x[:, ::3] *= -1
    norm(g, x, 0.0)


@pytest.mark.parametrize("eps", [1e-45, 1e-42, 1e-38, 1e-30, 1e-24])
@pytest.mark.parametrize("N", WIDTHS)
def test_an_eps_of_the_squares_size(g, N, eps):
    """Rows whose mean square is about eps, and far above and below it: the squares are subnormal, or zero in fp32."""
    x = eps ** 0.5 * torch.randn(7, N, generator=gen(N)) * torch.tensor([1e-6, 0.01, 0.3, 1.0, 3.0, 100.0, 1e6])[:, None]
    norm(g, x, eps)


@pytest.mark.parametrize("eps", [1e-5, 1e30, 1e38, 3.4e38])
def test_an_eps_and_squares_at_the_end_of_the_range(g, eps):
    x = torch.randn(6, 512, generator=gen(1)) * torch.tensor([0.0, 1.0, 1e10, 1e18, 1e19, 1e35])[:, None]
    norm(g, x, eps)


@pytest.mark.parametrize("N", [16, 4096])
def test_a_row_of_zeros_without_eps(g, N):
    """0 times infinity: r is infinite and the row NaN; the rows beside it are as ever."""
    x = torch.ones(3, N)
    x[1] = 0
    got = g.coda_add_rmsnorm(x.cuda(), torch.ones(N, device="cuda"), 0.0, want_q=True)
    assert torch.isinf(got["r"][1]) and got["scale"][1] == 1
    assert torch.isnan(got["y"][1]).all() and torch.isnan(got["q"].view(E4)[1].float()).all()
    for i in (0, 2):
        assert (got["r"][i] == 1).all() and (got["y"][i] == 1).all()
        assert (got["q"].view(E4)[i].float() * got["scale"][i] == 1).all()
    # with any eps at all it is a row of zeros, with scale 1
    got = g.coda_add_rmsnorm(x.cuda(), torch.ones(N, device="cuda"), 1e-45, want_q=True)
    assert (got["y"][1] == 0).all() and (got["q"][1] & 0x7F == 0).all() and got["scale"][1] == 1
