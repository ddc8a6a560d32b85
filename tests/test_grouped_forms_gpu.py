"""Every grouped product in every form of its kernels, whichever the rule would
take: lone CTAs, pairs, and 32-row tiles whose contraction 1, 2, 4 or 8 CTAs
split, each forced by its variable, on ragged groups against 64 bits."""
import pytest
import torch

from experts_util import BF, E4, HALF, check, codes, gen, grouped, offsets_of, sum_bound, swiglu, swiglu_backward

pytestmark = pytest.mark.gpu

FORMS = {"lone": ("CODA_CTA_GROUP", "1"), "pair": ("CODA_CTA_GROUP", "2"),
         **{f"split_{n}": ("CODA_GROUP_SPLIT", str(n)) for n in (1, 2, 4, 8)}}
COUNTS = {"one_row": [1], "edges": [0, 31, 32, 33, 0, 1, 64, 65, 2], "last_only": [0, 0, 0, 40],
          "uneven": [150, 0, 7, 300], "many": [(5 * i * i + 3 * i) % 23 for i in range(60)]}
# one k-block (fewer than the CTAs of a split), a part-filled last one, more than the stages; ragged columns
SIZES = [(136, 16), (264, 144), (520, 1040)]
DEEP = (72, 4112)  # k-blocks for every CTA of a split, and rounds of its stages


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield g
    assert g.coda_get_device_status() == g.CODA_OK


@pytest.fixture(params=FORMS)
def form(request, monkeypatch):
    monkeypatch.delenv("CODA_CTA_GROUP", raising=False)
    monkeypatch.setenv(*FORMS[request.param])
    return request.param


def filled(*shape):
    return torch.full(shape, 7.0, dtype=BF, device="cuda")


class Case:
    """Ragged groups with five rows of no expert behind them; bf16 or e4m3 operands, scales for rows and experts."""

    def __init__(self, counts, N, K, e4m3, seed):
        r = gen(seed)
        c = COUNTS[counts]
        self.n, self.E, self.o = sum(c), len(c), offsets_of(c)
        X, W = torch.randn(self.n + 5, K, generator=r), torch.randn(self.E, N, K, generator=r) / K ** 0.5
        self.rs = torch.rand(self.n + 5, generator=r) + 0.5
        self.ws = torch.rand(self.E, generator=r) + 0.5 if e4m3 else None
        self.X, self.W = (codes(64 * X), codes(64 * W)) if e4m3 else (X.to(BF), W.to(BF))
        if e4m3:  # back to values of about one
            self.rs, self.ws = self.rs / 64, self.ws / 64
        self.scales = {"row_scale": self.rs.cuda(), **({"w_scale": self.ws.cuda()} if e4m3 else {})}
        self.host = (self.X.float(), self.W.float(), self.o, self.rs, self.ws)
        self.dev = (self.X.cuda(), self.W.cuda(), self.o.cuda())

    def same(self, got, ref, tol, what):
        check(got[:self.n], ref[:self.n], tol[:self.n], what)
        assert (got[self.n:].float() == 7.0).all(), f"{what}: rows of no expert were written"


def plain(g, case, K):
    ref, S = grouped(*case.host)
    # two scales are two roundings more, of the product and of their own
    tol = ref.abs() * (HALF[BF] + 2.0 ** -22) + sum_bound(S, K) * 1.01 + 1e-37
    for _ in range(2):
        Y = filled(len(case.X), case.W.shape[1])
        g.coda_grouped_gemm(*case.dev, Y=Y, **case.scales)
        case.same(Y, ref, tol, "Y")
    return Y, ref, tol


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N, K", SIZES + [DEEP])
def test_bf16(g, form, counts, N, K):
    case = Case(counts, N, K, False, 1)
    Y, ref, tol = plain(g, case, K)
    T = filled(*Y.shape)
    g.coda_grouped_gemm(case.dev[0], case.dev[1].transpose(1, 2).contiguous(), case.dev[2], b_mn=True, Y=T, **case.scales)
    case.same(T, ref, tol, "Y, b_mn")


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N, K", SIZES + [DEEP])
def test_e4m3(g, form, counts, N, K):
    plain(g, Case(counts, N, K, True, 2), K)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I, K", SIZES + [DEEP])
def test_swiglu(g, form, counts, I, K, e4m3):
    case = Case(counts, 2 * I, K, e4m3, 3)
    act, tol, Z, ztol = swiglu(*case.host)
    A = filled(len(case.X), I)
    g.coda_grouped_gemm_swiglu(*case.dev, Act=A, **case.scales)
    case.same(A, act, tol, "act")
    if not e4m3:
        B, GU = filled(len(case.X), I), filled(len(case.X), 2 * I)
        g.coda_grouped_gemm_swiglu(*case.dev, Act=B, GU=GU, **case.scales)
        case.same(GU, Z, ztol, "GU")
        assert torch.equal(A, B)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I, K", SIZES + [DEEP])
def test_swiglu_backward(g, form, counts, I, K):
    case = Case(counts, K, I, False, 4)  # its weights are Wd [E, K, I]
    dY = torch.randn(case.n + 5, K, generator=gen(5)).to(BF)
    GU = torch.randn(case.n + 5, 2 * I, generator=gen(6)).to(BF)
    ref, tol = swiglu_backward(dY, case.W, GU, case.o)
    dGU = filled(case.n + 5, 2 * I)
    g.coda_grouped_gemm_swiglu_backward(dY.cuda(), case.dev[1], GU.cuda(), case.dev[2], dGU)
    case.same(dGU, ref, tol, "dGU")


@pytest.mark.parametrize("e4m3", [False, True])
def test_replayed_with_other_offsets(g, form, e4m3):
    """One captured SwiGLU product, replayed on groups of other sizes."""
    case, I, K = Case("uneven", 2 * 200, 1040, e4m3, 7), 200, 1040
    X, W, o = case.dev
    A = filled(len(case.X), I)
    g.coda_grouped_gemm_swiglu(X, W, o, Act=A, **case.scales)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.coda_grouped_gemm_swiglu(X, W, o, Act=A, **case.scales)
    for c in ([0, 0, 0, 0], [457, 0, 0, 0], [1, 2, 33, 400], [100, 100, 100, 100]):
        case.o, case.n = offsets_of(c), sum(c)
        o.copy_(case.o)
        A.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        act, tol, _, _ = swiglu(case.X.float(), case.W.float(), case.o, case.rs, case.ws)
        case.same(A, act, tol, f"act of {c}")


@pytest.mark.parametrize("split", ["1", "8"])
def test_as_many_columns_as_wrapped_the_band(g, monkeypatch, split):
    """2^24 output columns, and 2^23 with SwiGLU: 65536 column tiles."""
    monkeypatch.setenv("CODA_GROUP_SPLIT", split)
    N, K, rows = 1 << 24, 8, 70
    X = torch.randn(rows, K, generator=gen(8)).to(BF)
    W = torch.randn(1, N, K, generator=torch.Generator("cuda").manual_seed(9), device="cuda").to(BF)
    o = torch.tensor([0, rows], dtype=torch.int32)
    pick = torch.cat((torch.arange(0, N, N // 97), torch.arange(N - 300, N)))
    Y = g.coda_grouped_gemm(X.cuda(), W, o.cuda())
    ref, S = grouped(X, W[:, pick.cuda()].cpu(), o)
    check(Y[:, pick.cuda()], ref, ref.abs() * HALF[BF] + sum_bound(S, K) * 1.01 + 1e-37, "Y")
    del Y
    pick = pick // 2
    A, _ = g.coda_grouped_gemm_swiglu(X.cuda(), W, o.cuda())
    act, tol, _, _ = swiglu(X, W[:, torch.cat((pick, pick + N // 2)).cuda()].cpu(), o)
    check(A[:, pick.cuda()], act, tol, "act")
