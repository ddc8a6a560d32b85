"""Log probabilities of given tokens, entropy and best alternatives, and their
gradient, on the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import decode_util as U

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield
    g.coda_get_device_status()


def padded(x):
    """x [M, V] on the GPU as a view of rows on 16-byte boundaries, NaN behind column V."""
    step = 16 // x.element_size()
    ld = -(-x.shape[1] // step) * step
    full = torch.full((x.shape[0], ld), math.nan, dtype=x.dtype)
    full[:, :x.shape[1]] = x
    return full.cuda()[:, :x.shape[1]]


def check_forward(x, targets, top):
    import gemm_epilogue_fusion_gb300 as gg
    got = gg.coda_logprobs(padded(x), targets.cuda(), top)
    assert gg.coda_get_device_status() == gg.CODA_OK
    got = {k: v.cpu() for k, v in got.items()}
    ref = U.logprobs(x, targets, top)
    b, be = U.logprobs_bounds(x, ref)
    for k, bound in (("lse", b), ("logp", 2 * b), ("entropy", be)):
        same = got[k].to(U.F64) == ref[k]  # infinities
        assert (same | ((got[k].to(U.F64) - ref[k]).abs() <= bound)).all(), k
    if top:
        assert torch.equal(got["top_ids"], ref["top_ids"])
        same = got["top_logp"].to(U.F64) == ref["top_logp"]
        assert (same | ((got["top_logp"].to(U.F64) - ref["top_logp"]).abs() <= 2 * b[:, None])).all()
    return got, ref


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,V,top", [(1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 7, 5), (5, 64, 64), (4, 100, 20), (1, 257, 3),
                                     (7, 1000, 1), (3, 4096, 50), (2, 8193, 64), (300, 515, 8), (1, 50257, 20),
                                     (5, 32000, 0), (160, 9999, 5), (1, 200001, 64), (20, 33001, 12),
                                     (1, 73729, 20), (2, 57345, 64), (1, 57344, 16), (40, 90001, 12), (500, 9999, 5),
                                     (460, 25001, 3), (1500, 603, 8)])
def test_logprobs_against_64_bits(dt, M, V, top):
    g = U.gen(M * 7 + V)
    x = (torch.randn(M, V, generator=g) * 3).to(dt)
    t = torch.randint(-1, V, (M,), generator=g, dtype=torch.int32)
    check_forward(x, t, top)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "few values", "blocks", "one large", "few threads", "nan"])
@pytest.mark.parametrize("M,V", [(2, 40000), (170, 6001), (100, 12001), (3, 100001), (500, 3001),
                                 (470, 13001)])
def test_alternatives_in_hard_orders(dt, kind, M, V):
    """Ties by the lower index, and orders in which every element beats those before it."""
    g = U.gen(V)
    j = torch.arange(V, dtype=torch.float32).expand(M, V)
    x = {"equal": torch.full((M, V), -1.5), "rising": j / V * 8, "falling": -j / V * 8,
         "few values": torch.randint(0, 3, (M, V), generator=g).float(),
         "blocks": (j // 97) % 11, "one large": torch.randn(M, V, generator=g),
         # thousands of elements above all others in one thread of six
         "few threads": torch.where((j // 8) % 128 < 20, 100 - (j // 8) % 128, torch.randn(M, V, generator=g)),
         "nan": j % 5}[kind].clone()
    if kind == "one large":
        x[:, V // 2] = 300.0
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    if kind == "nan":
        import gemm_epilogue_fusion_gb300 as gg
        x[:, 50::2] = math.nan
        got = gg.coda_logprobs(padded(x.to(dt)), t.cuda(), 33)
        assert torch.isnan(got["lse"]).all()
        assert (got["top_ids"].cpu() == torch.arange(50, 50 + 2 * 33, 2)).all()
        return
    check_forward(x.to(dt), t, 33)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [20, 5000, 70000, 150001])
def test_masked_logits(dt, V):
    """Rows with -inf, with the type's lowest value, with nothing left, and with one value left."""
    low = torch.finfo(dt).min
    g = U.gen(V)
    x = (torch.randn(6, V, generator=g) * 2).to(dt)
    x[0, ::2] = -math.inf
    x[1, : V - 3] = low
    x[2] = low                  # all equal: an ordinary uniform row
    x[3] = -math.inf            # nothing left
    x[4] = -math.inf
    x[4, V // 3] = 1.25         # one value left
    x[5, 1:] = -math.inf
    x[5, 0] = low
    t = torch.tensor([0, V - 1, 5, 2, V // 3, 0], dtype=torch.int32)
    import gemm_epilogue_fusion_gb300 as gg
    got = gg.coda_logprobs(padded(x), t.cuda(), 7)
    got = {k: v.cpu() for k, v in got.items()}
    keep = [0, 1, 2, 4, 5]
    ref = U.logprobs(x[keep], t[keep], 7)
    b, be = U.logprobs_bounds(x[keep], ref)
    b = b.clamp(max=1e-3) + ref["lse"].abs() * 2.0 ** -23  # the lowest value's own size bounds nothing of the others
    for k, bound in (("lse", b), ("logp", 2 * b)):
        a = got[k][keep].to(U.F64)
        assert ((a == ref[k]) | ((a - ref[k]).abs() <= bound + ref[k].abs() * 2.0 ** -22)).all(), k
    # 64-bit lse is lowest + log V there: its own rounding hides log V, the entropy does not
    want = ref["entropy"].clone()
    want[2] = math.log(V)
    assert ((got["entropy"][keep].to(U.F64) - want).abs() <= 1e-3).all()
    assert torch.equal(got["top_ids"][keep], ref["top_ids"])
    assert got["lse"][3] == -math.inf and got["logp"][3] == -math.inf and got["entropy"][3] == 0
    assert torch.isneginf(got["top_logp"][3]).all()
    assert got["top_ids"][3].tolist() == list(range(7))
    assert got["logp"][4] == 0 and got["entropy"][4] == 0 and got["logp"][5] == 0


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,V", [(5, 300), (500, 300), (5, 40001), (5, 90001)])
def test_logits_at_the_limit_of_the_packed_arithmetic(dt, M, V):
    """Rows whose largest logit is -2^126 or 2^126, beside -inf, equal and ordinary ones."""
    x = torch.full((M, V), -math.inf)
    x[0, 7] = -2.0 ** 126
    x[1] = -2.0 ** 126
    x[2, 3:9] = 2.0 ** 126
    x[3, ::3] = torch.randn(x[3, ::3].shape, generator=U.gen(V))
    x[3, 1] = -2.0 ** 126
    x[4:] = 0.0
    import gemm_epilogue_fusion_gb300 as gg
    t = torch.full((M,), 7, dtype=torch.int32)
    t[3] = 3
    got = {k: v.cpu() for k, v in gg.coda_logprobs(padded(x.to(dt)), t.cuda(), 6).items()}
    ref = U.logprobs(x.to(dt), t, 6)
    lp = [0.0, -math.log(V), -math.log(6), float(ref["logp"][3])] + [-math.log(V)] * (M - 4)
    ent = [0.0, math.log(V), math.log(6), float(ref["entropy"][3])] + [math.log(V)] * (M - 4)
    # log V plus the sums' 2^-20, and x - lse's rounding at the size of row 3
    for k, want in (("logp", lp), ("entropy", ent)):
        assert ((got[k].to(U.F64) - torch.tensor(want, dtype=U.F64)).abs() <= 2.0 ** -16).all(), k
    assert torch.equal(got["top_ids"], ref["top_ids"])


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_nan_infinite_and_unscored(dt):
    import gemm_epilogue_fusion_gb300 as gg
    V = 3001
    g = U.gen(1)
    x = torch.randn(5, V, generator=g).to(dt)
    x[0, 77] = math.nan
    x[1, 5] = math.inf
    t = torch.tensor([3, 3, -1, V, 2147483647], dtype=torch.int32)
    got = gg.coda_logprobs(padded(x), t.cuda(), 3)
    with pytest.raises(gg.CodaError, match="out of range"):
        gg.coda_get_device_status()
    got = {k: v.cpu() for k, v in got.items()}
    assert torch.isnan(got["lse"][:2]).all() and torch.isnan(got["entropy"][:2]).all()
    assert got["top_ids"][0, 0] == 77 and got["top_ids"][1, 0] == 5
    assert (got["logp"][2:] == 0).all() and torch.isfinite(got["lse"][2:]).all()
    assert gg.coda_get_device_status() == gg.CODA_OK


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (2, 7), (5, 64), (1, 50257), (40, 1003), (200, 4096), (3, 128256)])
@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
def test_gradient_against_64_bits(dt, M, V, which):
    import gemm_epilogue_fusion_gb300 as gg
    g = U.gen(M + V)
    x = (torch.randn(M, V, generator=g) * 3).to(dt)
    if V > 3:
        x[0, 1] = -math.inf
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    t[M // 2] = -1
    xd = padded(x)
    fwd = gg.coda_logprobs(xd, t.cuda())
    dl = torch.randn(M, generator=g) if which != "entropy" else None
    dh = torch.randn(M, generator=g) if which != "logp" else None
    c = lambda a: None if a is None else a.cuda()  # noqa: E731
    step = 16 // x.element_size()
    full = torch.full((M, -(-V // step) * step + step), 7.0, dtype=dt).cuda()
    out = gg.coda_logprobs_backward(xd, t.cuda(), fwd["lse"], fwd["entropy"] if dh is not None else None, c(dl), c(dh),
                                    dlogits=full[:, :V])
    assert out.data_ptr() == full.data_ptr()
    assert (full[:, V:] == 7.0).all()
    z = torch.zeros(M)
    ref, size, lp = U.logprobs_grad(x, t, fwd["lse"].cpu(), fwd["entropy"].cpu(), z if dl is None else dl,
                                    z if dh is None else dh)
    # p is off by x - lse's rounding (2^-24 of it) and the exponential's 2^-21; four more fp32 roundings
    bound = U.HALF[dt] * ref.abs() + size * (2.0 ** -20 + (lp.abs() + 32) * 2.0 ** -23) + 1e-36
    if dl is not None:
        bound += 2.0 ** -23 * dl.abs().to(U.F64)[:, None] * (ref.abs() > size * 1.0001)
    assert ((out.cpu().to(U.F64) - ref).abs() <= bound).all()
    alloc = gg.coda_logprobs_backward(xd, t.cuda(), fwd["lse"], fwd["entropy"], c(dl), c(dh))
    assert torch.equal(alloc, out)


def test_gradient_of_empty_and_unscored_rows():
    import gemm_epilogue_fusion_gb300 as gg
    x = torch.randn(4, 64, generator=U.gen(0)).to(BF)
    x[1] = -math.inf
    t = torch.tensor([2, 2, -1, 64], dtype=torch.int32).cuda()
    xd = x.cuda()
    lse = torch.logsumexp(x.double(), 1).float().cuda()
    ent = torch.zeros(4).cuda()
    dl = torch.tensor([1.0, 1.0, math.nan, math.nan]).cuda()
    d = gg.coda_logprobs_backward(xd, t, lse, None, dl, None).cpu()
    with pytest.raises(gg.CodaError, match="out of range"):
        gg.coda_get_device_status()
    assert torch.isfinite(d).all() and torch.count_nonzero(d[0]) == 64
    assert (d[1:] == 0).all()
    assert (gg.coda_logprobs_backward(xd, t.clamp(max=63), lse).cpu() == 0).all()  # no upstream gradient at all
    assert torch.equal(gg.coda_logprobs_backward(xd, t.clamp(max=63), lse, ent, None, torch.zeros(4).cuda()).cpu(),
                       torch.zeros(4, 64, dtype=BF))


def test_gradient_against_differences():
    """Central differences of the 64-bit forward along random directions."""
    import gemm_epilogue_fusion_gb300 as gg
    g = U.gen(3)
    M, V = 4, 257
    x = torch.randn(M, V, generator=g) * 2
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    a, b = torch.randn(M, generator=g), torch.randn(M, generator=g)
    xd = padded(x)
    f = gg.coda_logprobs(xd, t.cuda())
    grad = gg.coda_logprobs_backward(xd, t.cuda(), f["lse"], f["entropy"], a.cuda(), b.cuda()).cpu().to(U.F64)

    def loss(y):
        r = U.logprobs(y, t, 0)
        return (r["logp"] * a).sum() + (r["entropy"] * b).sum()

    for _ in range(5):
        u = torch.randn(M, V, generator=g, dtype=U.F64)
        h = 1e-5
        want = (loss(x.double() + h * u) - loss(x.double() - h * u)) / (2 * h)
        # the fp32 gradient's own error (2^-18 of its terms' size) and the differences' (h^2 and 2^-52 / h)
        assert abs((grad * u).sum() - want) <= 1e-5 * (1 + (grad * u).abs().sum())


@pytest.mark.parametrize("M,V", [(30, 5001), (1, 50257), (100, 20000), (2, 128256), (500, 5001)])
def test_logprobs_on_another_stream_and_in_a_graph(M, V):
    """Captured and replayed on other values in the same buffer, the bits are the eager calls'."""
    import gemm_epilogue_fusion_gb300 as gg
    g = U.gen(4)
    xs = [padded((torch.randn(M, V, generator=g) * 3).to(BF)) for _ in range(2)]
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32).cuda()
    dl = torch.randn(M, generator=g).cuda()
    want = []
    for x in xs:
        f = gg.coda_logprobs(x, t, 5)
        want.append({**{k: v.clone() for k, v in f.items()},
                     "d": gg.coda_logprobs_backward(x, t, f["lse"], f["entropy"], dl, dl)})
    buf = torch.empty(M, -(-V // 8) * 8, dtype=BF, device="cuda")[:, :V]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = gg.coda_logprobs(buf, t, 5)
        d = gg.coda_logprobs_backward(buf, t, f["lse"], f["entropy"], dl, dl)
    for x, w in list(zip(xs, want)) * 2:
        buf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        for k in f:
            assert torch.equal(f[k], w[k]), k
        assert torch.equal(d, w["d"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f = gg.coda_logprobs(xs[1], t, 5)
    side.synchronize()
    assert torch.equal(f["logp"], want[1]["logp"]) and torch.equal(f["top_ids"], want[1]["top_ids"])


def test_rows_behind_2_to_the_31_elements():
    import gemm_epilogue_fusion_gb300 as gg
    M, ld = 17000, 128256
    big = torch.empty(M, ld, dtype=BF, device="cuda")
    big[-2:] = 0.0
    big[-1, 77] = 4.0
    sub = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    sub[-1] = 77
    f = gg.coda_logprobs(big[-2:], sub[-2:], 2)
    whole = gg.coda_logprobs(big.zero_().index_put_((torch.tensor([M - 1]).cuda(), torch.tensor([77]).cuda()),
                                                    torch.tensor(4.0, dtype=BF).cuda()), sub, 2)
    assert torch.equal(whole["logp"][-2:], f["logp"]) and whole["top_ids"][-1].tolist() == [77, 0]
    g2 = torch.zeros_like(big)
    gg.coda_logprobs_backward(big, sub, whole["lse"], None, torch.ones(M, device="cuda"), None, dlogits=g2)
    p = math.exp(float(whole["logp"][-1]))
    assert abs(float(g2[-1, 77]) - (1 - p)) <= 2.0 ** -8 * (1 - p) + 1e-6 and (g2[-2] == 0).all()


@pytest.mark.parametrize("M,V", [(1, 20011), (7, 20011), (100, 20011), (700, 20011), (700, 30011), (5, 100003)])
def test_the_same_bits_on_every_call(M, V):
    import gemm_epilogue_fusion_gb300 as gg
    x = (torch.randn(M, V, generator=U.gen(M)) * 3).to(BF)
    x[:, 5000:9000] = x[:, 4999:5000]  # thousands of ties
    xd, t = padded(x), torch.full((M,), 17, dtype=torch.int32).cuda()
    first = {k: v.clone() for k, v in gg.coda_logprobs(xd, t, 30).items()}
    for _ in range(5):
        for k, v in gg.coda_logprobs(xd, t, 30).items():
            assert torch.equal(v, first[k]), k
