"""Decode attention with scores of every finite size: the largest weight of a
row is 1 whatever the scores' own rounding, so nothing overflows or vanishes."""
import math

import pytest
import torch

import decode_util as U
from test_paged_gpu import BF, E4, IDS, TYPES, make, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield
    g.coda_get_device_status()


def put(cache, table, b, t, page, col, x):
    raw = cache.view(torch.uint8) if cache.element_size() == 1 else cache
    raw[table[b, t // page], :, t % page, col] = torch.tensor(x).to(cache.dtype).view(raw.dtype)


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("hq,d", [(2, 64), (8, 64), (16, 128), (4, 256)], ids=str)
@pytest.mark.parametrize("size", [1e5, 1.1e7, 1e8, 1e10, 1e12, 1e20, 1e30, -1e6, -3e7, -1e8, -1e10, -1e20, -1e30], ids=str)
def test_equal_scores_of_every_size(types, hq, d, size):
    """Column 0 alone makes the scores, the same for every key: the output is the values' mean."""
    import gemm_epilogue_fusion_gb300 as gg
    page, lens = 16, [1, 5, 70, 2000, 0]
    q, k, v, table, ln, s = make(hq, 1, d, page, lens, types, hq + d)
    one = 48.0 if types[1] == E4 else 1.0
    q = torch.zeros_like(q)
    q[:, :, 0] = size / (one * s[0])
    for b, n in enumerate(lens):
        for t in range(n):
            put(k, table, b, t, page, 0, one)
    ws = gg.paged_attention_workspace(hq, 1, d, "cuda")
    lse = torch.empty(len(lens), hq).cuda()
    o = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, lse=lse, scale=1.0,
                                **scales(types[1], s)).cpu().view(len(lens), hq, d).to(U.F64)
    assert gg.coda_get_device_status() == gg.CODA_OK
    lse = lse.cpu().to(U.F64)
    score = q[0, 0, 0].to(U.F64) * one * float(torch.tensor(s[0]))
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[b] == 0).all() and torch.isneginf(lse[b]).all()
            continue
        ids = table[b, :-(-n // page)].long()
        vals = U.pages(v, ids, 0).reshape(-1, d)[:n].to(U.F64) * s[1]
        # equal weights: the products' and sums' additions, the division, one rounding
        bound = U.HALF[types[0]] * vals.mean(0).abs() + vals.abs().mean(0) * ((n + 16) * 2.0 ** -23 + 2.0 ** -20)
        assert ((o[b] - vals.mean(0)).abs() <= bound * 1.01).all()
        assert ((lse[b] - (score + math.log(n))).abs() <= score.abs() * 2.0 ** -21 + 1e-4).all()


@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("hq,d", [(2, 64), (8, 64), (16, 128), (4, 256)], ids=str)
@pytest.mark.parametrize("far", [1e8, 1e10, 1e20, 1e30], ids=str)
def test_keys_of_far_scores_beside_ordinary_ones(types, hq, d, far):
    """Column 0 puts most keys at a score of -far, whole tiles of them too: the ordinary keys alone make the output."""
    import gemm_epilogue_fusion_gb300 as gg
    page, lens = 16, [70, 700, 3000, 40]
    keep = [[3], [5, 600, 601], list(range(1000, 1040)), [0, 39]]
    q, k, v, table, ln, s = make(hq, 1, d, page, lens, types, hq + d + 1)
    # an e4m3 cache's queries are held relative to their largest value: the far column takes it, the others are zero
    q[:, :, 1:] = 0
    q[:, :, 0] = far / (48.0 * s[0] if types[1] == E4 else 1.0)
    for b, n in enumerate(lens):
        for t in range(n):
            put(k, table, b, t, page, 0, 0.0 if t in keep[b] else -48.0 if types[1] == E4 else -1.0)
    ws = gg.paged_attention_workspace(hq, 1, d, "cuda")
    lse = torch.empty(len(lens), hq).cuda()
    o = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, lse=lse, scale=1.0,
                                **scales(types[1], s)).cpu().view(len(lens), hq, d).to(U.F64)
    assert gg.coda_get_device_status() == gg.CODA_OK
    for b, at in enumerate(keep):
        vals = torch.stack([U.pages(v, table[b, t // page].long()[None], 0)[0, t % page] for t in at]).to(U.F64) * s[1]
        bound = U.HALF[types[0]] * vals.mean(0).abs() + vals.abs().mean(0) * 2.0 ** -16
        assert ((o[b] - vals.mean(0)).abs() <= bound * 1.01).all()
        assert ((lse[b].cpu().to(U.F64) - math.log(len(at))).abs() <= 2.0 ** -18).all()
