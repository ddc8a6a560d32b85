"""The weights of the decode attention are held in two 16-bit parts: inputs
whose outputs cancel (a key's value is the negative of its neighbour's), so
that the outputs' own rounding does not hide the weights'.

The bound is that of the other attention tests with 2^-16 for the weights.  The
keys are many and their scores small, so the scores' own fp32 error stays well
below that, and a host test shows that weights rounded once would not pass."""
import pytest
import torch

import decode_util as U
from test_paged_gpu import BF, E4, make, scales

LENS = [64, 1, 150, 0, 33]
HEADS = {BF: [(4, 16), (3, 64), (8, 16), (5, 128), (7, 192), (6, 256), (16, 16), (9, 64), (16, 128), (12, 192),
              (16, 256), (32, 32)],
         E4: [(4, 16), (1, 64), (8, 16), (6, 128), (2, 192), (5, 256), (8, 128), (16, 16), (9, 64), (16, 128), (12, 192),
              (16, 256), (32, 32)]}
CASES = [(ct, hq, d) for ct, heads in HEADS.items() for hq, d in heads]
NAME = {BF: "bf16", E4: "e4m3"}


def inputs(ct, hq, d):
    """Scores of a standard deviation of about 0.1."""
    q, k, v, table, ln, s = make(hq, 1, d, 16, LENS, (BF, ct), hq * 1000 + d, q_scale=0.1)
    odd = (-v[:, :, 0::2].float()).to(ct)  # a page begins at an even position
    live = ~torch.isnan(v[:, :, 1::2].float())
    v = v.float()
    v[:, :, 1::2] = torch.where(live, odd.float(), v[:, :, 1::2])
    v = v.to(ct)
    return q, k, v, table, ln, s


def reference(ct, hq, d):
    q, k, v, table, ln, s = inputs(ct, hq, d)
    o, lse, slack, spread = U.attention(q, k, v, table, ln, range(len(LENS)), d ** -0.5, *s)
    bound, _ = U.attention_bounds(o, slack, spread, lse, d, max(LENS), BF, 2.0 ** -16)
    return o, bound


def once_rounded(ct, hq, d):
    """The same outputs with each weight rounded once: to bf16, or 2^15 times as large to f16 (an e4m3 cache)."""
    q, k, v, table, ln, s = inputs(ct, hq, d)
    half, up = (torch.float16, 2.0 ** 15) if ct == E4 else (BF, 1.0)
    o = torch.zeros(len(LENS), hq, d, dtype=U.F64)
    for i, n in enumerate(LENS):
        if n == 0:
            continue
        ids = table[i, :-(-n // 16)].long()
        kk, vv = (U.pages(t, ids, 0).reshape(-1, d)[:n].to(U.F64) * f for t, f in zip((k, v), s))
        w = q[i].to(U.F64) @ kk.T * d ** -0.5
        w = torch.exp(w - w.amax(1, keepdim=True))
        o[i] = (w.float() * up).to(half).to(U.F64) / up @ vv / w.sum(1, keepdim=True)
    return o.to(BF)


@pytest.mark.parametrize("ct,hq,d", CASES, ids=lambda v: NAME.get(v, str(v)))
def test_a_single_rounding_would_show(ct, hq, d):
    o, bound = reference(ct, hq, d)
    assert ((once_rounded(ct, hq, d).to(U.F64) - o).abs() > bound).sum() >= 3


def on_the_gpu(ct, hq, d):
    import gemm_epilogue_fusion_gb300 as gg
    q, k, v, table, ln, s = inputs(ct, hq, d)
    ws = gg.paged_attention_workspace(hq, 1, d, "cuda")
    got = gg.coda_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda(), ln.cuda(), ws, **scales(ct, s))
    assert gg.coda_get_device_status() == gg.CODA_OK
    o, bound = reference(ct, hq, d)
    error = (got.cpu().view_as(o).to(U.F64) - o).abs()
    assert (error <= bound).all(), (error / bound).max()


@pytest.mark.gpu
@pytest.mark.parametrize("hq,d", HEADS[E4])
def test_weights_of_an_e4m3_cache(hq, d):
    on_the_gpu(E4, hq, d)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,d", HEADS[BF])
def test_weights_of_a_bf16_cache(hq, d):
    on_the_gpu(BF, hq, d)
