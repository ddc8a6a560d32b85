"""Log probabilities and their gradient of logits of every finite size, beside
ordinary ones and by themselves: masks of -1e10 or -1e30, rows that are huge as
a whole.  References are taken from the differences to the row's largest logit
in 64 bits, which hold log V where the logits themselves no longer do."""
import math

import pytest
import torch

import decode_util as U
from test_logprobs_gpu import BF, F32, padded

pytestmark = pytest.mark.gpu
# V below and above a vector for every thread, and rows that a cluster shares; M for 512, 256 and 128 threads a row
SHAPES = [(6, 300), (6, 5001), (6, 90001), (340, 601), (400, 30001)]
FAR = [1e9, 1e10, 3.3e20, 1e30, 5e37, 1.3 * 2.0 ** 25, 2.0 ** 25, 2.0 ** 24 + 2, 2.0 ** 23 - 2, 123456.0]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield
    g.coda_get_device_status()


def reference(x, t):
    """(logp, entropy, log sum exp(x - max), max, log probabilities) of rows without NaN and +inf, in 64 bits."""
    x = x.to(U.F64)
    top = x.amax(1, keepdim=True)
    d = x - top
    total = torch.logsumexp(d, 1, keepdim=True)
    lp = d - total
    p = torch.exp(lp)
    ent = -(torch.where(p > 0, lp, torch.zeros((), dtype=U.F64)) * p).sum(1)
    logp = torch.where(t >= 0, lp.gather(1, t.long().clamp(min=0)[:, None])[:, 0], torch.zeros((), dtype=U.F64))
    return logp, ent, total[:, 0], top[:, 0], lp


def check(x, t, top=5):
    import gemm_epilogue_fusion_gb300 as gg
    got = {k: v.cpu() for k, v in gg.coda_logprobs(padded(x), t.cuda(), top).items()}
    assert gg.coda_get_device_status() == gg.CODA_OK
    logp, ent, total, high, lp = reference(x, t)
    V = x.shape[1]
    # as in decode_util.logprobs_bounds, with the parts' sizes of x - max instead of x itself
    rel = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -20
    b = rel + total * 2.0 ** -22
    assert ((got["logp"].to(U.F64) - logp).abs() <= 2 * b + logp.abs() * 2.0 ** -22).all()
    assert ((got["entropy"].to(U.F64) - ent).abs() <= 4 * rel * (ent + total + math.log(V) + 1) + total * 2.0 ** -22).all()
    assert ((got["lse"].to(U.F64) - (high + total)).abs() <= 2 * b + high.abs() * 2.0 ** -23).all()
    order = torch.sort(x.to(U.F64), dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(got["top_ids"], order.int())
    want = lp.gather(1, order)
    assert ((got["top_logp"].to(U.F64) - want).abs() <= 2 * b[:, None] + want.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,V", SHAPES, ids=str)
@pytest.mark.parametrize("far", FAR, ids=lambda v: f"{v:g}")
def test_finite_masks_beside_ordinary_logits(dt, M, V, far):
    """All but a few columns masked with -far, a masked half, single masked columns, and a logit of -far as the target."""
    g = U.gen(V)
    x = (torch.randn(M, V, generator=g) * 2).to(dt)
    x[0, 3:] = -far
    x[1, : V // 2] = -far
    x[2, V // 2:] = -far
    x[3, ::97] = -far
    x[4, : V - 1] = -far
    x[5::2, 8:V - 8] = -far
    t = torch.randint(0, 3, (M,), generator=g, dtype=torch.int32)
    t[2] = V - 1
    check(x, t)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,V", SHAPES, ids=str)
@pytest.mark.parametrize("far", FAR, ids=lambda v: f"{v:g}")
def test_rows_whose_largest_logit_is_huge(dt, M, V, far):
    """Every logit at -far or far, or next to it, alone or beside much smaller ones."""
    g = U.gen(V + 1)
    size = torch.tensor(far).to(dt)
    # the next value of the type towards 0, and the one behind it: 0 or a few units away where far is near 2^24
    bits = size.view(torch.int16 if dt == BF else torch.int32)
    near = torch.stack([(bits - i).view(dt) for i in range(3)])
    x = near[torch.randint(0, 3, (M, V), generator=g)]
    x[0] = size
    x[1] = -size
    x[2] = -x[2]
    x[3, ::3] = -2 * size.float().clamp(max=8e37)
    x[4] = -x[4]
    x[4, ::2] = -torch.inf
    x[5::3] = -x[5::3]
    t = torch.randint(0, V, (M,), generator=g, dtype=torch.int32)
    t[4] = 1
    check(x, t)


def test_one_warp_of_huge_logits_at_every_place():
    """A stretch of a few threads' logits at -1e10 moves over the row; the maximum lies beside it."""
    V = 4096
    x = torch.zeros(64, V)
    for i in range(64):
        x[i, i * 64:(i + 1) * 64] = -1e10
        x[i, (i * 64 + 80) % V] = 5.0
    t = torch.tensor([(i * 64 + 80) % V for i in range(64)], dtype=torch.int32)
    check(x, t)
    check(x.to(BF), t)
