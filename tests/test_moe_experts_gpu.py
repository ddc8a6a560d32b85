"""chain.moe_block and its backward for numbers of experts that are no multiple
of 8, whose logits' rows end inside 16 bytes, against 64 bits."""
import pytest
import torch

from experts_util import BF, F64, gen, route
from test_moe_chain_gpu import EPS, Block, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield g
    assert g.coda_get_device_status() == g.CODA_OK


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("M, E, top", [(1, 5, 2), (33, 12, 3), (70, 60, 4), (9, 1, 1), (20, 15, 15)])
def test_block_and_backward(g, M, E, top, renormalize):
    from gemm_epilogue_fusion_gb300 import chain
    H, I = 264, 72
    b = Block(M, H, E, I, M)
    f = b.run(chain, top, renormalize=renormalize, save=True)
    assert f["logits"].shape == (M, E)
    ids, _, slots, offsets = route(f["logits"].cpu().float(), top, renormalize)
    assert torch.equal(f["ids"].cpu(), ids) and torch.equal(f["slots"].cpu(), slots)
    assert torch.equal(f["offsets"].cpu(), offsets)
    dH2 = torch.randn(M, H, generator=gen(4)).to(BF)
    d = chain.moe_block_backward(b.dev["gamma"], b.dev["Wr"], b.dev["Wgu"], b.dev["Wd"], f, dH2.cuda(),
                                 renormalize=renormalize)
    assert d["dWrt"].shape == (E, H) and d["dlogits"].shape == (M, E)
    leaves = {k: getattr(b, k).to(F64).requires_grad_(True) for k in ("X", "R", "gamma", "Wr", "Wgu", "Wd")}
    _, h2 = b.exact(ids, renormalize, leaves)
    near(f["h2"], h2)
    (h2 * dH2.to(F64)).sum().backward()
    for name, leaf in (("dX", "X"), ("dX", "R"), ("dgamma", "gamma"), ("dWgut", "Wgu"), ("dWdt", "Wd")):
        near(d[name], leaves[leaf].grad)
    if renormalize and top == 1:  # the only choice has all the weight whatever its logit
        assert (d["dWrt"] == 0).all()
    else:
        near(d["dWrt"], leaves["Wr"].grad)


def test_a_logits_buffer(g):
    from gemm_epilogue_fusion_gb300 import chain
    b = Block(20, 128, 12, 64, 3)
    want = b.run(chain, 2)
    logits = torch.empty(20, 16, dtype=BF, device="cuda")
    got = b.run(chain, 2, bufs={"logits": logits})
    assert got["logits"].data_ptr() == logits.data_ptr() and torch.equal(got["logits"], want["logits"])
    assert torch.equal(got["h2"], want["h2"])


@pytest.mark.parametrize("E", [8, 12])
def test_no_rows(g, E):
    """An empty batch: nothing comes out, and the weights' gradients are zeros."""
    from gemm_epilogue_fusion_gb300 import chain
    b = Block(0, 128, E, 64, 5)
    f = b.run(chain, 2, save=True, want_p=True)
    assert f["h2"].shape == (0, 128) and f["logits"].shape == (0, E) and (f["offsets"] == 0).all()
    dH2 = torch.empty(0, 128, dtype=BF, device="cuda")
    d = chain.moe_block_backward(b.dev["gamma"], b.dev["Wr"], b.dev["Wgu"], b.dev["Wd"], f, dH2)
    assert d["dX"].shape == (0, 128)
    for name, like in (("dgamma", "gamma"), ("dWrt", "Wr"), ("dWgut", "Wgu"), ("dWdt", "Wd")):
        assert d[name].shape == b.dev[like].shape and (d[name] == 0).all(), name
