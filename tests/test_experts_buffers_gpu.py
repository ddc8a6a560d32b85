"""One set of buffers for layers of both types, on the GPU: what an e4m3 layer
leaves in it does not reach a bf16 one."""
import pytest
import torch

from experts_util import BF, E4, gen, route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gemm_epilogue_fusion_gb300 as g
    g.load_library()
    yield g
    assert g.coda_get_device_status() == g.CODA_OK


def layer(seed, M=37, H=128, E=8, I=64, top=2):
    r = gen(seed)
    n = lambda *s: torch.randn(*s, generator=r).to(BF)  # noqa: E731
    _, w, slots, offsets = route(torch.randn(M, E, generator=r), top, True)
    return {"X": n(M, H).cuda(), "slots": slots.cuda(), "offsets": offsets.cuda(), "weights": w.float().cuda(),
            "Wgut": (n(E, 2 * I, H) / H ** 0.5).cuda(), "Wdt": (n(E, H, I) / I ** 0.5).cuda(), "R": n(M, H).cuda()}


@pytest.mark.parametrize("save", [False, True])
def test_scales_in_the_buffers(g, save):
    from gemm_epilogue_fusion_gb300 import chain
    a = layer(1)
    want = chain.expert_layer(**a, save=save)
    for stale in (0.25, float("nan")):
        sxs = torch.full((len(a["X"]) * 2,), stale, device="cuda")
        got = chain.expert_layer(**a, save=save, bufs={"sxs": sxs})
        assert got["sxs"] is None
        for k in ("act", "y", "h") + (("GU",) if save else ()):
            assert torch.equal(got[k], want[k]), k


def test_layers_of_both_types_in_turn(g):
    from gemm_epilogue_fusion_gb300 import chain
    a = layer(2)
    q, scale = g.coda_quantize_rows_e4m3(a["X"])
    w8 = {k: (a[k].float() * 100).to(E4) for k in ("Wgut", "Wdt")}
    s8 = torch.full((8,), 0.01, device="cuda")
    fp8 = {**a, **w8, "X": q, "scale_x": scale, "scale_wgu": s8, "scale_wd": s8}
    want, want8 = chain.expert_layer(**a), chain.expert_layer(**fp8)
    bufs = {"sxs": torch.empty(74, device="cuda"), "act": torch.empty_like(want["act"]), "y": torch.empty_like(want["y"])}
    for _ in range(2):
        assert torch.equal(chain.expert_layer(**fp8, bufs=bufs)["h"], want8["h"])
        assert torch.equal(chain.expert_layer(**a, bufs=bufs)["h"], want["h"])
