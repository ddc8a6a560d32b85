"""Buffers handed to the mixture-of-experts calls beyond what a call writes, on
the host: the library's calls are replaced by a recorder, so only the binding
and the composition run."""
import pytest
import torch

import gemm_epilogue_fusion_gb300 as g
from gemm_epilogue_fusion_gb300 import chain

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Recorder:
    """Stands in for the C marshalling: every call succeeds, its arguments are kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return g.CODA_OK
        return call

    def args(self, name):
        return [a for n, a in self.calls if n == name]


@pytest.fixture
def recorder(monkeypatch):
    g.load_library()
    r = Recorder()
    monkeypatch.setattr(g, "_fast", r)
    return r


def test_dispatch_returns_no_scale_that_it_has_not_written(recorder):
    X, slots, stale = torch.zeros(3, 16, dtype=BF), torch.zeros(3, 2, dtype=I32), torch.full((6,), 9.0)
    _, got = g.coda_expert_dispatch(X, slots, scale_s=stale)
    assert got is None
    assert recorder.args("expert_dispatch")[0][4] is None
    _, got = g.coda_expert_dispatch(X, slots, scale=torch.ones(3), scale_s=stale)
    assert got is stale


@pytest.mark.parametrize("save", [False, True])
def test_a_bf16_layer_ignores_the_scales_buffer(recorder, save):
    """One set of buffers for bf16 and e4m3 layers: the e4m3 one's row scales are no scale of the bf16 one's rows."""
    X, slots = torch.zeros(3, 16, dtype=BF), torch.zeros(3, 2, dtype=I32)
    Wgu, Wd = torch.zeros(4, 16, 16, dtype=BF), torch.zeros(4, 16, 8, dtype=BF)
    out = chain.expert_layer(X, slots, torch.zeros(5, dtype=I32), torch.ones(3, 2), Wgu, Wd, save=save,
                             bufs={"sxs": torch.full((6,), 9.0)})
    assert out["sxs"] is None
    assert recorder.args("grouped_swiglu")[0][3] is None
    assert all(a[3] is None for a in recorder.args("grouped_gemm"))


def test_an_e4m3_layer_uses_it(recorder):
    X, slots = torch.zeros(3, 16, dtype=U8), torch.zeros(3, 2, dtype=I32)
    Wgu, Wd, one, sxs = torch.zeros(4, 32, 16, dtype=U8), torch.zeros(4, 16, 16, dtype=U8), torch.ones(4), torch.zeros(6)
    out = chain.expert_layer(X, slots, torch.zeros(5, dtype=I32), torch.ones(3, 2), Wgu, Wd, scale_x=torch.ones(3),
                             scale_wgu=one, scale_wd=one, bufs={"sxs": sxs})
    assert out["sxs"] is sxs and recorder.args("grouped_swiglu")[0][3] is sxs


def test_the_norm_returns_no_scale_that_it_has_not_written(recorder):
    X, stale = torch.zeros(3, 16, dtype=BF), torch.full((3,), 9.0)
    got = g.coda_add_rmsnorm(X, torch.ones(16), 1e-5, scale=stale)
    assert got["q"] is None and got["scale"] is None
    assert recorder.args("add_rmsnorm")[0][6] is None
    got = g.coda_add_rmsnorm(X, torch.ones(16), 1e-5, scale=stale, want_q=True)
    assert got["scale"] is stale
    codes = torch.zeros(3, 16, dtype=U8)
    assert g.coda_add_rmsnorm(X, torch.ones(16), 1e-5, Yq=codes, scale=stale)["scale"] is stale
