"""Two findings between two reads of the device status: neither is lost."""
import pytest
import torch

import gemm_epilogue_fusion_gb300 as g

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["timeout", "index"])
def test_a_timeout_does_not_hide_a_bad_index(first):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g.load_library()
    assert g.coda_get_device_status() == g.CODA_OK
    logits, t = torch.zeros(1, 64, device="cuda"), torch.tensor([64], dtype=torch.int32, device="cuda")
    for what in ([0, 1] if first == "timeout" else [1, 0]):
        g.coda_selftest_wait_timeout(1_000_000) if what == 0 else g.coda_logprobs(logits, t)
    with pytest.raises(g.CodaError) as err:
        g.coda_get_device_status()
    assert err.value.status == g.CODA_ERR_TIMEOUT
    with pytest.raises(g.CodaError) as err:
        g.coda_get_device_status()
    assert err.value.status == g.CODA_ERR_INVALID_ARG
    assert g.coda_get_device_status() == g.CODA_OK
