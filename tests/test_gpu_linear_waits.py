"""The linear kernel's waits where a sum is taken over in parts of eight slabs: whether one of them outlasts the hardware's own
patience hangs on the memory (14 to 20 of 20 calls did whose W comes from HBM), so one of 40 calls has to be reported."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300 import _abi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [17, 128])
def test_waits_for_a_part_of_a_sum_are_reported(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, 7168, generator=g, device="cuda").bfloat16()
    w = torch.randn(131072, 7168, generator=g, device="cuda", dtype=torch.bfloat16)
    want = dsa.dsa_linear(x, w, dtype=torch.float32)
    assert dsa.dsa_check_device_error()[0] == _abi.DSA_OK
    for _ in range(40):
        try:
            dsa.dsa_set_wait_limit(1)
            dsa.dsa_linear(x, w, dtype=torch.float32)
            status, site = dsa.dsa_check_device_error()
        finally:
            dsa.dsa_set_wait_limit(0)
        if status != _abi.DSA_OK:
            break
    assert status == _abi.DSA_ERR_TIMEOUT and 61 <= site <= 66
    assert torch.equal(dsa.dsa_linear(x, w, dtype=torch.float32), want)
    assert dsa.dsa_check_device_error()[0] == _abi.DSA_OK
