"""The linear kernel's waits for a sum, in the forms that take it over in parts or whose warps make the slabs themselves: a limit of one
cycle is polled for, and the sum is not there when its epilogue looks for it, so every such call has to be reported."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300 import _abi

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("M,N,K,dt,out", [(17, 20000, 7168, BF16, F32), (128, 20000, 7168, BF16, F32), (16, 1024, 16384, BF16, F32),
                                          (300, 8000, 8192, BF16, F32), (70, 1024, 8192, F32, F32), (900, 2048, 4096, F32, F32),
                                          (64, 40000, 4096, F32, BF16),
                                          (500, 260, 1536, F32, F32), (500, 260, 1536, F32, BF16), (33, 70, 200, BF16, F32)])
def test_waits_for_a_sum_are_reported(M, N, K, dt, out):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(dt)
    w = torch.randn(N, K, generator=g, device="cuda").to(dt)
    want = dsa.dsa_linear(x, w, dtype=out)
    assert "linear" in dsa.last_kernels() and dsa.dsa_check_device_error()[0] == _abi.DSA_OK
    for _ in range(5):
        try:
            dsa.dsa_set_wait_limit(1)
            dsa.dsa_linear(x, w, dtype=out)
            status, site = dsa.dsa_check_device_error()
        finally:
            dsa.dsa_set_wait_limit(0)
        assert status == _abi.DSA_ERR_TIMEOUT and 61 <= site <= 66
    assert torch.equal(dsa.dsa_linear(x, w, dtype=out), want)
    assert dsa.dsa_check_device_error()[0] == _abi.DSA_OK
