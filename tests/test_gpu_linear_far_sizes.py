"""Linear layers whose sizes end just below what the interface admits, at 2^31 - 1026: one column of W each way, so that every
value of y is one product, rounded once."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 - 1026


def same(y, a, b):
    """y = a b^T for columns a and b, a part at a time; rows of one value would be laid out on their own."""
    step = 1 << 26
    for i in range(0, y.shape[0], step):
        for j in range(0, y.shape[1], step):
            if not torch.equal(y[i:i + step, j:j + step], a[i:i + step] * b[j:j + step].T):
                return False
    return True


def test_features_up_to_2_31():
    """W off 16 bytes, laid out in 512 parts whose last ends 4 million features from where 32 bits do."""
    x = torch.randn(5, 1, device="cuda").bfloat16()
    w = torch.randint(-512, 513, (FAR, 1), dtype=torch.int16, device="cuda").bfloat16()
    y = dsa.dsa_linear(x, w)
    assert dsa.last_kernels() == {"linear", "linear_layout"}
    assert same(y, x, w)


def test_tokens_up_to_2_31():
    """More tokens than their number and that of their tiles add up to in 32 bits."""
    x = torch.randint(-512, 513, (FAR, 1), dtype=torch.int16, device="cuda").bfloat16()
    w = torch.randn(5, 1, device="cuda").bfloat16()
    y = dsa.dsa_linear(x, w)
    assert dsa.last_kernels() == {"linear", "linear_layout"}
    assert same(y, x, w)
