"""Arguments of another kind than a tensor are refused in words, whichever argument it is.  No GPU: the tensors beside them only
say that they are on one."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa


class OnGpu(torch.Tensor):
    """A host tensor that names a device; it never gets as far as a launch."""

    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


X, W, H, L = on_gpu(4, 8), on_gpu(6, 8), on_gpu(4, 8), on_gpu(4, 9, dtype=torch.float32)
U = on_gpu(4, dtype=torch.float32)
OTHERS = [3, [1.0, 2.0], "x", torch.bfloat16]


@pytest.mark.parametrize("other", OTHERS + [None])
@pytest.mark.parametrize("call,name", [
    (lambda o: dsa.dsa_linear(o, W), "x"), (lambda o: dsa.dsa_linear(X, o), "weight"),
    (lambda o: dsa.dsa_linear_workspace_size(o, W), "x"), (lambda o: dsa.dsa_linear_workspace_size(X, o), "weight"),
    (lambda o: dsa.dsa_block_norm(o), "h"), (lambda o: dsa.dsa_sample(o, U), "logits"),
])
def test_what_a_call_cannot_do_without(call, name, other):
    with pytest.raises(TypeError, match=f"{name} must be a tensor"):
        call(other)


@pytest.mark.parametrize("other", OTHERS)
@pytest.mark.parametrize("call,name", [
    (lambda o: dsa.dsa_linear(X, W, bias=o), "bias"), (lambda o: dsa.dsa_linear(X, W, residual=o), "residual"),
    (lambda o: dsa.dsa_linear(X, W, y=o), "y"), (lambda o: dsa.dsa_linear(X, W, workspace=o), "workspace"),
    (lambda o: dsa.dsa_block_norm(H, u=o), "u"), (lambda o: dsa.dsa_block_norm(H, u=H, gate=o), "gate"),
    (lambda o: dsa.dsa_block_norm(H, y=o), "y"), (lambda o: dsa.dsa_block_norm(H, h_out=o), "h_out"),
    (lambda o: dsa.dsa_block_norm(H, dsa.Norm("rms", o)), "pre.gain"),
    (lambda o: dsa.dsa_block_norm(H, u=H, post=dsa.Norm("layer", None, o)), "post.bias"),
    (lambda o: dsa.dsa_sample(L, o), "uniform"), (lambda o: dsa.dsa_sample(L, U, temperature=o), "temperature"),
    (lambda o: dsa.dsa_sample(L, U, top_k=o), "top_k"), (lambda o: dsa.dsa_sample(L, U, top_p=o), "top_p"),
    (lambda o: dsa.dsa_sample(L, U, min_p=o), "min_p"), (lambda o: dsa.dsa_sample(L, U, token=o), "token"),
])
def test_what_may_be_left_out(call, name, other):
    with pytest.raises(TypeError, match=f"{name} must be a tensor"):
        call(other)


def test_norms_and_matrices_of_another_kind():
    with pytest.raises(TypeError, match="pre must be a Norm"):
        dsa.dsa_block_norm(H, "rms")
    with pytest.raises(TypeError, match="post must be a Norm"):
        dsa.dsa_block_norm(H, u=H, post=torch.ones(8))
    for w in (on_gpu(), on_gpu(8), on_gpu(1, 6, 8)):
        with pytest.raises(ValueError, match="weight must be 2-D"):
            dsa.dsa_linear(X, w)
