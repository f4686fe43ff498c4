"""Refusals of the linear layer, the block norm and the sampling, without a GPU: an invalid call returns its status
before anything is launched, and the binding raises before the call."""
import ctypes

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300 import _abi

BAD, NOT, WORKSPACE = _abi.DSA_ERR_INVALID_ARG, _abi.DSA_ERR_UNSUPPORTED, _abi.DSA_ERR_WORKSPACE
A, B, C, D = (1 << 20), (2 << 20), (3 << 20), (4 << 20)  # addresses that are never read


def linear(**k):
    d = dict(x=A, ld_x=64, W=B, ld_w=64, dtype=1, M=4, N=32, K=64, bias=None, act=0, res=None, ld_r=32, y=C, ld_y=32,
             y_dtype=1, ws=None, ws_bytes=0)
    d.update(k)
    return _abi.load().dsa_linear(d["x"], d["ld_x"], d["W"], d["ld_w"], d["dtype"], d["M"], d["N"], d["K"], d["bias"],
                                  d["act"], d["res"], d["ld_r"], d["y"], d["ld_y"], d["y_dtype"], d["ws"], d["ws_bytes"], None)


@pytest.mark.parametrize("k,status", [
    (dict(x=None), BAD), (dict(W=None), BAD), (dict(y=None), BAD), (dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD),
    (dict(x=A + 1), BAD), (dict(W=B + 1), BAD), (dict(y=C + 1), BAD), (dict(bias=D + 2), BAD), (dict(res=D + 1), BAD),
    (dict(dtype=2), NOT), (dict(y_dtype=2), NOT), (dict(act=5), NOT), (dict(act=-1), NOT), (dict(ld_y=31), BAD),
    (dict(y=A), BAD), (dict(y=B), BAD), (dict(res=C, ld_r=64), BAD), (dict(ld_x=-64), BAD), (dict(ld_w=-1), BAD),
    (dict(M=2 ** 31 - 1), NOT), (dict(N=2 ** 31 - 1), NOT), (dict(K=2 ** 31 - 1), NOT), (dict(dtype=0, K=400000000), NOT),
    (dict(M=40, ld_x=65), WORKSPACE), (dict(M=70, W=B + 2), WORKSPACE), (dict(M=70, dtype=0, x=A + 4), WORKSPACE),
    (dict(M=70, dtype=0, x=A + 4, ws=D, ws_bytes=70 * 384 + 32 * 384 - 1), WORKSPACE), (dict(M=70, dtype=0, x=A + 4, ws=D + 16, ws_bytes=1 << 30), WORKSPACE),
    (dict(M=0), 0), (dict(M=0, x=None, W=None, y=None), 0),
])
def test_linear_refusals(k, status):
    assert linear(**k) == status
    assert dsa.last_launch_count() == 0


def test_linear_workspace():
    """Nothing where the tensor cores take the rows as they are; a copy of x, of W (a part at a time) and both."""
    size = lambda x, ld_x, W, ld_w, dt, M, N, K: _abi.load().dsa_linear_workspace_size(x, ld_x, W, ld_w, dt, M, N, K)  # noqa: E731
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert size(A, 64, B, 64, 1, 40, 32, 64) == 0
    assert size(A, 64, B, 64, 1, 0, 32, 64) == 0
    assert size(A + 2, 64, B, 64, 1, 40, 32, 64) == 40 * 128
    assert size(A, 64, B, 65, 1, 70, 32, 64) == 32 * 128
    assert size(A, 33, B, 33, 1, 70, 32, 33) == up(70 * 80) + up(32 * 80)
    assert size(A + 4, 64, B, 64, 0, 70, 32, 64) == up(70 * 384) + 32 * 384
    # fp32 rows on 16 bytes: little work, and few tokens of a large W
    assert size(A, 64, B, 64, 0, 70, 32, 64) == 0 and size(A, 9000, B, 9000, 0, 64, 9000, 9000) == 0
    assert size(A, 9000, B, 9000, 0, 65, 9000, 9000) > 0 and size(A, 9000, B, 9000, 0, 64, 900, 9000) > 0
    # few tokens, or little work, read W as it is
    assert size(A, 9999, B, 9999, 1, 4, 9999, 9999) == 0 and size(A, 9999, B, 9999, 1, 5, 9999, 9999) > 0
    assert size(A, 9999, B, 9999, 0, 4, 9999, 9999) == 0 and size(A, 9999, B, 9999, 0, 5, 9999, 9999) > 0
    assert size(A, 64, B, 65, 1, 64, 32, 64) == 0 and size(A, 64, B, 64, 0, 64, 32, 64) == 0
    assert size(A, 64, B, 64, 0, 70, 1 << 20, 64) < (1 << 20) * 384  # not all of W at once
    assert size(A, 64, B, 64, 2, 40, 32, 64) == 0 and size(A, 64, B, 64, 1, 40, 0, 64) == 0


def test_block_norm_bytes():
    """The packed form is the structure's."""
    v = list(range(1, 25))
    flat = _abi.block_norm_bytes.pack(*v)
    st = _abi.dsa_block_norm_args(*v[:11], _abi.dsa_norm(*v[11:14]), _abi.dsa_norm(*v[14:17]), *v[17:])
    got = _abi.dsa_block_norm_args.from_buffer_copy(flat)
    for name, _ in st._fields_:
        a, b = getattr(got, name), getattr(st, name)
        if isinstance(a, ctypes.Structure):
            assert [getattr(a, n) for n, _ in a._fields_] == [getattr(b, n) for n, _ in a._fields_]
        else:
            assert a == b and a
    assert len(flat) == ctypes.sizeof(st)


def norm(**k):
    d = dict(rows=4, D=64, h_dtype=1, x_dtype=1, h=A, ld_h=64, u=B, ld_u=64, gate=None, ld_gate=64, gate_act=0,
             post=(0, None, None), pre=(1, None, None), skip=1.0, scale=1.0, eps=1e-6, h_out=C, ld_ho=64, y=D, ld_y=64)
    d.update(k)
    d["post"], d["pre"] = _abi.dsa_norm(*d["post"]), _abi.dsa_norm(*d["pre"])
    return _abi.load().dsa_block_norm(ctypes.byref(_abi.dsa_block_norm_args(**d)), None)


@pytest.mark.parametrize("k,status", [
    (dict(rows=-1), BAD), (dict(D=0), BAD), (dict(D=16385), NOT), (dict(h=None), BAD), (dict(h_out=None, y=None), BAD),
    (dict(u=None, gate=B), BAD), (dict(u=None, post=(1, None, None)), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(h_dtype=2), NOT), (dict(x_dtype=3), NOT), (dict(pre=(3, None, None)), NOT), (dict(post=(-1, None, None)), NOT),
    (dict(gate_act=1), NOT), (dict(gate_act=4), NOT), (dict(h=A + 1), BAD), (dict(u=B + 1), BAD), (dict(y=D + 1), BAD),
    (dict(pre=(1, D + 2, None)), BAD), (dict(post=(2, None, D + 1)), BAD), (dict(ld_ho=63), BAD), (dict(ld_y=0), BAD),
    (dict(h_out=A, ld_ho=128), BAD), (dict(y=B, ld_y=128), BAD), (dict(y=A), BAD), (dict(y=C), BAD), (dict(h_out=B), BAD),
    (dict(gate=D), BAD), (dict(gate=C), BAD), (dict(rows=0), 0), (dict(rows=0, h=None), 0),
])
def test_block_norm_refusals(k, status):
    assert norm(**k) == status
    assert dsa.last_launch_count() == 0
    assert _abi.load().dsa_block_norm(None, None) == BAD


def sample(**k):
    d = dict(logits=A, ld=100, dtype=0, R=3, V=100, u=B, T=None, k=None, p=None, m=None, token=C, logprob=None, kept=None)
    d.update(k)
    return _abi.load().dsa_sample(*d.values(), None)


@pytest.mark.parametrize("k,status", [
    (dict(logits=None), BAD), (dict(u=None), BAD), (dict(token=None), BAD), (dict(R=-1), BAD), (dict(V=0), BAD),
    (dict(V=262145), NOT), (dict(dtype=2), NOT), (dict(R=2 ** 31 - 1), NOT), (dict(ld=-1), BAD), (dict(logits=A + 2), BAD),
    (dict(u=B + 2), BAD), (dict(T=B + 1), BAD), (dict(k=B + 3), BAD), (dict(p=B + 2), BAD), (dict(m=B + 1), BAD),
    (dict(token=C + 2), BAD), (dict(logprob=C + 1), BAD), (dict(kept=C + 2), BAD), (dict(dtype=1, logits=A + 1), BAD),
    (dict(R=0), 0), (dict(R=0, logits=None, u=None, token=None), 0),
])
def test_sample_refusals(k, status):
    assert sample(**k) == status
    assert dsa.last_launch_count() == 0


def test_binding_refuses_host_tensors_and_wrong_names():
    t = torch.zeros(4, 8)
    for call in (lambda: dsa.dsa_linear(t, t), lambda: dsa.dsa_block_norm(t, dsa.Norm()), lambda: dsa.dsa_sample(t, t[:, 0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="kind must be"):
        dsa.Norm("batch")
