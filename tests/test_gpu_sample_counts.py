"""Sampling where the kept tokens are hard to count: outputs are filled before the call, so that one which is not written
shows, and token and count have to equal the 64-bit form's (the kernel's sums are off by less than 2^-36 of the whole)."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300 import _abi
from tests import next_token_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def on(values, dt=F32):
    return None if values is None else torch.as_tensor(values, dtype=dt, device="cuda")


def sample(x, u, T=None, k=None, p=None, m=None):
    """The C call, into outputs that hold something else before."""
    n, V = x.shape
    u, T, k, p, m = on(u), on(T), on(k, torch.int32), on(p), on(m)
    token, kept = torch.full((n,), -77, dtype=torch.int32, device="cuda"), torch.full((n,), -78, dtype=torch.int32, device="cuda")
    logprob = torch.full((n,), 79.0, device="cuda")
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rc = _abi.load().dsa_sample(x.data_ptr(), x.stride(0), _abi.DSA_F32 if x.dtype == F32 else _abi.DSA_BF16, n, V, at(u), at(T), at(k),
                                at(p), at(m), at(token), at(logprob), at(kept), torch.cuda.current_stream().cuda_stream)
    assert rc == _abi.DSA_OK
    return token.tolist(), logprob.tolist(), kept.tolist()


def check(x, u, T=None, k=None, p=None, m=None, rows=None):
    got = sample(x, u, T, k, p, m)
    f = lambda v, i, d: d if v is None else float(torch.tensor(float(v[i]), dtype=F32))  # noqa: E731
    for i in range(x.shape[0]) if rows is None else rows:
        want = R.sample_row(x[i], f(u, i, 0.0), f(T, i, 1.0), 0 if k is None else int(k[i]), f(p, i, 1.0), f(m, i, 0.0))
        assert (got[0][i], got[2][i]) == (want[0], want[2]), f"row {i}: {[g[i] for g in got]}, expected {want}"
        assert abs(got[1][i] - want[1]) <= 8 * 2.0 ** -24 * (abs(want[1]) + 2.0 ** -20), f"row {i}: {[g[i] for g in got]}, expected {want}"
    return got


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,V", [(12, 131072), (10, 6007), (300, 20011), (200, 131072), (700, 6007)])
def test_nucleus_that_reaches_behind_min_p(n, V, dt):
    """Without top-k: 300 to 1900 tokens pass min-p, and the run that reaches top_p of all tokens ends among them or behind
    them.  Rows of one CTA and of several, kept in shared memory or not."""
    g = torch.Generator(device="cuda").manual_seed(n + V)
    x = torch.randn(n, V, generator=g, device="cuda").to(dt)
    T = [0.9, 0.8, 1.0, 1.3]
    rows = list(range(n)) if n <= 12 else list(range(0, n, max(1, n // 40)))
    T, p, m, behind = [T[i % 4] for i in range(n)], [], [], 0
    for i in range(n):
        t = float(torch.tensor(T[i], dtype=F32))
        l = x[i].double().sort(descending=True)[0]  # noqa: E741
        w = ((l - l[0]) / t).exp()
        many = 300 + i * 331 % 1600
        m.append(float((w[many - 1] * w[many]).sqrt()) if dt == F32 else float(w[many]) * 0.999)
        share = float(w[:many].sum() / w.sum())
        p.append([0.999, 0.95, 0.5 + 0.5 * share, 0.5 * share, share * 0.999][i % 5])
        behind += p[-1] > share
    assert behind >= n // 2
    check(x, torch.rand(n, generator=g, device="cuda").tolist(), T, None, p, m, rows)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,V", [(10, 64), (10, 5000), (10, 131072), (300, 131072), (900, 3001)])
def test_masks_of_finite_numbers(n, V, dt):
    """The type's lowest number, or another far below the rest, is a token like any other: it weighs nothing and counts.
    top_k below, at and above the number of tokens without a mask."""
    g = torch.Generator(device="cuda").manual_seed(n * V)
    low = [torch.finfo(dt).min, -1e30, -1e9, -1e38]
    x = torch.empty(n, V, dtype=dt, device="cuda")
    for i in range(n):
        x[i] = low[i % 4]
        at = torch.randperm(V, generator=g, device="cuda")[:40]
        x[i, at] = (2 * torch.randn(40, generator=g, device="cuda")).to(dt)
    u = torch.rand(n, generator=g, device="cuda").tolist()
    T = [[1.0, 0.5, 1.0, 2.0, 1e-4][i % 5] for i in range(n)]
    pick = lambda *v: [v[i // 4 % len(v)] for i in range(n)]  # noqa: E731
    rows = list(range(n)) if n <= 12 else list(range(0, n, 31))
    for k in ([50] * n, [1000] * n, pick(3, 40, 41, V - 1)):
        got = check(x, u, T, k, None, None, rows)
        assert all(got[2][i] == min(k[i], V) for i in range(n))
    check(x, u, T, [50] * n, pick(0.9, 0.999, 1.0), None, rows)
    check(x, u, T, [50] * n, None, pick(0.0, 0.01, 1e-20), rows)
    check(x, u, T, None, pick(0.9, 0.999), None, rows)
    check(x, u, T, None, None, pick(0.01, 1e-20, 1e-44), rows)
    check(x, u, T, None, pick(0.9, 0.999), pick(0.01, 1e-20, 1e-44), rows)
    assert check(x, u, T, None, None, None, rows)[2] == [V] * n


@pytest.mark.parametrize("V", [200, 1500, 20011, 131072])
def test_min_p_below_every_weight_that_counts(V):
    """min_p below 2^-46, where weights are too small to be drawn: their tokens are counted all the same, however many
    candidates there are."""
    g = torch.Generator(device="cuda").manual_seed(V)
    n = 16
    x = -90 * torch.rand(n, V, generator=g, device="cuda")
    x[::2] -= 300  # most of the row far below its highest token
    x[:, 7] = 1.0
    x[::2, 50:150] = -60 * torch.rand(8, 100, generator=g, device="cuda")
    u = torch.rand(n, generator=g, device="cuda").tolist()
    m = [[1e-13, 2e-14, 1e-14, 1e-16, 1e-20, 1e-25, 1e-30, 1e-37][i // 2] for i in range(n)]
    T = [[1.0, 0.75][i % 2] for i in range(n)]
    check(x, u, T, None, None, m)
    for k in (20, 120, 700, 5000):
        check(x, u, T, [k] * n, None, m)
    check(x, u, T, None, [0.9999] * n, m)
