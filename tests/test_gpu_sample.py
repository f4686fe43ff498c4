"""Sampling against the 64-bit form, row by row.

Tokens and counts have to be equal: the kernel's sums are off by less than 2^-36 of the whole, so a random number would
have to fall that near to a border.  The log-probability is rounded a few times in fp32, from two parts of one sign."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import next_token_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def on(values, dt=F32):
    return None if values is None else torch.tensor(values, dtype=dt, device="cuda")


def check(logits, u, T=None, k=None, p=None, m=None, stream=None):
    n = logits.shape[0]
    token, logprob, kept = dsa.dsa_sample(logits.cuda(), on(u), on(T), on(k, torch.int32), on(p), on(m), want_kept=True,
                                          stream=stream)
    torch.cuda.synchronize()
    assert dsa.last_kernels() == {"sample"} and dsa.last_launch_count() == 1
    assert token.dtype == torch.int32 and logprob.dtype == F32 and kept.dtype == torch.int32
    at = lambda v, i, d: d if v is None else float(torch.tensor(v[i], dtype=F32))  # noqa: E731
    for i in range(n):
        want = R.sample_row(logits[i], at(u, i, 0.0), at(T, i, 1.0), 0 if k is None else k[i], at(p, i, 1.0), at(m, i, 0.0))
        got = int(token[i]), float(logprob[i]), int(kept[i])
        assert got[0] == want[0] and got[2] == want[2], f"row {i}: {got}, expected {want}"
        if want[1] > -INF:
            assert abs(got[1] - want[1]) <= 8 * 2.0 ** -24 * (abs(want[1]) + 2.0 ** -20), f"row {i}: {got}, expected {want}"
        else:
            assert got[1] == -INF
    return token


def draw(R_, V, g, dt=F32, std=2.0, peaks=10):
    x = std * torch.randn(R_, V, generator=g)
    at = torch.randint(0, V, (R_, peaks), generator=g)
    x.scatter_add_(1, at, 3 + 3 * torch.rand(R_, peaks, generator=g))
    return x.to(dt)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 32, 33, 511, 512, 513, 4095, 4096, 4097, 10007, 32768, 50001, 131072, 200003, 262144])
def test_sizes(V, dt):
    g = torch.Generator().manual_seed(V)
    n = 9
    u = torch.rand(n, generator=g).tolist()
    check(draw(n, V, g, dt), u)
    check(draw(n, V, g, dt), u, [0.7, 1.0, 1.3, 0.0, 0.3, 2.0, 1.0, 0.9, 0.05], [0, 1, 5, 7, 50, V, V + 5, V // 2, 1000],
          [0.9, 1.0, 0.5, 0.2, 0.95, 0.999, 0.0, 0.3, 0.99], [0.0, 0.1, 0.0, 0.0, 0.01, 0.001, 0.0, 0.2, 0.0])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("which", ["k", "p", "m", "kp", "pm", "km", "kpm"])
def test_rules(which, dt):
    g = torch.Generator().manual_seed(len(which) + 17 * ord(which[0]))
    n, V = 40, 7001
    pick = lambda vals: [vals[int(i)] for i in torch.randint(0, len(vals), (n,), generator=g)]  # noqa: E731
    check(draw(n, V, g, dt, std=1.5), torch.rand(n, generator=g).tolist(), pick([0.5, 0.8, 1.0, 1.5, 3.0]),
          pick([0, 1, 2, 10, 100, 3000, 6999, 7001]) if "k" in which else None,
          pick([0.05, 0.3, 0.9, 0.99, 0.9999, 1.0]) if "p" in which else None,
          pick([0.0, 1e-4, 0.01, 0.3, 1.0, 2.0]) if "m" in which else None)


@pytest.mark.parametrize("V", [64, 1024, 5000, 65536, 262144])
def test_equal_logits(V):
    """All weights are one, so every border is a whole number: the k-th, the share of p, and the draw itself."""
    n = 8
    x = torch.full((n, V), 3.25)
    u = [0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.5, 0.125, 0.0]
    k = [0, 0, 0, 0, 0, 48, 32, 0]
    p = [1.0, 1.0, 1.0, 0.5, 0.25, 1.0, 0.5, 0.75]
    token = check(x, u, None, k, p).tolist()
    assert token[:4] == [0, V // 4, V // 2, V // 2 * 3 // 4] and token[5:7] == [24, 2]
    token, logprob, kept = dsa.dsa_sample(x.cuda(), on(u), top_k=on(k, torch.int32), top_p=on(p), want_kept=True)
    assert kept.tolist() == [V, V, V, V // 2, V // 4, 48, 16, V * 3 // 4]


def test_ties_go_to_the_lowest_index():
    """Few distinct values: the k-th token and the end of the nucleus lie among equals."""
    g = torch.Generator().manual_seed(3)
    n, V = 30, 20011
    x = torch.randint(-3, 3, (n, V), generator=g).float()
    x[5] = -0.0
    x[6, ::2], x[6, 1::2] = 0.0, -0.0
    check(x, torch.rand(n, generator=g).tolist(), [0.7 + 0.05 * i for i in range(n)], [i * 61 for i in range(n)],
          [0.31 + 0.02 * i for i in range(n)])


@pytest.mark.parametrize("V", [5, 4097, 131072])
def test_masks_nan_and_infinities(V):
    g = torch.Generator().manual_seed(V)
    n = 10
    x = draw(n, V, g, peaks=2)
    x[0] = -INF
    x[1] = float("nan")
    x[2] = -INF
    x[2, V - 1] = -3e38
    x[3, : V // 2] = float("nan")
    x[4, torch.randperm(V, generator=g)[: V - 2]] = -INF
    x[5, 1], x[5, V - 2] = INF, INF
    x[6, :3] = torch.tensor([INF, float("nan"), -INF])
    x[7] = torch.finfo(F32).min
    x[8] = torch.finfo(F32).min
    x[8, V // 3] = 0.0
    x[9] = -INF
    x[9, ::2] = torch.finfo(F32).min
    u = [0.3, 0.3, 0.9, 0.7, 0.6, 0.6, 0.99, 0.51, 0.999, 0.5]
    token = check(x, u)
    assert token[:3].tolist() == [-1, -1, V - 1]
    check(x, u, [0.0] * n)
    check(x, u, None, [2] * n, [0.6] * n, [0.1] * n)
    if V > 5:
        check(x.bfloat16(), u, [0.8] * n, [3] * n)


def test_settings_at_their_ends():
    """Settings without a meaning of their own: what the documentation says of them."""
    g = torch.Generator().manual_seed(11)
    n, V = 16, 3001
    x = draw(n, V, g)
    nan = float("nan")
    u = [0.0, 1.0, 2.0, -1.0, nan, 1 - 2.0 ** -24, 2.0 ** -30, 1e-40] + [0.4] * 8
    T = [1.0] * 8 + [nan, -1.0, 1e-6, 1e-5, 1e30, INF, 1e-4, 100.0]
    check(x, u, T)
    one = [1.0] * n
    check(x, u, one, [0, -1, -5, 1, 2, 2 ** 31 - 1, V, V - 1] * 2)
    check(x, u, one, None, [0.0, -1.0, nan, 1.0, 1.5, 1e-30, 1 - 2.0 ** -24, 2.0 ** -20] * 2)
    check(x, u, one, None, None, [0.0, -1.0, nan, 1.0, 1.5, 1e-30, 1 - 2.0 ** -24, 2.0 ** -20] * 2)


def test_every_token_is_drawn_where_it_should():
    """Random numbers on both sides of every border of a short row."""
    x = torch.tensor([1.0, -2.0, 0.5, -INF, 3.0, 0.25, 3.0, -1.0])
    w = torch.exp(x.double() - 3)
    ends = torch.cumsum(w, 0) / w.sum()
    u, want = [], []
    for i in range(8):
        if w[i] > 0:
            lo, hi = (float(ends[i - 1]) if i else 0.0), float(ends[i])
            u += [lo + 1e-6, hi - 1e-6]
            want += [i, i]
    token, logprob, _ = dsa.dsa_sample(x.expand(len(u), 8).cuda(), on(u))
    assert token.tolist() == want
    for t, p in zip(want, logprob.tolist()):
        assert abs(p - math.log(float(w[t] / w.sum()))) < 1e-6


def test_strides_rows_behind_and_outputs():
    """Rows of a wider tensor that start anywhere, one row for all, a token buffer of the caller's, nothing to do."""
    g = torch.Generator().manual_seed(2)
    for dt in (F32, BF16):
        for off in (0, 1, 3):
            wide = draw(12, 6013 + 16, g, dt).cuda()
            view = wide[:, off:off + 6013]
            check(view, torch.rand(12, generator=g).tolist(), None, [17] * 12, [0.9] * 12)
    one = draw(1, 9001, g).expand(64, 9001)
    check(one.cuda(), torch.rand(64, generator=g).tolist())
    out = torch.full((10,), -7, dtype=torch.int32, device="cuda")
    x = draw(6, 100, g).cuda()
    token, logprob, kept = dsa.dsa_sample(x, on([0.5] * 6), token=out[2:8], want_logprob=False)
    assert logprob is None and kept is None and token.data_ptr() == out[2:8].data_ptr()
    assert out[:2].tolist() == [-7, -7] and out[8:].tolist() == [-7, -7] and int(out[2:8].min()) >= 0
    empty = dsa.dsa_sample(x[:0], on([]), want_kept=True)
    assert all(t.shape == (0,) for t in empty) and dsa.last_launch_count() == 0


def test_many_rows_and_far_ones():
    """More rows than fit the GPU at once, and rows past 2^31 values; the same call gives the same answer."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, V = 2000, 5003
    x = torch.randn(n, V, generator=g, device="cuda") * 3
    u, p = torch.rand(n, generator=g, device="cuda"), torch.full((n,), 0.9, device="cuda")
    token, logprob, kept = dsa.dsa_sample(x, u, top_p=p, want_kept=True)
    again = dsa.dsa_sample(x, u, top_p=p, want_kept=True)
    assert torch.equal(token, again[0]) and torch.equal(logprob, again[1]) and torch.equal(kept, again[2])
    for i in range(0, n, 97):
        assert R.sample_row(x[i], float(u[i]), p=float(p[i]))[::2] == (int(token[i]), int(kept[i]))
    far = torch.zeros(3, 1200000000, dtype=BF16, device="cuda")
    far[:, 5:5 + V] = x[:3]
    got = dsa.dsa_sample(far[:, 5:5 + V], u[:3])
    assert torch.equal(got[0], dsa.dsa_sample(x[:3].bfloat16(), u[:3])[0])


def test_streams_and_graphs():
    g = torch.Generator().manual_seed(8)
    x = draw(20, 30011, g)
    u, p = torch.rand(20, generator=g).tolist(), [0.9] * 20
    side = torch.cuda.Stream()
    want = check(x, u, None, None, p)
    assert torch.equal(check(x, u, None, None, p, stream=side), want)
    xd, ud, pd = x.cuda(), on(u), on(p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token, _, _ = dsa.dsa_sample(xd, ud, top_p=pd)
    xd.copy_(xd.flip(0))
    ud.copy_(ud.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(token, want.flip(0))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,V", [(256, 131072), (90, 262141), (700, 20011)])
def test_large_batches(n, V, dt):
    """Many long rows, of every kind side by side: the same rules whichever way a row's CTAs share it."""
    g = torch.Generator(device="cuda").manual_seed(n + V)
    x = 2 * torch.randn(n, V, generator=g, device="cuda")
    x.scatter_add_(1, torch.randint(0, V, (n, 20), generator=g, device="cuda"), 4 + 3 * torch.rand(n, 20, generator=g, device="cuda"))
    x[3], x[4, V - 5:], x[5] = -INF, INF, 1.5
    x[6, : V // 3] = float("nan")
    x[7] = torch.randint(-2, 3, (V,), generator=g, device="cuda").float()
    x[8].masked_fill_(torch.rand(V, generator=g, device="cuda") < 0.99, -INF)
    x = x.to(dt)
    pick = lambda vals: [vals[i % len(vals)] for i in range(n)]  # noqa: E731
    u = torch.rand(n, generator=g, device="cuda").tolist()
    T, k = pick([0.0, 0.5, 0.8, 1.0, 1.3]), pick([0, 1, 20, 0, 170, 200, 0, 1000, 5000, V - 1, 0])
    p, m = pick([1.0, 0.9, 0.5, 0.95, 0.999, 1.0, 0.8]), pick([0.0, 0.0, 0.05])
    token, logprob, kept = dsa.dsa_sample(x, on(u), on(T), on(k, torch.int32), on(p), on(m), want_kept=True)
    f = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
    for i in list(range(60)) + list(range(60, n, 7)):
        want = R.sample_row(x[i], f(u[i]), f(T[i]), k[i], f(p[i]), f(m[i]))
        assert (int(token[i]), int(kept[i])) == want[::2], f"row {i}"
        if want[1] > -INF:
            assert abs(float(logprob[i]) - want[1]) <= 8 * 2.0 ** -24 * (abs(want[1]) + 2.0 ** -20)


def test_large_batches_of_equal_logits():
    """Long rows whose every token has the same weight: nothing that counts them may run over."""
    n, V = 320, 262144
    x = torch.full((n, V), -2.5, dtype=BF16, device="cuda")
    p = [0.25, 0.5, 0.75, 0.125] * (n // 4)
    token, logprob, kept = dsa.dsa_sample(x, on([0.5] * n), top_p=on(p), want_kept=True)
    assert kept.tolist() == [int(V * v) for v in p] and token.tolist() == [int(V * v) // 2 for v in p]
    assert torch.all((logprob.cpu() + torch.tensor([math.log(V * v) for v in p])).abs() < 1e-5)
