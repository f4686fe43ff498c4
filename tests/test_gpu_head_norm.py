"""Per-head norm and rotation against the 64-bit form.

A result is rounded once to its type; before that its fp32 sums of D squares (and of D
values) are off by at most about D roundings of 2^-24, relative to the largest value that
enters, and the norm's division, gain, bias and rotation add a few more: 4 (D + 16) 2^-24
of the row's largest possible result."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def tables(n_pos, d_r):
    ang = torch.arange(n_pos).double()[:, None] * 10000.0 ** (-torch.arange(d_r // 2).double() / max(d_r // 2, 1))
    return ang.cos().float(), ang.sin().float()


def check(got, x, norm, gain, bias, eps, cos, sin, pos, rope, first, split, y_dt):
    D, d_r = x.shape[2], 2 * cos.shape[1]
    g = None if gain is None else gain.double()
    b = None if bias is None else bias.double()
    keep, turn = R.norm_rope(x.double(), norm, g, b, eps, cos.double(), sin.double(), pos, rope, first)
    want = (keep, turn) if split else torch.cat([turn, keep] if first else [keep, turn], -1)
    xd = x.double()
    spread = xd.abs().amax(-1, keepdim=True)
    if norm != "none":
        mean = xd.mean(-1, keepdim=True) if norm == "layer" else 0.0
        spread = 2 * spread / ((xd - mean).pow(2).mean(-1, keepdim=True) + eps).sqrt()
        spread = spread * (1.0 if g is None else g.abs().max()) + (0.0 if b is None else b.abs().max())
    slack = 4 * (D + 16) * 2.0 ** -24 * 2 * spread
    for a, w in zip(got if split else (got,), want if split else (want,)):
        assert a.dtype == y_dt and a.shape == w.shape
        assert torch.all((a.cpu().double() - w).abs() <= R.U[y_dt] * w.abs() + slack)


CASES = [
    # D, d_r, Hq, Hk, norm q, norm k, rope, first, split
    (192, 64, 8, 1, "rms", "rms", "pairs", False, True),
    (192, 64, 3, 2, "none", "layer", "halves", False, True),
    (128, 64, 64, 1, "layer", "layer", "halves", True, False),
    (128, 128, 5, 0, "rms", None, "pairs", False, True),
    (64, 32, 1, 1, "layer", "rms", "pairs", True, True),
    (256, 0, 4, 1, "rms", "none", "pairs", False, False),
    (512, 64, 2, 3, "layer", "rms", "halves", False, False),
    (40, 16, 7, 1, "rms", "rms", "halves", True, True),
    # widths that go value by value
    (33, 6, 3, 1, "rms", "layer", "pairs", False, True),
    (511, 22, 2, 1, "layer", "none", "halves", True, False),
    (1, 0, 2, 2, "rms", "rms", "pairs", False, False),
    (2, 2, 3, 1, "none", "rms", "halves", False, True),
]


@pytest.mark.parametrize("x_dt,y_dt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("given", [False, True])
def test_against_the_formula(case, x_dt, y_dt, given):
    D, d_r, Hq, Hk, nq, nk, rope, first, split = case
    split = split and d_r > 0
    g = torch.Generator().manual_seed(D + d_r)
    T, P = [3, 0, 14], [0, 5, 31]
    N = sum(T)
    seqs = dsa.Seqs.from_lengths(T, [t + p for t, p in zip(T, P)], P)
    cos, sin = tables(45, d_r)
    pos = [p + t for n, p in zip(T, P) for t in range(n)]
    if given:  # depths of a tree, the same position twice, padding rows
        pos = [int(v) for v in torch.randint(0, 45, (N,), generator=g)]
        pos[2], pos[3], pos[5] = -1, 45, pos[4]

    def make(n, norm):
        x = torch.randn(N, n, D, generator=g).to(x_dt)
        gain = 1 + 0.2 * torch.randn(D, generator=g) if norm != "none" and n != 3 else None
        bias = torch.randn(D, generator=g) if norm == "layer" and n != 2 else None
        return x, norm, gain, bias

    q = make(Hq, nq)
    k = make(Hk, nk) if Hk else None

    def heads(a):
        return None if a is None else dsa.Heads(a[0].cuda(), a[1], *(None if t is None else t.cuda() for t in a[2:]))

    got = dsa.dsa_head_norm_rope(heads(q), heads(k), cos.cuda(), sin.cuda(), seqs, rope=rope, rope_first=first,
                                 split=split, dtype=y_dt,
                                 pos=torch.tensor(pos, dtype=torch.int32).cuda() if given else None)
    assert dsa.last_kernels() == {"head_norm"} and dsa.last_launch_count() == 1
    assert (got[1] is None) == (k is None)
    for a, r in ((q, got[0]), (k, got[1])):
        if a is not None:
            check(r, a[0], a[1], a[2], a[3], 1e-6, cos, sin, pos, rope, first, split, y_dt)


@pytest.mark.parametrize("rope", ["pairs", "halves"])
@pytest.mark.parametrize("off", [0, 1])
def test_in_place_and_strided(rope, off):
    """x as slices of one projection's output, y over x; off = 1: rows off 16 bytes."""
    N, D, d_r = 37, 192, 64
    g = torch.Generator().manual_seed(5)
    cos, sin = tables(60, d_r)
    buf = torch.randn(N, 5 * D + 8, generator=g).bfloat16()
    seqs = dsa.Seqs([0, N], [0, 60], [20])
    dev = buf.cuda()
    view = lambda b, h0, n: b[:, off + h0 * D:off + (h0 + n) * D].unflatten(1, (n, D))  # noqa: E731
    q, k = view(dev, 0, 4), view(dev, 4, 1)
    got = dsa.dsa_head_norm_rope(dsa.Heads(q, "rms", y=q), dsa.Heads(k, "layer", y=k), cos.cuda(), sin.cuda(), seqs,
                                 rope=rope)
    assert got[0].data_ptr() == q.data_ptr()
    pos = list(range(20, 20 + N))
    check(view(dev, 0, 4), view(buf, 0, 4), "rms", None, None, 1e-6, cos, sin, pos, rope, False, False, BF16)
    check(view(dev, 4, 1), view(buf, 4, 1), "layer", None, None, 1e-6, cos, sin, pos, rope, False, False, BF16)
    rest = torch.cat([dev[:, :off], dev[:, off + 5 * D:]], 1).cpu()
    assert torch.equal(rest, torch.cat([buf[:, :off], buf[:, off + 5 * D:]], 1))


def test_zero_rows_and_far_positions():
    """A head of zeros normalises to zeros (layer: to the bias); a position far out takes its own angles."""
    N, D = 4, 128
    cos, sin = tables(70000, 64)
    x = torch.zeros(N, 2, D)
    bias = torch.arange(D).float() / D
    seqs = dsa.Seqs([0, N], [0, 70000], [69996])
    got = dsa.dsa_head_norm_rope(dsa.Heads(x.cuda(), "rms"), dsa.Heads(x.cuda(), "layer", bias=bias.cuda()), cos.cuda(),
                                 sin.cuda(), seqs)
    assert torch.count_nonzero(got[0]) == 0
    check(got[1], x, "layer", None, bias, 1e-6, cos, sin, list(range(69996, 70000)), "pairs", False, False, F32)


def test_graph_and_side_stream():
    N, D = 9, 192
    g = torch.Generator().manual_seed(6)
    cos, sin = tables(40, 64)
    x = torch.randn(N, 4, D, generator=g).bfloat16()
    xd, cd, sd = x.cuda(), cos.cuda(), sin.cuda()
    pos = torch.arange(N, dtype=torch.int32).cuda()
    seqs = dsa.Seqs([0, N], [0, 40], [31])
    eager = dsa.dsa_head_norm_rope(dsa.Heads(xd), None, cd, sd, seqs, pos=pos, split=True)[0]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dsa.dsa_head_norm_rope(dsa.Heads(xd), None, cd, sd, seqs, pos=pos, split=True)[0]
    graph.replay()
    assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])
    pos += 5
    graph.replay()
    check((out[0], out[1]), x, "rms", None, None, 1e-6, cos, sin, list(range(5, 5 + N)), "pairs", False, True, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_head_norm_rope(dsa.Heads(xd), None, cd, sd, seqs, pos=pos, split=True, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], out[0]) and torch.equal(got[1], out[1])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rope", ["pairs", "halves"])
@pytest.mark.parametrize("D,d_r", [(64, 64), (128, 64), (192, 64), (256, 128), (512, 64)])
def test_heads_on_16_but_not_32_bytes(dt, rope, D, d_r):
    """The same bits whether heads start on 32 bytes or on 16 only, for every number of lanes and vectors a head."""
    g = torch.Generator().manual_seed(D)
    T, n = [5, 0, 30], 9
    seqs = dsa.Seqs([0, 5, 5, 35], [0, 5, 6, 40], [0, 1, 4])
    cos, sin = (t.cuda() for t in tables(64, d_r))
    x = torch.randn(35, n, D, generator=g).to(dt).cuda()
    gain, bias = torch.randn(D, generator=g).cuda(), torch.randn(D, generator=g).cuda()
    want, _ = dsa.dsa_head_norm_rope(dsa.Heads(x, norm="layer", gain=gain, bias=bias), None, cos, sin, seqs, rope=rope)
    pad = 16 // x.element_size()
    wide = torch.full((35, n, D + pad), 9.0, dtype=dt, device="cuda")
    view = wide[:, :, pad:]
    view.copy_(x)
    got, _ = dsa.dsa_head_norm_rope(dsa.Heads(view, norm="layer", gain=gain, bias=bias, y=view), None, cos, sin, seqs, rope=rope)
    assert torch.equal(got, want) and torch.all(wide[:, :, :pad] == 9)
    check(want, x.cpu(), "layer", gain.cpu(), bias.cpu(), 1e-6, cos.cpu(), sin.cpu(), [0, 1, 2, 3, 4] + list(range(4, 34)), rope,
          False, False, dt)
