"""The norms around a block with its gate and residual against the 64-bit form.

h' and y are rounded once each (U).  Before that a norm's fp32 sums of D values are off by at most about D roundings of
2^-24, relative to the largest value that enters, its division, gain and bias add a few more: E = 8 (D + 16) 2^-24 of the
row's largest possible result; a gate, the scale and the addition to h add a few roundings of what they work on; and y
inherits what h' is off by, as many times as the norm enlarges it."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import next_token_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def gained(v, kind, gain, bias, eps):
    """How large a row's results may be, and by how much the norm enlarges."""
    if kind in (None, "none"):
        return v.abs().amax(-1, keepdim=True), 1.0
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
    inv = 1 / ((v - mean).pow(2).mean(-1, keepdim=True) + eps).sqrt()
    if gain is not None:
        inv = inv * gain.double().abs().max()
    top = 2 * v.abs().amax(-1, keepdim=True) * inv
    return top + (bias.double().abs().max() if bias is not None else 0.0), inv


def check(got, h, u, gate, gate_act, post, pre, skip, scale, eps, dtypes):
    r, y = R.block_norm(h, u, gate, gate_act, post, pre, skip, scale, eps)
    D = h.shape[1]
    E = 8 * (D + 16) * 2.0 ** -24
    off = 4 * 2.0 ** -24 * (skip * h.double()).abs().amax(-1, keepdim=True)
    if u is not None:
        top, _ = gained(u.double(), *post, eps)
        times = abs(scale) * (1.0 if gate is None else R.act(gate.double(), gate_act).abs().amax(-1, keepdim=True))
        off = off + (E if post[0] not in (None, "none") else 8 * 2.0 ** -24) * top * times
    top, inv = gained(r, *pre, eps)
    off_y = (E if pre[0] not in (None, "none") else 0.0) * top + 4 * off * inv
    for a, want, dt, slack in ((got[0], r, dtypes[0], off), (got[1], y, dtypes[1], off_y)):
        if a is None:
            continue
        assert a.dtype == dt and a.shape == want.shape
        over = (a.double() - want).abs() - R.U[dt] * want.abs() - slack
        assert float(over.max()) <= 0, f"off by {float(over.max()):.3e} more than derived"


def make(N, D, h_dt, x_dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(N + D + seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return (3 * r(N, D)).to(h_dt), r(N, D).to(x_dt), r(N, D).to(x_dt), 1 + 0.2 * r(D), r(D), 1 + 0.1 * r(D), 0.5 * r(D)


WIDTHS = [1, 2, 7, 8, 31, 33, 64, 255, 256, 257, 264, 1000, 1024, 1025, 1032, 2049, 4096, 4097, 7168, 8192, 8193, 8200, 16383, 16384]


@pytest.mark.parametrize("h_dt,x_dt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, h_dt, x_dt):
    N = 6
    h, u, g, a, b, c, d = make(N, D, h_dt, x_dt)
    pre_kind, post_kind = ("rms", "layer")[D % 2], ("layer", "rms", "none")[D % 3]
    post, pre = (post_kind, a, b if post_kind == "layer" else None), (pre_kind, c, d if pre_kind == "layer" else None)
    got = dsa.dsa_block_norm(h, dsa.Norm(*pre), u=u, post=dsa.Norm(*post), gate=g, gate_act="sigmoid", scale=0.5)
    assert dsa.last_kernels() == {"block_norm"} and dsa.last_launch_count() == 1
    check(got, h, u, g, "sigmoid", post, pre, 1.0, 0.5, 1e-6, (h_dt, x_dt))


@pytest.mark.parametrize("D", [40, 333, 1536, 7168])
@pytest.mark.parametrize("N", [1, 5, 400])
def test_forms(N, D):
    """With and without a block, its norm, its gate and either output; more rows than SMs."""
    h, u, g, a, b, c, d = make(N, D, BF16, BF16)
    none = ("none", None, None)
    for post in (none, ("rms", None, None), ("layer", a, b)):
        for pre in (none, ("rms", c, None), ("layer", None, d)):
            for gate, gate_act in ((None, None), (g, None), (g[:1], "silu"), (g, "sigmoid")):
                got = dsa.dsa_block_norm(h, dsa.Norm(*pre), u=u, post=dsa.Norm(*post), gate=gate, gate_act=gate_act, skip=0.7,
                                         scale=-1.3, eps=1e-5)
                check(got, h, u, gate, gate_act, post, pre, 0.7, -1.3, 1e-5, (BF16, BF16))
    got = dsa.dsa_block_norm(h, dsa.Norm("rms", c))
    assert torch.equal(got[0], h)
    check(got, h, None, None, None, none, ("rms", c, None), 1.0, 1.0, 1e-6, (BF16, BF16))
    only = dsa.dsa_block_norm(h, dsa.Norm("rms", c), u=u, want_h=False)
    both = dsa.dsa_block_norm(h, dsa.Norm("rms", c), u=u)
    assert only[0] is None and torch.equal(only[1], both[1])
    h_only = dsa.dsa_block_norm(h, u=u, want_y=False)
    assert h_only[1] is None and torch.equal(h_only[0], both[0])


@pytest.mark.parametrize("D", [48, 200, 1024, 2047, 7168])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strides_and_in_place(D, off):
    """Slices of wider rows, h' over h and y over u, gate rows far apart; what lies beside stays."""
    N = 9
    g = torch.Generator(device="cuda").manual_seed(D + off)
    wide = lambda: torch.randn(N, D + 24, generator=g, device="cuda").bfloat16()  # noqa: E731
    bh, bu, bg = wide(), wide(), wide()
    cut = lambda t: t[:, off:off + D]  # noqa: E731
    h, u, gate = cut(bh).clone(), cut(bu).clone(), cut(bg).clone()
    keep_h, keep_u = bh.clone(), bu.clone()
    pre = dsa.Norm("layer")
    got = dsa.dsa_block_norm(cut(bh), pre, u=cut(bu), gate=cut(bg), h_out=cut(bh), y=cut(bu))
    assert got[0].data_ptr() == cut(bh).data_ptr() and got[1].data_ptr() == cut(bu).data_ptr()
    apart = [cut(torch.empty_like(bh)) for _ in range(2)]  # rows that start on the same bytes: the same sums
    want = dsa.dsa_block_norm(cut(keep_h), pre, u=cut(keep_u), gate=cut(bg), h_out=apart[0], y=apart[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(got, h, u, gate, None, ("none", None, None), ("layer", None, None), 1.0, 1.0, 1e-6, (BF16, BF16))
    for now, then in ((bh, keep_h), (bu, keep_u)):
        assert torch.equal(now[:, :off], then[:, :off]) and torch.equal(now[:, off + D:], then[:, off + D:])


@pytest.mark.parametrize("h_dt,x_dt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("D", [1, 2, 5, 253, 254, 509, 510, 2050, 4093, 4094, 8191, 16381, 16382])
def test_rows_that_start_off_16_bytes(D, h_dt, x_dt):
    """All tensors alike, with NaN beside every row, gain, bias and gate row: none gets in, and what lies there stays."""
    N = 21
    for off in range(4):
        h, u, gate, pg, pb, qg, qb = make(N, D, h_dt, x_dt, seed=off)
        pad = 9 - D % 4 + off

        def beside(t, at=off):
            buf = torch.full((t.shape[0], D + pad) if t.dim() == 2 else (D + 11,), float("nan"), dtype=t.dtype, device="cuda")
            return buf, (buf[:, at:at + D] if t.dim() == 2 else buf[at:at + D]).copy_(t)

        row = beside(gate[0], 3)[1][None]
        post, pre = ("layer", beside(pg, 1)[1], beside(pb, 2)[1]), ("rms", beside(qg, 3)[1], None)
        for gate_, act in ((beside(gate)[1], "silu"), (row, "sigmoid"), (None, None)):
            (bh, ch), (bu, cu) = beside(h), beside(u)
            for outs in ((beside(torch.zeros_like(h)), beside(torch.zeros_like(u))), ((bh, ch), (bu, cu))):
                got = dsa.dsa_block_norm(ch, dsa.Norm(*pre), u=cu, post=dsa.Norm(*post), gate=gate_, gate_act=act, skip=0.5, scale=2.0,
                                         h_out=outs[0][1], y=outs[1][1])
                check(got, h, u, gate_, act, post, pre, 0.5, 2.0, 1e-6, (h_dt, x_dt))
                for buf, _ in outs:
                    assert bool(buf[:, :off].isnan().all()) and bool(buf[:, off + D:].isnan().all())


def test_large_means_zeros_and_nan():
    """A mean far above the spread costs layer norm nothing that fp32 has; zeros give the bias; a NaN stays in its row."""
    N, D = 4, 4096
    h = torch.randn(N, D, device="cuda") + 1000.0
    bias = torch.randn(D, device="cuda")
    got = dsa.dsa_block_norm(h, dsa.Norm("layer", None, bias))
    want = R.norm(h.double(), "layer", None, bias, 1e-6)
    # a value near 1000 is held to 2^-14 already; its mean to as much
    assert float((got[1] - want).abs().max()) <= 2.0 ** -13
    z = torch.zeros(N, D, device="cuda")
    assert torch.equal(dsa.dsa_block_norm(z, dsa.Norm("layer", None, bias))[1], bias.expand(N, D))
    assert torch.equal(dsa.dsa_block_norm(z, dsa.Norm("rms"))[1], z)
    clean = dsa.dsa_block_norm(h, dsa.Norm("rms"))[1]
    h[2, 77] = float("nan")
    got = dsa.dsa_block_norm(h, dsa.Norm("rms"))[1]
    assert bool(got[2].isnan().all()) and torch.equal(got[[0, 1, 3]], clean[[0, 1, 3]])


def test_gates_at_their_ends():
    """sigmoid and silu of numbers far out are their limits, not NaN."""
    D = 64
    gate = torch.tensor([-1e30, -200.0, -90.0, 0.0, 90.0, 200.0, 1e30, 1.0], device="cuda").repeat(8)[None]
    h, u = torch.zeros(2, D, device="cuda"), torch.ones(2, D, device="cuda")
    got = dsa.dsa_block_norm(h, u=u, gate=gate, gate_act="sigmoid", want_y=False)[0]
    check((got, None), h, u, gate, "sigmoid", ("none", None, None), ("none", None, None), 1.0, 1.0, 1e-6, (F32, F32))
    got = dsa.dsa_block_norm(h, u=u, gate=gate, gate_act="silu", want_y=False)[0]
    assert bool(got.isfinite().all()) and float(got[0, 6]) == float(gate[0, 6]) and float(got[0, 0]) == 0.0


def test_offsets_past_32_bits():
    """Rows past 2^31 values, and rows further than 2^31 apart."""
    N, D = 140000, 16384
    h = torch.randn(N, 64, device="cuda").bfloat16().repeat(1, D // 64)
    got = dsa.dsa_block_norm(h, dsa.Norm("rms"), want_h=False)[1]
    for r in (0, 1, 131071, 131072, 139999):
        check((None, got[r:r + 1]), h[r:r + 1], None, None, None, ("none", None, None), ("rms", None, None), 1.0, 1.0, 1e-6, (BF16, BF16))
    del got, h
    far = torch.zeros(3, 1200000000, dtype=BF16, device="cuda")
    x = torch.randn(3, 512, device="cuda").bfloat16()
    far[:, 16:528] = x
    got = dsa.dsa_block_norm(far[:, 16:528], dsa.Norm("rms"))
    assert torch.equal(got[1], dsa.dsa_block_norm(x, dsa.Norm("rms"))[1])


def test_streams_graphs_and_nothing_to_do():
    h, u, g, a, b, c, d = make(33, 1536, BF16, BF16)
    pre = dsa.Norm("rms", c)
    want = dsa.dsa_block_norm(h, pre, u=u, gate=g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dsa.dsa_block_norm(h, pre, u=u, gate=g, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dsa.dsa_block_norm(h, pre, u=u, gate=g)
    for t in (h, u, g):
        t.copy_(t.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0].flip(0)) and torch.equal(got[1], want[1].flip(0))
    empty = dsa.dsa_block_norm(h[:0], pre, u=u[:0])
    assert empty[1].shape == (0, 1536) and dsa.last_launch_count() == 0
