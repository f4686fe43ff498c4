"""Writing the latent cache and reading it back: bit for bit what the 64-bit form
gives, every other byte of the cache as it was."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R

pytestmark = pytest.mark.gpu
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8


def make_cache(rows, d_c, d_r, dtype, seed, packed=False):
    """Arbitrary bytes in every row (NaN patterns among them): what is not written has to keep them."""
    g = torch.Generator().manual_seed(seed)
    if dtype == U8:
        kv = torch.randint(0, 256, (rows, d_c), generator=g).to(U8)
        sc = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, d_c // 128), generator=g).to(torch.int32).view(F32)
        pe = torch.randint(-2 ** 15, 2 ** 15, (rows, d_r), generator=g).to(torch.int16).view(BF16)
        return [kv.cuda(), pe.cuda(), sc.cuda()]
    word, size = (torch.int32, 2 ** 31) if dtype == F32 else (torch.int16, 2 ** 15)
    w = d_c + d_r if packed else d_c
    kv = torch.randint(-size, size, (rows, w), generator=g).to(word).view(dtype).cuda()
    if packed:
        return [kv[:, :d_c], kv[:, d_c:], None]
    return [kv, torch.randint(-size, size, (rows, d_r), generator=g).to(word).view(dtype).cuda(), None]


def bits(t):
    return t.contiguous().view(U8).cpu() if t is not None else None


def stored(x, pe, dtype):
    """What the cache holds for fp32 / bf16 inputs on the CPU: (kv, pe, scale)."""
    if dtype == U8:
        codes, scale = R.quantise(x.double())
        return codes, pe.to(BF16), scale
    return x.to(dtype), pe.to(dtype), None


LAYOUTS = [0, 16, 48, 64]
WIDTHS = [(512, 64), (128, 0), (384, 40), (256, 3)]


def inputs(N, d_c, d_r, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, d_c, generator=g) * torch.exp(2 * torch.randn(N, 1, generator=g))).to(dt)
    return x, torch.randn(N, d_r, generator=g).to(dt)


@pytest.mark.parametrize("page", LAYOUTS)
@pytest.mark.parametrize("cache_dt", [F32, BF16, U8])
@pytest.mark.parametrize("x_dt", [F32, BF16])
@pytest.mark.parametrize("d_c,d_r", WIDTHS)
def test_write(page, cache_dt, x_dt, d_c, d_r):
    # a rotary width that is no multiple of 16 bytes needs rows padded to 16 bytes: a slice of wider ones
    bt = R.Batch([5, 0, 1, 70], [0, 7, 63, 40], page, seed=1, slack=2)
    x, pe = inputs(bt.N, d_c, d_r, x_dt, 2)
    wide = -(-d_r // 8) * 8
    kv, full, sc = make_cache(bt.rows, d_c, wide, cache_dt, 3)
    before = [bits(t) for t in (kv, full, sc)]
    want = [t.cpu().clone() if t is not None else None for t in (kv, full, sc)]
    c, p, s = stored(x, pe, cache_dt)
    for b in range(4):
        rows = bt.rows_at(b, range(bt.P[b], bt.P[b] + bt.T[b]))
        n0, n1 = bt.cu_q[b], bt.cu_q[b + 1]
        want[0][rows], want[1][rows, :d_r] = c[n0:n1], p[n0:n1]
        if s is not None:
            want[2][rows] = s[n0:n1]
    cache = dsa.LatentCache(kv, full[:, :d_r], sc)
    dsa.dsa_latent_cache_write(x.cuda(), pe.cuda(), cache, bt.seqs(), pages=bt.pages())
    assert dsa.last_kernels() == {"cache_write"}
    for got, exp, old in zip((kv, full, sc), want, before):
        if got is not None:
            assert torch.equal(bits(got), bits(exp))
            assert got.numel() == 0 or not torch.equal(bits(got), old)


@pytest.mark.parametrize("page", [0, 48])
@pytest.mark.parametrize("cache_dt", [F32, BF16, U8])
@pytest.mark.parametrize("out_dt", [F32, BF16])
@pytest.mark.parametrize("by_pos", [False, True])
@pytest.mark.parametrize("d_c,d_r", [(512, 64), (128, 0), (384, 40)])
def test_read(page, cache_dt, out_dt, by_pos, d_c, d_r):
    bt = R.Batch([5, 0, 1, 70], [0, 7, 63, 40], page, seed=4, slack=30)
    x, pe = inputs(bt.rows, d_c, d_r, F32, 5)
    c, p, s = stored(x, pe, cache_dt)
    cache = dsa.LatentCache(c.cuda(), p.cuda(), None if s is None else s.cuda())
    lat = R.dequantise(c, s) if s is not None else c.double()
    pos, want_c, want_p = [], torch.zeros(bt.N, d_c).double(), torch.zeros(bt.N, d_r).double()
    g = torch.Generator().manual_seed(6)
    for b in range(4):
        for t in range(bt.T[b]):
            at = bt.P[b] + t
            if by_pos:  # the same token twice, tokens that are none, the first and the last
                at = [-1, bt.S[b], 0, bt.S[b] - 1, -2 ** 31, 2 ** 31 - 1][t] if t < 6 else int(
                    torch.randint(0, bt.S[b], (1,), generator=g))
            if 0 <= at < bt.S[b]:
                row = bt.rows_at(b, [at])[0]
                want_c[len(pos)], want_p[len(pos)] = lat[row], p[row].double()
            pos.append(at)
    got_c, got_p = dsa.dsa_latent_cache_read(cache, bt.seqs(), pages=bt.pages(), dtype=out_dt,
                                             pos=torch.tensor(pos, dtype=torch.int32).cuda() if by_pos else None)
    assert dsa.last_kernels() == {"cache_read"}
    assert torch.equal(got_c.cpu(), want_c.to(out_dt)) and torch.equal(got_p.cpu(), want_p.to(out_dt))


@pytest.mark.parametrize("x_dt", [F32, BF16])
def test_quantised_blocks_at_the_borders(x_dt):
    """Block maxima at and next to 448 * 2^e, zeros, one value, the smallest and largest numbers; codes equal the
    library's own quantiser's and reading back twice changes nothing."""
    tops = [0.0, 448.0, 449.0, 446.0, 1.0, 0.875, 0.8750001, 2.0 ** -133, 2.0 ** -126, 1e-40, 3e38, 2.0 ** 127, 7 * 2.0 ** -20]
    x = torch.zeros(len(tops), 512)
    g = torch.Generator().manual_seed(7)
    for i, t in enumerate(tops):
        x[i] = (torch.rand(512, generator=g) * 2 - 1) * t
        x[i, ::128] = t if i % 2 else -t
    x[:, 130:256] = 0
    x = x.to(x_dt)
    N = len(tops)
    kv, pe, sc = make_cache(N, 512, 64, U8, 8)
    cache = dsa.LatentCache(kv, pe, sc)
    seqs = dsa.Seqs([0, N], [0, N], [0])
    zero = torch.zeros(N, 64, dtype=x_dt).cuda()
    dsa.dsa_latent_cache_write(x.cuda(), zero, cache, seqs)
    codes, scale = R.quantise(x.double())
    own_codes, own_scale = dsa.dsa_quant_e4m3_ue8m0(x.cuda())
    assert torch.equal(kv, own_codes) and torch.equal(sc.flatten(), own_scale)
    normal = scale.flatten() >= 2.0 ** -126  # 2^-127 is no normal fp32 number to compare the codes' division with
    assert torch.equal(sc.cpu().flatten(), scale.flatten())
    a, b = kv.cpu().view(-1, 128)[normal], codes.view(-1, 128)[normal]
    zeros = (a & 0x7f == 0) & (b & 0x7f == 0)
    assert torch.equal(torch.where(zeros, 0, a), torch.where(zeros, 0, b))
    first, _ = dsa.dsa_latent_cache_read(cache, seqs, dtype=F32)
    dsa.dsa_latent_cache_write(first, zero.float(), cache, seqs)
    second, _ = dsa.dsa_latent_cache_read(cache, seqs, dtype=F32)
    big = first.abs() >= 2.0 ** -126
    assert torch.equal(first[big], second[big])


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_entries_that_name_no_page(cache_dt):
    bt = R.Batch([40, 33], [20, 100], 16, seed=9)
    bad = {0: [2, 3], 1: [7]}
    x, pe = inputs(bt.N, 512, 64, F32, 10)
    kv, pe_c, sc = make_cache(bt.rows, 512, 64, cache_dt, 11)
    want = [t.cpu().clone() if t is not None else None for t in (kv, pe_c, sc)]
    for n, (b, ks) in enumerate(bad.items()):
        for k in ks:
            bt.table[b, k] = [-1, bt.n_pages, 2 ** 31 - 1][(n + k) % 3]
    c, p, s = stored(x, pe, cache_dt)
    out_c, out_p = torch.zeros(bt.N, 512).double(), torch.zeros(bt.N, 64).double()
    lat = R.dequantise(c, s) if s is not None else c.double()
    for b in range(2):
        for t in range(bt.T[b]):
            at, r = bt.P[b] + t, bt.cu_q[b] + t
            if at // 16 in bad[b]:
                continue
            row = int(bt.table[b, at // 16]) * 16 + at % 16
            want[0][row], want[1][row] = c[r], p[r]
            if s is not None:
                want[2][row] = s[r]
            out_c[r], out_p[r] = lat[r], p[r].double()
    cache = dsa.LatentCache(kv, pe_c, sc)
    dsa.dsa_latent_cache_write(x.cuda(), pe.cuda(), cache, bt.seqs(), pages=bt.pages())
    for got, exp in zip((kv, pe_c, sc), want):
        assert got is None or torch.equal(bits(got), bits(exp))
    got_c, got_p = dsa.dsa_latent_cache_read(cache, bt.seqs(), pages=bt.pages(), dtype=F32)
    assert torch.equal(got_c.cpu().double(), out_c) and torch.equal(got_p.cpu().double(), out_p)


@pytest.mark.parametrize("cache_dt", [F32, BF16, U8])
def test_strides_and_alignment(cache_dt):
    """Dense rows off 16 bytes and with odd strides, cache rows as slices of wider ones: same bytes."""
    bt = R.Batch([9, 4], [3, 60], 64, seed=12)
    x, pe = inputs(bt.N, 512, 64, BF16, 13)
    odd = torch.zeros(bt.N, 700, dtype=BF16, device="cuda")[:, 1:]
    odd[:, :512], odd[:, 520:584] = x.cuda(), pe.cuda()
    got = []
    for a, b in ((x.cuda(), pe.cuda()), (odd[:, :512], odd[:, 520:584])):
        kv, p, sc = make_cache(bt.rows, 576, 128, cache_dt if cache_dt != U8 else BF16, 14)
        if cache_dt == U8:
            kv = torch.zeros(bt.rows, 640, dtype=U8, device="cuda")[:, 64:576]
            sc = torch.zeros(bt.rows, 4, device="cuda")
        cache = dsa.LatentCache(kv[:, :512], p[:, 64:], sc)
        dsa.dsa_latent_cache_write(a, b, cache, bt.seqs(), pages=bt.pages())
        dense = torch.full((bt.N, 601), 7.0, dtype=F32, device="cuda")
        dsa.dsa_latent_cache_read(cache, bt.seqs(), pages=bt.pages(), c_kv=dense[:, 3:515], k_pe=dense[:, 530:594])
        assert torch.all(dense[:, :3] == 7) and torch.all(dense[:, 515:530] == 7) and torch.all(dense[:, 594:] == 7)
        got.append((bits(kv), bits(p), bits(dense)))
    assert all(torch.equal(u, v) for u, v in zip(*got))


def test_graph_and_side_stream():
    """Captured and replayed on new inputs; called on a stream of its own."""
    bt = R.Batch([3, 2], [10, 64], 16, seed=15)
    kv, pe, sc = make_cache(bt.rows, 512, 64, U8, 16)
    cache, pages, seqs = dsa.LatentCache(kv, pe, sc), bt.pages(), bt.seqs()
    x, p = (t.cuda() for t in inputs(bt.N, 512, 64, BF16, 17))
    dsa.dsa_latent_cache_write(x, p, cache, seqs, pages=pages)
    dsa.dsa_latent_cache_read(cache, seqs, pages=pages)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_latent_cache_write(x, p, cache, seqs, pages=pages)
        out = dsa.dsa_latent_cache_read(cache, seqs, pages=pages)
    x2, p2 = (t.cuda() for t in inputs(bt.N, 512, 64, BF16, 18))
    x.copy_(x2)
    p.copy_(p2)
    graph.replay()
    codes, scale = R.quantise(x2.cpu().double())
    assert torch.equal(out[0].cpu(), R.dequantise(codes, scale).to(BF16)) and torch.equal(out[1], p2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_latent_cache_read(cache, seqs, pages=pages, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], out[0]) and torch.equal(got[1], out[1])


@pytest.mark.parametrize("cache_dt", [F32, BF16, U8])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T", [[9, 4], [3000, 4000]])
def test_rows_on_16_but_not_32_bytes(cache_dt, dt, T):
    """The same bytes whether rows start on 32 bytes or on 16 only; few tokens (one a warp) and many (four a warp)."""
    bt = R.Batch(T, [3, 60], 64, seed=19)
    x, pe = inputs(bt.N, 512, 64, dt, 20)
    pad = 16 // x.element_size()
    got = []
    for extra in (0, pad):
        wide = torch.zeros(bt.N, 576 + extra, dtype=dt, device="cuda")[:, extra:]
        wide[:, :512], wide[:, 512:] = x.cuda(), pe.cuda()
        kv, p, sc = make_cache(bt.rows, 512, 64, cache_dt, 21)
        cache = dsa.LatentCache(kv, p, sc)
        dsa.dsa_latent_cache_write(wide[:, :512], wide[:, 512:], cache, bt.seqs(), pages=bt.pages())
        dense = torch.full((bt.N, 576 + extra), 7.0, dtype=dt, device="cuda")[:, extra:]
        dsa.dsa_latent_cache_read(cache, bt.seqs(), pages=bt.pages(), c_kv=dense[:, :512], k_pe=dense[:, 512:])
        got.append((bits(kv), bits(p), bits(dense.contiguous())))
    assert all(torch.equal(u, v) for u, v in zip(*got))
    if cache_dt != U8:
        assert torch.equal(got[0][2], bits(torch.cat([x, pe], 1).to(cache_dt).to(dt).cuda()))
