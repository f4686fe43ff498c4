"""Tree attention at the edges of what a call may be given: scales of the softmax
and of the cache, NaN that some rows see, caches past 2^32 bytes, the most
sequences, wide block tables, graphs side by side, waits that run out."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from sparse_latent_attention_indexer_gb300 import _abi
from tests import latent_reference as R
from tests.test_gpu_tree_mla import BF16, TC, U8, Case, random_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1e-30, 1.0])
def test_softmax_scales(cache_dt, generic, scale, monkeypatch):
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([3, 1], [130, 64], 32, 4, TC, BF16, cache_dt, "tree", seed=21)
    c.scale = scale
    out, lse = c.call()
    c.check(out, lse, exchange=not generic)


@pytest.mark.parametrize("e", [-40, -9, 9, 12, 40])
def test_block_scales(e):
    """Latents times 2^e (block scales from far below to far above the range of one bf16 factor) and scores of the usual
    size: what a softmax scale of 2^-e makes of them."""
    c = Case([3, 2], [130, 300], 16, 4, TC, BF16, U8, "odd", seed=22)
    f = 2.0 ** e
    c.sc = torch.where(torch.isfinite(c.sc), c.sc * f, c.sc)
    c.lat = torch.where(torch.isfinite(c.lat), c.lat * f, c.lat)
    c.pe = (c.pe.float() * f).to(BF16)
    c.scale /= f
    out, lse = c.call()
    # everything past the scores scales with the latents
    c.check(out, lse)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 2.0 ** 127, -2.0 ** 20, -1e30, 1e30, -2.0 ** -140])
@pytest.mark.parametrize("masks", ["tree", "chain", "odd"])
def test_hidden_scales(bad, masks):
    """Any scale beside any code in rows that nobody sees, or that only some rows do not see."""
    c = Case([5, 70], [64, 1], 48, 4, TC, BF16, U8, masks, seed=23, slack=3)
    c.sc[torch.isinf(c.sc)] = bad
    out, lse = c.call()
    c.check(out, lse)


@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("P", [40, 3000])
def test_a_nan_reaches_the_rows_that_see_it(generic, P, monkeypatch):
    """Node 2's latents hold a NaN: its descendants are NaN, the other nodes are what they were without it (up to the
    rounding of probabilities that were taken against another reference: twice the final rounding and P's)."""
    def same(got, want):
        a, b = got.double(), want.double()
        return bool(((a - b).abs() <= 4 * R.U[BF16] * b.abs().amax(-1, keepdim=True)).all())

    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([9, 2], [P, 30], 0, 3, TC, BF16, BF16, "tree", seed=24)
    out, lse = c.call()
    c.kv[c.bt.rows_at(0, [P + 2])[0], 77] = math.nan
    got, got_lse = c.call()
    hit = torch.tensor([bool(r >> 2 & 1) for r in random_tree(9, 24)] + [False, False])
    assert hit.any() and not hit[:9].all()
    assert torch.isnan(got[hit.cuda()]).all() and torch.isnan(got_lse[hit.cuda()]).all()
    assert same(got[~hit.cuda()], out[~hit.cuda()]) and same(got_lse[~hit.cuda()][..., None], lse[~hit.cuda()][..., None])
    c.q_nope[4, 1, 5] = math.nan  # one head of one node
    got, _ = c.call()
    assert torch.isnan(got[4, 1]).all()
    still = ~hit
    still[4] = False
    assert same(got[still.cuda()], out[still.cuda()])


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_cache_past_32_bit_offsets(cache_dt):
    """Pages at the end of a cache whose rows lie more than 2^32 bytes (e4m3: 2^31) from its start: written, attended
    over and read there."""
    rows, page = 4_400_000 // 64 * 64, 64
    c = Case([3, 1], [150, 64], page, 4, TC, BF16, cache_dt, "tree", seed=25)
    shift = rows // page - c.bt.n_pages
    small = c.cache()
    kv = torch.zeros(rows, 512, dtype=small.kv.dtype, device="cuda")
    pe = torch.zeros(rows, 64, dtype=BF16, device="cuda")
    sc = None if small.kv_scale is None else torch.ones(rows, 4, device="cuda")
    n = c.bt.n_pages * page
    for big, t in ((kv, small.kv), (pe, small.k_pe), (sc, small.kv_scale)):
        if big is not None:
            big[shift * page:shift * page + n] = t[:n]
    far = dsa.LatentCache(kv, pe, sc)
    table = torch.where(c.bt.table >= 0, c.bt.table + shift, c.bt.table).cuda()
    pages = dsa.Pages(table, page, rows // page)
    args = c.q_nope.cuda(), c.q_pe.cuda()
    W = c.W_UK.cuda(), c.W_UV.cuda()
    want = dsa.dsa_tree_mla_fwd(*args, small, *W, c.bt.seqs(), c.scale, tree_mask=c.mask(), pages=c.bt.pages())
    got = dsa.dsa_tree_mla_fwd(*args, far, *W, c.bt.seqs(), c.scale, tree_mask=c.mask(), pages=pages)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    x, xp = torch.randn(c.bt.N, 512, device="cuda").to(BF16), torch.randn(c.bt.N, 64, device="cuda").to(BF16)
    back = []
    for cache, pg in ((small, c.bt.pages()), (far, pages)):
        dsa.dsa_latent_cache_write(x, xp, cache, c.bt.seqs(), pages=pg)
        back.append(dsa.dsa_latent_cache_read(cache, c.bt.seqs(), pages=pg))
    assert all(torch.equal(a, b) for a, b in zip(*back))
    assert torch.equal(back[0][1], xp)


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("page", [0, 16])
def test_most_sequences(cache_dt, page):
    T = [(b * 7 + 3) % 4 for b in range(1024)]
    P = [(b * 13) % 40 for b in range(1024)]
    c = Case(T, P, page, 2, TC, BF16, cache_dt, "chain", seed=26)
    out, lse = c.call()
    assert "tree_tc" in dsa.last_kernels()
    c.check(out, lse, heads=[1])


def test_block_table_wider_than_the_call_needs():
    c = Case([2, 3], [100, 20], 16, 4, TC, BF16, U8, "tree", seed=27)
    out, lse = c.call()
    wide = torch.full((2, c.bt.table.shape[1] + 5), 2 ** 30, dtype=torch.int32)
    wide[:, :c.bt.table.shape[1]] = c.bt.table
    for table in (wide.cuda(), wide.cuda()[:, :c.bt.table.shape[1]]):
        got = dsa.dsa_tree_mla_fwd(c.q_nope.cuda(), c.q_pe.cuda(), c.cache(), c.W_UK.cuda(), c.W_UV.cuda(), c.bt.seqs(),
                                   c.scale, tree_mask=c.mask(), pages=dsa.Pages(table, 16, c.bt.n_pages))
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)


def test_two_graphs_with_their_own_workspaces():
    """Two captured calls that split their contexts run at the same time, again and again."""
    cases = [Case([2, 3], [2500, 700], 64, 16, TC, BF16, dt, "tree", seed=28 + i) for i, dt in enumerate((BF16, U8))]
    graphs, outs, want = [], [], []
    for c in cases:
        held = c.q_nope.cuda(), c.q_pe.cuda(), c.cache(), c.W_UK.cuda(), c.W_UV.cuda(), c.mask(), c.bt.pages(), c.bt.seqs()
        need = dsa.dsa_tree_mla_workspace_size(_abi.DSA_BF16, 16, *TC, held[7])
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def call(held=held, ws=ws, c=c):
            return dsa.dsa_tree_mla_fwd(*held[:5], held[7], c.scale, tree_mask=held[5], pages=held[6], workspace=ws)

        want.append([t.clone() for t in call()])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append((g, held, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_waits_that_run_out_are_reported(cache_dt):
    """With a wait limit of 64 cycles the first wait that is not already over gives up, both CTAs of the unit drain and
    exit, the site is reported, and with the limit restored the same call gives the same result."""
    c = Case([3, 2], [900, 130], 64, 16, TC, BF16, cache_dt, "tree", seed=30)
    out, lse = c.call()
    assert dsa.dsa_check_device_error() == (_abi.DSA_OK, 0)
    try:
        dsa.dsa_set_wait_limit(64)
        c.call()
        st, site = dsa.dsa_check_device_error()
    finally:
        dsa.dsa_set_wait_limit(0)
    assert st == _abi.DSA_ERR_TIMEOUT and site > 0
    for _ in range(8):  # a word for each kernel
        dsa.dsa_check_device_error()
    again = c.call()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert dsa.dsa_check_device_error() == (_abi.DSA_OK, 0)


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("generic", [False, True])
def test_bits_of_nodes_that_are_not_there(cache_dt, generic, monkeypatch):
    """Mask bits from the sequence's last node on, and words that no node needs, change nothing."""
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([5, 70, 64], [100, 7, 64], 16, 3, TC, BF16, cache_dt, "tree", seed=31, slack=9)
    out, lse = c.call()
    T = [t for t in c.bt.T for _ in range(t)]
    words = 4
    rows = [(v | (1 << 64 * words) - (1 << t)) for v, t in zip(c.bits, T)]
    sign = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
    mask = torch.tensor([[sign(v >> 64 * w & (1 << 64) - 1) for w in range(words)] for v in rows]).cuda()
    got = dsa.dsa_tree_mla_fwd(c.q_nope.cuda(), c.q_pe.cuda(), c.cache(), c.W_UK.cuda(), c.W_UV.cuda(), c.bt.seqs(), c.scale,
                               tree_mask=mask, pages=c.bt.pages())
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
