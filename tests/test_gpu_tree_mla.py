"""Tree attention over the latent cache against the 64-bit form (bands: see
latent_reference).  Rows that nobody sees, and what a row does not see, hold NaN
and Inf throughout."""
import math
import random

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R

pytestmark = pytest.mark.gpu
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
TC = (128, 64, 512, 128)  # d_n, d_r, d_c, d_v of the tensor-core kernel


def random_tree(T, seed):
    r, rows = random.Random(seed), []
    for t in range(T):
        up = r.randint(max(-1, t - 4), t - 1)
        rows.append(1 << t | (rows[up] if up >= 0 else 0))
    return rows


class Case:
    def __init__(self, T, P, page, H, dims, dt, cache_dt, masks="tree", seed=0, slack=0, logits=1.0):
        g = torch.Generator().manual_seed(seed)
        self.bt = bt = R.Batch(T, P, page, seed=seed, slack=slack)
        d_n, d_r, d_c, d_v = dims
        self.H, self.dims, self.dt = H, dims, dt
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q_nope, self.q_pe = (n(bt.N, H, d_n) * logits).to(dt), (n(bt.N, H, d_r) * logits).to(dt)
        self.W_UK, self.W_UV = (n(H, d_n, d_c) / math.sqrt(d_c)).to(dt), (n(H, d_c, d_v) / math.sqrt(d_c)).to(dt)
        self.scale = 1.0 / math.sqrt(d_n + d_r)
        lat, pe = n(bt.rows, d_c), n(bt.rows, d_r).to(dt)
        if cache_dt == U8:
            self.kv, self.sc = R.quantise(lat.double())
            self.lat = R.dequantise(self.kv, self.sc)
        else:
            self.kv, self.sc = lat.to(cache_dt), None
            self.lat = self.kv.double()
        self.pe, self.kinds = pe, masks
        self.see, self.bits = [], []
        for b in range(len(T)):
            rows = {"tree": random_tree(T[b], seed + b), "chain": None,
                    # nothing, itself only, everything, later nodes only, the last node only
                    "odd": [[0, 1 << t, (1 << T[b]) - 1, (1 << T[b]) - (1 << t), 1 << (T[b] - 1)][(t + b) % 5]
                            for t in range(T[b])]}[masks]
            self.bits += rows or []
            self.see.append(R.visible(T[b], P[b], rows))
        used = torch.zeros(bt.rows, dtype=torch.bool)
        for b in range(len(T)):
            n_b = P[b] + T[b]
            seen = self.see[b].any(0)
            at = bt.rows_at(b, range(n_b))
            used[[r for r, s in zip(at, seen.tolist()) if s]] = True
        if self.sc is not None:
            self.kv[~used] = 0x7f
            self.sc[~used] = math.inf
        else:
            self.kv[~used] = math.nan
            self.kv[~used, 1] = math.inf
        self.pe = torch.where(used[:, None], pe, torch.tensor(-math.inf).to(dt))

    def mask(self):
        if self.kinds == "chain":
            return None
        words = max(1, -(-max(self.bt.T) // 64))
        sign = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
        rows = [[sign(v >> 64 * w & (1 << 64) - 1) for w in range(words)] for v in self.bits]
        return torch.tensor(rows, dtype=torch.int64).reshape(-1, words).cuda()

    def cache(self, packed=False):
        if packed and self.sc is None:
            buf = torch.cat([self.kv, self.pe], 1).cuda()
            return dsa.LatentCache(buf[:, :self.dims[2]], buf[:, self.dims[2]:])
        return dsa.LatentCache(self.kv.cuda(), self.pe.cuda(), None if self.sc is None else self.sc.cuda())

    def call(self, **kw):
        return dsa.dsa_tree_mla_fwd(self.q_nope.cuda(), self.q_pe.cuda(), kw.pop("cache", None) or self.cache(),
                                    self.W_UK.cuda(), self.W_UV.cuda(), self.bt.seqs(), self.scale,
                                    tree_mask=self.mask(), pages=self.bt.pages(), **kw)

    def check(self, out, lse, heads=None, exchange=True):
        heads = list(range(self.H)) if heads is None else heads
        u = R.U[self.dt]
        for b in range(len(self.bt.T)):
            n0, n1 = self.bt.cu_q[b], self.bt.cu_q[b + 1]
            if n0 == n1:
                continue
            at = self.bt.rows_at(b, range(self.bt.P[b] + self.bt.T[b]))
            ok = torch.tensor([r >= 0 for r in at])
            at = [max(r, 0) for r in at]
            ref, tol, l, lt = R.tree_attention(
                self.q_nope[n0:n1, heads].double(), self.q_pe[n0:n1, heads].double(), self.lat[at],
                self.pe[at].double(), self.see[b] & ok, self.W_UK[heads].double(), self.W_UV[heads].double(),
                self.scale, u, exchange=exchange)
            got = out[n0:n1].cpu().double()[:, heads]
            assert torch.all(torch.isfinite(got))
            err, band = (got - ref).abs(), tol + u * ref.abs()
            assert torch.all(err <= band), f"sequence {b}: error {err.max():.3e}, {(err / band.clamp(min=1e-30)).max():.2f} of its band"
            empty = ~(self.see[b] & ok).any(1)
            assert torch.all(got[empty] == 0)
            if lse is not None:
                gl = lse[n0:n1].cpu().double()[:, heads]
                assert torch.all(gl[empty] == -math.inf)
                assert torch.all((gl - l)[~empty].abs() <= lt[~empty]), ((gl - l)[~empty].abs() / lt[~empty]).max()


# --- generic kernel: any widths, fp32, and the tensor-core shapes when told so -----------------------------------
@pytest.mark.parametrize("dt,cache_dt,dims", [
    (F32, F32, (32, 16, 64, 32)), (F32, F32, (16, 0, 36, 5)), (BF16, BF16, (24, 8, 104, 40)),
    (BF16, U8, (32, 16, 128, 32)), (F32, F32, (128, 64, 512, 128))])
@pytest.mark.parametrize("masks", ["tree", "chain", "odd"])
@pytest.mark.parametrize("page", [0, 16])
def test_generic(dt, cache_dt, dims, masks, page):
    c = Case([5, 0, 1, 33], [0, 3, 31, 70], page, 3, dims, dt, cache_dt, masks, seed=1, slack=2)
    out, lse = c.call()
    assert "tree_simt" in dsa.last_kernels()
    c.check(out, lse, exchange=False)


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_generic_at_the_tensor_core_shape(cache_dt, monkeypatch):
    monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([4, 9], [100, 7], 32, 4, TC, BF16, cache_dt, "tree", seed=2)
    out, lse = c.call()
    assert dsa.last_kernels() == {"tree_simt", "absorb_simt"}
    c.check(out, lse, exchange=False)


# --- the released model's shape -----------------------------------------------------------------------------------
@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("masks", ["tree", "chain", "odd"])
@pytest.mark.parametrize("page", [0, 16, 32, 48, 64, 128])
def test_released_shape(cache_dt, masks, page):
    """Contexts of 0, 1, one tile and its neighbours, a few tiles; trees inside, over and behind a tile's end."""
    c = Case([1, 5, 3, 0, 2, 7], [0, 1, 64, 9, 63, 150], page, 16, TC, BF16, cache_dt, masks, seed=3, slack=1)
    out, lse = c.call()
    c.check(out, lse, heads=[0, 7, 15])
    # the rows the packed layout of the bf16 cache gives are the same
    if cache_dt == BF16:
        again, _ = c.call(cache=c.cache(packed=True))
        assert torch.equal(out, again)


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("H", [1, 5, 64, 128, 200])
def test_head_counts(cache_dt, H):
    c = Case([3, 1], [20, 200], 64, H, TC, BF16, cache_dt, "tree", seed=4)
    out, lse = c.call()
    c.check(out, lse, heads=sorted({0, H // 2, H - 1}))


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("T,P,masks", [([1], [2999], "chain"), ([2, 1], [2500, 700], "tree"), ([66, 130], [300, 5], "tree"),
                                       ([70], [0], "chain"), ([65], [1], "odd"), ([1, 1, 1], [64, 65, 4000], "odd")])
def test_long_contexts_and_trees(cache_dt, T, P, masks):
    """Contexts that are split and joined again, trees of more than a word and a tile."""
    c = Case(T, P, 64, 8, TC, BF16, cache_dt, masks, seed=5)
    out, lse = c.call()
    c.check(out, lse, heads=[1, 6])


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_peaked_scores_rescale(cache_dt):
    """Scores forty times the usual size, whose running maximum moves many times."""
    c = Case([4, 3], [900, 130], 32, 16, TC, BF16, cache_dt, "tree", seed=6, logits=6.0)
    out, lse = c.call()
    c.check(out, lse, heads=[0, 9])


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_entries_that_name_no_page(cache_dt):
    c = Case([3, 2], [200, 30], 16, 8, TC, BF16, cache_dt, "tree", seed=7)
    for b, k, e in ((0, 2, -1), (0, 7, c.bt.n_pages), (1, 0, -5), (1, 1, 2 ** 31 - 1)):
        c.bt.table[b, k] = e
    rows_at = c.bt.rows_at

    def masked(b, pos):
        return [r if 0 <= int(c.bt.table[b, s // 16]) < c.bt.n_pages else -1 for r, s in zip(rows_at(b, pos), pos)]

    c.bt.rows_at = masked
    out, lse = c.call()
    c.check(out, lse)


def test_rows_beside_the_outputs_stay():
    """Outputs inside larger buffers: the rows before and behind keep their values."""
    c = Case([3, 2], [70, 10], 16, 5, TC, BF16, BF16, "tree", seed=8)
    N, big = c.bt.N, torch.full((c.bt.N + 8, 5, 128), 3.0, dtype=BF16, device="cuda")
    lse = torch.full((N + 8, 5), 3.0, device="cuda")
    c.call(out=big[4:4 + N], lse=lse[4:4 + N])
    c.check(big[4:4 + N], lse[4:4 + N])
    assert torch.all(big[:4] == 3) and torch.all(big[4 + N:] == 3)
    assert torch.all(lse[:4] == 3) and torch.all(lse[4 + N:] == 3)


@pytest.mark.parametrize("cache_dt", [BF16, U8])
def test_same_bits_again_in_a_graph_and_beside_another_call(cache_dt):
    c = Case([3, 6], [1500, 64], 64, 16, TC, BF16, cache_dt, "tree", seed=9)
    args = [t.cuda() for t in (c.q_nope, c.q_pe)], c.cache(), [t.cuda() for t in (c.W_UK, c.W_UV)]
    mask, pages, seqs = c.mask(), c.bt.pages(), c.bt.seqs()

    def call(**kw):
        return dsa.dsa_tree_mla_fwd(*args[0], args[1], *args[2], seqs, c.scale, tree_mask=mask, pages=pages, **kw)

    out, lse = call()
    again, lse2 = call()
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_out, g_lse = call()
    graph.replay()
    assert torch.equal(out, g_out) and torch.equal(lse, g_lse)
    args[0][0].mul_(0.5)
    graph.replay()
    half, half_lse = call()
    assert torch.equal(half, g_out) and torch.equal(half_lse, g_lse) and not torch.equal(half, out)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    got = [call(stream=s) for s in (a, b, a, b)]
    for s in (a, b):
        torch.cuda.current_stream().wait_stream(s)
    for o, l in got:
        assert torch.equal(o, half) and torch.equal(l, half_lse)
