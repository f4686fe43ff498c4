"""Tree attention where a score's two halves of columns are large beside the score's spread, and where scores are
large altogether.

What a softmax cancels must cancel: a latent column that is the same for all tokens, whose share of the scores is
hundreds of nats in one half of the columns; and halves of the columns that are large, different for every token, and
opposite.  Bands as in latent_reference, with nothing for the exchange between the halves, and without the rounding of
those absorbed queries that are bf16 values as they are (their products are exact).

With whole numbers for queries and latents every product and sum is exact in fp32, so with a softmax scale of 1e3 and
more the result is the mean of the tokens that share the highest score, and nothing else: the others count 0 (e^-1000).
Of those that share it each counts 1 up to a rounding of its probability to bf16 (2^-8; the row sum adds the rounded
ones), which moves the mean by at most 2^-8 of its tokens' mean distance from it.  The mean is rounded to bf16 (2^-8),
multiplied by W_UV in fp32 (up to 512 terms, 2^-15 of their absolute sum) and rounded to bf16 again."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R
from tests.test_gpu_tree_mla import Case, TC

pytestmark = pytest.mark.gpu
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
A0, A1 = 5, 400  # a latent column of each half


def put(c, col, values):
    """Latent column `col` of every row that some row sees := values [rows] (exact in bf16 and in e4m3 with its scale)."""
    if c.sc is None:
        ok = torch.isfinite(c.kv[:, 0].float())
        c.kv[ok, col] = values[ok].to(c.kv.dtype)
        c.lat = c.kv.double()
    else:
        ok = torch.isfinite(c.sc[:, 0])
        tight = ok & (values.abs() > 448 * c.sc[:, col // 128])  # blocks of small values: their scale doubles, and they with it
        c.sc[tight, col // 128] *= 2
        codes = (values / c.sc[:, col // 128]).to(torch.float8_e4m3fn)
        c.kv[ok, col] = codes.view(U8)[ok]
        c.lat = R.dequantise(c.kv, c.sc)
    got = c.lat[ok, col]
    assert torch.equal(got, values[ok].double())


def query_column(c, col, w):
    """The absorbed query's column `col` is w for every row and head: bf16 products 1 w and 0."""
    w = float(torch.tensor(w).to(BF16))
    c.q_nope[:, :, 0] = 1.0
    c.W_UK[:, :, col] = 0.0
    c.W_UK[:, 0, col] = w
    c.W_UV[:, col] = 0.0  # the column shapes scores, not values
    return w


def form(q_nope, q_pe, lat, pe, see, W_UK, W_UV, scale, exact):
    """One sequence in 64 bits: out, its band, lse, its band (latent_reference says how), `exact`: columns of the
    absorbed queries that are not rounded."""
    T, H, _ = q_nope.shape
    v, n = R.U[BF16] / math.sqrt(3.0), lat.shape[0]
    acc = 2.0 ** -24 * math.sqrt(lat.shape[1] + pe.shape[1] + n)
    rounded = torch.ones(lat.shape[1], dtype=torch.float64)
    rounded[exact] = 0.0
    out, tol = torch.zeros(T, H, W_UV.shape[2]).double(), torch.zeros(T, H, W_UV.shape[2]).double()
    lse, ltol = torch.zeros(T, H).double(), torch.zeros(T, H).double()
    for h in range(H):
        qt = q_nope[:, h] @ W_UK[h]
        for t in range(T):
            c, r = lat[see[t]], pe[see[t]]
            z = (c @ qt[t] + r @ q_pe[t, h]) * scale
            lse[t, h] = torch.logsumexp(z, 0)
            p = torch.exp(z - lse[t, h])
            o = p @ c
            out[t, h] = o @ W_UV[h]
            d = c @ W_UV[h] - out[t, h]
            var_z = (acc * (c.abs() @ qt[t].abs() + r.abs() @ q_pe[t, h].abs()) * scale) ** 2
            var = (v * scale) ** 2 * (rounded * qt[t] ** 2) @ ((p[:, None] * c).T @ d) ** 2
            var += (p ** 2 * (var_z + v ** 2 + acc ** 2)) @ d ** 2 + v ** 2 * o ** 2 @ W_UV[h] ** 2
            tol[t, h] = R.SIGMAS * (var.sqrt() + acc * (o.abs() @ W_UV[h].abs()))
            lvar = (v * scale) ** 2 * (rounded * (qt[t] * o) ** 2).sum() + (p ** 2 * (var_z + v ** 2)).sum()
            ltol[t, h] = R.SIGMAS * lvar.sqrt() + 2.0 ** -20 * (1 + lse[t, h].abs())
    return out, tol, lse, ltol


def check(c, out, lse, exact):
    for b in range(len(c.bt.T)):
        n0, n1 = c.bt.cu_q[b], c.bt.cu_q[b + 1]
        at = c.bt.rows_at(b, range(c.bt.P[b] + c.bt.T[b]))
        ref, tol, l, lt = form(c.q_nope[n0:n1].double(), c.q_pe[n0:n1].double(), c.lat[at], c.pe[at].double(), c.see[b],
                               c.W_UK.double(), c.W_UV.double(), c.scale, exact)
        err = (out[n0:n1].cpu().double() - ref).abs()
        band = tol + R.U[BF16] * ref.abs()
        assert torch.all(err <= band), f"sequence {b}: {(err / band).max():.2f} of its band"
        lerr = (lse[n0:n1].cpu().double() - l).abs()
        assert torch.all(lerr <= lt), f"sequence {b}: lse {(lerr / lt).max():.2f} of its band"


@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("nats", [100.0, -300.0, 1000.0])
@pytest.mark.parametrize("where", [[A0], [A1], [A0, A1]])
def test_an_offset_that_all_tokens_share(generic, cache_dt, nats, where, monkeypatch):
    """One latent column (of either half, or of both with opposite signs) is 2 in every token."""
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([3, 2], [300, 130], 16, 8, TC, BF16, cache_dt, "tree", seed=50)
    for i, col in enumerate(where):
        query_column(c, col, (nats if i == 0 else -nats) / (2.0 * c.scale))
        put(c, col, torch.full((c.bt.rows,), 2.0))
    out, lse = c.call()
    assert ("tree_simt" if generic else "tree_tc") in dsa.last_kernels()
    check(c, out, lse, where)


@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("nats", [100.0, 300.0, 1000.0])
def test_halves_that_cancel(generic, cache_dt, nats, monkeypatch):
    """A column of each half holds the same value (another for every token), and the queries' columns are opposite."""
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([3, 2], [300, 130], 16, 8, TC, BF16, cache_dt, "tree", seed=51)
    g = torch.Generator().manual_seed(51)
    x = 2.0 ** torch.randint(-1, 2, (c.bt.rows,), generator=g) * (1 - 2 * torch.randint(0, 2, (c.bt.rows,), generator=g))
    for sign, col in ((1, A0), (-1, A1)):
        query_column(c, col, sign * nats / (2.0 * c.scale))
        put(c, col, x)
    out, lse = c.call()
    check(c, out, lse, [A0, A1])


@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("scale", [1e3, 3e3, 1e4, -1e4, 1e6])
@pytest.mark.parametrize("P", [130, 2500])
def test_whole_numbers_at_large_scales(generic, cache_dt, scale, P, monkeypatch):
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([3, 2], [P, 40], 64, 4, TC, BF16, cache_dt, "tree", seed=52)
    g = torch.Generator().manual_seed(53)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g).float()  # noqa: E731
    rows = c.bt.rows
    seen = c.pe[:, 0].float() > -math.inf
    lat = ints(-3, 3, rows, 512)
    if cache_dt == U8:
        c.kv[seen] = lat.to(torch.float8_e4m3fn).view(U8)[seen]
        c.sc[seen] = 1.0
    else:
        c.kv[seen] = lat.to(BF16)[seen]
    c.lat = lat.double()
    c.pe[seen] = ints(-3, 3, rows, 64).to(BF16)[seen]
    c.q_nope, c.q_pe = ints(-2, 2, c.bt.N, 4, 128).to(BF16), ints(-2, 2, c.bt.N, 4, 64).to(BF16)
    # column j of the absorbed query is value j % 128 of the query: whole numbers again
    c.W_UK = torch.eye(128).repeat(1, 4).expand(4, 128, 512).to(BF16).contiguous()
    c.W_UV = ints(-2, 2, 4, 512, 128).to(BF16)
    c.scale = scale
    out, lse = c.call()
    assert ("tree_simt" if generic else "tree_tc") in dsa.last_kernels()
    for b in range(2):
        n = c.bt.P[b] + c.bt.T[b]
        at = c.bt.rows_at(b, range(n))
        for t in range(c.bt.T[b]):
            r = c.bt.cu_q[b] + t
            see = c.see[b][t]
            for h in range(4):
                z = (c.lat[at] @ c.q_nope[r, h].double().repeat(4) + c.pe[at].double().nan_to_num(neginf=0) @ c.q_pe[r, h].double())
                z = torch.where(see, z * (1 if scale > 0 else -1), torch.tensor(-math.inf).double())
                top = z == z.max()
                o = c.lat[at][top].mean(0)
                want = o @ c.W_UV[h].double()
                apart = (c.lat[at][top] - o).abs().mean(0)
                band = ((2.0 ** -8 + 2.0 ** -15) * o.abs() + 2.0 ** -8 * apart) @ c.W_UV[h].double().abs()
                got = out[r, h].cpu().double()
                assert torch.all((got - want).abs() <= band + 2.0 ** -8 * (want.abs() + band)), (b, t, h)
                l = float(z.max()) * abs(scale) + math.log(int(top.sum()))
                assert abs(float(lse[r, h]) - l) <= 2.0 ** -21 * abs(l) + 2.0 ** -8
