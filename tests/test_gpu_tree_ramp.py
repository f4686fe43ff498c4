"""Tree attention whose running maximum moves from tile to tile (bands: see latent_reference, without a term for the
exchange of half scores).

The queries' latent part is 0, so scores come from the rotary keys alone: their first value puts a tile of 64 tokens on
a level, 9.16 powers of two above the level below (88 softmax_scale log2(e)); a reference moves by more than 8.  The
latents of a level are 2^9 times smaller than those of the level below, so every tile has about the same weight in the
result, however far the maximum has moved since: a factor that is missing, late or applied twice shows in full."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R
from tests.test_gpu_tree_mla import Case, TC

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8
TOP = 12
RAMPS = {
    "every tile": lambda t: t % (TOP + 1),
    "every second": lambda t: t // 2 % (TOP + 1),
    "every third": lambda t: t // 3 % (TOP + 1),
    "down": lambda t: TOP - t % (TOP + 1),
    "up 3, down 2": lambda t: t // 2 % 10 + (3 if t % 2 else 0),
    "anyhow": lambda t: t * 7919 % 104729 % (TOP + 1),
}
ROWS = {  # rows (node * heads + head) that the ramp lifts; of 32 rows a CTA of the pair finishes 16
    "all rows": lambda i: i >= 0, "every third row": lambda i: i % 3 == 0,
    "one CTA's rows": lambda i: i % 32 < 16, "the other CTA's rows": lambda i: i % 32 >= 16,
}


def ramp(c, level, lifted):
    T_H = [(r - c.bt.cu_q[b]) * c.H for b in range(len(c.bt.T)) for r in range(c.bt.cu_q[b], c.bt.cu_q[b + 1])]
    i = torch.tensor(T_H)[:, None] + torch.arange(c.H)
    c.q_nope.zero_()
    c.q_pe[..., 0] = lifted(i).to(BF16)
    for b in range(len(c.bt.T)):
        n = c.bt.P[b] + c.bt.T[b]
        at = torch.tensor(c.bt.rows_at(b, range(n)))
        seen = c.pe[at, 0].float() > -float("inf")
        at, lv = at[seen], torch.tensor([level(s // 64) for s in range(n)]).float()[seen]
        c.pe[at, 0] = (88 * lv).to(BF16)
        assert torch.equal(c.pe[at, 0].float(), 88 * lv)
        f = 2.0 ** (9 * (TOP - lv))
        if c.sc is None:
            c.kv[at] = (c.kv[at].float() * f[:, None]).to(BF16)
        else:
            c.sc[at] *= f[:, None]
    c.lat = c.kv.double() if c.sc is None else R.dequantise(c.kv, c.sc)


PAIRS = [(r, "all rows") for r in RAMPS] + [(r, w) for r in ("every tile", "up 3, down 2") for w in ROWS if w != "all rows"]


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("which,rows", PAIRS)
def test_whole_sequences(cache_dt, which, rows):
    """13 to 15 tiles in one piece, trees of 16 nodes with 128 heads."""
    c = Case([16] * 5, [830, 880, 900, 839, 896], 64, 128, TC, BF16, cache_dt, "tree", seed=70)
    ramp(c, RAMPS[which], ROWS[rows])
    out, lse = c.call()
    assert "tree_tc" in dsa.last_kernels() and "tree_combine" not in dsa.last_kernels()
    c.check(out, lse, heads=[0, 20, 77, 127], exchange=False)


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("which,rows", PAIRS)
def test_split_sequences(cache_dt, which, rows):
    """57 tiles in three ranges that are joined again."""
    c = Case([2] * 12, [3600 - 5 * b for b in range(12)], 64, 128, TC, BF16, cache_dt, "chain", seed=71)
    ramp(c, RAMPS[which], ROWS[rows])
    out, lse = c.call()
    assert {"tree_tc", "tree_combine"} <= dsa.last_kernels()
    c.check(out, lse, heads=[0, 20, 127], exchange=False)
