"""The operators as a step of speculative decoding uses them, one after another:
norm and rotate the queries' heads and the drafted tokens' keys, write the keys
into the cache, attend over prefix and tree, read the accepted path back, write
it where the sequence goes on, and decode the next token over the result.

Each stage is held to the 64-bit form of what the stage before it left (bands:
see latent_reference), the moves to the bit."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R
from tests.test_gpu_tree_mla import random_tree

pytestmark = pytest.mark.gpu
F32, BF16, U8 = torch.float32, torch.bfloat16, torch.uint8
H, D_N, D_R, D_C, D_V = 16, 128, 64, 512, 128
EPS = 1e-6


def rows_of(cache, bt, b, n):
    """Latents and rotary keys of the first n tokens of sequence b, as the cache holds them (fp64)."""
    at = torch.tensor(bt.rows_at(b, range(n)))
    kv = cache.kv.cpu()[at]
    lat = kv.double() if cache.kv_scale is None else R.dequantise(kv, cache.kv_scale.cpu()[at])
    return lat, cache.k_pe.cpu()[at].double()


def attend(bt, q_nope, q_pe, cache, W_UK, W_UV, T, first, masks, words):
    cu = [0]
    for t in T:
        cu.append(cu[-1] + t)
    seqs = dsa.Seqs(cu, bt.cu_k, first)
    scale = 1.0 / math.sqrt(D_N + D_R)
    mask = None
    if masks is not None:
        sign = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
        mask = torch.tensor([[sign(v >> 64 * w & (1 << 64) - 1) for w in range(words)] for m in masks for v in m]).cuda()
    out, lse = dsa.dsa_tree_mla_fwd(q_nope, q_pe, cache, W_UK, W_UV, seqs, scale, tree_mask=mask, pages=bt.pages())
    for b in range(len(T)):
        lat, pe = rows_of(cache, bt, b, first[b] + T[b])
        rows = slice(cu[b], cu[b + 1])
        heads = [0, H - 1]
        see = R.visible(T[b], first[b], None if masks is None else masks[b])
        ref, tol, l, lt = R.tree_attention(q_nope[rows][:, heads].cpu().double(), q_pe[rows][:, heads].cpu().double(), lat, pe,
                                           see, W_UK[heads].cpu().double(), W_UV[heads].cpu().double(), scale, R.U[BF16],
                                           exchange=True)
        got = out[rows][:, heads].cpu().double()
        assert torch.all((got - ref).abs() <= tol + R.U[BF16] * ref.abs())
        assert torch.all((lse[rows][:, heads].cpu().double() - l).abs() <= lt)
    return out, seqs


@pytest.mark.parametrize("cache_dt", [BF16, U8])
@pytest.mark.parametrize("page", [0, 32])
def test_draft_step(cache_dt, page):
    T, P = [7, 1, 66], [100, 33, 250]
    bt = R.Batch(T, P, page, seed=40, slack=2)
    g = torch.Generator().manual_seed(40)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n_pos = max(P) + max(T) + 8
    ang = torch.arange(n_pos).double()[:, None] * 10000.0 ** (-torch.arange(D_R // 2).double() / (D_R // 2))
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    kv = torch.zeros(bt.rows, D_C, dtype=cache_dt)
    cache = dsa.LatentCache(kv.cuda(), torch.zeros(bt.rows, D_R, dtype=BF16).cuda(),
                            torch.ones(bt.rows, D_C // 128).cuda() if cache_dt == U8 else None)
    W_UK, W_UV = (n(H, D_N, D_C) / math.sqrt(D_C)).to(BF16).cuda(), (n(H, D_C, D_V) / math.sqrt(D_C)).to(BF16).cuda()
    gain_q, gain_c = (1 + 0.1 * n(D_N + D_R)).cuda(), (1 + 0.1 * n(D_C)).cuda()
    pages = bt.pages()

    def keys(seqs, pos):
        """Norm latents and rotate rotary keys of new tokens, and write them."""
        c, pe = n(seqs.total_q, 1, D_C).to(BF16).cuda(), n(seqs.total_q, 1, D_R).to(BF16).cuda()
        # a norm alone has no rotary dims; the rotation alone no norm
        lat, _ = dsa.dsa_head_norm_rope(dsa.Heads(c, norm="rms", gain=gain_c), None, cos[:, :0].contiguous(),
                                        sin[:, :0].contiguous(), seqs, eps=EPS)
        rot, _ = dsa.dsa_head_norm_rope(dsa.Heads(pe, norm="none"), None, cos, sin, seqs, pos=pos)
        dsa.dsa_latent_cache_write(lat[:, 0], rot[:, 0], cache, seqs, pages=pages)
        return lat[:, 0], rot[:, 0]

    # the prompts
    prompt = dsa.Seqs([0] + [sum(P[:i + 1]) for i in range(len(P))], bt.cu_k, [0] * len(P))
    keys(prompt, None)
    # the drafts: a node sits at its depth
    masks = [random_tree(t, 41 + b) for b, t in enumerate(T)]
    depth = [bin(v).count("1") - 1 for m in masks for v in m]
    seq_of = [b for b, t in enumerate(T) for _ in range(t)]
    pos = torch.tensor([P[b] + d for b, d in zip(seq_of, depth)], dtype=torch.int32).cuda()
    seqs = bt.seqs()
    lat, rot = keys(seqs, pos)
    x = n(bt.N, H, D_N + D_R).to(BF16).cuda()
    (q_nope, q_pe), none = dsa.dsa_head_norm_rope(dsa.Heads(x, norm="rms", gain=gain_q), None, cos, sin, seqs, pos=pos,
                                                  eps=EPS, split=True)
    assert none is None
    keep, turn = R.norm_rope(x.cpu().double(), "rms", gain_q.cpu().double(), None, EPS, cos.cpu().double(),
                             sin.cpu().double(), pos.tolist(), "pairs", False)
    for got, want in ((q_nope, keep), (q_pe, turn)):
        # one rounding, and fp32 sums of 192 squares of values below 5
        assert torch.all((got.cpu().double() - want).abs() <= R.U[BF16] * want.abs() + 1e-4)
    words = -(-max(T) // 64)
    out, _ = attend(bt, q_nope, q_pe, cache, W_UK, W_UV, T, P, masks, words)

    # the accepted path: of each tree its last node's ancestors
    paths = [[j for j in range(t) if m[-1] >> j & 1] for t, m in zip(T, masks)]
    at = torch.tensor([P[b] + j for b, p in enumerate(paths) for j in p], dtype=torch.int32).cuda()
    cu = [0]
    for p in paths:
        cu.append(cu[-1] + len(p))
    accepted = dsa.Seqs(cu, bt.cu_k, P)
    c_path, pe_path = dsa.dsa_latent_cache_read(cache, accepted, pages=pages, pos=at)
    rows = [bt.cu_q[b] + j for b, p in enumerate(paths) for j in p]
    assert torch.equal(pe_path, rot[rows])
    if cache_dt == BF16:
        assert torch.equal(c_path, lat[rows])
    prefix = [rows_of(cache, bt, b, P[b]) for b in range(len(P))]
    dsa.dsa_latent_cache_write(c_path, pe_path, cache, accepted, pages=pages)
    for b, p in enumerate(paths):
        l, r = rows_of(cache, bt, b, P[b] + len(p))
        assert torch.equal(l[:P[b]], prefix[b][0]) and torch.equal(r[:P[b]], prefix[b][1])
        assert torch.equal(l[P[b]:], c_path[cu[b]:cu[b + 1]].cpu().double())
        assert torch.equal(r[P[b]:], pe_path[cu[b]:cu[b + 1]].cpu().double())

    # the path as a chain is what the tree said of its nodes: the last node again, now over the moved keys
    last = torch.tensor([bt.cu_q[b + 1] - 1 for b in range(len(T))])
    first = [P[b] + len(p) - 1 for b, p in enumerate(paths)]
    again, _ = attend(bt, q_nope[last.cuda()].contiguous(), q_pe[last.cuda()].contiguous(), cache, W_UK, W_UV, [1] * len(T), first,
                      None, 0)
    # both are within their bands of one value (checked above), which are a few roundings wide
    a, b = again.double(), out[last.cuda()].double()
    assert torch.all((a - b).abs() <= 0.03 * b.abs().amax(-1, keepdim=True))
