"""The operators between two attentions and after the last as a step uses them, one after another: the attention's
output through wo onto the residual stream, the norms around the next block, a layer of that block with its gate, the
final norm, the logits, and the next token of every sequence.

Each stage is held to the 64-bit form of what the stage before it left."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as L
from tests import next_token_reference as R
from tests.test_gpu_block_norm import check as check_norm
from tests.test_gpu_linear import check as check_linear

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
H, D_N, D_R, D_C, D_V, DIM, V = 16, 128, 64, 512, 128, 1536, 5003


def weights(g):
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(UK=(r(H, D_N, D_C) / math.sqrt(D_C)).bfloat16(), UV=(r(H, D_C, D_V) / math.sqrt(D_C)).bfloat16(),
                wo=(r(DIM, H * D_V) / math.sqrt(H * D_V)).bfloat16(), up=(r(DIM, DIM) / math.sqrt(DIM)).bfloat16(),
                gate=(r(DIM, DIM) / math.sqrt(DIM)).bfloat16(), bias=0.1 * r(DIM), head=(r(V, DIM) / math.sqrt(DIM)).bfloat16(),
                gain=[1 + 0.1 * r(DIM) for _ in range(3)])


@pytest.mark.parametrize("B", [1, 37])
def test_end_of_step(B):
    g = torch.Generator(device="cuda").manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    w = weights(g)
    P = [20 + 7 * b for b in range(B)]
    bt = L.Batch([1] * B, P, 32, seed=B)
    rows = bt.rows
    cache = dsa.LatentCache(r(rows, D_C).bfloat16(), r(rows, D_R).bfloat16())
    seqs = dsa.Seqs(list(range(B + 1)), bt.cu_k, P)
    pages = bt.pages()
    q_nope, q_pe, h = r(B, H, D_N).bfloat16(), r(B, H, D_R).bfloat16(), r(B, DIM).bfloat16()
    u, T, p = torch.rand(B, generator=g, device="cuda"), torch.full((B,), 0.8, device="cuda"), torch.full((B,), 0.9, device="cuda")

    def run():
        out, _ = dsa.dsa_tree_mla_fwd(q_nope, q_pe, cache, w["UK"], w["UV"], seqs, 1 / math.sqrt(D_N + D_R), pages=pages)
        flat = out.view(B, H * D_V)
        h1 = dsa.dsa_linear(flat, w["wo"], residual=h)
        _, x = dsa.dsa_block_norm(h1, dsa.Norm("rms", w["gain"][0]), want_h=False)
        a = dsa.dsa_linear(x, w["up"], bias=w["bias"], act="silu")
        gt = dsa.dsa_linear(x, w["gate"])
        h2, y = dsa.dsa_block_norm(h1, dsa.Norm("rms", w["gain"][2]), u=a, post=dsa.Norm("rms", w["gain"][1]), gate=gt,
                                   gate_act="sigmoid", scale=0.5)
        logits = dsa.dsa_linear(y, w["head"], dtype=F32)
        return (flat, h1, x, a, gt, h2, y, logits) + dsa.dsa_sample(logits, u, temperature=T, top_p=p, want_kept=True)

    flat, h1, x, a, gt, h2, y, logits, token, logprob, kept = got = run()
    none = ("none", None, None)
    gains = [("rms", v, None) for v in w["gain"]]
    check_linear(h1, flat, w["wo"], res=h)
    check_norm((None, x), h1, None, None, None, none, gains[0], 1.0, 1.0, 1e-6, (BF16, BF16))
    check_linear(a, x, w["up"], w["bias"], "silu")
    check_linear(gt, x, w["gate"])
    check_norm((h2, y), h1, a, gt, "sigmoid", gains[1], gains[2], 1.0, 0.5, 1e-6, (BF16, BF16))
    check_linear(logits, y, w["head"])
    f = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
    for b in range(B):
        want = R.sample_row(logits[b], float(u[b]), f(0.8), 0, f(0.9), 0.0)
        assert (int(token[b]), int(kept[b])) == want[::2]
        assert abs(float(logprob[b]) - want[1]) <= 8 * 2.0 ** -24 * (abs(want[1]) + 2.0 ** -20)
    # the same step from a graph, on the next inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = run()
    q_nope.copy_(q_nope.flip(0))
    h.mul_(0.5)
    want = [t.clone() for t in run()]
    graph.replay()
    torch.cuda.synchronize()
    for i, j in zip(again, want):
        assert torch.equal(i, j)
    assert not torch.equal(want[7], got[7])


def test_sizes_that_do_not_fit_32_bits_are_refused():
    """Views of 2^32 + 3 rows or columns (of one row's memory) would otherwise count as 3."""
    many = 2 ** 32 + 3
    x, w = torch.zeros(1, 8, device="cuda", dtype=BF16), torch.zeros(4, 8, device="cuda", dtype=BF16)
    wide = torch.zeros(1, 1, device="cuda", dtype=BF16).expand(2, many)
    for call in (lambda: dsa.dsa_linear(x.expand(many, 8), w), lambda: dsa.dsa_linear(x, w[:1].expand(many, 8)),
                 lambda: dsa.dsa_linear_workspace_size(x.expand(many, 8), w), lambda: dsa.dsa_linear(wide, wide),
                 lambda: dsa.dsa_sample(x.expand(many, 8), torch.zeros(3, device="cuda")),
                 lambda: dsa.dsa_sample(wide, torch.zeros(2, device="cuda")), lambda: dsa.dsa_block_norm(wide)):
        with pytest.raises(ValueError):
            call()
        torch.cuda.synchronize()
