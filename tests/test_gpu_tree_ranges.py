"""Tree attention over latents and block scales at the end of their range (bands: see latent_reference, without a term
for the exchange of half scores)."""
import math

import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R
from tests.test_gpu_tree_mla import Case, TC

pytestmark = pytest.mark.gpu
BF16, U8 = torch.bfloat16, torch.uint8


@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("masks", ["tree", "chain", "odd"])
@pytest.mark.parametrize("P", [64, 70, 700])
def test_large_scales_beside_hidden_tokens(generic, masks, P, monkeypatch):
    """Tokens that rows see, with scales up to the largest one (2^120, small codes), in a tile with tokens that rows do
    not see (other nodes; rows behind the last token, whose scales are Inf)."""
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    c = Case([5], [P], 16, 4, TC, BF16, U8, masks, seed=60, slack=2)
    g = torch.Generator().manual_seed(60)
    n = P + 5
    for r in c.bt.rows_at(0, range(n // 64 * 64, n)):
        if not torch.isfinite(c.sc[r, 0]):
            continue  # seen by nobody
        # subnormal codes: 1 to 7 times 2^-9
        c.kv[r] = (torch.randint(1, 8, (512,), generator=g) | 128 * torch.randint(0, 2, (512,), generator=g)).to(U8)
        c.sc[r] = torch.tensor([2.0 ** 120, 2.0 ** 119, 2.0 ** 100, 2.0 ** 118])
    c.lat = R.dequantise(c.kv, c.sc)
    c.q_nope = (c.q_nope.float() * 2.0 ** -112).to(BF16)  # scores of the usual size
    out, lse = c.call()
    assert ("tree_simt" if generic else "tree_tc") in dsa.last_kernels()
    c.check(out, lse, exchange=False)


@pytest.mark.parametrize("generic", [False, True])
def test_large_values_written_and_attended(generic, monkeypatch):
    """A decode step whose new token's values make scales of 2^119.  Queries of 0 weigh all 65 tokens alike: its values
    are the mean's, up to two roundings to bf16 (context, output; W_UV picks 128 of the columns)."""
    if generic:
        monkeypatch.setenv("DSA_FORCE_GENERIC", "1")
    g = torch.Generator().manual_seed(61)
    kv = torch.randint(0, 120, (80, 512), generator=g).to(U8).cuda()
    cache = dsa.LatentCache(kv, torch.zeros(80, 64, dtype=BF16, device="cuda"), torch.ones(80, 4, device="cuda"))
    seqs = dsa.Seqs([0, 1], [0, 65], [64])
    x = (1.5e38 + 0.1e38 * torch.rand(1, 512, generator=g)).to(BF16) * (1 - 2 * torch.randint(0, 2, (1, 512), generator=g)).to(BF16)
    dsa.dsa_latent_cache_write(x.cuda(), torch.zeros(1, 64, dtype=BF16, device="cuda"), cache, seqs)
    assert torch.all(cache.kv_scale[64] == 2.0 ** 119)
    lat = R.dequantise(cache.kv.cpu(), cache.kv_scale.cpu())[:65]
    W_UK = torch.zeros(2, 128, 512, dtype=BF16, device="cuda")
    W_UV = torch.zeros(2, 512, 128, dtype=BF16, device="cuda")
    for h in range(2):
        W_UV[h, 256 * h:256 * h + 128] = torch.eye(128, device="cuda").to(BF16)
    zero = lambda d: torch.zeros(1, 2, d, dtype=BF16, device="cuda")  # noqa: E731
    out, lse = dsa.dsa_tree_mla_fwd(zero(128), zero(64), cache, W_UK, W_UV, seqs, 0.07)
    for h in range(2):
        want = lat[:, 256 * h:256 * h + 128].mean(0)
        assert torch.all((out[0, h].cpu().double() - want).abs() <= 2.02 * 2.0 ** -8 * want.abs())
        assert abs(float(lse[0, h]) - math.log(65)) <= 1e-5
