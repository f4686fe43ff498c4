"""What a norm's sums leave out, which a bound by the width does not show.

A thread adds at most 32 squares one after the other, two shuffles of five steps and a product with 1 / D (itself off by
2^-24) follow: a sum of squares is off by at most (32 + 10 + 3) 2^-24 of itself, its root's inverse by half of that and rsqrt's
two units (4 of 2^-24), and the products with it and the gain add two more: 29 of 2^-24 of a value (E is 32).  The mean is off by (32 + 10 + 2)
2^-24 of the mean of the absolute values, and the subtraction by 2^-24 of its result and that of the mean; a bias adds a rounding of what it gives.
A value that no sum takes in shows in a row in which it is nearly all of the sum."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import next_token_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
E = 32 * 2.0 ** -24
WIDTHS = [1, 3, 32, 33, 253, 254, 256, 264, 509, 510, 1025, 1536, 2049, 4093, 4097, 5120, 5128, 7167, 7168, 8192, 8200, 10001, 16381, 16383, 16384]


def check(y, v, kind, gain, bias, rounding):
    v = v.double()
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
    inv = 1 / ((v - mean).pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    scale = inv * (1.0 if gain is None else gain.double().abs())
    want = R.norm(v, kind, gain, bias, 1e-6)
    slack = rounding * want.abs() + E * (v - mean).abs() * scale
    if kind == "layer":
        slack = slack + 48 * 2.0 ** -24 * v.abs().mean(-1, keepdim=True) * scale + 2.0 ** -23 * want.abs()
    over = (y.double() - want).abs() - slack
    assert float(over.max()) <= 0, f"off by {float(over.max()):.3e} more than derived"


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("h_dt", [F32, BF16])
@pytest.mark.parametrize("N", [5, 400])
@pytest.mark.parametrize("D", WIDTHS)
def test_sums_to_the_last_digits(D, N, h_dt, kind):
    """fp32 results of rows of ordinary values; of both norms."""
    g = torch.Generator(device="cuda").manual_seed(D + N)
    h = (1 + 3 * torch.randn(N, D, generator=g, device="cuda")).to(h_dt)
    gain, bias = 1 + 0.2 * torch.randn(D, generator=g, device="cuda"), torch.randn(D, generator=g, device="cuda")
    bias = bias if kind == "layer" else None
    got = dsa.dsa_block_norm(h, dsa.Norm(kind, gain, bias), dtype=F32, want_h=False)[1]
    check(got, h, kind, gain, bias, 2.0 ** -24)
    u = h.float()
    got = dsa.dsa_block_norm(torch.zeros_like(u), u=u, post=dsa.Norm(kind, gain, bias), want_y=False)[0]
    check(got, u, kind, gain, bias, 2.0 ** -24)


@pytest.mark.parametrize("h_dt,x_dt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("D", WIDTHS)
def test_every_value_is_in_the_sum(D, h_dt, x_dt):
    """Row r holds one value that is nearly all of its sums, in column r: for every column, in few rows and in many."""
    h = torch.randn(D, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(D)).to(h_dt)
    h.diagonal().fill_(512.0 if D <= 256 else 4096.0)
    for parts in ([(0, D)], [(a, min(D, a + 100)) for a in range(0, D, 100)]):
        for a, b in parts:
            rows = h[a:b]
            y = dsa.dsa_block_norm(rows, dsa.Norm("rms"), dtype=x_dt, want_h=False)[1]
            for c in range(0, b - a, 2048):
                check(y[c:c + 2048], rows[c:c + 2048], "rms", None, None, R.U[x_dt])
            if x_dt == h_dt:
                v = dsa.dsa_block_norm(torch.zeros_like(rows), u=rows, post=dsa.Norm("layer"), want_y=False)[0]
                for c in range(0, b - a, 2048):
                    check(v[c:c + 2048], rows[c:c + 2048], "layer", None, None, R.U[h_dt])
