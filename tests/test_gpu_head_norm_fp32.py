"""Per-head norm and rotation held to what fp32 arithmetic may lose, so that a norm or rotation done in fewer bits shows.

With u = 2^-24, for heads of up to 512 values that are summed in chains of at most 32, then in at most 5 steps:
  RMS     the sum of squares (no cancellation) is off by at most 37 u of itself, with 1/D, the product and eps 40 u; the
          root halves that; rsqrtf adds 2 ulp (CUDA's documented bound, 4 u), two products 2 u: 26 u of the result.
  layer   the mean is off by at most 39 u of the mean size of the values (which moves the deviations, not the variance,
          to first order); subtracting adds u of the deviation: 27 u of the normed value, 39 u gain / sigma times the
          mean size of the values, and u of the sum with the bias.
  turn    each value's own error through cos and sin, and 3 u of the two products.
Then the one rounding to the output's type.  (Rounding to fp16 on the way would be 2^-11: 8000 u.)"""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import latent_reference as R
from tests.test_gpu_head_norm import CASES, tables

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
u = 2.0 ** -24


def error_of_norm(x, norm, gain, bias, eps):
    """What the normed heads [N, n, D] (64 bits) may be off by."""
    if norm == "none":
        return x, torch.zeros_like(x)
    g = torch.ones(x.shape[-1]).double() if gain is None else gain.double()
    if norm == "rms":
        y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * g
        return y, 26 * u * y.abs()
    sigma = (x.var(-1, unbiased=False, keepdim=True) + eps).sqrt()
    z = (x - x.mean(-1, keepdim=True)) / sigma * g
    y = z + (0.0 if bias is None else bias.double())
    return y, 27 * u * z.abs() + 39 * u * g.abs() / sigma * x.abs().mean(-1, keepdim=True) + u * y.abs()


def check(got, x, norm, gain, bias, eps, cos, sin, pos, rope, first, y_dt):
    """`got`: all D dims, the rotary ones first or last."""
    y, e = error_of_norm(x.double(), norm, gain, bias, eps)
    D, d_r = x.shape[2], 2 * cos.shape[1]
    keep, turn = R.norm_rope(y, "none", None, None, eps, cos.double(), sin.double(), pos, rope, first)
    e_keep, _ = R.norm_rope(e, "none", None, None, eps, cos.double(), sin.double(), pos, rope, first)
    at = 0 if first else D - d_r
    part = lambda t: ((t[..., ::2], t[..., 1::2]) if rope == "pairs" else (t[..., :d_r // 2], t[..., d_r // 2:]))  # noqa: E731
    (a, b), (ea, eb) = part(y[..., at:at + d_r]), part(e[..., at:at + d_r])
    ok = torch.tensor([0 <= p < cos.shape[0] for p in pos])[:, None, None]
    p0 = [p if 0 <= p < cos.shape[0] else 0 for p in pos]
    c = torch.where(ok, cos.double()[p0][:, None].abs(), torch.ones(()).double())
    s = torch.where(ok, sin.double()[p0][:, None].abs(), torch.zeros(()).double())
    e_turn = torch.cat([(ea + 3 * u * a.abs()) * c + (eb + 3 * u * b.abs()) * s,
                        (ea + 3 * u * a.abs()) * s + (eb + 3 * u * b.abs()) * c], -1)
    want, band = (torch.cat([t, k] if first else [k, t], -1) for k, t in ((keep, turn), (e_keep, e_turn)))
    err = (got.cpu().double() - want).abs()
    band = band + R.U[y_dt] * (want.abs() + band)
    assert torch.all(err <= band), f"{(err / band.clamp(min=1e-300)).max():.2f} of the band"


@pytest.mark.parametrize("x_dt,y_dt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("size,shift,pad", [(1.0, 0.0, 0), (1.0, 50.0, 0), (1e-4, 0.0, 1), (1e4, 0.0, 0)])
def test_fp32_arithmetic(case, x_dt, y_dt, size, shift, pad):
    """Values of any size, with a mean far above their spread; pad 1: rows off 16 bytes (one warp a head)."""
    D, d_r, Hq, Hk, nq, nk, rope, first, _ = case
    g = torch.Generator().manual_seed(7 * D + d_r)
    N, cos, sin = 17, *tables(45, d_r)
    pos = [int(v) for v in torch.randint(-1, 46, (N,), generator=g)]
    seqs = dsa.Seqs([0, 3, N], [0, 20, 50], [0, 5])
    parts = []
    for n, norm in ((Hq, nq), (Hk, nk)):
        if n:
            x = (torch.randn(N, n, D, generator=g) * size + shift).to(x_dt)
            gain = 1 + 0.2 * torch.randn(D, generator=g) if norm != "none" else None
            bias = torch.randn(D, generator=g) if norm == "layer" else None
            parts.append((x, norm, gain, bias))

    def heads(x, norm, gain, bias):
        buf = torch.zeros(N, x.shape[1] * D + pad, dtype=x_dt, device="cuda")
        view = buf[:, pad:].unflatten(1, (x.shape[1], D))
        view.copy_(x)
        return dsa.Heads(view, norm, *(None if t is None else t.cuda() for t in (gain, bias)))

    got = dsa.dsa_head_norm_rope(heads(*parts[0]), heads(*parts[1]) if len(parts) > 1 else None, cos.cuda(), sin.cuda(), seqs,
                                 pos=torch.tensor(pos, dtype=torch.int32).cuda(), rope=rope, rope_first=first, dtype=y_dt)
    for p, r in zip(parts, got):
        check(r, *p, 1e-6, cos, sin, pos, rope, first, y_dt)
