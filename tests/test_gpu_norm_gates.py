"""Gates of the norms around a block: their digits, and gates that share memory with what they gate."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import next_token_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("h_dt,x_dt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("D", [5, 201, 509, 2049, 4097, 9999])
@pytest.mark.parametrize("N", [1, 2, 7, 300])
def test_gate_that_is_the_block_output(N, D, h_dt, x_dt):
    """u as its own gate, and u's first row as the gate of all rows, where u starts elsewhere within 16 bytes than the stream and
    its rows are as far apart or not: no call reads u by the stream's alignment.  h' adds one to the other, rounded a few
    times in fp32 and once to its type."""
    g = torch.Generator(device="cuda").manual_seed(N + D)
    for off in range(4):
        for pad in (0, 1, 3, 4):
            buf = torch.randn(N, D + 8 + pad, generator=g, device="cuda").to(x_dt)
            h, u = torch.randn(N, D + 8, generator=g, device="cuda").to(h_dt)[:, :D], buf[:, off:off + D]
            for gate in (u, u[:1], buf[:1, 1:1 + D]):
                got, y = dsa.dsa_block_norm(h, u=u, gate=gate)
                want = h.double() + u.double() * gate.double()
                slack = 2.0 ** -23 * (h.double().abs() + (u.double() * gate.double()).abs())
                assert float(((got.double() - want).abs() - R.U[h_dt] * want.abs() - slack).max()) <= 0
                assert float(((y.double() - want).abs() - R.U[x_dt] * want.abs() - slack).max()) <= 0
        one = torch.randn(1, D + 8, generator=g, device="cuda").to(x_dt)[:, off:off + D].expand(N, D)
        got, _ = dsa.dsa_block_norm(h, u=one, gate=one)
        want = h.double() + one.double() ** 2
        assert float(((got.double() - want).abs() - R.U[h_dt] * want.abs() - 2.0 ** -23 * (h.double().abs() + one.double() ** 2)).max()) <= 0


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("x_dt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 1000, 2049, 4096, 7168, 16384])
def test_gates_of_an_fp32_stream(D, x_dt, act):
    """h' = gate alone, in fp32 whatever the gate's type: expf is good to 1 unit of 2^-23, 1 + e to a rounding, the quotient to 2
    units, silu's product, u's and the sum round once each: 3.5 + 1.5 units at most."""
    gate = torch.linspace(-80, 80, 7 * D, device="cuda").reshape(7, D).to(x_dt)
    h, u = torch.zeros(7, D, device="cuda"), torch.ones(7, D, dtype=x_dt, device="cuda")
    for g in (gate, gate[3:4]):
        got = dsa.dsa_block_norm(h, u=u, gate=g, gate_act=act, want_y=False)[0]
        want = R.act(g.double(), act)
        over = (got.double() - want).abs() / want.abs().clamp(min=2.0 ** -110)
        assert got.dtype == F32 and got.shape == h.shape
        assert float(over.max()) <= 5 * 2.0 ** -23, f"{float(over.max()) * 2 ** 23:.1f} units"
