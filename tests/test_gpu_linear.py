"""The linear layer with its epilogue against the 64-bit form.

A result is rounded once to its type (U).  Before that a sum of K products passes through at most K / 16 + 32 additions
of which each may cut off 2^-23 of what it adds to, which is never above the sum A of the absolute products; fp32 layers
add six products of terms, 6 K / 16 such steps, and leave out terms of at most 2^-25 A in all.  Results in fp32 are
summed in parts of 32 such steps, which are added to nearest (few tokens: K / 32 steps a lane, each to nearest, half of 2^-23).
No activation moves by more than 1.13 where its argument moves by 1, and its own arithmetic adds a few roundings of its
argument and result."""
import pytest
import torch

import sparse_latent_attention_indexer_gb300 as dsa
from tests import next_token_reference as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def bound(y, spread, K, dt, out):
    steps = (6 if dt == F32 else 1) * K / 16 + 32
    if out == F32:
        steps = min(steps, 64 + steps / 32 + K / 64)
    return R.U[out] * y.abs() + 1.13 * (steps * 2.0 ** -23 + 2.0 ** -25) * spread + 2.0 ** -20 * spread.clamp(max=1) + 2.0 ** -21 * y.abs()


def check(got, x, w, bias=None, act=None, res=None):
    want, spread = R.linear(x, w, bias, act, res)
    assert got.shape == want.shape
    over = (got.double() - want).abs() - bound(want, spread, x.shape[1], x.dtype, got.dtype)
    assert float(over.max()) <= 0, f"off by {float(over.max()):.3e} more than derived"


def make(M, N, K, dt, seed=0, bias=False, res=None):
    g = torch.Generator(device="cuda").manual_seed(1000 * M + 10 * N + K + seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(dt)
    w = (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).to(dt)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    r = torch.randn(M, N, generator=g, device="cuda").to(res) if res else None
    return x, w, b, r


SIZES = [(1, 1, 1), (1, 128, 64), (1, 300, 8), (3, 129, 65), (15, 64, 1000), (16, 127, 200), (17, 1000, 7), (31, 260, 512),
         (33, 8, 2048), (64, 768, 4096), (100, 5, 63), (255, 257, 72), (256, 128, 640), (257, 131, 129), (300, 1024, 96),
         (513, 40, 2), (1000, 136, 264), (60, 1000, 1001), (40, 130, 16384), (7, 72, 20001), (5, 2500, 2999), (20, 2000, 1999),
         (80, 500, 576), (81, 129, 257), (161, 300, 64), (400, 5200, 4100),
         (1000, 520, 1040), (2000, 250, 640)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(M, N, K, dt, out):
    x, w, b, r = make(M, N, K, dt, bias=M % 2 == 1, res=out if N % 2 == 1 else None)
    act = ACTS[(M + N + K) % 5]
    got = dsa.dsa_linear(x, w, bias=b, act=act, residual=r, dtype=out)
    assert got.dtype == out
    check(got, x, w, b, act, r)
    kernels = dsa.last_kernels()
    if dt == BF16 and K % 8 == 0:
        assert kernels == {"linear"}
    elif (dt == F32 or N > 1) and (M <= 4 or (M <= 64 and M * N * K <= (3.5e7 if dt == F32 else 6e6))):
        assert kernels == {"linear_simt"}
    elif dt == F32 and K % 4 == 0 and K <= 4096 and M * N * K <= 3e8:
        assert kernels == {"linear"}
    elif N > 1:
        assert kernels == {"linear", "linear_layout"}


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M", [4, 40, 700])
def test_epilogues(M, dt, act):
    for bias in (False, True):
        for res in (None, dt):
            x, w, b, r = make(M, 392, 320, dt, seed=7, bias=bias, res=res)
            check(dsa.dsa_linear(x * 3, w, bias=b, act=act, residual=r), x * 3, w, b, act, r)


@pytest.mark.parametrize("M,N,K", [(1, 7168, 1536), (64, 7168, 2048), (9, 20000, 128), (2048, 1536, 512), (300, 4104, 1024)])
def test_many_tiles_and_shared_ones(M, N, K):
    """Tiles on every SM and more, and tiles whose K a cluster shares; the same call gives the same bits."""
    x, w, b, r = make(M, N, K, BF16, bias=True, res=F32)
    got = dsa.dsa_linear(x, w, bias=b, residual=r)
    check(got, x, w, b, None, r)
    for _ in range(3):
        assert torch.equal(dsa.dsa_linear(x, w, bias=b, residual=r), got)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M", [2, 16, 50])
def test_strides(M, dt):
    """Column slices of wider tensors, on and off 16 bytes, one row for all of x; what lies beside y stays."""
    N, K = 130, 136
    g = torch.Generator(device="cuda").manual_seed(M)
    for off in (0, 1, 8):
        wide = lambda n, k: torch.randn(n, k + 24, generator=g, device="cuda").to(dt)  # noqa: E731
        bx, bw, by, br = wide(M, K), wide(N, K), wide(M, N), wide(M, N)
        x, w, y, r = bx[:, off:off + K], bw[:, off:off + K], by[:, off:off + N], br[:, off:off + N]
        before = by.clone()
        assert dsa.dsa_linear(x, w, act="silu", residual=r, y=y) is y
        check(y, x, w, None, "silu", r)
        assert torch.equal(by[:, :off], before[:, :off]) and torch.equal(by[:, off + N:], before[:, off + N:])
        same = bx[:1, off:off + K].expand(M, K)
        check(dsa.dsa_linear(same, w), same, w)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(100, 200, 301), (130, 150, 1040), (3, 70, 77)])
def test_rows_at_every_offset(M, N, K, dt):
    """Rows that start anywhere within 16 bytes, with NaN beside each."""
    x, w, _, _ = make(M, N, K, dt)
    for off in range(9):
        bufs = [torch.full((n, K + 10 + off % 2), float("nan"), dtype=dt, device="cuda") for n in (M, N)]
        cx, cw = bufs[0][:, off:off + K].copy_(x), bufs[1][:, 8 - off:8 - off + K].copy_(w)
        check(dsa.dsa_linear(cx, cw), x, w)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(5, 2048, 4096), (16, 2049, 4099), (17, 4100, 2052), (33, 20000, 448), (50, 9000, 1000), (64, 3000, 7001),
                                   (48, 140000, 60), (63, 40000, 321)])
def test_few_tokens_of_a_large_fp32_layer(M, N, K, out):
    """W read as it is: rows with NaN beside them, every part of the epilogue, y over the residual, the same bits again."""
    x, w, b, r = make(M, N, K, F32, bias=True, res=out)
    ld = (K + 7) // 4 * 4
    bufs = [torch.full((n, ld), float("nan"), device="cuda") for n in (M, N)]
    cx, cw = bufs[0][:, :K].copy_(x), bufs[1][:, :K].copy_(w)
    assert dsa.dsa_linear_workspace_size(cx, cw) == 0
    y = r.clone()
    assert dsa.dsa_linear(cx, cw, bias=b, act="silu", residual=y, y=y) is y and dsa.last_kernels() == {"linear"}
    check(y, x, w, b, "silu", r)
    assert torch.equal(dsa.dsa_linear(cx, cw, bias=b, act="silu", residual=r), y)
    check(dsa.dsa_linear(cx, cw, dtype=out), x, w)
    cx[1, 5], cw[7, 9] = float("nan"), float("inf")
    got = dsa.dsa_linear(cx, cw, bias=b, act="silu", residual=r)
    assert bool(got[1].isnan().all()) and not bool(got[:, 7].isfinite().any())
    rows, cols = [i for i in range(M) if i != 1], [i for i in range(N) if i != 7]
    assert torch.equal(got[rows][:, cols], y[rows][:, cols])


@pytest.mark.parametrize("M", [1, 20, 600])
def test_in_place_residual(M):
    x, w, b, r = make(M, 264, 192, BF16, bias=True, res=BF16)
    want = dsa.dsa_linear(x, w, bias=b, act="gelu", residual=r)
    y = r.clone()
    assert dsa.dsa_linear(x, w, bias=b, act="gelu", residual=y, y=y) is y
    assert torch.equal(y, want)


def test_rows_behind_the_last_stay():
    """M and N end inside a tile: nothing behind them is written."""
    for M, N, K, dt in ((5, 130, 64, BF16), (200, 100, 72, BF16), (300, 132, 40, F32), (7, 33, 20, F32)):
        buf = torch.full((M + 40, N + 60), 7.0, dtype=dt, device="cuda")
        x, w, _, _ = make(M, N, K, dt)
        dsa.dsa_linear(x, w, y=buf[:M, :N])
        check(buf[:M, :N], x, w)
        assert bool((buf[M:] == 7).all()) and bool((buf[:, N:] == 7).all())


@pytest.mark.parametrize("M", [3, 40, 400])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_nan_and_infinity_stay_in_their_rows(M, dt):
    """A NaN or infinity of a token or feature reaches that row or column and no other."""
    x, w, _, _ = make(M, 260, 128, dt)
    clean = dsa.dsa_linear(x, w)
    x[1, 5], x[2, 0], w[7, 9] = float("nan"), float("inf"), float("nan")
    got = dsa.dsa_linear(x, w, act="relu")
    assert bool(got[1].isnan().all()) and bool(got[:, 7].isnan().all())
    assert not bool(got[2].isfinite().all())
    rows = [i for i in range(M) if i not in (1, 2)]
    cols = [i for i in range(260) if i != 7]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols].clamp(min=0))


def test_fp32_values_at_the_ends_of_their_range():
    """Numbers that the nearest bf16 would make infinite, and small ones, keep their digits."""
    K = 64
    x = torch.zeros(20, K, device="cuda")
    w = torch.zeros(30, K, device="cuda")
    x[:, 0] = 3.4028234e38
    x[:, 1] = 1.2345678e-20
    w[:, 0] = torch.linspace(0.01, 0.99, 30, device="cuda")
    w[5:, 1] = 9.8765432e-3
    check(dsa.dsa_linear(x, w), x, w)
    x[:, 0] = 0
    got = dsa.dsa_linear(x, w)
    want = x.double() @ w.double().T
    assert float(((got - want).abs() - 2.0 ** -21 * want.abs()).max()) <= 0


def test_zero_rows_and_empty_batches():
    x, w, b, _ = make(4, 72, 64, BF16, bias=True)
    assert dsa.dsa_linear(x[:0], w).shape == (0, 72) and dsa.last_launch_count() == 0
    got = dsa.dsa_linear(torch.zeros_like(x), w, bias=b, dtype=F32)
    assert torch.equal(got, b.expand(4, 72))


def test_offsets_past_32_bits():
    """y of more than 2^31 values, and x and W whose rows lie further than 2^31 apart."""
    M, N, K = 16500, 131072, 64
    x, w, _, _ = make(M, N, K, BF16)
    got = dsa.dsa_linear(x, w)
    rows = torch.tensor([0, 1, 8191, 16384, 16499], device="cuda")
    check(got[rows], x[rows], w)
    del got
    far = torch.zeros(3, 1200000000, dtype=BF16, device="cuda")
    x, w, _, _ = make(3, 40, 64, BF16)
    far[:, 8:72] = x
    check(dsa.dsa_linear(far[:, 8:72], w), x, w)
    far[:, 1:65] = x
    check(dsa.dsa_linear(w, far[:, 1:65]), w, x)


def test_streams_and_graphs():
    """Another stream than the current one; two captured calls with a workspace of their own, replayed on new inputs."""
    side = torch.cuda.Stream()
    for M, K, dt in ((40, 129, BF16), (300, 256, BF16), (50, 96, F32), (3, 96, F32)):
        x, w, b, _ = make(M, 200, K, dt, bias=True)
        want = dsa.dsa_linear(x, w, bias=b)
        torch.cuda.synchronize()
        got = dsa.dsa_linear(x, w, bias=b, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
        need = dsa.dsa_linear_workspace_size(x, w)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                y = dsa.dsa_linear(x, w, bias=b, workspace=ws)
            graphs.append((g, y))
        x.copy_(x.flip(0))
        for g, y in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, y in graphs:
            assert torch.equal(y, want.flip(0))


@pytest.mark.parametrize("M,N,K,dt,out", [(64, 7168, 16384, BF16, BF16), (16, 1024, 16384, BF16, F32), (700, 4096, 8192, BF16, BF16),
                                          (300, 8000, 8192, BF16, F32), (70, 1024, 8192, F32, F32), (900, 2048, 4096, F32, BF16),
                                          (40, 4096, 8192, F32, F32), (64, 40000, 4096, F32, BF16), (10, 40000, 4096, F32, F32)])
def test_waits_that_run_out_are_reported(M, N, K, dt, out):
    """Clusters that share a tile and the persistent kernel, summed in parts or not: with a limit of 64 cycles on their waits
    they give up, drain and leave; the device reports it, and the next call gives the same bits as before."""
    from sparse_latent_attention_indexer_gb300 import _abi

    x, w, b, _ = make(M, N, K, dt, bias=True)
    want = dsa.dsa_linear(x, w, bias=b, dtype=out)
    torch.cuda.synchronize()
    assert dsa.dsa_check_device_error()[0] == _abi.DSA_OK
    try:
        dsa.dsa_set_wait_limit(64)
        dsa.dsa_linear(x, w, bias=b, dtype=out)
        status, site = dsa.dsa_check_device_error()
    finally:
        dsa.dsa_set_wait_limit(0)
    # a sum in parts waits for eight slabs at a time, and warps that make the slabs
    # themselves for one, which may be there within the hardware's own patience
    assert (status == _abi.DSA_ERR_TIMEOUT and 61 <= site <= 66) or ((out == F32 or (dt == F32 and M <= 64)) and status == _abi.DSA_OK)
    assert torch.equal(dsa.dsa_linear(x, w, bias=b, dtype=out), want)
    assert dsa.dsa_check_device_error()[0] == _abi.DSA_OK
