"""int8 products on the GPU against the definition in 64 bits (serving_ref).

Tolerance: the integer sum is exact; the two scale products and the bias add
round in fp32 (three operations, 2^-24 each) and the result once to the
element type."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from group_wise_affine_amd.devio import TORCH_DT
from tests import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def rows(M, K, dt, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (sigma * torch.randn(M, K, generator=g)).to(TORCH_DT[dt])


def check(y, y64, mag, dt, what):
    y = y.double().cpu().numpy()
    tol = R.UNIT[dt] * np.abs(y64) * (1 + 2.0 ** -10) + 4 * 2.0 ** -24 * mag + R.TINY[dt]
    bad = np.abs(y - y64) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(y - y64)[bad].max()}"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (5, 2048), (2, 2064), (7, 8192), (2, 8208), (1, 40000)])
def test_quantize_rows(M, K, dt):
    x = rows(M, K, dt, M + K)
    x[0, : K // 2] *= 30
    c, s = Q.i8_quantize(x.cuda())
    rc, rs = R.i8_quantize(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(c.cpu().numpy(), rc)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_quantize_ties_zeros_and_extremes(dt):
    """Quotients on and next to half-integers, zero rows, the smallest and the
    largest finite values, infinities and NaN."""
    x = torch.zeros(9, 256)
    x[0] = torch.arange(256) - 128.0            # amax 128: nothing divides evenly
    x[1] = (torch.arange(256) - 127.0) * 0.5    # amax 64
    x[2, 0], x[2, 1:255] = 254.0, torch.arange(254) + 1.0   # scale 2: every odd value a tie
    x[3] = 2.0 ** -24 if dt == "f16" else 2.0 ** -133       # subnormal
    x[3, ::2] = 0
    x[4, 5] = 65504.0 if dt == "f16" else 3.38953e38
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7] = torch.linspace(-1, 1, 256)
    x = x.to(TORCH_DT[dt])
    c, s = Q.i8_quantize(x.cuda())
    rc, rs = R.i8_quantize(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.isnan(rs[5]) and np.isnan(rs[6]) and rs[8] == 0
    assert np.array_equal(c.cpu().numpy(), rc)


def test_quantize_strided_rows():
    x = rows(9, 512, "bf16", 3).cuda()
    part = x[:, 64:320]
    c, s = Q.i8_quantize(part)
    rc, rs = R.i8_quantize(part.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(c.cpu().numpy(), rc)


SHAPES = [(1, 1, 16), (1, 17, 64), (2, 100, 144), (4, 300, 1040), (15, 33, 4096), (16, 64, 128), (17, 250, 272),
          (31, 130, 2064), (33, 129, 256), (64, 500, 1024), (65, 256, 80), (100, 66, 16384), (129, 131, 144),
          (200, 1024, 4112), (257, 640, 2048), (300, 2050, 1008), (1025, 260, 512), (1030, 515, 272),
          (1300, 1027, 1552)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dt):
    x, w = rows(M, K, dt, M + 1), rows(N, K, "f16", N + 2, 0.05)
    wc, ws = R.i8_quantize(w.float().numpy())
    bias = rows(1, N, dt, 5)[0] if (M + N) % 2 else None
    y = Q.i8_linear(x.cuda(), torch.from_numpy(wc).cuda(), torch.from_numpy(ws).cuda(),
                    bias=None if bias is None else bias.cuda())
    xc, xs = R.i8_quantize(x.float().numpy())
    y64, mag = R.i8_t(xc, xs, wc, ws, None if bias is None else bias.double().numpy())
    check(y, y64, mag, dt, f"linear {M}x{N}x{K} {dt}")


# more rows than the GEMV's one pass over W, on both sides of where it ends
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(65, 64, 528), (65, 64, 512), (130, 515, 2064), (300, 1000, 1504), (320, 1640, 1024),
                                   (320, 1639, 1024), (1000, 50, 2048), (4100, 17, 1040), (8200, 9, 1040)])
def test_linear_many_rows_little_work(M, N, K, dt):
    test_linear(M, N, K, dt)


@pytest.mark.parametrize("M,N,K", [(1, 40, 131056), (40, 40, 131056), (300, 300, 131056)])
def test_largest_sums_are_exact(M, N, K):
    """Every code at its bound and the longest row: the sum 131056 * 127^2 =
    2113802224 is 98% of 2^31; an alternating sign leaves exact zeros."""
    xq = torch.full((M, K), 127, dtype=torch.int8)
    wq = torch.full((N, K), -127, dtype=torch.int8)
    wq[1, ::2] = 127
    wq[2] = -128
    sx = torch.full((M,), 2.0 ** -20)
    sw = torch.full((N,), 2.0 ** -3)
    y = Q.i8_t(xq.cuda(), sx.cuda(), wq.cuda(), sw.cuda(), dtype=torch.bfloat16)
    y64, mag = R.i8_t(xq.numpy(), sx.numpy(), wq.numpy(), sw.numpy())
    assert np.all(y64[:, 1] == 0)
    check(y, y64, mag, "bf16", f"largest sums {M}x{N}")


@pytest.mark.parametrize("M", [1, 20, 70, 1100])
def test_non_finite_rows_stay_in_their_rows(M):
    x, w = rows(M, 256, "f16", 1), rows(300, 256, "f16", 2)
    x[M // 2, 3] = float("inf")
    wc, ws = Q.i8_quantize(w.cuda())
    y = Q.i8_linear(x.cuda(), wc, ws).cpu()
    assert torch.isnan(y[M // 2]).all()
    keep = torch.arange(M) != M // 2
    assert torch.isfinite(y[keep]).all()


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (13, 300, 2048), (100, 200, 8192), (1030, 300, 512)])
def test_linear_is_the_two_calls_and_repeats(M, N, K):
    x, w = rows(M, K, "bf16", 7).cuda(), rows(N, K, "bf16", 8).cuda()
    wc, ws = Q.i8_quantize(w)
    y = Q.i8_linear(x, wc, ws)
    xc, xs = Q.i8_quantize(x)
    assert torch.equal(y, Q.i8_t(xc, xs, wc, ws))
    for _ in range(3):
        assert torch.equal(y, Q.i8_linear(x, wc, ws))


def test_strided_x_and_other_stream():
    big = rows(40, 1536, "f16", 4).cuda()
    x = big[:, 256:1280]
    wc, ws = Q.i8_quantize(rows(96, 1024, "f16", 5).cuda())
    want = Q.i8_linear(x.contiguous(), wc, ws)
    assert torch.equal(want, Q.i8_linear(x, wc, ws))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = Q.i8_linear(x, wc, ws, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(want, y)


@pytest.mark.parametrize("M", [1, 48])
def test_graph_replays(M):
    """Captured once, replayed on changed inputs with eager calls in between."""
    x = rows(M, 4096, "bf16", 1).cuda()
    wc, ws = Q.i8_quantize(rows(128, 4096, "bf16", 2).cuda())
    Q.i8_linear(x, wc, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = Q.i8_linear(x, wc, ws)
    for i in range(4):
        x.copy_(rows(M, 4096, "bf16", 10 + i))
        want = Q.i8_linear(x, wc, ws)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, y)


def test_graph_of_two_streams():
    """A capture that forks to a side stream: the scratch of the call there (arrival
    counters, codes, parts of K) is ordered on that stream, and memory that the
    capture gives out meanwhile on its own stream is other memory."""
    M, N, K = 128, 1030, 12288
    assert Q.lib().qmm_i8_t_work(M, N, K) > 0   # K is cut: counters are used
    x = rows(M, K, "bf16", 1).cuda()
    wc, ws = Q.i8_quantize(rows(N, K, "bf16", 2).cuda())
    side, out = torch.cuda.Stream(), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    Q.i8_linear(x, wc, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        for _ in range(3):
            Q.i8_linear(x, wc, ws, out=out, stream=side)
            other = [torch.empty(1 << n, dtype=torch.uint8, device="cuda").fill_(255) for n in range(16, 24)]
        mine = Q.i8_linear(x, wc, ws)
        here.wait_stream(side)
    for i in range(4):
        x.copy_(rows(M, K, "bf16", 10 + i))
        want = Q.i8_linear(x, wc, ws)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out) and torch.equal(want, mine)
    assert all(int(t.min()) == 255 for t in other)


def test_graph_of_calls_that_cut_k():
    """Counters and parts in a graph's own scratch, on the current stream."""
    M, N, K = 100, 1100, 8192
    assert Q.lib().qmm_i8_t_work(M, N, K) > 0
    x = rows(M, K, "f16", 1).cuda()
    wc, ws = Q.i8_quantize(rows(N, K, "f16", 2).cuda())
    Q.i8_linear(x, wc, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ys = [Q.i8_linear(x, wc, ws) for _ in range(3)]
    for i in range(4):
        x.copy_(rows(M, K, "f16", 10 + i))
        want = Q.i8_linear(x, wc, ws)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want, y) for y in ys)


def test_one_row_of_a_wider_tensor():
    """The distance to a next row, which is none, is no condition: a row of a tensor
    whose rows are not a multiple of 8 long."""
    big = rows(3, 260, "bf16", 1).cuda()
    wc, ws = Q.i8_quantize(rows(40, 256, "bf16", 2).cuda())
    part = big[:1, :256]
    assert part.stride(0) == 260
    c, s = Q.i8_quantize(part)
    c2, s2 = Q.i8_quantize(part.contiguous())
    assert torch.equal(c, c2) and torch.equal(s, s2)
    assert torch.equal(Q.i8_linear(part, wc, ws), Q.i8_linear(part.contiguous(), wc, ws))
    with pytest.raises(Q.QmmError):
        Q.i8_linear(big[:2, :256], wc, ws)


# many tiles: those of 128 x 128 beyond one round of the chip, and those of 256 x
# 256; ragged in M, N and K, rows of y that start on 2, 4 and 16 bytes
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(2100, 2201, 208), (2100, 2198, 272), (2100, 2200, 1040),
                                   (3900, 3901, 208), (3971, 3898, 272), (3900, 3904, 1040)])
def test_many_tiles(M, N, K, dt):
    g = torch.Generator().manual_seed(M + N + K)
    codes = lambda n: torch.randint(-127, 128, (n, K), generator=g).to(torch.int8)  # noqa: E731
    xq, wq = codes(M), codes(N)
    sx, sw = torch.rand(M, generator=g) * 0.1, torch.rand(N, generator=g) * 0.01
    bias = rows(1, N, dt, 5)[0] if K != 272 else None
    y = Q.i8_t(xq.cuda(), sx.cuda(), wq.cuda(), sw.cuda(), dtype=TORCH_DT[dt],
               bias=None if bias is None else bias.cuda())
    y64 = (xq.double() @ wq.double().t()) * (sx.double()[:, None] * sw.double())   # sums below 2^53: exact
    mag = y64.abs()
    if bias is not None:
        y64, mag = y64 + bias.double(), mag + bias.double().abs()
    check(y, y64.numpy(), mag.numpy(), dt, f"{M}x{N}x{K} {dt}")
