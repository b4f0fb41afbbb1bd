"""Log probabilities and entropy of rows whose finite logits are far from zero: masks of
any value, peaks, both forms of the sums; and the accuracy of long rows' sums."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests.test_gpu_logprobs import DT, check, rows, toks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e20, -1e30])
def test_entropy_and_log_probability_agree_on_nan(mask, dt):
    """An entropy is a number where the token's log probability is one, and no number
    where that is none."""
    x = rows(4, 4096, dt, 3)
    x[:, 30:] = mask
    x[2, 7] = float("nan")
    lp, h, _, _ = Q.logprobs(x, toks(4, 30), top=5)
    assert torch.equal(torch.isnan(lp), torch.isnan(h)) and bool(torch.isnan(h[2]))


MASKS = [-1e4, -6e4, -65535.0, -65536.0, -1e5, -1e6, -1e9, -5e9, -1e10, -1e12, -1e20, -1e30, -1e37, -9e37, -1.1e38, -2e38]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 70, 300, 5000, 70001])
def test_finite_masks_of_any_value(V, dt):
    """Masked before and behind the allowed logits, between them, all but one and all; the
    same numbers as single peaks."""
    up = torch.linspace(-4, 4, V)
    for top in (0, 3, 5):
        x = []
        for m in MASKS:
            tail, head, every, one, whole, peak = up.clone(), up.clone(), up.clone(), torch.full((V,), m), torch.full((V,), m), up.clone()
            tail[V // 3:], head[:V - 2], every[::2] = m, m, m
            one[V // 2] = 2.0
            peak[V - 2] = -m
            x += [tail, head, every, one, whole, peak]
        x = torch.stack(x).to(DT[dt]).cuda()
        t = toks(len(x), V, 1)
        t[::2] = 0
        t[1::6] = V - 1
        check(x, t, top, Q.logprobs(x, t, top=top), f"V{V} {dt} top {top}")


@pytest.mark.parametrize("top", [0, 7])
@pytest.mark.parametrize("V", [40, 3000, 60000])
def test_logits_on_both_sides_of_a_sums_form(V, top):
    """Maxima near +-2^16, from where differences come before products: lanes and
    wavefronts of one row hold their sums in one form and the other, and join them."""
    g = torch.Generator().manual_seed(V)
    x = torch.cat([a + b * torch.rand(6, V, generator=g) for a in (65536.0, -65536.0, 65500.0, -65500.0) for b in (1.0, 9.0, 60.0)])
    x = torch.cat([x - 4.5, x, x.sort(1).values, x.sort(1, descending=True).values]).cuda()
    t = toks(len(x), V, 2)
    check(x, t, top, Q.logprobs(x, t, top=top), f"V{V} top {top}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [70, 5000, 70001])
def test_probabilities_of_the_lowest_logits(V, dt):
    """Tokens under a mask of the type's lowest value, asked for and among the top:
    x - lse is finite wherever fp32 can hold it."""
    low = float(torch.finfo(DT[dt]).min)
    x = torch.full((4, V), low).to(DT[dt])
    x[0, :3] = torch.tensor([1.0, 2.0, 3.0])
    x[1, V // 2] = -2.9e38
    x[2, V - 1] = 3.0e38   # the others: past the range of fp32
    x[3, 1] = -2.4e38
    t = torch.tensor([V - 1, 0, 0, 0], dtype=torch.int32)
    lp, _, ids, tl = (o.double().cpu().numpy() for o in Q.logprobs(x.cuda(), t.cuda(), top=6))
    d = x.double().numpy()
    for r, lse in enumerate((3.40760596444438, d[1].max(), d[2].max(), d[3].max())):
        for got, want in ((lp[r], d[r, t[r]] - lse), *zip(tl[r], np.sort(d[r])[::-1][:6] - lse)):
            if want < -3.4028235e38:
                assert got == -np.inf
            else:
                assert abs(got - want) <= 2.0 ** -22 * abs(want) + 1e-5, (r, got, want)


def final(lp):
    """Roundings behind the sums, of a log probability `lp`: the logarithm's (an ulp), the
    token's exponent, the difference's, the product's and its factor's."""
    return 6 * 2.0 ** -24 * np.maximum(np.abs(lp), 1.0)


def lane_sum(rest, n0, n1, N):
    """Half an ulp of each partial sum of a lane that adds n0 ones and n1 terms `rest`, N of
    them at a time, relative to its sum."""
    s, off = np.zeros_like(rest), np.zeros_like(rest)
    for k in range((n0 + n1) // N):
        s = s + N * (1.0 if k < n0 // N else rest)
        off += 2.0 ** (np.floor(np.log2(s)) - 24)
    return off / s


@pytest.mark.parametrize("dt,N", [("bf16", 8), ("f32", 4)])
def test_long_sums_are_not_taken_term_by_term(dt, N):
    """Rows of a plateau behind some larger logits, many plateaus: added one by one, its
    terms are rounded the same way in every step of a lane, up to 1000 times. Bound: half
    an ulp of each of a lane's partial sums, a load's N terms added first (N - 1
    roundings, as many as 2^-24 each); the exponential's ulp and its exponent's rounding
    (4 * 2^-24); lanes and wavefronts joined (7 sums, and as many scalings)."""
    M, lanes = 2048, 128
    V = 1000 * lanes
    n0 = 4 * N   # terms of a lane's first four loads
    c = torch.linspace(-0.7, -0.2, M).to(DT[dt])
    x = c[:, None].repeat(1, V)
    x[:, :n0 * lanes] = 0.0
    t = torch.full((M,), V - 1, dtype=torch.int32)
    t[::2] = 0
    lp, h, _, _ = (o.double().cpu().numpy() for o in Q.logprobs(x.cuda(), t.cuda(), top=3))
    c = c.double().numpy()
    s = lanes * (n0 + (1000 - n0) * np.exp(c))
    want = np.where(t.numpy() == 0, 0.0, c) - np.log(s)
    u = lane_sum(np.exp(c), n0, 1000 - n0, N) + (N - 1 + 4 + 14) * 2.0 ** -24
    off = np.abs(lp - want) / (u + final(want))
    assert off.max() <= 1, f"log probability off by {off.max()} tolerances"
    # the mean of x - max: numerator (as many additions, 2^-24 each, a product more) and
    # denominator
    mean = lanes * (1000 - n0) * np.exp(c) * -c / s
    v = (1000 / N + N + 20) * 2.0 ** -24
    off = np.abs(h - (np.log(s) + mean)) / (u + (u + v) * mean + final(np.log(s)) + final(mean))
    assert off.max() <= 1, f"entropy off by {off.max()} tolerances"


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,V", [(1, 131071), (3, 20000), (40, 50001), (300, 9999), (2048, 32000), (2100, 5001)])
def test_accuracy_of_plain_rows(M, V, dt):
    """Rows without masks, a bound from the number of additions that there are: a lane
    takes A loads of N elements, and its sums are raised at most once per load (three
    roundings); then as above, with 14 joins of four roundings at most. An exponent's
    rounding and its factor's make a term off by 2^-23 |x - max| of it. The mean of x -
    max has such a sum above and below the line."""
    N = 4 if dt == "f32" else 8
    lanes = 512 if M < 2048 else 128
    A = -(-V // (N * lanes)) + 2
    x, t = rows(M, V, dt, M + V), toks(M, V, 5)
    d = x.double().cpu().numpy()
    top = d.max(1)
    z = np.exp(d - top[:, None])
    s = z.sum(1)
    mag, square = (z * (top[:, None] - d)).sum(1) / s, (z * (top[:, None] - d) ** 2).sum(1) / s
    lp, h = d[np.arange(M), t.cpu().numpy()] - top - np.log(s), np.log(s) + mag
    u = (4 * A + N - 1 + 4 + 56) * 2.0 ** -24
    for n in (0, 5):
        a, b, _, _ = (o.double().cpu().numpy() for o in Q.logprobs(x, t, top=n))
        off = np.abs(a - lp) / (u + 2.0 ** -23 * mag + final(lp))
        assert off.max() <= 1, f"log probability, top {n}: {off.max()} tolerances"
        off = np.abs(b - h) / (u * (1 + 2 * mag) + 2.0 ** -23 * (mag + mag ** 2 + square) + final(np.log(s)) + final(mag))
        assert off.max() <= 1, f"entropy, top {n}: {off.max()} tolerances"


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M", [256, 257, 1536, 1537])
def test_rows_beside_a_change_of_workgroups(M, dt):
    """Numbers of rows on both sides of where a row is no longer cut, and of where a
    workgroup has fewer wavefronts."""
    V = 8500
    x, t = rows(M, V, dt, M), toks(M, V, 6)
    x[M - 1, V // 2:] = -1e4
    for top in (0, 20):
        check(x, t, top, Q.logprobs(x, t, top=top), f"{M}x{V} {dt} top {top}")
