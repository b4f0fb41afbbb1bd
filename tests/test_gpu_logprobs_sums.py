"""Log probabilities and entropy of rows whose finite logits are far from zero: masks of
any value, peaks, both forms of the sums."""
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
