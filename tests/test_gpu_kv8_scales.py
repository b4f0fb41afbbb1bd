"""Attention over pages whose value scales differ: the weights keep their bits
whichever page carries a row's result, and no row depends on what it does not
see.

Tolerances, relative to a row's own sum mag = sum p vs |c| / sum p:
 * scores as fp32 sums: e = (2 D + 8) 2^-24 of the largest sum of magnitudes,
   in the numerator and in the normaliser: 2 e.
 * weights p vs as f16: 2^-11 for bf16 results, two terms (2^-22) for f16 ones;
   weights below 2^-14 of the row's largest p vs to 2^-25 of that, for every
   key with codes up to 127.
 * exponentials whose argument is a difference of logarithms up to span = 8 +
   log2(largest / smallest value scale): 2^-23 (span + 2), and fp32 sums of n
   terms: (n + 64) 2^-24.
 * the result's rounding to the element type."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests import serving_ref as R
from tests.test_gpu_kv8 import fresh, i32, make, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


def heaviest(ref, q, tab, lens, cu, scale):
    """Largest p vs of each row, over sum p, in float64."""
    T, Hq, _ = q.shape
    G, B = Hq // ref.H, ref.B
    top = np.zeros((T, Hq))
    for s, n in enumerate(lens):
        pages = [j for j in range(-(-n // B)) if 0 <= tab[s][j] < ref.P]
        if not pages:
            continue
        pos = np.concatenate([np.arange(j * B, (j + 1) * B) for j in pages])
        for h in range(ref.H):
            k = np.concatenate([ref.values(tab[s][j], h)[0] for j in pages])
            vs = np.repeat([np.float64(ref.vs[tab[s][j], h]) for j in pages], B)
            for t in range(cu[s], cu[s + 1]):
                see = pos <= n - cu[s + 1] + t
                for g in range(h * G, h * G + G):
                    x = scale * (k[see] @ q[t, g].astype(np.float64))
                    p = np.exp(x - x.max())
                    top[t, g] = (p * vs[see]).max() / p.sum()
    return top


def check(got, ref, q, tab, lens, cu, scale, dt, what):
    want, _, mag, smag = ref.attention(q, tab, lens, cu, scale)
    top, D, n = heaviest(ref, q, tab, lens, cu, scale), q.shape[2], max(lens)
    vs = ref.vs[np.isfinite(ref.vs) & (ref.vs > 0)].astype(np.float64)
    span = 8 + np.log2(vs.max() / vs.min())
    e = (2 * D + 8) * 2.0 ** -24 * smag
    weight = 2.0 ** -11 if dt == "bf16" else 2.0 ** -22
    rel = weight + 2.0 ** -23 * (span + 2) + (n + 64) * 2.0 ** -24 + 2 * e
    tol = R.UNIT[dt] * np.abs(want) + rel[..., None] * mag + (127 * n * 2.0 ** -25 * top)[..., None] + R.TINY[dt]
    off = np.abs(got.double().cpu().numpy() - want) / (tol * (1 + 2.0 ** -7))
    assert (off <= 1).all(), f"{what}: {(off > 1).sum()} of {off.size} off, by up to {np.nanmax(off)} tolerances"


# value scales by page; the codes' magnitudes are alike
FAR = {"bf16": [1e-6, 3.0, 0.0, 1e6, 1e-2], "f16": [1e-5, 3.0, 0.0, 60.0, 1e-2]}


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,G", [(16, 64, 4), (32, 128, 2), (64, 256, 1)])
@pytest.mark.parametrize("new", [1, 2, 70])
@pytest.mark.parametrize("loud", [0, 1, 2, 4])
def test_the_page_that_carries_a_row(loud, new, B, D, G, dt):
    """Scores favour the pages of one value scale, the smallest among them, in any
    place of the row's pages."""
    n = 12 * B - 5
    dev, ref = make(30, 1, B, D, 17 + loud)
    tab = tables([n], B, 30, 18)
    for j, p in enumerate(tab[0]):
        ref.vs[p, 0] = FAR[dt][(j * 7 + j // 3) % 5]
        ref.ks[p, 0] = 0.02 if ref.vs[p, 0] != np.float32(FAR[dt][loud]) else 0.12
    dev.v_scales.copy_(torch.from_numpy(ref.vs))
    dev.k_scales.copy_(torch.from_numpy(ref.ks))
    q = fresh(new, G, D, dt, 19)
    out = Q.kv8_attention(dev, q.cuda(), i32(tab), i32([n]), i32([0, new]), scale=0.5)
    check(out, ref, q.float().numpy(), tab, [n], [0, new], 0.5, dt, f"loud {loud} new {new} B{B} D{D} G{G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,G", [(16, 64, 4), (32, 128, 2), (64, 256, 1)])
@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("loud", [0, 3])
def test_parts_whose_scales_differ(loud, new, B, D, G, dt):
    """A context cut into parts, each with a value scale of its own."""
    n = 2501
    held = -(-n // B)
    dev, ref = make(held + 3, 1, B, D, 41 + loud)
    tab = tables([n], B, held + 3, 42)
    for j, p in enumerate(tab[0]):
        x = j * 5 // held
        ref.vs[p, 0] = FAR[dt][x]
        ref.ks[p, 0] = 0.02 if x != loud else 0.12
    dev.v_scales.copy_(torch.from_numpy(ref.vs))
    dev.k_scales.copy_(torch.from_numpy(ref.ks))
    assert Q.lib().qmm_kv8_attention_work(dev._at, new, G, 1, held) > 0
    q = fresh(new, G, D, dt, 43)
    out = Q.kv8_attention(dev, q.cuda(), i32(tab), i32([n]), i32([0, new]), scale=0.5)
    check(out, ref, q.float().numpy(), tab, [n], [0, new], 0.5, dt, f"parts, loud {loud} new {new} B{B} D{D} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D,new", [(16, 256, 1), (16, 64, 9), (32, 128, 33), (16, 128, 80)])
def test_weights_keep_the_bits_of_the_result(B, D, new, dt):
    """Few keys of like scales, whose values cancel: an f16 result needs more than
    the 11 bits of one f16 weight."""
    dev, ref = make(8, 1, B, D, 21)
    n = new + 7
    tab = tables([n], B, 8, 22)
    q = fresh(new, 16 // (16 if D == 256 else 4), D, dt, 23)
    out = Q.kv8_attention(dev, q.cuda(), i32(tab), i32([n]), i32([0, new]), scale=0.01)
    check(out, ref, q.float().numpy(), tab, [n], [0, new], 0.01, dt, f"B{B} D{D} new {new} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,D", [(16, 64), (16, 128), (32, 128), (16, 256)])
@pytest.mark.parametrize("new", [4, 40])
def test_later_pages_do_not_reach_earlier_rows(new, B, D, dt):
    """A page that later rows alone see gets a value scale of 1e8, louder keys, or
    both: the rows before it keep their bits."""
    n = 3 * B + 2 if new == 4 else 64 + B + 2
    G = 20 if new == 4 else 2      # (more rows than the kernel of few rows takes; the last page inside a tile)
    dev, ref = make(12, 1, B, D, 31)
    tab = tables([n], B, 12, 32)
    q = fresh(new, G, D, dt, 33).cuda()
    args = (i32(tab), i32([n]), i32([0, new]))
    want, wlse = Q.kv8_attention(dev, q, *args, return_lse=True)
    last = tab[0][-1]              # tokens n - 2, n - 1
    for vs, ks in ((1e8, 0.02), (1e-8, 3.0), (1e8, 3.0)):
        dev.v_scales[last], dev.k_scales[last] = vs, ks
        got, lse = Q.kv8_attention(dev, q, *args, return_lse=True)
        assert torch.equal(got[:new - 2], want[:new - 2]) and torch.equal(lse[:new - 2], wlse[:new - 2])
        assert not torch.equal(got[new - 2:], want[new - 2:])
