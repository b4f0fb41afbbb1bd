"""f16 results of attention over the 8-bit cache: the weights of the second product are two
f16 terms, 22 bits, in every kernel."""
import numpy as np
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests import serving_ref as R
from tests import step_ref as S
from tests.test_gpu_kv8 import fresh, i32, make
from tests.test_gpu_kv8_masks import grown

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("mask", ["causal", "window", "tree"])
@pytest.mark.parametrize("S_,new,G", [(150, 1, 64), (250, 2, 16), (250, 8, 4), (80, 20, 8)])
def test_weights_of_few_tokens(S_, new, G, mask, D):
    """Many rows that see a few tokens with weights of about one size, of every query
    count that the kernels differ by. Where the values cancel, a term of a weight that is
    off by a bit of 11 is above the result's own rounding: a few in ten thousand rows
    have one if the two terms come from two roundings of a weight. Bound: the result's
    rounding; scores as elsewhere (e); two terms and their fp32 arithmetic, 2^-20 of the
    magnitudes, and the smallest numbers of f16 relative to the largest weight."""
    lens, news = [new + 3] * S_, [new] * S_
    dev, ref = make(S_ * 2, 1, 16, D, S_ + new)
    tab = [[2 * s] + ([2 * s + 1] if lens[s] > 16 else []) for s in range(S_)]
    cu = [int(c) for c in np.cumsum([0] + news)]
    q, scale = fresh(cu[-1], G, D, "f16", 5).clamp(-3, 3), 0.5 / D
    args = (dev, q.cuda(), i32(tab), i32(lens), i32(cu))
    parent = grown(news, 3)
    out = {"causal": lambda: Q.kv8_attention(*args, scale=scale),
           "window": lambda: Q.kv8_attention_window(*args, new + 2, scale=scale),
           "tree": lambda: Q.kv8_attention_tree(*args, i32(parent), scale=scale)}[mask]()
    sees = S.window_sees(lens, cu, new + 2 if mask == "window" else 1 << 30, 0) if mask != "tree" else S.tree_sees(lens, cu, parent)
    want, _, mag, smag = S.Masked.of(ref, sees).attention(q.float().numpy(), tab, lens, cu, scale)
    n, top = lens[0], 127 * ref.vs.max()
    e = (2 * D + 8) * 2.0 ** -24 * smag
    tol = R.UNIT["f16"] * np.abs(want) * (1 + 2.0 ** -7) + (2 * e[..., None] + 2.0 ** -20) * mag + n * 2.0 ** -25 * top + R.TINY["f16"]
    off = np.abs(out.double().cpu().numpy() - want) / tol
    rows = (off > 1).any(2).sum()
    assert rows == 0, f"{rows} of {off.shape[0] * off.shape[1]} rows off, by up to {off.max()} tolerances"
