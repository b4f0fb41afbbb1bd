"""Attention over pages whose value scales differ: no row depends on what it does
not see."""
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests.test_gpu_kv8 import fresh, i32, make, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


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
