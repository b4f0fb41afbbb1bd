"""Window and tree attention of heads of 256 over contexts that are cut into parts, and
trees whose parents are any number, against the definition (step_ref)."""
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests.test_gpu_kv8_masks import batch, grown, tree, window

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("B,H,G", [(16, 1, 4), (64, 2, 3)])
@pytest.mark.parametrize("lens,new", [([5003, 40], [7, 1]), ([3000], [40]), ([1700, 5, 2100], [33, 1, 20]), ([2600, 1700, 3100], [3, 1, 2])])
def test_trees_of_wide_heads_in_parts(lens, new, B, H, G, dt):
    """Few query rows and many, for the decode kernel and the prompt kernel."""
    b = batch(lens, new, B, 256, H, G, dt)
    assert Q.lib().qmm_kv8_attention_tree_work(b[0]._at, sum(new), H * G, len(lens), len(b[2][0])) > 0   # cut into parts
    tree(*b[:3], lens, b[3], b[4], dt, grown(new, 7), f"{lens} {new} B{B} H{H} G{G} {dt}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("w,sinks", [(2600, 100), (1 << 40, 7)])
@pytest.mark.parametrize("B,H,G", [(16, 1, 4), (64, 1, 3)])
@pytest.mark.parametrize("lens,new", [([5003, 40], [1, 1]), ([3000], [30]), ([4300, 5, 3100], [20, 1, 2])])
def test_windows_of_wide_heads_in_parts(lens, new, B, H, G, w, sinks, dt):
    b = batch(lens, new, B, 256, H, G, dt)
    assert Q.lib().qmm_kv8_attention_window_work(b[0]._at, sum(new), H * G, len(lens), len(b[2][0]), w, sinks) > 0
    window(*b[:3], lens, b[3], b[4], dt, w, sinks, f"{lens} {new} B{B} H{H} G{G} {dt}")


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("G", [1, 4])
def test_parents_of_any_number_behind_causal_tokens(G, D):
    """The ends of the type's range where the tree does not start with the first new
    token: all of them roots."""
    n = 90
    lens, new = [n + 70], [n]
    b = batch(lens, new, 16, D, 1, G, "f16")
    for parent in ([-2 ** 31] * n, [2 ** 31 - 1] * n, [-2 ** 31 + i for i in range(n)], [25] * n, [26 + i for i in range(n)],
                   [[-2 ** 31, i - 1, 2 ** 31 - 1, 20][i % 4] for i in range(n)]):
        tree(*b[:3], lens, b[3], b[4], "f16", parent, f"{parent[:5]}")
