"""Tree attention whose parents are any number, against the definition (step_ref)."""
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests.test_gpu_kv8_masks import batch, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()


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
