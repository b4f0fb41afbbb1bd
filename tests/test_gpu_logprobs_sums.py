"""Log probabilities and entropy of rows whose finite logits are far from zero."""
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from tests.test_gpu_logprobs import rows, toks

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
