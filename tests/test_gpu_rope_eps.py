"""Norms of heads that hold nothing but zeros or subnormal numbers, under the smallest eps
that there are."""
import pytest
import torch

from group_wise_affine_amd import qmm as Q
from group_wise_affine_amd.devio import TORCH_DT
from tests.test_gpu_rope import check, draw, freqs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.1754942e-38, 1e-37, 1e-30])
@pytest.mark.parametrize("D", [8, 64, 264])
def test_zero_heads_under_any_eps(D, eps, dt):
    """0 / sqrt(0 + eps) is 0 for the subnormal eps of fp32 too; the heads beside them are
    as ever, the smallest ones among them."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    q = draw(3, 4, D, dt, 1)
    q[0, 1] = q[1] = 0
    q[2, 3] = torch.finfo(TORCH_DT[dt]).smallest_normal
    k, w = q[:, 1:3].contiguous(), draw(1, 1, D, dt, 2)[0, 0]
    pos, f = torch.arange(3, dtype=torch.int32), freqs(D)
    qo, ko = Q.qk_norm_rope(*[t.cuda() for t in (q, k, pos, f, w, w)], eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    check(qo, q, pos, f, w, eps, False, dt, f"q eps {eps}")
    check(ko, k, pos, f, w, eps, False, dt, f"k eps {eps}")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-20])
@pytest.mark.parametrize("D", [8, 64, 264, 512])
def test_heads_of_subnormal_numbers(D, eps, dt):
    """Whole heads and single elements of the type's smallest numbers: the mean of their
    squares is far below the range of fp32 (bf16)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    least = float(torch.finfo(TORCH_DT[dt]).smallest_normal) * float(torch.finfo(TORCH_DT[dt]).eps)
    q = torch.zeros(4, 2, D, dtype=torch.float64)
    q[0, 0], q[0, 1, D - 1], q[1, 0, 3], q[1, 1, ::3] = least, -least, 5 * least, 60 * least
    q[2] = least * torch.randint(1, 120, (2, D), generator=torch.Generator().manual_seed(D))
    q[3] = (2.0 ** -80 if dt == "bf16" else 2.0 ** -20) * torch.randn(2, D, generator=torch.Generator().manual_seed(D), dtype=torch.float64)
    q = q.to(TORCH_DT[dt])
    assert bool((q != 0).any(2).all())
    k, w = q[:, :1].contiguous(), torch.ones(D, dtype=TORCH_DT[dt])
    pos, f = torch.arange(4, dtype=torch.int32), freqs(D)
    qo, ko = Q.qk_norm_rope(*[t.cuda() for t in (q, k, pos, f, w, w)], eps=eps)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    check(qo, q, pos, f, w, eps, False, dt, f"q eps {eps}")
    check(ko, k, pos, f, w, eps, False, dt, f"k eps {eps}")
