"""The example runs: int8 projections, 8-bit cache, forks and packing together,
against the dense fp32 block.

Bound: int8 codes under a scale amax / 127 round a normal value by amax / (127
sqrt(12)) ~ 4 / 440 of its deviation, 0.9%; six such roundings (activations and
weights of two products, keys, values) add up as sqrt(6) * 0.9% = 2.2%, the
bf16 roundings in between stay below 1%; single rows differ from the mean by
less than a factor of two."""
import os
import sys

import pytest
import torch

from group_wise_affine_amd import qmm as Q

pytestmark = pytest.mark.gpu


def test_int8_decoder_block():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    Q.lib()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import int8_decoder_block as ex
    worst, used = ex.run(steps=8)
    assert worst < 0.06
    # 77 + 10 .. tokens of two forks share two pages: 4 + 3 - 2 pages + 1
    assert 0 < used < 12
