"""Attention over a 4-bit cache without tokens: nothing is read or written but the status word."""
import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark
from fp4 import BF16, F32, make
from test_gpu_fp4_attention import attend

pytestmark = pytest.mark.gpu
BAD = dspark.binding.DEV_BAD_INPUT


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
def test_calls_without_tokens(dtype, D):
    for Hq in (2, 80):
        i = make(dtype, [0, 0, 0], [50, 20, 0], Hq, 2, D, 16, seed=81)
        r = attend(i)
        assert r["out"].shape == (0, Hq, D) and r["lse"].shape == (0, Hq)
        for at, n in ((0, 2), (1, 3), (3, 1), (2, -1)):  # offsets past the rows given, or out of order
            i["off"].zero_()
            i["off"][at] = n
            attend(i, status=BAD)
        i["off"].zero_()
        i["lens"][1] = -1
        attend(i, status=BAD)
        i["lens"][1] = 20
        i["table"][:] = -7  # (no page is looked at)
        attend(i)
