"""Attention of bf16 queries over a 4-bit cache, where queries are subnormal numbers: rows are multiplied by a power of
two and the scores' factor takes it back, so queries 2^-n and a scale 2^n times another call's give that call's results."""
import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark
from fp4 import BF16, make
from test_gpu_fp4_attention import attend, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunks", [[1, 1, 1], [2, 1, 2], [4, 1, 40]], ids=["one block", "two blocks", "many rows"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_subnormal_queries(chunks, D, sign):
    i = make(BF16, chunks, [90, 260, 300], 8, 2, D, 16, seed=71)
    g = torch.Generator().manual_seed(72)
    T = sum(chunks)
    whole = torch.randint(-3, 4, (T, 8, D), generator=g)
    whole[0, 0] = 0
    i["scale"] = sign * 2.0 ** -6
    i["q"] = whole.to(BF16).cuda()
    want = attend(i)
    check(i, want)
    small = (whole.double() * 2.0 ** -131).to(BF16)  # multiples of 2^-133, all below 2^-126
    assert torch.equal(small.double(), whole.double() * 2.0 ** -131)
    small[-1] = whole[-1].to(BF16) * 2.0 ** -100  # (and rows that are not, beside them)
    wide = small.cuda()
    cache = dspark.PagedCacheFp4(i["k"], i["v"], *i["factors"])
    got = dspark.dspark_paged_attention(wide, cache, 0, i["off"], i["lens"], i["table"], sign * 2.0 ** 125)
    assert torch.equal(got["out"][:T - 1], want["out"][:T - 1]) and torch.equal(got["lse"][:T - 1], want["lse"][:T - 1])
