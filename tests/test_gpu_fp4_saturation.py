"""A 4-bit cache's bytes where quotients of elements and scale leave fp32's range: a group's scale is at most
448, so an element may be far more than 2^128 times its scale and factor, and is stored as the largest code of its sign."""
import pytest
import torch

import fp4
from fp4 import BF16, F32
from test_gpu_rotary import append, check, make, rotated

pytestmark = pytest.mark.gpu


def rows_of(T, big, factor):
    """[T, 1, 64] whose groups hold +-big between elements of the range that 448 covers, ties of two codes among them."""
    unit = 448 * factor
    x = torch.zeros(T, 1, 64, dtype=torch.float64)
    for t in range(T):
        for d in range(64):
            x[t, 0, d] = (0.25, -0.75, 1.0, -2.5, 3.5, 6.0, -6.0, 0.0)[(3 * t + d) % 8] * unit
        for d in range(0, 64, 16):  # each group's place and sign, and how many
            for n in range(1 + (t + d // 16) % 3):
                x[t, 0, d + (5 * t + 7 * n) % 16] = big * (-1) ** (t + n)
    return x


@pytest.mark.parametrize("big, factor", [(3e38, 2.0 ** -12), (1e24, 2.0 ** -60), (3e38, 2.0 ** -60), (3e38, 0.5)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rotation", ["none", "whole", "half", "interleaved", "any", "misaligned"])
def test_elements_far_past_the_largest_code_keep_their_sign(rotation, dtype, big, factor):
    T, D = 40, 64
    i = make("fp4", dtype, [T], [T], 1, 1, D, 16, factors=(factor, factor))
    for name in ("kn", "vn"):
        x = rows_of(T, big, factor).to(dtype).cuda()
        if rotation == "misaligned":  # rows that are no 16-byte vectors
            x = torch.cat((x.new_zeros(T, 1, 1), x), 2)[:, :, 1:]
        i[name] = x
    before = dict(k=i["k"].clone(), v=i["v"].clone())
    dim = {"none": 0, "whole": 64, "half": 32, "interleaved": 64, "any": 6, "misaligned": 64}[rotation]
    tab = None
    if dim:  # no turn, a half and quarters of one: rotated values are elements, so that ties stay ties
        c, s = torch.tensor([1.0, -1.0, 0.0, 0.0]), torch.tensor([0.0, 0.0, 1.0, -1.0])
        tab = torch.cat((c[:, None].expand(4, dim // 2), s[:, None].expand(4, dim // 2)), 1).contiguous().cuda()
    pos = (torch.arange(T, dtype=torch.int32) % 4).cuda()
    inter = rotation == "interleaved"
    append(i, tab, **(dict(positions=pos, interleaved=inter) if dim else {}))
    check(i, tab[pos.long()] if dim else None, inter, before)


def test_the_inputs_reach_both_signs():
    """(Of the test above: what is stored has the largest code of either sign, by the definition alone.)"""
    x = rows_of(40, 3e38, 2.0 ** -12).to(BF16).double()
    codes, scales = fp4.encode(x, 2.0 ** -12)
    assert (scales == 126).all()
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    assert (n[x > 1e38] == 7).all() and (n[x < -1e38] == 15).all() and (x < -1e38).any() and (x > 1e38).any()
    assert rotated(x, torch.ones(40, 64, dtype=torch.float64), False)[0].isfinite().all()
