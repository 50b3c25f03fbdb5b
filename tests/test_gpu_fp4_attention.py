"""dspark_paged_attention over a 4-bit cache against the definition in 64 bits.

Codes times scales are exact in fp16, so tolerances are those of fp32 sums and of what is rounded on the way
(``fp4.reference``): scores (D + 3) 2^-24 scale sum |q k|, sums over L keys (2 L + 16) 2^-24, and with bf16
queries each probability 2^-11 (fp16) and the output 2^-8, relative.
"""
import math

import pytest
import torch

import fp4
import speculative_decoding_draft_05_gb300 as dspark
from fp4 import BF16, F32, make, reference

pytestmark = pytest.mark.gpu


def attend(i, layer=0, status=0, **kw):
    cache = dspark.PagedCacheFp4(i["k"], i["v"], *i["factors"])
    r = dspark.dspark_paged_attention(i["q"], cache, layer, i["off"], i["lens"], i["table"], i["scale"], **kw)
    assert dspark.dspark_read_device_status(r["workspace"], kw.get("stream")) == status
    return r


def check(i, res, layer=0):
    out, lse, tol, tol_lse = reference(i, layer)
    got, got_lse = res["out"].cpu().double(), res["lse"].cpu().double()
    assert not got.isnan().any()
    bad = (got - out).abs() > tol
    assert not bad.any(), f"out: {int(bad.sum())} off, worst {(got - out).abs()[bad].max():.3g}"
    none = torch.isinf(lse)
    assert (got_lse[none] == -math.inf).all() and (got[none] == 0).all()
    bad = (got_lse - lse).abs()[~none] > tol_lse[~none]
    assert not bad.any(), f"lse: {int(bad.sum())} off, worst {(got_lse - lse).abs()[~none][bad].max():.3g}"


SHAPES = [
    # chunks, lens, Hq, Hkv, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [1], 8, 2, 128, 16),
    ([1, 1, 1], [1, 2, 17], 4, 4, 32, 16),
    ([1] * 5, [127, 128, 129, 1, 300], 8, 2, 128, 16),
    ([3, 0, 2], [5, 0, 40], 4, 2, 64, 16),            # a request without tokens
    ([5, 4], [3, 4], 4, 2, 64, 16),                   # the first two tokens see nothing
    ([2, 0, 3, 200, 0], [0, 0, 40, 0, 7], 8, 2, 64, 16),  # requests without positions
    ([17, 1, 9], [255, 256, 257], 32, 8, 128, 64),
    ([17, 17], [400, 17], 40, 8, 128, 32),            # 5 query heads a K/V head
    ([16, 3], [131, 64], 7, 1, 96, 16),
    ([2, 5], [33, 250], 6, 3, 64, 128),
    ([4, 4], [70, 513], 16, 1, 128, 256),             # a page longer than a tile
    ([2, 3], [65, 100], 4, 2, 32, 48),                # a page size that is no power of two
    ([2, 1], [65, 34], 4, 2, 256, 16),                # wide heads
    ([3, 40], [65, 340], 6, 2, 160, 16),
    ([300], [300], 8, 1, 128, 64),                    # several row blocks, causal from the start
    ([129, 40], [700, 40], 16, 2, 64, 16),
    ([1], [5000], 8, 1, 128, 64),                     # one item over many CTAs
    ([20], [6001], 32, 2, 128, 16),
    ([1] * 130, [(7 * r) % 300 + 1 for r in range(130)], 4, 2, 64, 16),
    ([2] * 700, [(r % 5) + 1 for r in range(700)], 2, 1, 64, 16),  # more requests than threads
    ([3, 1], [200, 20], 130, 1, 64, 16),              # more query heads a K/V head than rows of a tile
    ([1, 1], [200, 20], 600, 2, 128, 16),
    ([20, 3], [400, 97], 8, 2, 96, 48),
    ([90, 1], [300, 641], 8, 2, 128, 160),
    ([60, 30, 1, 70], [60, 300, 900, 70], 12, 4, 128, 16),  # pieces of one and of two row tiles in turn
    ([1, 200, 1, 1, 300, 2], [50, 200, 1300, 7, 900, 2], 20, 4, 64, 64),
    ([64, 1] * 64, [900, 61] * 64, 32, 8, 128, 16),   # long chunks and single tokens in turn
    ([40, 1, 1, 33] * 40, [40, 90, 1, 33] * 40, 8, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", range(len(SHAPES)))
def test_attention_matches_the_definition(dtype, n):
    i = make(dtype, *SHAPES[n], seed=n, strided=n % 3 == 1)
    check(i, attend(i))


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 11, 15, 16, 17, 24, 33, 64, 65, 128, 129, 300])
def test_query_heads_of_a_head(G):
    for chunks in ([1, 1, 1, 1], [1, 2, 5, 9]):
        i = make(BF16, chunks, [140, 2, 30, 260], 2 * G, 2, 128, 16, seed=61)
        check(i, attend(i))


@pytest.mark.parametrize("D, dtype", [(32, F32), (64, F32), (96, F32), (128, F32), (160, F32), (256, F32), (192, BF16),
                                      (256, BF16)])
def test_query_heads_of_a_head_in_fp32_and_of_wide_heads(D, dtype):
    for G in (1, 2, 4, 5, 8, 9, 16, 33, 65):
        for chunks in ([1, 1, 1, 1], [1, 2, 5, 9]):
            i = make(dtype, chunks, [140, 2, 30, 260], 2 * G, 2, D, 16, seed=62)
            check(i, attend(i))


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_head_dims(D):
    for dtype in (F32, BF16):
        for chunks in ([1, 1, 1], [3, 1, 40]):
            i = make(dtype, chunks, [150, 20, 300], 8, 2, D, 16, seed=60)
            check(i, attend(i))


@pytest.mark.parametrize("page", [16, 32, 48, 80, 112, 128, 144, 256, 272])
def test_page_sizes(page):
    for chunks in ([1, 1, 1], [17, 1, 60]):
        i = make(BF16, chunks, [500, 129, 260], 8, 2, 128, page, seed=62, strided=True)
        check(i, attend(i))


@pytest.mark.parametrize("chunks,lens", [([300, 1, 700], [900, 50, 700]), ([257, 256, 255], [257, 300, 4000]), ([1100], [1100])])
def test_long_chunks_of_one_query_head(chunks, lens):
    for D in (64, 128):
        i = make(BF16, chunks, lens, 2, 2, D, 16, seed=63)
        check(i, attend(i))


def test_later_layer_given_outputs_and_rows_past_the_last_request():
    for dtype in (F32, BF16):
        for chunks in ([1, 1], [3, 1], [30, 40]):
            i = make(dtype, chunks, [90, 50], 8, 2, 128, 16, layers=3, seed=5)
            T = sum(chunks)
            i["q"] = torch.cat((i["q"], i["q"].new_full((4, 8, 128), math.nan)))  # padding
            out = torch.full((T + 4, 8, 128), 7.0, dtype=dtype, device="cuda")
            lse = torch.full((T + 4, 8), 7.0, device="cuda")
            r = attend(i, layer=2, out=out, lse=lse)
            assert r["out"] is out and r["lse"] is lse
            assert (out[T:] == 7).all() and (lse[T:] == 7).all()
            check(i, dict(out=out[:T], lse=lse[:T]), layer=2)


@pytest.mark.parametrize("level", [-3000.0, -300.0, -20.0, -9.0, 9.0, 20.0, 300.0, 3000.0])
def test_scores_far_from_zero_and_a_growing_maximum(level):
    # scores of a row from 0.6 level to level in the order of the keys, and back
    for dtype in (F32, BF16):
        for chunks in ([1, 1], [4, 40]):
            i = make(dtype, chunks, [1000, 1500], 4, 2, 64, 16, seed=9, factors=(1.0, 0.25))
            codes, scales = fp4.parts(i["k"])
            codes[:], scales[:] = 0, 0x38
            for r, L in enumerate(i["L"]):
                pos = torch.arange(L, device="cuda")
                pg, slot = i["table"][r, pos // 16].long(), pos % 16
                x = torch.zeros(L, 2, 64, device="cuda")
                x[:, :, 0] = 0.6 + 0.4 * (pos if r == 0 else pos.flip(0))[:, None] / L
                c, s = fp4.encode(x, 1.0)
                codes[0, pg, :, 0, slot], scales[0, pg, :, 0, slot] = c, s
            i["qkv"][:] = 0
            i["qkv"][:, :, 0] = level
            i["scale"] = 1.0
            check(i, attend(i))


@pytest.mark.parametrize("big", [1e-30, 1e-6, 1e30])
def test_queries_far_outside_fp16(big):
    i = make(BF16, [1, 3, 50], [100, 200, 300], 8, 2, 128, 16, seed=10)
    i["qkv"].mul_(big)
    i["scale"] /= big
    check(i, attend(i))
    i = make(BF16, [1, 3, 50], [100, 200, 300], 8, 2, 128, 16, seed=11)
    i["scale"] = -i["scale"]
    check(i, attend(i))
    i["scale"] = 0.0
    check(i, attend(i))


HIDDEN = [
    # chunks, lens, Hq, Hkv, D, page, tokens of the first request whose K or V is not finite
    ([4], [400], 2, 2, 128, 16, (0, 1, 3)),
    ([2], [33], 16, 2, 128, 16, (0, 1)),
    ([17], [400], 8, 2, 128, 16, (0, 9, 16)),
    ([17, 3], [130, 40], 8, 2, 64, 16, (1, 2, 14)),   # the chunk lies over two tiles
    ([10], [4], 4, 2, 64, 16, (6, 9)),                # the first tokens see nothing
    ([300], [300], 8, 1, 128, 64, (0, 31, 32, 130, 299)),
    ([129, 40], [700, 40], 16, 2, 96, 16, (5, 128)),
    ([20], [6001], 32, 2, 128, 16, (19, 4)),          # many CTAs, cut pieces
    ([20], [90], 4, 2, 256, 16, (7, 19)),
    ([300], [700], 2, 2, 128, 16, (0, 130, 299)),     # masks over several tiles
]


@pytest.mark.parametrize("what", ["v", "k"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", range(len(HIDDEN)))
def test_later_tokens_that_are_not_finite_stay_out_of_earlier_rows(dtype, what, n):
    *shape, places = HIDDEN[n]
    i = make(dtype, *shape, seed=50 + n)
    out, lse, tol, tol_lse = reference(i)
    count, L, G = shape[0][0], shape[1][0], shape[2] // shape[3]
    clean = [i[x].clone() for x in "kv"]
    for a in places:
        i["k"].copy_(clean[0])
        i["v"].copy_(clean[1])
        p = L - count + a
        page, slot = i["table"][0, p // i["page"]].long(), p % i["page"]
        fp4.parts(i[what])[1][0, page, 0, slot // 16, slot % 16, 1] = 0xff if a % 2 else 0x7f  # elements 16 .. 31
        r = attend(i)
        got, got_lse = r["out"].cpu().double(), r["lse"].cpu().double()
        sees = torch.zeros(lse.shape, dtype=torch.bool)  # rows of the first K/V head from token a on
        sees[a:count, :G] = True
        assert not got[sees][:, 16:32].isfinite().any(), a
        rest, none = ~sees, torch.isinf(lse)
        assert ((got - out).abs() <= tol)[rest].all(), a
        assert (got_lse[rest & none] == -math.inf).all()
        assert ((got_lse - lse).abs() <= tol_lse)[rest & ~none].all(), a


def test_queries_that_are_not_finite_stay_in_their_rows():
    for dtype in (F32, BF16):
        for chunks in ([1, 1, 1], [2, 3, 60]):
            i = make(dtype, chunks, [50, 200, 300], 8, 2, 128, 16, seed=12)
            out, lse, tol, tol_lse = reference(i)
            i["qkv"][1, 2, 7] = math.nan
            i["qkv"][2, 5, 9] = math.inf
            r = attend(i)
            got = r["out"].cpu().double()
            hit = torch.zeros(lse.shape, dtype=torch.bool)
            hit[1, 2] = hit[2, 5] = True
            assert not got[hit].isfinite().any()
            assert ((got - out).abs() <= tol)[~hit].all()
            assert ((r["lse"].cpu().double() - lse).abs() <= tol_lse)[~hit].all()


def test_equal_inputs_give_equal_results_beside_other_work():
    i = make(BF16, [17] * 20, [(331 * r) % 3000 + 17 for r in range(20)], 32, 8, 128, 16, seed=13)
    r = attend(i)
    for _ in range(20):
        b = attend(i, workspace=r["workspace"])
        assert torch.equal(r["out"], b["out"]) and torch.equal(r["lse"], b["lse"])


def test_bad_pages_and_lengths_are_flagged_and_stay_inside():
    for dtype in (F32, BF16):
        for chunks in ([1, 1], [30, 2]):
            i = make(dtype, chunks, [90, 50], 8, 2, 128, 16, seed=14)
            good = i["table"].clone()
            for at, value in (((0, 1), -1), ((1, 3), 1 << 30), ((0, 5), i["k"].shape[1])):
                i["table"].copy_(good)
                i["table"][at] = value
                attend(i, status=dspark.binding.DEV_BAD_INPUT)
            i["table"].copy_(good)
            for lens in ([1 << 30, 50], [-5, 50], [90, 0x7fffffff]):
                i["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
                i["table"].clamp_(min=0)
                attend(i, status=dspark.binding.DEV_BAD_INPUT)


@pytest.mark.parametrize("chunks", [[1, 1, 1], [3, 2, 4], [20, 3, 150]])
def test_queries_of_other_strides_and_alignments(chunks):
    i = make(BF16, chunks, [50, 200, 300], 8, 2, 128, 16, seed=20)
    want = attend(i)
    T = sum(chunks)
    for wide in (torch.zeros(T, 8, 131, dtype=BF16, device="cuda")[:, :, 1:129],
                 torch.zeros(8, T, 136, dtype=BF16, device="cuda").transpose(0, 1)[:, :, 8:]):
        wide.copy_(i["q"])
        r = attend(dict(i, q=wide))
        assert torch.equal(r["out"], want["out"]) and torch.equal(r["lse"], want["lse"])


def test_requests_of_both_kinds_of_rows_in_one_call():
    # the kernel is chosen by the mean: some requests have far more rows than that, some fewer
    for Hq in (8, 32):
        for chunks in ([1] * 60 + [300, 90], [100, 1, 1, 1], [1] * 10 + [64], [5, 0, 0, 0, 0, 0, 0, 0]):
            lens = [max(n, (37 * r) % 700 + 1) for r, n in enumerate(chunks)]
            i = make(BF16, chunks, lens, Hq, 2, 128, 16, seed=21)
            check(i, attend(i))


@pytest.mark.parametrize("chunk, dtype", [(1, BF16), (2, BF16), (40, BF16), (2, F32)])
def test_a_request_of_2_to_the_31_positions(chunk, dtype):
    """The longest request there is, of one page many times over: K is 0 and V is 1, so that every partial sum is
    a number of positions (times a power of two), exact up to 2^24.  304 or fewer partial results meet: (304 + 16)
    2^-24."""
    L, page = 2 ** 31 - 2 ** 16, 65536
    P = 32768
    k = torch.zeros(1, 1, 1, page // 16, 9 * 32, dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, 0x22)
    fp4.parts(v)[1].fill_(0x38)
    i32 = dict(dtype=torch.int32, device="cuda")
    i = dict(k=k, v=v, factors=(1.0, 1.0), q=torch.ones(chunk, 4, 32, dtype=dtype, device="cuda"), scale=0.2,
             off=torch.tensor([0, chunk], **i32), lens=torch.tensor([L], **i32), table=torch.zeros(1, P, **i32))
    r = attend(i)
    tol = 320 * 2.0 ** -24
    want = torch.tensor([math.log(L - chunk + 1 + t) for t in range(chunk)], dtype=torch.float64)[:, None]
    assert ((r["out"].double() - 1).abs() <= tol + (2.0 ** -8 if dtype == BF16 else 0)).all()
    assert ((r["lse"].cpu().double() - want).abs() <= tol + 8 * 2.0 ** -24 * want).all()
