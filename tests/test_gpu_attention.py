"""dspark_paged_attention and dspark_cache_append against the definition in 64 bits.

Tolerances, per output element, from the formulas.  With u = 2^-24, scores of
the fp32 sums are off by at most ds = (D + 3) u scale sum |q k| (plus the
rounding of the exponent's argument, 2 u max|s|), so a probability is off by
the factor e^{+-2 ds}; sums over L keys add (L + 8) u; the bf16 kernel rounds
each probability and the output to 8 bits (2^-8 relative each).  All of it is relative
to sum_j p_j |v_j|, which the reference computes.
"""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def make(dtype, chunks, lens, Hq, Hkv, D, page, layout="thd", seed=0, layers=1, spare=2, poison=True):
    """Random inputs; everything past kv_len in the cache, and unused pages, hold NaN."""
    g = torch.Generator().manual_seed(seed)
    R = len(lens)
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + spare
    P = max(held + [1]) + 1
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((R, P), -1, dtype=torch.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = perm[at:at + h].int()
        at += h
    shape = [layers, n_pages, page, Hkv, D]
    k, v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    if poison:
        live = torch.zeros(n_pages, page, dtype=torch.bool)
        for r, n in enumerate(lens):
            for j in range(held[r]):
                live[table[r, j], : min(page, n - j * page)] = True
        k[:, ~live] = math.nan
        v[:, ~live] = math.nan
    T = sum(chunks)
    # q is a part of a wider projection, so its rows are strided
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype)
    dev = "cuda"

    def put(t):
        if layout == "htd":
            return t.transpose(2, 3).contiguous().to(dev).transpose(2, 3)
        return t.to(dev)

    off = torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32)
    return dict(k=put(k), v=put(v), qkv=qkv.to(dev), q=qkv.to(dev)[:, :Hq], off=off.to(dev),
                lens=torch.tensor(lens, dtype=torch.int32).to(dev), table=table.to(dev), scale=1 / math.sqrt(D),
                chunks=chunks, L=lens, Hq=Hq, Hkv=Hkv, D=D, page=page)


def reference(i, layer=0):
    T, Hq, D, G = sum(i["chunks"]), i["Hq"], i["D"], i["Hq"] // i["Hkv"]
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    table, q = i["table"].cpu().long(), i["q"].cpu().double()
    k, v = i["k"][layer].cpu(), i["v"][layer].cpu()
    bf = i["k"].dtype == BF16
    t = 0
    for r, (n, L) in enumerate(zip(i["chunks"], i["L"])):
        pg = table[r, : -(-L // i["page"])]
        K = k[pg].reshape(-1, i["Hkv"], D)[:L].double()
        V = v[pg].reshape(-1, i["Hkv"], D)[:L].double()
        for a in range(n):
            p = L - n + a
            if p >= 0:
                Kh, Vh = (x[: p + 1].repeat_interleave(G, 1) for x in (K, V))
                s = torch.einsum("hd,jhd->hj", q[t], Kh) * i["scale"]
                ds = ((D + 3) * U * abs(i["scale"]) * torch.einsum("hd,jhd->hj", q[t].abs(), Kh.abs())).amax(1)
                ds = ds + 2 * U * s.abs().amax(1)
                lse[t] = torch.logsumexp(s, 1)
                pr = torch.exp(s - lse[t][:, None])
                out[t] = torch.einsum("hj,jhd->hd", pr, Vh)
                mix = torch.einsum("hj,jhd->hd", pr, Vh.abs())
                rel = 4 * ds + (2 * p + 16) * U + (2.0 ** -8 if bf else 0)
                tol[t] = rel[:, None] * mix + (2.0 ** -8 * out[t].abs() if bf else 0)
                tol_lse[t] = 2 * ds + (2 * p + 16) * U + 4 * U * lse[t].abs()
            t += 1
    return out, lse, tol, tol_lse


def reference_on_gpu(i):
    """``reference`` of layer 0, a request at a time in 64 bits on the GPU (what only goes into tolerances: 32)."""
    Hq, D, G, scale = i["Hq"], i["D"], i["Hq"] // i["Hkv"], i["scale"]
    bf = i["k"].dtype == BF16
    table, parts, t = i["table"].long(), [], 0
    for r, (n, L) in enumerate(zip(i["chunks"], i["L"])):
        pg = table[r, : -(-L // i["page"])]
        K, V = (x[0][pg].reshape(-1, i["Hkv"], D)[:L].double().repeat_interleave(G, 1) for x in (i["k"], i["v"]))
        q = i["q"][t:t + n].double()
        t += n
        if n == 0:
            continue
        if L == 0:  # nothing to see
            z = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
            parts.append((z, z[..., 0] - math.inf, z, z[..., 0]))
            continue
        pos = torch.arange(L - n, L, device="cuda")
        see = torch.arange(L, device="cuda") <= pos[:, None, None]  # [n, 1, L]
        s = torch.einsum("nhd,jhd->nhj", q, K) * scale
        sa = torch.einsum("nhd,jhd->nhj", q.float().abs(), K.float().abs()) * abs(scale)
        ds = (D + 3) * U * torch.where(see, sa, 0.0).amax(2) + 2 * U * torch.where(see, s.abs(), 0.0).amax(2)
        s = torch.where(see, s, -math.inf)
        lse = torch.logsumexp(s, 2)
        pr = torch.where(see, torch.exp(s - lse[..., None].nan_to_num(neginf=0.0)), 0.0)
        out = torch.einsum("nhj,jhd->nhd", pr, V)
        mix = torch.einsum("nhj,jhd->nhd", pr.float(), V.float().abs())
        sums = ((2 * pos + 16) * U)[:, None]
        tol = (4 * ds + sums + (2.0 ** -8 if bf else 0))[..., None] * mix + (2.0 ** -8 * out.abs() if bf else 0)
        parts.append((out, lse, tol, 2 * ds + sums + 4 * U * lse.abs()))
    return [torch.cat(x).cpu() for x in zip(*parts)]


def check(i, res, layer=0, want=None):
    out, lse, tol, tol_lse = reference(i, layer) if want is None else want
    got, got_lse = res["out"].cpu().double(), res["lse"].cpu().double()
    assert not got.isnan().any()
    bad = (got - out).abs() > tol
    assert not bad.any(), f"out: {int(bad.sum())} off, worst {(got - out).abs()[bad].max():.3g}"
    none = torch.isinf(lse)
    assert (got_lse[none] == -math.inf).all() and (got[none] == 0).all()
    bad = (got_lse - lse).abs()[~none] > tol_lse[~none]
    assert not bad.any(), f"lse: {int(bad.sum())} off, worst {(got_lse - lse).abs()[~none][bad].max():.3g}"


def attend(i, layer=0, **kw):
    cache = dspark.PagedCache(i["k"], i["v"])
    r = dspark.dspark_paged_attention(i["q"], cache, layer, i["off"], i["lens"], i["table"], i["scale"], **kw)
    assert dspark.dspark_read_device_status(r["workspace"], kw.get("stream")) == 0
    return r


SHAPES = [
    # chunks, lens, Hq, Hkv, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [1], 8, 2, 128, 16),
    ([1, 1, 1], [1, 2, 17], 4, 4, 64, 1),
    ([1] * 5, [127, 128, 129, 1, 300], 8, 2, 128, 16),
    ([3, 0, 2], [5, 0, 40], 4, 2, 64, 16),            # a request without tokens
    ([5, 4], [3, 4], 4, 2, 64, 16),                   # the first two tokens see nothing
    ([17, 1, 9], [255, 256, 257], 32, 8, 128, 64),
    ([17, 17], [400, 17], 40, 8, 128, 32),            # 5 query heads a K/V head
    ([16, 3], [131, 64], 7, 1, 96, 16),
    ([2, 5], [33, 250], 6, 3, 80, 128),
    ([4, 4], [70, 513], 16, 1, 128, 256),             # a page longer than a tile
    ([4, 7], [70, 50], 8, 4, 64, 8),
    ([2, 3], [65, 100], 4, 2, 40, 24),                # a page size that is no power of two
    ([2, 1], [65, 34], 4, 2, 256, 16),                # wider than the tensor-core kernel takes
    ([3, 2], [19, 40], 2, 2, 12, 5),
    ([300], [300], 8, 1, 128, 64),                    # several row blocks, causal from the start
    ([129, 40], [700, 40], 16, 2, 64, 16),
    ([1], [5000], 8, 1, 128, 64),                     # one item over many CTAs
    ([20], [6001], 32, 2, 128, 16),
    ([1] * 130, [(7 * r) % 300 + 1 for r in range(130)], 4, 2, 64, 16),
    ([2] * 700, [(r % 5) + 1 for r in range(700)], 2, 1, 64, 16),  # more requests than threads
    ([3, 2], [70, 300], 4, 2, 40, 16),                # narrower than a swizzled row
    ([2, 40], [9, 200], 3, 1, 16, 32),
    ([3, 1], [200, 20], 130, 1, 64, 16),              # more query heads a K/V head than rows of a tile
    ([2, 17, 1], [65, 300, 24], 4, 2, 128, 24),       # pages of whole boxes of 8 tokens
    ([20, 3], [400, 97], 8, 2, 64, 48),
    ([90, 1], [300, 641], 8, 2, 128, 160),            # a page longer than a tile, not a multiple of it
    ([60, 30, 1, 70], [60, 300, 900, 70], 12, 4, 128, 16),  # pieces of one and of two row tiles in turn
    ([1, 200, 1, 1, 300, 2], [50, 200, 1300, 7, 900, 2], 20, 4, 64, 64),
]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", range(len(SHAPES)))
def test_attention_matches_the_definition(dtype, n):
    i = make(dtype, *SHAPES[n], layout="htd" if n % 2 else "thd", seed=n)
    check(i, attend(i))


def mixed(kind):
    """Long chunks and young requests in turn: (chunks, lens, Hq, Hkv, D, page)."""
    g = torch.Generator().manual_seed(31)
    young = torch.randint(5, 121, (400,), generator=g).tolist()
    if kind == "chunks of 64, single tokens":
        return [64, 1] * 128, sum(([900, n] for n in young[:128]), []), 32, 8, 128, 16
    if kind == "prompts of 448, single tokens":
        return [448, 1] * 32, sum(([448, n] for n in young[:32]), []), 32, 8, 128, 64
    if kind == "verify chunks, all young":
        c = [n % 17 + 1 for n in young[:256]]
        return c, [max(a, n) for a, n in zip(c, young)], 32, 4, 128, 16
    if kind == "one head, three kinds":
        return [32, 9, 16] * 120, sum(([300, n, 129 + n] for n in young[:120]), []), 8, 1, 64, 16
    # every second request has two row blocks of one tile, or one of one tile
    return [40, 1, 1, 33] * 90, sum(([40, n, 1, 33] for n in young[:90]), []), 8, 1, 128, 8


@pytest.mark.parametrize("kind", ["chunks of 64, single tokens", "prompts of 448, single tokens",
                                  "verify chunks, all young", "one head, three kinds", "single tiles"])
def test_shares_of_many_pieces_of_both_kinds(kind):
    # A CTA's share holds a piece of two row blocks, one of a single tile and one
    # more, in this order: the last one must not overwrite what the first one's
    # results are still read from.
    i = make(BF16, *mixed(kind), seed=31)
    r = attend(i)
    check(i, r, want=reference_on_gpu(i))
    for _ in range(40):
        b = attend(i, workspace=r["workspace"])
        assert torch.equal(r["out"], b["out"]) and torch.equal(r["lse"], b["lse"])


def test_attention_of_a_later_layer_and_given_outputs():
    i = make(BF16, [3, 1], [90, 20], 8, 2, 128, 16, layers=3, seed=5)
    T = 4
    out = torch.full((T, 8, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((T, 8), 7.0, device="cuda")
    r = attend(i, layer=2, out=out, lse=lse)
    assert r["out"] is out and r["lse"] is lse
    check(i, r, layer=2)


def test_requests_without_positions():
    for dtype in (F32, BF16):
        i = make(dtype, [2, 0, 3, 200, 0], [0, 0, 40, 0, 7], 8, 2, 64, 16, seed=64)
        check(i, attend(i), want=reference_on_gpu(i))
        check(i, attend(i))


@pytest.mark.parametrize("D", [8, 24, 56, 72, 104, 120, 136, 248])
def test_head_dims(D):
    for dtype in (F32, BF16):
        i = make(dtype, [3, 1, 40], [150, 20, 300], 8, 2, D, 16, seed=60)
        check(i, attend(i))


@pytest.mark.parametrize("G", [3, 11, 33, 43, 64, 65, 100, 127, 128, 129, 300])
def test_query_heads_of_a_head(G):
    # row blocks of whole tokens that do not fill 128 rows, and tokens of more rows than a block
    for dtype in (F32, BF16):
        i = make(dtype, [1, 2, 5, 9], [140, 1, 30, 260], 2 * G, 2, 64, 16, seed=61)
        check(i, attend(i), want=reference_on_gpu(i))


@pytest.mark.parametrize("chunks,lens", [([300, 1, 700], [900, 50, 700]), ([257, 256, 255], [257, 300, 4000]), ([1100], [1100])])
def test_long_chunks_of_one_query_head(chunks, lens):
    # a row block is 128 or 256 tokens: the causal mask lies over several tiles
    for dtype in (F32, BF16):
        for D in (64, 128):
            i = make(dtype, chunks, lens, 2, 2, D, 16, seed=63)
            check(i, attend(i), want=reference_on_gpu(i))


@pytest.mark.parametrize("page", [1, 3, 8, 40, 56, 72, 104, 128, 136, 200, 264])
def test_page_sizes(page):
    for dtype in (F32, BF16):
        i = make(dtype, [17, 1, 60], [500, 129, 260], 8, 2, 128, page, layout="htd", seed=62)
        check(i, attend(i), want=reference_on_gpu(i))


HIDDEN = [
    # chunks, lens, Hq, Hkv, D, page, tokens of the first request whose K or V is not finite
    ([17], [400], 8, 2, 128, 16, (0, 9, 16)),
    ([17, 3], [130, 40], 8, 2, 64, 16, (1, 2, 14)),   # the chunk lies over two tiles
    ([5, 2], [5, 30], 4, 2, 64, 16, (0, 1, 4)),
    ([10], [4], 4, 2, 64, 16, (6, 9)),                # the first tokens see nothing
    ([64, 1], [900, 50], 32, 8, 128, 16, (3, 62)),
    ([300], [300], 8, 1, 128, 64, (0, 31, 32, 130, 299)),
    ([129, 40], [700, 40], 16, 2, 96, 16, (5, 128)),
    ([20], [6001], 32, 2, 128, 16, (19, 4)),          # many CTAs, cut pieces
    ([80], [3000], 10, 2, 40, 24, (79, 0, 44)),
    ([4, 2], [9, 3], 130, 1, 64, 16, (1, 3)),
    ([20], [90], 4, 2, 256, 16, (7, 19)),
    ([3], [20], 2, 1, 12, 5, (1,)),
    ([300], [700], 2, 2, 128, 16, (0, 130, 299)),     # one query head a K/V head: masks over several tiles
    ([700], [700], 1, 1, 64, 64, (0, 200, 511, 699)),
    ([260, 2], [3000, 5], 2, 2, 128, 24, (1, 255)),
]


@pytest.mark.parametrize("what", ["v nan", "v inf", "v -inf", "k nan"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n", range(len(HIDDEN)))
def test_later_tokens_that_are_not_finite_stay_out_of_earlier_rows(dtype, what, n):
    *shape, places = HIDDEN[n]
    i = make(dtype, *shape, layout="thd" if n % 2 else "htd", seed=50 + n)
    out, lse, tol, tol_lse = reference(i)
    count, L, G = shape[0][0], shape[1][0], shape[2] // shape[3]
    clean = [i[x].clone() for x in "kv"]
    for a in places:
        i["k"].copy_(clean[0])
        i["v"].copy_(clean[1])
        p = L - count + a
        page = i["table"][0, p // i["page"]].long()
        if what[0] == "v":
            i["v"][0, page, p % i["page"], 0, 3] = float(what[2:])
        else:
            i["k"][0, page, p % i["page"], 0, 5] = math.nan
        r = attend(i)
        got, got_lse = r["out"].cpu().double(), r["lse"].cpu().double()
        sees = torch.zeros(lse.shape, dtype=torch.bool)  # rows of the first K/V head from token a on
        sees[a:count, :G] = True
        assert not got[sees][:, 3].isfinite().any(), a
        rest, none = ~sees, torch.isinf(lse)
        assert ((got - out).abs() <= tol)[rest].all(), a
        assert (got_lse[rest & none] == -math.inf).all()
        assert ((got_lse - lse).abs() <= tol_lse)[rest & ~none].all(), a


def test_attention_with_large_scores_and_a_growing_maximum():
    # keys in order of rising score: every tile raises the running maximum
    for dtype in (F32, BF16):
        i = make(dtype, [4], [1000], 4, 2, 64, 16, seed=9)
        ramp = torch.linspace(0, 30, 1008)
        pages = i["table"][0, :63].long()
        unit = torch.zeros(64)
        unit[0] = 1
        k = (ramp.view(63, 16, 1, 1) * unit).expand(63, 16, 2, 64).to(dtype)
        i["k"][0][pages] = k.cuda()
        i["qkv"][:] = 0
        i["qkv"][:, :, 0] = 16.0
        check(i, attend(i))


@pytest.mark.parametrize("level", [-300.0, -90.0, 90.0, 300.0])
def test_scores_far_from_zero(level):
    # every score of a row is near `level`: nothing may under- or overflow
    for dtype in (F32, BF16):
        i = make(dtype, [4, 20], [500, 150], 4, 2, 64, 16, seed=22)
        i["qkv"][:, :, 0] = 16.0
        i["k"][..., 0] = torch.where(i["k"][..., 0].isnan(), i["k"][..., 0], level * 8 / 16.0)
        check(i, attend(i))


def test_rows_that_fall_and_rise():
    # a run of low tiles, one far above them, then low ones again
    for dtype in (F32, BF16):
        i = make(dtype, [3], [1100], 4, 2, 64, 16, seed=23)
        pages = i["table"][0, :69].long()
        lev = torch.full((69, 16), -200.0)
        lev[30:33] = 150.0
        lev[50] = 155.0
        i["qkv"][:, :, 0] = 16.0
        k = i["k"][0][pages]
        k[..., 0] = (lev * 8 / 16.0)[:, :, None].to(dtype).cuda()
        i["k"][0][pages] = k
        check(i, attend(i))


@pytest.mark.parametrize("chunks", [[3], [70]], ids=["few", "many"])
@pytest.mark.parametrize("rise", [[64], [100, 230], [64, 192, 320, 448], [192, 193, 700]])
def test_a_maximum_that_rises_inside_a_tile(rise, chunks):
    # the level goes up by 50 (72 in units of log2) at each of these positions
    for dtype in (F32, BF16):
        i = make(dtype, chunks, [1100], 8, 2, 128, 16, seed=24)
        pages = i["table"][0, :69].long()
        pos = torch.arange(69 * 16)
        lev = sum(((pos >= x).float() * 50.0 for x in rise), -20.0 + 0 * pos)
        i["qkv"][:, :, 0] = 16.0
        k = i["k"][0][pages]
        k[..., 0] = (lev * math.sqrt(128) / 16.0).view(69, 16, 1).to(dtype).cuda()
        i["k"][0][pages] = k
        check(i, attend(i))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_scales(scale):
    for dtype in (F32, BF16):
        i = make(dtype, [3, 20], [300, 40], 8, 2, 128, 16, seed=21)
        i["scale"] = scale
        check(i, attend(i))


def test_padding_rows_are_left_alone():
    i = make(BF16, [2, 3], [40, 60], 8, 2, 128, 16, seed=11)
    q = torch.cat([i["q"], torch.full_like(i["q"][:2], math.nan)])
    out = torch.full((7, 8, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((7, 8), 7.0, device="cuda")
    cache = dspark.PagedCache(i["k"], i["v"])
    r = dspark.dspark_paged_attention(q, cache, 0, i["off"], i["lens"], i["table"], i["scale"], out=out, lse=lse)
    assert dspark.dspark_read_device_status(r["workspace"]) == 0
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    check(i, dict(out=out[:5], lse=lse[:5]))


def test_results_do_not_change_between_calls_or_with_a_used_workspace():
    i = make(BF16, [17, 1, 5], [3000, 900, 77], 32, 8, 128, 16, seed=12)
    a = attend(i)
    ws = torch.randint(0, 255, (a["workspace"].numel(),), dtype=torch.uint8, device="cuda")
    b = attend(i, workspace=ws)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_another_stream():
    i = make(BF16, [17, 1], [600, 90], 32, 8, 128, 16, seed=13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = attend(i, stream=s)
    s.synchronize()
    check(i, r)


@pytest.mark.parametrize("layout", ["thd", "htd"])
def test_pools_past_32_bit_offsets(layout):
    # 2.7 G elements in K and in V; the pages in use are the last ones
    n_pages, page, Hkv, D = 41000, 64, 8, 128
    shape = (1, n_pages, page, Hkv, D) if layout == "thd" else (1, n_pages, Hkv, page, D)
    free, _ = torch.cuda.mem_get_info()
    if free < 4 * n_pages * page * Hkv * D + (4 << 30):
        pytest.skip("not enough free device memory")
    i = make(BF16, [17, 1], [200, 130], 16, Hkv, D, page, seed=14, spare=0)
    k, v = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(2))
    kk, vv = (t if layout == "thd" else t.transpose(2, 3) for t in (k, v))
    m = i["k"].shape[1]
    kk[:, -m:] = i["k"]
    vv[:, -m:] = i["v"]
    big = dict(i, k=kk, v=vv, table=torch.where(i["table"] >= 0, i["table"] + (n_pages - m), -1).int())
    r = attend(big)
    check(i, r)


def test_bad_device_inputs_are_flagged_and_stay_in_bounds():
    i = make(BF16, [2, 3], [40, 60], 8, 2, 128, 16, seed=15, poison=False)
    cache = dspark.PagedCache(i["k"], i["v"])
    n_pages = i["k"].shape[1]

    def status(**kw):
        a = dict(i, **kw)
        r = dspark.dspark_paged_attention(a["q"], cache, 0, a["off"], a["lens"], a["table"], a["scale"])
        return dspark.dspark_read_device_status(r["workspace"])

    bad = i["table"].clone()
    bad[0, 1] = n_pages
    assert status(table=bad) == 1
    bad[0, 1] = -1
    assert status(table=bad) == 1
    assert status(lens=torch.tensor([40, 1 << 20], dtype=torch.int32, device="cuda")) == 1
    assert status(lens=torch.tensor([-3, 60], dtype=torch.int32, device="cuda")) == 1
    assert status(off=torch.tensor([0, 2, 9], dtype=torch.int32, device="cuda")) == 1
    assert status(off=torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda")) == 1
    assert status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_request_of_2_to_the_31_positions(dtype):
    # The longest request there is, 2^31 - 2^16 positions, whose table names one
    # page of 65,536 again and again: 32,767 times its keys, so the same
    # probabilities over it.  Chains of sums: l adds 2^26 / 304 tiles of 32 keys
    # a lane (bf16: 2^24 / 152 / 2 tiles of 64 pairs), out 2^31 / 304 keys one
    # after another (bf16: 8 products a tile, truncated at 2^-23).
    longest = 2 ** 31 - 2 ** 16
    i = make(dtype, [1], [65536], 2, 1, 16, 65536, seed=33, poison=False)
    i["table"] = torch.full((1, 32768), int(i["table"][0, 0]), dtype=torch.int32, device="cuda")
    cache = dspark.PagedCache(i["k"], i["v"])

    def call(L):
        r = dspark.dspark_paged_attention(i["q"], cache, 0, i["off"], torch.tensor([L], dtype=torch.int32, device="cuda"),
                                          i["table"], i["scale"])
        return r, dspark.dspark_read_device_status(r["workspace"])

    want, lse, tol, tol_lse = reference(i)
    lse = lse + math.log(longest // 65536)
    r, status = call(longest)
    assert status == 0
    chain = (2 ** 31 / 304 * U) if dtype == F32 else 2 ** 24 / 152 * 8 * 2 * U
    mix = 1.0  # sum p |v| of normal values: 0.8
    assert ((r["out"].cpu().double() - want).abs() <= tol + chain * mix).all()
    assert ((r["lse"].cpu().double() - lse).abs() <= tol_lse + 2 ** 26 / 304 * U + 4 * U * lse.abs()).all()
    for L in (longest + 1, 2 ** 31 - 1):
        b, status = call(L)
        assert status == 1 and torch.equal(b["out"], r["out"])  # clamped


def test_offsets_that_do_not_start_at_zero_are_flagged():
    # rows before the first offset belong to no request and get no result
    for dtype in (F32, BF16):
        i = make(dtype, [2, 3], [40, 60], 8, 2, 64, 16, seed=36)
        cache = dspark.PagedCache(i["k"], i["v"])
        for off, want in (([1, 2, 5], 1), ([2, 2, 5], 1), ([0, 0, 5], 0), ([0, 2, 4], 0)):
            r = dspark.dspark_paged_attention(i["q"], cache, 0, torch.tensor(off, dtype=torch.int32, device="cuda"),
                                              i["lens"], i["table"], i["scale"])
            assert dspark.dspark_read_device_status(r["workspace"]) == want, off


def test_no_rows_and_offsets_past_them_are_flagged():
    i = make(BF16, [2, 3], [40, 60], 8, 2, 64, 16, seed=37)
    cache = dspark.PagedCache(i["k"], i["v"])
    for off, want in (([0, 0, 0], 0), ([0, 0, 1], 1)):
        r = dspark.dspark_paged_attention(i["q"][:0], cache, 0, torch.tensor(off, dtype=torch.int32, device="cuda"),
                                          i["lens"], i["table"], i["scale"])
        assert dspark.dspark_read_device_status(r["workspace"]) == want, off


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("L", [2 ** 31 - 2 ** 16, 2 ** 31 - 2 ** 16 + 1, 2 ** 31 - 1])
def test_append_at_the_last_positions(L):
    i = make(BF16, [2], [2], 2, 2, 8, 65536, seed=34, poison=False, spare=1)
    k0, longest = i["k"].clone(), 2 ** 31 - 2 ** 16
    table = torch.full((1, 32768), 1, dtype=torch.int32, device="cuda")
    kn, vn = i["qkv"][:, 2:4], i["qkv"][:, 4:]
    r = dspark.dspark_cache_append(dspark.PagedCache(i["k"], i["v"]), 0, kn, vn, i["off"],
                                   torch.tensor([L], dtype=torch.int32, device="cuda"), table)
    assert dspark.dspark_read_device_status(r["workspace"]) == (0 if L <= longest else 1)
    for a, p in enumerate((L - 2, L - 1)):
        if p < longest:
            k0[0, 1, p % 65536] = kn[a]
    assert torch.equal(i["k"], k0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["thd", "htd"])
@pytest.mark.parametrize("chunks,lens,Hkv,D,page", [
    ([1], [1], 1, 64, 16), ([17, 0, 1, 5], [17, 3, 40, 64], 8, 128, 16), ([3, 2], [3, 9], 2, 12, 5),
    ([1] * 300, [r % 7 + 1 for r in range(300)], 2, 64, 4), ([200, 300], [200, 900], 4, 128, 64), ([7], [7], 3, 20, 1),
])
def test_append_writes_the_chunk_and_nothing_else(dtype, layout, chunks, lens, Hkv, D, page):
    i = make(dtype, chunks, lens, Hkv, Hkv, D, page, layout=layout, layers=2, seed=3, poison=False)
    k0, v0 = i["k"].clone(), i["v"].clone()
    kn, vn = i["qkv"][:, Hkv:2 * Hkv], i["qkv"][:, 2 * Hkv:]
    r = dspark.dspark_cache_append(dspark.PagedCache(i["k"], i["v"]), 1, kn, vn, i["off"], i["lens"], i["table"])
    assert dspark.dspark_read_device_status(r["workspace"]) == 0
    table, t = i["table"].cpu(), 0
    for q, (n, L) in enumerate(zip(chunks, lens)):
        for a in range(n):
            p = L - n + a
            pg = int(table[q, p // page])
            k0[1, pg, p % page] = kn[t]
            v0[1, pg, p % page] = vn[t]
            t += 1
    assert torch.equal(i["k"], k0) and torch.equal(i["v"], v0)


def test_append_leaves_out_what_is_out_of_range():
    i = make(BF16, [4, 2], [2, 30], 2, 2, 64, 16, seed=4, poison=False)
    k0 = i["k"].clone()
    kn, vn = i["qkv"][:, 2:4], i["qkv"][:, 4:]
    cache = dspark.PagedCache(i["k"], i["v"])
    r = dspark.dspark_cache_append(cache, 0, kn, vn, i["off"], i["lens"], i["table"])  # positions -2, -1
    assert dspark.dspark_read_device_status(r["workspace"]) == 1
    t = i["table"].cpu()
    for row, (q, p) in zip((2, 3, 4, 5), ((0, 0), (0, 1), (1, 28), (1, 29))):
        k0[0, int(t[q, p // 16]), p % 16] = kn[row]
    assert torch.equal(i["k"], k0)
    bad = i["table"].clone()
    bad[1, 1] = 99
    r = dspark.dspark_cache_append(cache, 0, kn[4:], vn[4:], torch.tensor([0, 0, 2], dtype=torch.int32, device="cuda"),
                                   i["lens"], bad)
    assert dspark.dspark_read_device_status(r["workspace"]) == 1
    assert torch.equal(i["k"], k0)


@pytest.mark.parametrize("chunks,lens", [([2] * 600, [(5 * r) % 40 + 2 for r in range(600)]), ([700, 3, 650], [700, 9, 700])])
def test_append_flags_any_page_out_of_range(chunks, lens):
    i = make(BF16, chunks, lens, 2, 2, 64, 16, seed=25, poison=False)
    cache = dspark.PagedCache(i["k"], i["v"])
    kn, vn = i["qkv"][:, 2:4], i["qkv"][:, 4:]

    def status(table):
        return dspark.dspark_read_device_status(
            dspark.dspark_cache_append(cache, 0, kn, vn, i["off"], i["lens"], table)["workspace"])

    assert status(i["table"]) == 0
    R = len(lens)
    for r in (0, R // 2, R - 1):
        first, last = (lens[r] - chunks[r]) // 16, (lens[r] - 1) // 16
        for j in {first, (first + last) // 2, last}:
            for bad in (-1, i["k"].shape[1]):
                t = i["table"].clone()
                t[r, j] = bad
                assert status(t) == 1, (r, j)
        t = i["table"].clone()
        t[r, last + 1:] = 1 << 30  # pages that no token goes to
        t[r, :first] = -5
        assert status(t) == 0, r


def test_append_flags_offsets_past_the_rows():
    # the requests' positions would be counted, and never written
    i = make(BF16, [2, 3], [40, 60], 2, 2, 64, 16, seed=35, poison=False)
    cache = dspark.PagedCache(i["k"], i["v"])
    kn, vn = i["qkv"][:, 2:4], i["qkv"][:, 4:]

    def status(*off):
        r = dspark.dspark_cache_append(cache, 0, kn, vn, torch.tensor(off, dtype=torch.int32, device="cuda"), i["lens"],
                                       i["table"])
        return dspark.dspark_read_device_status(r["workspace"])

    assert status(0, 2, 5) == 0 and status(0, 2, 4) == 0
    assert status(0, 2, 6) == 1 and status(0, 2, 9) == 1     # the last one
    assert status(0, 6, 6) == 1 and status(0, 6, 7) == 1     # one before it
    assert status(0, 9, 5) == 1 and status(0, -1, 5) == 1
    none = kn[:0]
    r = dspark.dspark_cache_append(cache, 0, none, none, torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda"),
                                   i["lens"], i["table"])
    assert dspark.dspark_read_device_status(r["workspace"]) == 1


def test_append_of_unaligned_rows():
    # rows that start one element off a 16-byte boundary, and a pool that does
    for dtype in (F32, BF16):
        i = make(dtype, [3, 4], [20, 9], 2, 2, 64, 16, seed=6, poison=False)
        flat = torch.zeros(i["k"].numel() + 1, dtype=dtype, device="cuda")
        flat_v = torch.zeros_like(flat)
        k, v = flat[1:].view(i["k"].shape), flat_v[1:].view(i["k"].shape)
        k.copy_(i["k"])
        v.copy_(i["v"])
        wide = torch.randn(7, 4 * 64 + 1, device="cuda").to(dtype)
        kn, vn = wide[:, 1:129].unflatten(1, (2, 64)), wide[:, 129:].unflatten(1, (2, 64))
        dspark.dspark_cache_append(dspark.PagedCache(k, v), 0, kn, vn, i["off"], i["lens"], i["table"])
        dspark.dspark_cache_append(dspark.PagedCache(i["k"], i["v"]), 0, kn.contiguous(), vn.contiguous(), i["off"],
                                   i["lens"], i["table"])
        assert torch.equal(k, i["k"]) and torch.equal(v, i["v"])
        i["q"] = wide[:, 1:129].unflatten(1, (2, 64))
        i["k"], i["v"] = k, v
        check(i, attend(i))


def test_strides_of_dimensions_of_one():
    # they say nothing, so they need not agree: pools of one layer cut from arrays
    # of different depth, one head, one page, and a single new token
    for Hkv, lens in ((2, [20]), (1, [9])):
        i = make(BF16, [1], lens, 4, Hkv, 64, 16, seed=38, spare=0)
        v = torch.empty(3, *i["v"].shape[1:], dtype=BF16, device="cuda")[::3]
        v.copy_(i["v"])
        assert v.stride() != i["k"].stride()
        j = dict(i, v=v)
        check(i, attend(j))
        kn = i["qkv"][:, 4:4 + Hkv]                                   # token stride of the projection
        vn = torch.randn(1, Hkv, 64, device="cuda").bfloat16()        # and of an array of its own
        assert kn.stride() != vn.stride()
        r = dspark.dspark_cache_append(dspark.PagedCache(i["k"], v), 0, kn, vn, i["off"], i["lens"], i["table"])
        assert dspark.dspark_read_device_status(r["workspace"]) == 0
        p = lens[0] - 1
        pg = int(i["table"][0, p // 16])
        assert torch.equal(i["k"][0, pg, p % 16], kn[0]) and torch.equal(v[0, pg, p % 16], vn[0])


# ------------------------------------------------------------------ refusals
def test_refusals():
    i = make(BF16, [2, 3], [40, 60], 8, 2, 128, 16, seed=7)
    k, v = i["k"], i["v"]
    with pytest.raises(ValueError):
        dspark.PagedCache(k, v[:, :-1])
    with pytest.raises(ValueError):
        dspark.PagedCache(k, v.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError):
        dspark.PagedCache(k[0], v[0])
    with pytest.raises(TypeError):
        dspark.PagedCache(k.cpu(), v.cpu())
    with pytest.raises(TypeError):
        dspark.PagedCache(k.half(), v.half())
    cache = dspark.PagedCache(k, v)
    a = dict(q=i["q"], cache=cache, layer=0, q_offsets=i["off"], kv_len=i["lens"], page_table=i["table"], scale=0.1)

    def refused(kind, **kw):
        with pytest.raises(kind):
            dspark.dspark_paged_attention(**{**a, **kw})

    refused(TypeError, q=i["q"].float())
    refused(ValueError, q=i["q"][:, :, :64])
    refused(dspark.DSparkError, q=i["q"][:, :7])          # not a multiple of the K/V heads
    refused(dspark.DSparkError, layer=1)
    refused(dspark.DSparkError, layer=-1)
    refused(dspark.DSparkError, scale=math.nan)
    refused(TypeError, kv_len=i["lens"].long())
    refused(ValueError, kv_len=i["lens"][:1])
    refused(ValueError, q_offsets=i["off"][:2])
    refused(ValueError, page_table=i["table"][0])
    refused(ValueError, page_table=i["table"][:, ::2])
    refused(ValueError, out=torch.empty(5, 8, 64, dtype=BF16, device="cuda"))
    refused(TypeError, lse=torch.empty(5, 8, dtype=BF16, device="cuda"))
    refused(ValueError, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    kn = i["qkv"][:, 8:10]
    with pytest.raises(ValueError):
        dspark.dspark_cache_append(cache, 0, kn, kn.contiguous(), i["off"], i["lens"], i["table"])
    with pytest.raises(ValueError):
        dspark.dspark_cache_append(cache, 0, i["qkv"][:, :3], i["qkv"][:, :3], i["off"], i["lens"], i["table"])
    empty = dspark.dspark_paged_attention(i["q"][:0], cache, 0, torch.zeros_like(i["off"]), i["lens"], i["table"], 0.1)
    assert empty["out"].shape == (0, 8, 128)
