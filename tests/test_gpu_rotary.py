"""dspark_cache_append_rotary and dspark_cache_read against the definitions in 64 bits; page management of a
4-bit cache; a run of them together.

Tolerances: a rotated value is two products and a sum in fp32, 3 2^-24 (|a c| + |b s|), and its rounding to the
type (bf16 2^-8 relative).  Into a 4-bit cache the bytes are those of the formula, whatever the inputs (with
factors that are powers of two).
"""
import math

import pytest
import torch

import fp4
import speculative_decoding_draft_05_gb300 as dspark
from fp4 import BF16, F32, U

pytestmark = pytest.mark.gpu
BAD = dspark.binding.DEV_BAD_INPUT


def table_of(n, dim, seed=0):
    inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv + seed
    return torch.cat((a.cos(), a.sin()), 1).float().cuda()


def rotated(x, cs, interleaved):
    """x [T, H, D] in 64 bits, cs [T, dim]; and the sum of the two products' magnitudes."""
    dim = cs.shape[1]
    half = dim // 2
    j = torch.arange(half, device=x.device)
    a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
    c, s = cs[:, None, :half], cs[:, None, half:]
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def near(got, want, mag):
    tol = 3 * U * mag + (2.0 ** -8 * want.abs() if got.dtype == BF16 else U * want.abs())
    assert ((got.double() - want).abs() <= tol).all()


def make(cache, dtype, chunks, lens, Hq, Hkv, D, page, seed=0, layers=1, layout="thd", strided=False, pad=0,
         factors=(0.5, 2.0)):
    g = torch.Generator().manual_seed(seed)
    table, n_pages = fp4.tables(lens, page, 2, g)
    if cache == "fp4":
        k, v = (fp4.pool_of([layers, n_pages, Hkv, page // 16, 9 * D], g, strided) for _ in range(2))
        c = dspark.PagedCacheFp4(k, v, *factors)
    else:
        shape = [layers, n_pages, page, Hkv, D]
        k, v = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
        if layout == "htd":
            k, v = (x.transpose(2, 3).contiguous().transpose(2, 3) for x in (k, v))
        c = dspark.PagedCache(k, v)
    T = sum(chunks) + pad
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    off = torch.tensor([sum(chunks[:r]) for r in range(len(chunks) + 1)], dtype=torch.int32).cuda()
    q, kn, vn = qkv.split([Hq, Hkv, Hkv], 1)
    pos = torch.cat([torch.arange(n - a, n) for a, n in zip(chunks, lens)] + [torch.zeros(0, dtype=torch.long)]).cuda()
    req = torch.repeat_interleave(torch.arange(len(chunks)), torch.tensor(chunks)).cuda()
    return dict(cache=c, k=k, v=v, qkv=qkv, q=q, kn=kn, vn=vn, off=off, lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                table=table.cuda(), page=page, pos=pos, req=req, T=sum(chunks), n=max(lens) + 1)


def append(i, cos_sin, layer=0, status=0, **kw):
    r = dspark.dspark_cache_append_rotary(i["cache"], layer, i["kn"], i["vn"], i["off"], i["lens"], i["table"], cos_sin,
                                          **kw)
    assert dspark.dspark_read_device_status(r["workspace"], kw.get("stream")) == status
    return r


def check(i, cs, interleaved, before, q=None, layer=0, keep=None):
    """The cache and q after an append; cs: each token's row of the table (None: no rotation); keep: tokens that
    were written."""
    T, fp = i["T"], isinstance(i["cache"], dspark.PagedCacheFp4)
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if keep is None else keep
    at = (i["pos"][keep], i["req"][keep])
    pg, slot = i["table"].long()[at[1], at[0] // i["page"]], at[0] % i["page"]
    turn = (lambda x: rotated(x, cs.double(), interleaved)) if cs is not None else (lambda x: (x, torch.zeros_like(x)))
    for name, new in (("k", i["kn"]), ("v", i["vn"])):
        want, mag = new[:T].double(), torch.zeros_like(new[:T], dtype=torch.float64)
        if name == "k":
            want, mag = turn(want)
        want, mag = want[keep], mag[keep]
        pool, old = i[name], before[name]
        if fp:
            codes, scales = fp4.parts(pool)
            c, s = fp4.encode(want, i["cache"].k_factor if name == "k" else i["cache"].v_factor)
            got = codes[layer, pg, :, slot // 16, slot % 16]
            # (the sign of a zero is its element's)
            z = lambda b: b & ~(((b & 7) == 0).to(torch.uint8) * 8 + ((b & 0x70) == 0).to(torch.uint8) * 128)  # noqa: E731
            assert torch.equal(scales[layer, pg, :, slot // 16, slot % 16], s)
            assert torch.equal(z(got), z(c))
            oc, os_ = fp4.parts(old)
            oc[layer, pg, :, slot // 16, slot % 16] = got
            os_[layer, pg, :, slot // 16, slot % 16] = s
            assert torch.equal(pool, old)  # nothing else changed
        else:
            got = pool[layer, pg, slot]
            if name == "k":
                near(got, want, mag)
            else:
                assert torch.equal(got, new[:T][keep])
            old[layer, pg, slot] = got
            assert torch.equal(pool, old)
    if q is not None:
        want, mag = turn(i["q"][:T].double())
        near(q[:T][keep], want[keep], mag[keep])


SHAPES = [
    # chunks, lens, Hq, Hkv, D, page, dim, interleaved
    ([1], [1], 1, 1, 64, 16, 64, False),
    ([1, 1, 1], [1, 16, 17], 8, 2, 128, 16, 128, False),
    ([3, 0, 2], [5, 0, 40], 4, 2, 64, 16, 64, True),
    ([17, 1, 9], [255, 256, 257], 32, 8, 128, 64, 128, False),
    ([17, 20], [400, 20], 40, 8, 128, 32, 64, False),     # half a head rotated
    ([5, 4], [50, 4], 12, 3, 96, 16, 96, False),
    ([5, 4], [50, 4], 4, 4, 96, 48, 48, True),
    ([5, 4], [50, 4], 4, 2, 96, 16, 16, False),           # pairs eight apart
    ([5, 4], [50, 4], 4, 2, 64, 16, 2, False),            # one pair
    ([5, 4], [50, 4], 4, 2, 64, 16, 6, True),
    ([5, 4], [50, 4], 4, 2, 64, 16, 34, False),
    ([2, 1], [65, 34], 4, 2, 256, 16, 256, False),
    ([2, 1], [65, 34], 4, 2, 160, 16, 160, True),
    ([300, 2], [300, 900], 7, 7, 32, 256, 32, False),
    ([1] * 300, [(r * 7) % 90 + 1 for r in range(300)], 6, 2, 128, 16, 128, False),
    ([2] * 1100, [(r % 30) + 2 for r in range(1100)], 2, 1, 64, 16, 64, False),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp4 of bf16", "fp4 of f32"])
@pytest.mark.parametrize("n", range(len(SHAPES)))
def test_append_matches_the_definition(kind, n):
    chunks, lens, Hq, Hkv, D, page, dim, inter = SHAPES[n]
    dtype = F32 if kind.endswith("f32") else BF16
    i = make("fp4" if "fp4" in kind else "rows", dtype, chunks, lens, Hq, Hkv, D, page, seed=n,
             layout="htd" if n % 2 else "thd", strided=n % 3 == 1, pad=3)
    before = dict(k=i["k"].clone(), v=i["v"].clone())
    tab = table_of(i["n"], dim)
    q0 = i["q"].clone()
    out = torch.full_like(q0, 7.0)
    r = append(i, tab, q=i["q"], q_out=out, interleaved=inter)
    assert r["q"] is out and torch.equal(i["q"], q0) and (out[i["T"]:] == 7).all()
    check(i, tab[i["pos"]], inter, before, out)
    # in place, with the same bytes
    again = dict(k=i["k"].clone(), v=i["v"].clone())
    i["kn"], i["vn"] = i["kn"].clone(), i["vn"].clone()
    append(i, tab, q=i["q"], q_out=i["q"], interleaved=inter)
    assert torch.equal(i["q"][:i["T"]], out[:i["T"]]) and torch.equal(i["q"][i["T"]:], q0[i["T"]:])
    assert torch.equal(i["k"], again["k"]) and torch.equal(i["v"], again["v"])


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp4 of bf16", "fp4 of f32"])
@pytest.mark.parametrize("dim, inter", [(128, False), (128, True), (64, False), (64, True), (96, True), (0, False), (48, False), (112, False),
                                        (12, False), (6, True)])
def test_from_few_tokens_to_more_than_run_at_once(kind, dim, inter):
    # a token's rows are dealt to one warp or to several, by the tokens there are
    dtype = F32 if kind.endswith("f32") else BF16
    for chunks, Hq, Hkv in (([2, 9], 32, 8), ([300, 1, 130], 32, 2), ([700], 20, 3), ([1300, 5], 9, 8), ([900, 1800], 4, 9)):
        i = make("fp4" if "fp4" in kind else "rows", dtype, chunks, [n + 30 for n in chunks], Hq, Hkv, 128, 16, seed=50,
                 layout="htd", pad=2)
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        tab = table_of(i["n"], dim) if dim else None
        out = torch.full_like(i["q"], 7.0)
        append(i, tab, q=i["q"], q_out=out, interleaved=inter)
        assert (out[i["T"]:] == 7).all()
        check(i, tab[i["pos"]] if dim else None, inter, before, out)
        append(i, tab, q=i["q"], q_out=i["q"], interleaved=inter)
        assert torch.equal(i["q"][:i["T"]], out[:i["T"]])


def test_rows_of_other_sizes_and_strides():
    # bf16 and fp32 caches of heads that are no multiple of 16, rows on odd addresses
    for dtype in (F32, BF16):
        for D, dim in ((12, 6), (40, 40), (80, 64), (7, 4), (129, 2)):
            for inter in (False, True):
                i = make("rows", dtype, [5, 2, 60], [50, 2, 60], 6, 3, D, 5, seed=D)
                wide = torch.randn(67, 12, D + 3).to(dtype).cuda()
                i["q"], i["kn"], i["vn"] = wide[:, :6, 1:D + 1], wide[:, 6:9, 1:D + 1], wide[:, 9:, 1:D + 1]
                before = dict(k=i["k"].clone(), v=i["v"].clone())
                tab = table_of(i["n"], dim)
                r = append(i, tab, q=i["q"], interleaved=inter)
                check(i, tab[i["pos"]], inter, before, r["q"])


def test_without_rotation_without_queries_and_a_later_layer():
    for cache, dtype in (("rows", F32), ("rows", BF16), ("fp4", F32), ("fp4", BF16)):
        i = make(cache, dtype, [5, 20], [50, 20], 4, 2, 64, 16, seed=3, layers=3)
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        append(i, None, layer=2)
        check(i, None, False, before, layer=2)
        if cache == "fp4":  # dspark_cache_append takes such a cache too
            again = dict(k=i["k"].clone(), v=i["v"].clone())
            r = dspark.dspark_cache_append(i["cache"], 2, i["kn"], i["vn"], i["off"], i["lens"], i["table"])
            assert dspark.dspark_read_device_status(r["workspace"]) == 0
            assert torch.equal(i["k"], again["k"]) and torch.equal(i["v"], again["v"])
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        tab = table_of(i["n"], 64)
        append(i, tab, layer=1)
        check(i, tab[i["pos"]], False, before, layer=1)


def test_given_positions():
    for cache, dtype in (("rows", BF16), ("fp4", BF16), ("rows", F32)):
        for D, dim in ((64, 64), (96, 20)):
            i = make(cache, dtype, [5, 20], [50, 20], 4, 2, D, 16, seed=4, pad=2)
            before = dict(k=i["k"].clone(), v=i["v"].clone())
            tab = table_of(100, dim)
            pos = torch.randint(0, 100, (27,), dtype=torch.int32).cuda()
            pos[25:] = 1 << 30  # padding
            r = append(i, tab, q=i["q"], positions=pos)
            check(i, tab[pos[:25].long()], False, before, r["q"])


def test_tokens_without_a_place_are_left_out():
    for cache, dtype in (("rows", BF16), ("fp4", BF16), ("fp4", F32)):
        for D, dim in ((64, 64), (96, 20)):
            tab = table_of(60, dim)
            # a page that is none; positions past the table, given or not
            for case in ("page", "short table", "positions"):
                i = make(cache, dtype, [5, 20], [50, 40], 4, 2, D, 16, seed=5)
                before = dict(k=i["k"].clone(), v=i["v"].clone())
                keep, kw, t = torch.ones(25, dtype=torch.bool, device="cuda"), {}, tab
                rows = tab[i["pos"].clamp(max=59)]
                if case == "page":
                    i["table"][1, 2] = 1 << 29
                    keep[5 + 12:] = False  # positions 32 .. 39 of request 1
                elif case == "short table":
                    t = tab[:47].contiguous()
                    keep[2:5] = False
                else:
                    pos = i["pos"].int()
                    pos[3], pos[7] = -1, 60
                    keep[3] = keep[7] = False
                    kw = dict(positions=pos)
                out = torch.full_like(i["q"], 7.0)
                append(i, t, status=BAD, q=i["q"], q_out=out, **kw)
                if case == "page":
                    i["table"][1, 2] = 0
                check(i, rows, False, before, out, keep=keep)
                assert (out[~keep] == 7).all()


def test_groups_that_are_not_finite_or_far_out():
    for dtype in (F32, BF16):
        i = make("fp4", dtype, [40], [40], 2, 2, 64, 16, seed=6, factors=(1.0, 0.25))
        i["qkv"][:] *= torch.logspace(-12, 8, 40, device="cuda")[:, None, None].to(dtype)
        kn, vn = i["kn"], i["vn"]
        kn[3, 0, 5], vn[4, 1, 40], vn[5, 0, 0] = math.nan, math.inf, -math.inf
        kn[6], vn[7] = 0, 0
        kn[8, 0, :16] = torch.tensor([0.0, -0.0] * 8)
        vn[9, 0, :16] = 3e38
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        append(i, None)
        check(i, None, False, before)


def test_borders_between_codes():
    # every bf16 multiple of a border: x / scale lies on a tie, or one step beside it
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    scale = fp4.E4M3[1:127]
    ties = (border[None] * scale[:, None]).flatten()
    for dtype in (F32, BF16):
        t = ties.to(dtype)
        t = t[t.double() == ties] if dtype == BF16 else t
        step = t.abs() * (2.0 ** -8 if dtype == BF16 else 2.0 ** -23)
        x = torch.stack((t, t + step, t - step, -t), 1).flatten()
        own = torch.stack((scale[:, None].expand(-1, 7).flatten(),) * 4, 1)[:len(t)].flatten() if dtype == F32 else None
        if own is None:
            keep = ties.to(dtype).double() == ties
            own = scale[:, None].expand(-1, 7).flatten()[keep][:, None].expand(-1, 4).flatten()
        x[-4 * 7:] = 0  # (scale 448: 6 times it is its own largest)
        n = len(x)
        rows = torch.zeros(-(-n // 64) * 64, 16, dtype=torch.float64)
        rows[:n, 0], rows[:n, 1] = x.double(), 6 * own  # the group's largest fixes its scale
        T = len(rows) // 4
        i = make("fp4", dtype, [T], [T], 1, 1, 64, 16, factors=(1.0, 4.0))
        i["kn"] = rows.view(T, 1, 64).to(dtype).cuda()
        i["vn"] = (4 * rows).view(T, 1, 64).to(dtype).cuda()
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        append(i, None)
        check(i, None, False, before)


def read(i, off, n, layer=0, status=0, **kw):
    r = dspark.dspark_cache_read(i["cache"], layer, off, i["lens"], i["table"], n, **kw)
    assert dspark.dspark_read_device_status(r["workspace"], kw.get("stream")) == status
    return r


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp4 as bf16", "fp4 as f32"])
def test_read_gives_back_what_the_cache_holds(kind):
    dtype = F32 if kind.endswith("f32") else BF16
    fp = "fp4" in kind
    for D, page, strided in ((64, 16, False), (128, 48, True), (96, 16, False), (256, 32, True)) + \
            (() if fp else ((12, 5, False), (7, 3, False))):
        i = make("fp4" if fp else "rows", dtype, [5, 0, 20], [50, 3, 130], 4, 3, D, page, seed=7, layers=2,
                 strided=strided, layout="htd" if strided else "thd")
        if fp:
            for x in "kv":
                fp4.parts(i[x])[1].random_(0, 256)
        for lens in ([5, 0, 20], [50, 3, 130]):
            off = torch.tensor([sum(lens[:r]) for r in range(4)], dtype=torch.int32).cuda()
            n = sum(lens)
            k, v = (torch.full((n + 2, 3, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
            r = read(i, off, n + 2, layer=1, dtype=dtype, k=k, v=v)
            assert r["k"] is k and (k[n:] == 7).all() and (v[n:] == 7).all()
            pos = torch.cat([torch.arange(L - a, L) for a, L in zip(lens, [50, 3, 130])]).cuda()
            req = torch.repeat_interleave(torch.arange(3), torch.tensor(lens)).cuda()
            pg, slot = i["table"].long()[req, pos // page], pos % page
            for name, got in (("k", k), ("v", v)):
                if fp:
                    f = i["cache"].k_factor if name == "k" else i["cache"].v_factor
                    want = fp4.values(i[name], f)[1, pg, slot].to(dtype)  # exact: six bits, powers of two
                else:
                    want = i[name][1, pg, slot]
                assert torch.equal(got[:n].nan_to_num(99.0), want.nan_to_num(99.0))
    i["table"][0, 0] = -1
    read(i, off, n, status=BAD)


def test_a_factor_that_is_no_power_of_two():
    # within half a step of fp32 the formula's: values next to a border may fall to its other side
    i = make("fp4", BF16, [300], [300], 4, 4, 128, 16, seed=8, factors=(0.3, 1.7))
    append(i, None)
    got = read(i, i["off"], 300, dtype=F32)
    for name, new, f in (("k", i["kn"], 0.3), ("v", i["vn"], 1.7)):
        c, s = fp4.encode(new, f)
        want = fp4.decode(c, s, f)
        y = new.double().unflatten(-1, (-1, 16))
        step = 2 * fp4.decode(c | 0x77, s, f).abs().unflatten(-1, (-1, 16)) / 6  # the widest gap between codes
        off = ((got[name].double() - want).abs() > 4 * U * want.abs())
        assert off.double().mean() < 1e-3
        assert ((got[name].double().unflatten(-1, (-1, 16)) - y).abs() <= 0.5 * step * (1 + 2.0 ** -3) + 4 * U * y.abs()).all()


# ---------------------------------------------------------------------------- pages
def test_pages_of_a_4_bit_cache_move_as_bytes():
    for strided in (False, True):
        for H, D in ((2, 64), (3, 32)):
            g = torch.Generator().manual_seed(9)
            lens = [40, 17, 64, 0, 0, 5]
            page = 16
            table, _ = fp4.tables(lens, page, 0, g)
            shape = [2, 24, H, 1, 9 * D]
            k, v = fp4.pool_of(shape, g, strided), fp4.pool_of(shape, g, strided)
            cache = dspark.PagedCacheFp4(k, v)
            rc = torch.zeros(24, dtype=torch.int32)
            rc[table[table >= 0].long()] = 1
            table, kv, rc = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), rc.cuda()

            def content(pool, t, r, n):
                return pool[:, t[r, : -(-n // page)].long()].clone()

            was = [[content(p, table, r, n) for r, n in enumerate(lens)] for p in (k, v)]
            f = dspark.dspark_pages_fork(cache, table, kv, torch.tensor([0, 1], dtype=torch.int32).cuda(),
                                         torch.tensor([3, 4], dtype=torch.int32).cuda(), rc)
            assert dspark.dspark_read_device_status(f["workspace"]) == 0
            assert f["kv_len"].tolist() == [40, 17, 64, 40, 17, 5]
            for p, w in zip((k, v), was):
                for r, a in ((3, 0), (4, 1), (0, 0), (2, 2)):
                    assert torch.equal(content(p, f["page_table"], r, lens[a]), w[a])
            new = torch.tensor([0, 20, 64, 60, 17, 5], dtype=torch.int32).cuda()
            s = dspark.dspark_pages_resize(cache, f["page_table"], f["kv_len"], new, f["refcount"])
            assert dspark.dspark_read_device_status(s["workspace"]) == 0
            assert s["kv_len"].tolist() == new.tolist()
            c = dspark.dspark_pages_compact(cache, s["page_table"], s["kv_len"], s["refcount"])
            assert dspark.dspark_read_device_status(c["workspace"]) == 0
            for p, w in zip((k, v), was):
                for r, a, n in ((3, 0, 40), (4, 1, 17), (2, 2, 64), (5, 5, 5)):
                    assert torch.equal(content(p, c["page_table"], r, n), w[a][:, : -(-n // page)])
            src, dst = torch.tensor([1], dtype=torch.int32).cuda(), torch.tensor([23], dtype=torch.int32).cuda()
            dspark.dspark_pages_copy(cache, src, dst)
            assert torch.equal(k[:, 1], k[:, 23]) and torch.equal(v[:, 1], v[:, 23])


# ---------------------------------------------------------------------------- together
@pytest.mark.parametrize("cache", ["rows", "fp4"])
def test_rounds_of_a_layer(cache):
    """Prompts, then rounds of drafted chunks with rejected suffixes: resize, append with K and Q rotated, attend;
    against the whole of it in 64 bits from what the cache was given."""
    R, Hq, Hkv, D, page, n_pages, most = 3, 8, 2, 128, 16, 40, 200
    g = torch.Generator().manual_seed(10)
    if cache == "fp4":
        c = dspark.PagedCacheFp4.zeros(1, n_pages, page, Hkv, D)
    else:
        c = dspark.PagedCache(*(torch.zeros(1, n_pages, page, Hkv, D, dtype=BF16, device="cuda") for _ in range(2)))
    tab = table_of(most, D)
    table = torch.full((R, 13), -1, dtype=torch.int32, device="cuda")
    kv, rc = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    K, V = [[torch.zeros(0, Hkv, D, dtype=torch.float64, device="cuda") for _ in range(R)] for _ in range(2)]
    ws = {}
    for chunks, cut in (([50, 33, 1], [0, 0, 0]), ([5, 1, 3], [2, 0, 1]), ([1, 1, 1], [0, 0, 0]), ([17, 4, 0], [9, 3, 0])):
        T = sum(chunks)
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(BF16).cuda()
        q, kn, vn = qkv.split([Hq, Hkv, Hkv], 1)
        off = torch.tensor([sum(chunks[:r]) for r in range(R + 1)], dtype=torch.int32).cuda()
        new = kv + off[1:] - off[:-1]
        st = dspark.dspark_pages_resize(c, table, kv, new, rc)
        table, kv, rc = st["page_table"], st["kv_len"], st["refcount"]
        a = dspark.dspark_cache_append_rotary(c, 0, kn, vn, off, kv, table, tab, q=q, workspace=ws.get("a"))
        ws["a"] = a["workspace"]
        r = dspark.dspark_paged_attention(a["q"], c, 0, off, kv, table, D ** -0.5, workspace=ws.get("r"))
        ws["r"] = r["workspace"]
        for w in (st["workspace"], ws["a"], ws["r"]):
            assert dspark.dspark_read_device_status(w) == 0
        for b in range(R):
            n, L = chunks[b], int(kv[b])
            at = slice(int(off[b]), int(off[b]) + n)
            kr, _ = rotated(kn[at].double(), tab[L - n:L].double(), False)
            stored = (lambda x: fp4.decode(*fp4.encode(x, 1.0), 1.0)) if cache == "fp4" else (lambda x: x.to(BF16).double())
            K[b], V[b] = torch.cat((K[b], stored(kr))), torch.cat((V[b], stored(vn[at].double())))
            assert len(K[b]) == L
            if n == 0:
                continue
            qr, mag = rotated(q[at].double(), tab[L - n:L].double(), False)
            near(a["q"][at], qr, mag)
            Kg, Vg = (x[b].repeat_interleave(Hq // Hkv, 1) for x in (K, V))
            s = torch.einsum("nhd,jhd->nhj", a["q"][at].double(), Kg) * D ** -0.5
            s.masked_fill_(torch.arange(L, device="cuda") > torch.arange(L - n, L, device="cuda")[:, None, None], -math.inf)
            p = torch.softmax(s, 2)
            want = torch.einsum("nhj,jhd->nhd", p, Vg)
            # (K's rotated rows may be a bf16 step off in a bf16 cache: 2^-8 of a score's terms)
            ds = 2.0 ** -8 * torch.einsum("nhd,jhd->nhj", a["q"][at].double().abs(), Kg.abs()).amax() * D ** -0.5
            tol = (2 * ds if cache == "rows" else 0) + 2.0 ** -7
            assert ((r["out"][at].double() - want).abs() <= tol * torch.einsum("nhj,jhd->nhd", p, Vg.abs()) + 1e-5).all()
        kept = kv - torch.tensor(cut, dtype=torch.int32).cuda()
        st = dspark.dspark_pages_resize(c, table, kv, kept, rc)
        table, kv, rc = st["page_table"], st["kv_len"], st["refcount"]
        for b in range(R):
            K[b], V[b] = K[b][:int(kv[b])], V[b][:int(kv[b])]


def test_in_a_graph_and_on_another_stream():
    side = torch.cuda.Stream()
    for cache, dtype in (("fp4", BF16), ("rows", BF16), ("fp4", F32)):
        for chunks, lens in (([1, 1], [50, 300]), ([20, 3], [50, 300])):
            i = make(cache, dtype, chunks, lens, 8, 2, 128, 16, seed=11)
            tab = table_of(i["n"], 128)
            every = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32).cuda()
            append_all = dict(i, off=every, T=sum(lens))
            qkv = torch.randn(sum(lens), 12, 128).to(dtype).cuda()
            _, append_all["kn"], append_all["vn"] = qkv.split([8, 2, 2], 1)
            append(append_all, tab)  # the cache is full

            def step(**kw):
                a = dspark.dspark_cache_append_rotary(i["cache"], 0, i["kn"], i["vn"], i["off"], i["lens"], i["table"],
                                                      tab, q=i["q"], workspace=kw.pop("wa", None), **kw)
                r = dspark.dspark_paged_attention(a["q"], i["cache"], 0, i["off"], i["lens"], i["table"], 0.1,
                                                  workspace=kw.pop("wr", None), **kw)
                b = dspark.dspark_cache_read(i["cache"], 0, i["off"], i["lens"], i["table"], i["T"], **kw)
                return a["q"], r["out"], r["lse"], b["k"], b["v"]

            want = [x.clone() for x in step()]
            side.wait_stream(torch.cuda.current_stream())
            got = step(stream=side)
            torch.cuda.current_stream().wait_stream(side)
            for x, y in zip(want, got):
                assert torch.equal(x, y)
            cap = torch.cuda.Stream()
            cap.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(cap):
                step()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=cap):
                    held = step()
            torch.cuda.current_stream().wait_stream(cap)
            i["k"].zero_(), i["v"].zero_()
            append(append_all, tab)
            for _ in range(3):
                for x in held:
                    x.fill_(3.0)
                graph.replay()
                torch.cuda.synchronize()
                for x, y in zip(want, held):
                    assert torch.equal(x, y)


def test_two_captured_graphs_share_workspaces():
    i = make("fp4", BF16, [17, 3], [900, 300], 8, 2, 128, 16, seed=12)
    j = make("fp4", BF16, [1, 1, 1], [700, 20, 90], 8, 2, 128, 16, seed=13)
    ws = torch.empty(dspark.paged_attention_workspace_bytes(i["cache"]), dtype=torch.uint8, device="cuda")
    for x in (i, j):
        for p in (x["k"], x["v"]):
            fp4.parts(p)[1].random_(0x28, 0x40)

    def step(x):
        return dspark.dspark_paged_attention(x["q"], x["cache"], 0, x["off"], x["lens"], x["table"], 0.1, workspace=ws)

    want, graphs = [], []
    for x in (i, j):
        r = step(x)
        want.append((r["out"].clone(), r["lse"].clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = step(x)
        graphs.append((g, r))
    for n in (0, 1, 1, 0, 1, 0, 0):
        graphs[n][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[n][1]["out"], want[n][0]) and torch.equal(graphs[n][1]["lse"], want[n][1])


# ---------------------------------------------------------------------------- the example
def dense_rotary(srv, tokens):
    """Logits [n, V] of a token sequence by the definition, positions by rotation."""
    s, m = srv.s, srv.m
    n = len(tokens)
    f = lambda x: x.double().cpu()  # noqa: E731
    h = f(m.embed)[tokens]
    mask = torch.ones(n, n).tril().bool()
    cs = f(m.cos_sin)[:n]
    for layer in range(s.layers):
        q, k, v = (h @ f(m.qkv[layer])).view(n, -1, s.D).split([s.Hq, s.Hkv, s.Hkv], dim=1)
        q, k = rotated(q, cs, False)[0], rotated(k, cs, False)[0]
        k, v = (x.repeat_interleave(s.Hq // s.Hkv, 1) for x in (k, v))
        a = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(s.D)
        p = torch.softmax(a.masked_fill(~mask, -math.inf), -1)
        h = h + torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1) @ f(m.out[layer])
    return h @ f(m.head)


def example():
    import importlib.util
    import os
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("paged_rounds_rotary", os.path.join(root, "examples", "paged_rounds.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules["paged_rounds_rotary"] = mod
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rows", "fp4"])
def test_the_serving_example_with_rotary_positions(kind, dtype):
    ex = example()
    srv = ex.Server(ex.Sizes(dtype=dtype, n_pages=40, rotary=True, fp4=kind == "fp4"), seed=3)
    g = torch.Generator().manual_seed(2)
    history = {}
    for slot, n in ((0, 3), (1, 17), (2, 40), (4, 2)):
        history[slot] = torch.randint(0, srv.s.V, (n,), generator=g).tolist()
        srv.prefill(slot, history[slot])
    # bf16: four products a layer and K's rotation round their results (2^-8 of values whose sums grow with two
    # layers of residuals); fp32: the same with 2^-24 and the sums' lengths.
    tol = 0.08 if dtype == BF16 else 1e-4
    for k in range(7):
        if k == 3:
            srv.fork(2, 5)
            history[5] = list(history[2])
        if k == 5:
            srv.end(1)
            del history[1]
            srv.compact()
        r = srv.round()
        off, chunk = r["offsets"].tolist(), r["chunk"].tolist()
        for slot in history:
            part = chunk[off[slot]: off[slot + 1]]
            got = r["logits"][off[slot]: off[slot + 1]].double().cpu()
            assert got.isfinite().all()
            if kind == "rows":
                want = dense_rotary(srv, history[slot][:-1] + part)[-len(part):]
                assert (got - want).norm() <= tol * want.norm(), (k, slot)
            history[slot] += [x for x in r["tokens"][slot].tolist() if x >= 0]
            assert srv.len[slot].item() == len(history[slot]) - 1
        held = torch.zeros(srv.s.n_pages, dtype=torch.int32)
        for row, n in zip(srv.table.tolist(), srv.len.tolist()):
            for p in row[: -(-n // srv.s.page)]:
                held[p] += 1
        assert torch.equal(held, srv.refcount.cpu())


# ---------------------------------------------------------------------------- what is easily forgotten
@pytest.mark.parametrize("interleaved", [False, True])
def test_borders_between_codes_with_rotation(interleaved):
    """Rotated values on a tie, and beside one by far less than fp32's step: K is a tie times a scale, and the
    other of its pair is turned in by a sine of 0 or of +-2^-40.  The bytes are the formula's."""
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    D, half = 64, 32
    for dtype in (F32, BF16):
        tab = torch.zeros(4, D, device="cuda")
        tab[:, :half] = 1.0
        tab[1, half:], tab[2, half:] = 2.0 ** -40, -2.0 ** -40
        tab[3, half:] = 1.0
        tab[3, :half] = 0.0  # a quarter turn: each of a pair becomes the other
        scales = fp4.E4M3[1:120]
        rows = torch.zeros(len(scales), D, dtype=torch.float64)
        for n, s in enumerate(scales.tolist()):
            for i in range(D):
                rows[n, i] = border[(n + i) % 7] * s * (-1) ** (i // 7)
            rows[n, ::16] = 6 * s  # fixes the groups' scales
        fits = (rows.to(dtype).double() == rows).all(1)
        rows = rows[fits] if fits.sum() > 20 else rows
        T = 4 * len(rows)
        i = make("fp4", dtype, [T], [T], 1, 1, D, 16, factors=(1.0, 1.0))
        i["kn"] = rows.repeat_interleave(4, 0).view(T, 1, D).to(dtype).cuda()
        i["vn"] = torch.zeros_like(i["kn"])
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        pos = (torch.arange(T, dtype=torch.int32) % 4).cuda()
        append(i, tab, positions=pos, interleaved=interleaved)
        check(i, tab[pos.long()], interleaved, before)


def test_large_chunks_take_whole_tokens_a_warp():
    for kind, dtype in (("rows", BF16), ("fp4", BF16), ("rows", F32), ("fp4", F32)):
        for D, dim, inter in ((128, 128, False), (128, 64, False), (64, 64, True), (96, 32, True)):
            i = make(kind, dtype, [700, 650], [900, 650], 12, 3, D, 32, seed=15, pad=1)
            before = dict(k=i["k"].clone(), v=i["v"].clone())
            tab = table_of(i["n"], dim)
            r = append(i, tab, q=i["q"], interleaved=inter)
            check(i, tab[i["pos"]], inter, before, r["q"])


def test_rows_of_queries_with_other_strides_than_the_new_ones():
    for kind in ("rows", "fp4"):
        i = make(kind, BF16, [5, 20], [50, 20], 8, 2, 64, 16, seed=16)
        tab = table_of(i["n"], 64)
        want = append(i, tab, q=i["q"])["q"]
        wide = torch.full((25, 9, 3, 64), 7.0, dtype=BF16, device="cuda")
        out = wide[:, 1:, 1]
        assert append(i, tab, q=i["q"], q_out=out)["q"] is out
        assert torch.equal(out, want) and (wide[:, 0] == 7).all() and (wide[:, :, [0, 2]] == 7).all()
        odd = torch.full((25, 8, 65), 7.0, dtype=BF16, device="cuda")[:, :, 1:]  # rows that are no 16-byte vectors
        assert torch.equal(append(i, tab, q=i["q"], q_out=odd)["q"], want)


def test_calls_without_tokens():
    for kind in ("rows", "fp4"):
        i = make(kind, BF16, [0, 0], [50, 20], 8, 2, 64, 16, seed=17)
        before = dict(k=i["k"].clone(), v=i["v"].clone())
        r = append(i, table_of(60, 64), q=i["q"])
        assert r["q"].shape == (0, 8, 64)
        assert read(i, i["off"], 0)["k"].shape == (0, 2, 64)
        a = dspark.dspark_paged_attention(i["q"], i["cache"], 0, i["off"], i["lens"], i["table"], 0.1)
        assert a["out"].shape == (0, 8, 64) and dspark.dspark_read_device_status(a["workspace"]) == 0
        assert torch.equal(i["k"], before["k"]) and torch.equal(i["v"], before["v"])
        i["off"][2] = 3  # rows that the call was not given
        append(i, table_of(60, 64), status=BAD, q=i["q"])
        read(i, i["off"], 0, status=BAD)


def test_pages_past_2_to_the_32_bytes():
    n_pages, page, Hkv, D = 60000, 16, 8, 128   # 9216 bytes a page and head: 4.4 GB each of K and V
    k, v = (torch.empty(1, n_pages, Hkv, 1, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    cache = dspark.PagedCacheFp4(k, v)
    lens = [100, 30, 700]
    held = [-(-n // page) for n in lens]
    ids = torch.randperm(2000)[:sum(held)].int() + n_pages - 2000
    table = torch.full((3, max(held)), -1, dtype=torch.int32)
    for r, h in enumerate(held):
        table[r, :h] = ids[sum(held[:r]): sum(held[:r + 1])]
    small = make("fp4", BF16, lens, lens, 32, Hkv, D, page, seed=18, factors=(1.0, 1.0))
    big = dict(small, cache=cache, k=k, v=v, table=table.cuda())
    tab = table_of(800, D)
    qs = [append(x, tab, q=x["q"])["q"] for x in (small, big)]
    assert torch.equal(*qs)
    a, b = (read(x, x["off"], x["T"]) for x in (small, big))
    assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"])
    for counts in ([1, 1, 1], [17, 5, 200]):
        for q in (qs[0], qs[0].float()):
            off = torch.tensor([sum(counts[:r]) for r in range(4)], dtype=torch.int32).cuda()
            a, b = (dspark.dspark_paged_attention(q[:sum(counts)], x["cache"], 0, off, x["lens"], x["table"], 0.1)
                    for x in (small, big))
            assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    moved = torch.tensor([n_pages - 1], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    dspark.dspark_pages_copy(cache, *moved)
    assert torch.equal(k[:, n_pages - 1], k[:, 3]) and torch.equal(v[:, n_pages - 1], v[:, 3])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_rotated_values_nearer_to_a_border_than_fp32_tells(dtype, interleaved):
    """For random a, b and sine the cosine is the float for which a c - b s comes nearest to a border between two
    codes: mostly within 2^-25 of it, on either side.  The bytes are the formula's."""
    g = torch.Generator().manual_seed(30)
    T, D, half = 1500, 64, 32
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    scale = fp4.E4M3[40:80][torch.randint(0, 40, (T, 1), generator=g)]
    target = border[torch.randint(0, 7, (T, half), generator=g)] * scale * (1 - 2 * torch.randint(0, 2, (T, half), generator=g))
    a, b = ((torch.rand(T, half, generator=g) + 0.5) * scale * 3).to(dtype).double(), \
        (torch.randn(T, half, generator=g) * scale).to(dtype).double()
    sin = torch.rand(T, half, generator=g).float()
    cos = ((target + b * sin.double()) / a).float()
    per = 8 if interleaved else 16  # pairs whose first outputs are in one group of 16
    fix = torch.arange(0, half, per)
    a[:, fix], b[:, fix], cos[:, fix], sin[:, fix] = 6 * scale, 0.0, 1.0, 0.0  # the group's scale
    if interleaved:  # the others of the pairs lie in the same group: keep them small
        small = torch.arange(half) % per != 0
        b[:, small], sin[:, small] = 0.0, sin[:, small] * 0.25
        sin = sin.to(torch.float32)
        cos[:, small] = (target[:, small] / a[:, small]).float()
    y = a * cos.double() - b * sin.double()
    near_ = ((y - target).abs() <= 2.0 ** -23 * target.abs()).float().mean()
    assert near_ > 0.5
    rows = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    i = make("fp4", dtype, [T], [T], 1, 1, D, 16, factors=(1.0, 1.0))
    i["kn"] = rows.view(T, 1, D).to(dtype).cuda()
    i["vn"] = torch.zeros_like(i["kn"])
    tab = torch.cat((cos, sin), 1).cuda()
    before = dict(k=i["k"].clone(), v=i["v"].clone())
    append(i, tab, interleaved=interleaved)
    check(i, tab[i["pos"]], interleaved, before)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [64, 32])
def test_a_table_of_more_than_cosines_and_sines(dtype, interleaved, dim):
    """Tables scaled for long contexts hold more than 1; here products up to a thousand times the value that is
    left of them, next to a border between two codes.  The bytes are the formula's."""
    g = torch.Generator().manual_seed(31)
    T, D, half = 1500, 64, dim // 2
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    target = border[torch.randint(0, 7, (T, half), generator=g)]
    a = (torch.rand(T, half, generator=g) + 0.5).to(dtype).double()
    b = torch.randn(T, half, generator=g).to(dtype).double()
    sin = (torch.randn(T, half, generator=g) * 500).float()
    cos = ((target + b * sin.double()) / a).float()
    a[:, ::16], b[:, ::16], cos[:, ::16], sin[:, ::16] = 6.0, 0.0, 1.0, 0.0  # a group's scale is 1 (if it has one output)
    i = make("fp4", dtype, [T], [T], 1, 1, D, 16, factors=(1.0, 1.0))
    k = torch.zeros(T, D, dtype=torch.float64)
    j = torch.arange(half)
    k[:, 2 * j if interleaved else j], k[:, 2 * j + 1 if interleaved else j + half] = a, b
    i["kn"] = k.view(T, 1, D).to(dtype).cuda()
    i["vn"] = torch.zeros_like(i["kn"])
    tab = torch.cat((cos, sin), 1).cuda()
    before = dict(k=i["k"].clone(), v=i["v"].clone())
    append(i, tab, interleaved=interleaved)
    check(i, tab[i["pos"]], interleaved, before)
