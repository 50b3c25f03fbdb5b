"""Page management (resize, fork, compact, copy) against a plain model of a pool.

All outputs are whole numbers or copied values: they have to be equal.
"""
import random

import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NO_PAGES, BAD = 4, 1


class Pool:
    """The state on the device, and the same operations written over lists."""

    def __init__(self, R, P, n_pages, S, Hkv=2, D=8, layers=2, dtype=BF16, layout="thd", seed=0):
        self.R, self.P, self.n, self.S = R, P, n_pages, S
        self.tab, self.len, self.rc = [[-1] * P for _ in range(R)], [0] * R, [0] * n_pages
        g = torch.Generator().manual_seed(seed)
        shape = [layers, n_pages, S, Hkv, D] if layout == "thd" else [layers, n_pages, Hkv, S, D]
        k, v = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
        if layout == "htd":
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        self.cache = dspark.PagedCache(k, v)
        self.k, self.v = k.clone(), v.clone()  # what the pool has to hold
        self.free_pages = n_pages

    def dev(self):
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return i(self.tab), i(self.len), i(self.rc)

    def move(self, pairs):
        if pairs:
            s, d = (torch.tensor(x, device="cuda") for x in zip(*pairs))
            self.k[:, d], self.v[:, d] = self.k[:, s].clone(), self.v[:, s].clone()

    def resize(self, new):
        S, pairs, short = self.S, [], False
        for r in range(self.R):
            for j in range(-(-new[r] // S), -(-self.len[r] // S)):
                self.rc[self.tab[r][j]] -= 1
                self.tab[r][j] = -1
        free = [p for p in range(self.n) if self.rc[p] == 0]
        before = list(self.rc)
        for r in range(self.R):
            L, N = self.len[r], new[r]
            if N <= L:
                self.len[r] = N
                continue
            if L % S and before[self.tab[r][L // S]] > 1:
                if not free:
                    short = True
                    continue
                old, p = self.tab[r][L // S], free.pop(0)
                pairs.append((old, p))
                self.rc[old] -= 1
                self.rc[p] = 1
                self.tab[r][L // S] = p
            held = -(-L // S)
            while held < -(-N // S):
                if not free:
                    short = True
                    break
                p = free.pop(0)
                self.tab[r][held], self.rc[p] = p, 1
                held += 1
            self.len[r] = min(N, held * S)
        self.move(pairs)
        self.free_pages = self.rc.count(0)
        return NO_PAGES if short else 0

    def fork(self, pairs):
        S, moves, short = self.S, [], False
        free = [p for p in range(self.n) if self.rc[p] == 0]
        was = list(self.len)  # parents as they are before the call
        for a, b in pairs:
            full = was[a] // S
            for j in range(full):
                self.tab[b][j] = self.tab[a][j]
                self.rc[self.tab[a][j]] += 1
            self.len[b] = full * S
            if was[a] % S:
                if not free:
                    short = True
                    continue
                p = free.pop(0)
                moves.append((self.tab[a][full], p))
                self.tab[b][full], self.rc[p] = p, 1
                self.len[b] = was[a]
        self.move(moves)
        self.free_pages = self.rc.count(0)
        return NO_PAGES if short else 0

    def compact(self):
        n_live = sum(c > 0 for c in self.rc)
        to = [p if c > 0 else -1 for p, c in enumerate(self.rc)]
        low = [p for p in range(n_live) if self.rc[p] == 0]
        high = [p for p in range(n_live, self.n) if self.rc[p] > 0]
        for a, b in zip(high, low):
            to[a], self.rc[b], self.rc[a] = b, self.rc[a], 0
        self.tab = [[to[p] if j < -(-self.len[r] // self.S) else p for j, p in enumerate(row)]
                    for r, row in enumerate(self.tab)]
        self.move(list(zip(high, low)))
        return n_live, to

    def check(self, res, status, want_len=True):
        assert dspark.dspark_read_device_status(res["workspace"]) == status
        assert res["page_table"].cpu().tolist() == self.tab
        assert res["refcount"].cpu().tolist() == self.rc
        if want_len:
            assert res["kv_len"].cpu().tolist() == self.len
            assert res["free_pages"].item() == self.free_pages
        assert torch.equal(self.cache.k, self.k) and torch.equal(self.cache.v, self.v)

    # one step on both sides; in place or into new tensors
    def do_resize(self, new, in_place=False):
        t, n, c = self.dev()
        kw = dict(page_table_out=t, kv_len_out=n, refcount_out=c) if in_place else {}
        src = [x.clone() for x in (t, n, c)]
        r = dspark.dspark_pages_resize(self.cache, t, n, torch.tensor(new, dtype=torch.int32, device="cuda"), c, **kw)
        self.check(r, self.resize(new))
        if not in_place:
            assert all(torch.equal(a, b) for a, b in zip(src, (t, n, c)))

    def do_fork(self, pairs, in_place=False):
        t, n, c = self.dev()
        kw = dict(page_table_out=t, kv_len_out=n, refcount_out=c) if in_place else {}
        i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        r = dspark.dspark_pages_fork(self.cache, t, n, i([a for a, _ in pairs]), i([b for _, b in pairs]), c, **kw)
        self.check(r, self.fork(pairs))

    def do_compact(self, in_place=False):
        t, n, c = self.dev()
        kw = dict(page_table_out=t, refcount_out=c) if in_place else {}
        r = dspark.dspark_pages_compact(self.cache, t, n, c, **kw)
        n_live, to = self.compact()
        self.check(r, 0, want_len=False)
        assert r["n_live"].item() == n_live and r["page_map"].cpu().tolist() == to


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layout,dtype,S,D", [("thd", BF16, 4, 8), ("htd", BF16, 16, 64), ("thd", F32, 1, 4),
                                              ("htd", F32, 5, 3), ("thd", BF16, 8, 5)])
def test_a_long_random_history(in_place, layout, dtype, S, D):
    rng = random.Random(S * 100 + D)
    R, P = 23, 12
    p = Pool(R, P, 150, S, D=D, dtype=dtype, layout=layout, seed=S)
    for step in range(40):
        u = rng.random()
        if u < 0.55 or step == 0:
            new = []
            for r in range(R):
                L, w = p.len[r], rng.random()
                new.append(0 if w < 0.1 else max(0, L - rng.randint(0, 2 * S + 1)) if w < 0.4
                           else min(P * S, L + rng.randint(0, 3 * S)))
            p.do_resize(new, in_place)
        elif u < 0.8:
            empty = [r for r in range(R) if p.len[r] == 0]
            rng.shuffle(empty)
            pairs = [(rng.randrange(R), b) for b in empty[: rng.randint(0, 6)]]
            pairs = [(a, b) for a, b in pairs if a not in empty[:6] or p.len[a] == 0]
            if pairs:
                p.do_fork(pairs, in_place)
        else:
            p.do_compact(in_place)


def test_a_request_cut_into_a_shared_page_gets_its_own_copy():
    p = Pool(4, 6, 30, 4)
    p.do_resize([16, 0, 0, 0])
    p.do_fork([(0, 1), (0, 2)])
    p.do_resize([16, 10, 9, 0])          # 1 and 2 end inside the shared third page
    p.do_resize([17, 11, 13, 3])         # growing copies it for both
    assert p.tab[0][2] != p.tab[1][2] != p.tab[2][2]


def test_all_holders_of_a_partial_page_grow():
    p = Pool(3, 6, 30, 4)
    p.do_resize([8, 0, 0])
    p.do_fork([(0, 1)])
    p.do_resize([6, 6, 0])
    before = p.free_pages
    p.do_resize([7, 7, 0])               # both copy, the old page is free afterwards
    assert p.free_pages == before - 1


def test_running_out_of_pages():
    p = Pool(5, 8, 7, 4)
    p.do_resize([9, 9, 9, 9, 0])         # 7 of 12 pages: 3, 3, 1, 0
    assert p.len == [9, 9, 4, 0, 0]
    p.do_resize([9, 9, 4, 1, 0])         # still none
    p.do_resize([0, 9, 4, 0, 0])
    p.do_fork([(1, 3), (1, 4)])          # one page each for the copied ends
    p.do_resize([1, 9, 4, 9, 9])
    p2 = Pool(3, 4, 3, 4)
    p2.do_resize([10, 0, 0])
    p2.do_fork([(0, 1)])                 # no page for the last one: 8 positions
    assert p2.len[1] == 8
    p2.do_resize([5, 8, 0])              # 0 ends inside a page that 1 shares; page 2 is free again
    p2.do_resize([6, 8, 0])
    p2.do_resize([6, 8, 9])              # nothing left


def test_nothing_to_do_and_everything_freed():
    p = Pool(6, 4, 20, 4)
    p.do_compact()
    p.do_resize([0] * 6)
    p.do_resize([16, 1, 4, 5, 0, 7])
    p.do_resize(list(p.len))
    p.do_compact()
    p.do_resize([0] * 6)
    assert p.free_pages == 20


@pytest.mark.parametrize("R,n_pages", [(1, 1), (1500, 9000), (3000, 70001)])
def test_many_requests_and_pages(R, n_pages):
    rng = random.Random(R)
    p = Pool(R, 6, n_pages, 2, Hkv=1, D=8, layers=1)
    p.do_resize([rng.randint(0, 12) for _ in range(R)])
    p.do_resize([rng.randint(0, 12) for _ in range(R)], in_place=True)
    p.do_compact()
    empty = [r for r in range(R) if p.len[r] == 0]
    full = [r for r in range(R) if p.len[r]]
    if empty and full:
        p.do_fork([(rng.choice(full), b) for b in empty])
    p.do_resize([rng.choice([0, n, min(12, n + 2)]) for n in p.len])
    p.do_compact(in_place=True)


def test_large_pages_and_large_tables():
    # shared pages of 256 KB each: their copies get a launch of their own
    p = Pool(70, 4, 220, 16, Hkv=8, D=128, layers=4)
    p.do_resize([40] + [0] * 69)
    p.do_fork([(0, b) for b in range(1, 70)])
    p.do_resize([24] * 70)               # all end inside the shared second page
    p.do_resize([25 + b % 9 for b in range(70)])
    p.do_resize([0] * 35 + [40] * 35, in_place=True)
    p.do_compact()
    # 1.2 M table entries: copied into the outputs by a launch of their own
    p = Pool(300, 4001, 2000, 1, Hkv=1, D=8, layers=1)
    p.do_resize([r % 13 for r in range(300)])
    p.do_fork([(1, 0), (12, 13), (11, 26)])
    p.do_compact()


def test_a_call_for_nothing_clears_the_status():
    p = Pool(3, 4, 16, 4)
    p.do_resize([5, 0, 3])
    t, n, c = p.dev()
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    r = dspark.dspark_pages_fork(p.cache, t, n, none, none, c, workspace=ws.clone())
    p.check(r, p.fork([]))
    r = dspark.dspark_pages_copy(p.cache, none, none, workspace=ws.clone())
    assert dspark.dspark_read_device_status(r["workspace"]) == 0
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    kv = torch.empty(0, 2, 8, dtype=BF16, device="cuda")
    r = dspark.dspark_cache_append(p.cache, 0, kv, kv, off, n, t, workspace=ws.clone())
    assert dspark.dspark_read_device_status(r["workspace"]) == 0
    big = torch.full((dspark.paged_attention_workspace_bytes(p.cache),), 255, dtype=torch.uint8, device="cuda")
    r = dspark.dspark_paged_attention(kv, p.cache, 0, off, n, t, 1.0, workspace=big)
    assert dspark.dspark_read_device_status(r["workspace"]) == 0 and r["out"].shape == (0, 2, 8)


def test_bad_device_inputs_are_flagged():
    p = Pool(4, 4, 16, 4)
    p.do_resize([9, 5, 0, 0])
    t, n, c = p.dev()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def status(r):
        return dspark.dspark_read_device_status(r["workspace"])

    r = dspark.dspark_pages_resize(p.cache, t, n, i(9, 99, -1, 0), c)  # 99 > 4 pages, -1
    assert status(r) == BAD and r["kv_len"].tolist() == [9, 16, 0, 0]
    bad = t.clone()
    bad[0, 2] = 77
    r = dspark.dspark_pages_resize(p.cache, bad, n, i(4, 5, 0, 0), c)
    assert status(r) == BAD
    # forks: a child that holds pages, one named twice, ids out of range
    r = dspark.dspark_pages_fork(p.cache, t, n, i(0, 0, 0, 9), i(1, 2, 2, 3), c)
    assert status(r) == BAD and r["kv_len"].tolist() == [9, 5, 9, 0]
    r = dspark.dspark_pages_fork(p.cache, t, n, i(0, 1), i(4, 3), c)
    assert status(r) == BAD and r["kv_len"].tolist() == [9, 5, 0, 5]
    r = dspark.dspark_pages_compact(p.cache, bad, n, c)
    assert status(r) == BAD and r["page_table"][0, 2] == 77
    r = dspark.dspark_pages_copy(p.cache, i(1, 2), i(16, 3))
    assert status(r) == BAD


LONGEST = 2 ** 31 - 2 ** 16  # positions of a request


@pytest.mark.parametrize("want,status", [(LONGEST, NO_PAGES), (LONGEST + 1, NO_PAGES | BAD), (2 ** 31 - 1, NO_PAGES | BAD)])
def test_lengths_near_2_to_the_31(want, status):
    # 65,536 positions a page: a table of 32,768 entries holds 2^31
    p = Pool(2, 32768, 5, 65536, Hkv=1, D=8, layers=1)
    t, n, c = p.dev()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for L in (0, 7):
        # the first request takes two pages, the second one all that are left
        a = dspark.dspark_pages_resize(p.cache, t, i(0, 0), i(70000, L), c)
        b = dspark.dspark_pages_resize(p.cache, a["page_table"], a["kv_len"], i(70000, want), a["refcount"])
        assert dspark.dspark_read_device_status(b["workspace"]) == status
        assert b["kv_len"].tolist() == [70000, 3 * 65536] and b["free_pages"].item() == 0
        assert b["page_table"][:, :4].tolist() == [[0, 1, -1, -1], [2, 3, 4, -1]]
        assert (b["page_table"][:, 4:] == -1).all() and b["refcount"].tolist() == [1] * 5
        # ... and gives them back
        e = dspark.dspark_pages_resize(p.cache, b["page_table"], b["kv_len"], i(0, 0), b["refcount"])
        assert dspark.dspark_read_device_status(e["workspace"]) == 0
        assert (e["page_table"] == -1).all() and e["free_pages"].item() == 5


@pytest.mark.parametrize("layout", ["thd", "htd"])
@pytest.mark.parametrize("dtype,S,Hkv,D,layers", [(BF16, 16, 8, 128, 3), (F32, 4, 2, 64, 1), (BF16, 3, 2, 5, 2),
                                                  (F32, 1, 1, 1, 1), (BF16, 64, 1, 128, 2)])
def test_copy(layout, dtype, S, Hkv, D, layers):
    p = Pool(1, 1, 40, S, Hkv, D, layers, dtype, layout)
    order = torch.randperm(40)
    src, dst = order[:13].int().cuda(), order[13:26].int().cuda()
    r = dspark.dspark_pages_copy(p.cache, src, dst)
    assert dspark.dspark_read_device_status(r["workspace"]) == 0
    p.move(list(zip(src.tolist(), dst.tolist())))
    assert torch.equal(p.cache.k, p.k) and torch.equal(p.cache.v, p.v)
    dspark.dspark_pages_copy(p.cache, src[:0], dst[:0])
    assert torch.equal(p.cache.k, p.k)


def test_copy_of_a_pool_with_gaps_and_k_v_in_one_array():
    kv = torch.randn(2, 20, 2, 4, 3, 20).bfloat16().cuda()  # [layers, pages, K/V, tokens, heads, dim], dim cut below
    k, v = kv[:, :, 0, :, :, :16], kv[:, :, 1, :, :, :16]
    want = kv.clone()
    s, d = torch.tensor([3, 7, 9]), torch.tensor([0, 19, 4])
    want[:, d, :, :, :, :16] = kv[:, s][:, :, :, :, :, :16]
    dspark.dspark_pages_copy(dspark.PagedCache(k, v), s.int().cuda(), d.int().cuda())
    assert torch.equal(kv, want)


def test_copy_past_32_bit_offsets():
    shape = (1, 41000, 64, 8, 128)  # 2.7 G elements in each pool
    free, _ = torch.cuda.mem_get_info()
    if free < 4 * 41000 * 65536 + (2 << 30):
        pytest.skip("not enough free device memory")
    k, v = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(2))
    for t in (k, v):
        t[:, 40998] = torch.randn(64, 8, 128).bfloat16().cuda()
    dspark.dspark_pages_copy(dspark.PagedCache(k, v), *(torch.tensor([x], dtype=torch.int32, device="cuda")
                                                        for x in (40998, 40999)))
    assert torch.equal(k[:, 40998], k[:, 40999]) and torch.equal(v[:, 40998], v[:, 40999])


def test_another_stream():
    p = Pool(4, 6, 30, 4)
    s = torch.cuda.Stream()
    t, n, c = p.dev()
    new = torch.tensor([9, 3, 0, 24], dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    r = dspark.dspark_pages_resize(p.cache, t, n, new, c, stream=s)
    assert dspark.dspark_read_device_status(r["workspace"], s) == 0
    p.resize(new.tolist())
    assert r["page_table"].tolist() == p.tab


def test_refusals():
    p = Pool(4, 4, 16, 4)
    t, n, c = p.dev()
    new = torch.zeros_like(n)
    with pytest.raises(TypeError):
        dspark.dspark_pages_resize(p.cache, t.long(), n, new, c)
    with pytest.raises(ValueError):
        dspark.dspark_pages_resize(p.cache, t, n[:3], new, c)
    with pytest.raises(ValueError):
        dspark.dspark_pages_resize(p.cache, t, n, new, c[:5])
    with pytest.raises(ValueError):
        dspark.dspark_pages_resize(p.cache, t, n, new, c, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        dspark.dspark_pages_resize(None, t, n, new, c)
    five = torch.zeros(5, dtype=torch.int32, device="cuda")
    with pytest.raises(dspark.DSparkError):
        dspark.dspark_pages_fork(p.cache, t, n, five, five, c)  # more pairs than requests
    with pytest.raises(ValueError):
        dspark.dspark_pages_fork(p.cache, t, n, five[:2], five[:3], c)
    with pytest.raises(ValueError):
        dspark.dspark_pages_copy(p.cache, five, five[:2])
    with pytest.raises(ValueError):
        dspark.dspark_pages_compact(p.cache, t, n, c, page_map=five)
