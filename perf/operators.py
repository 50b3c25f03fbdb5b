"""Measured cases of the serving operators: attention over the paged K/V cache,
writing to it, page management, and log-probabilities of emitted tokens.

``run`` computes an operator either in its plain form (``own`` false: elementary
torch operations in 32 bits) or through the package's public calls (``own``
true).  ``exact`` gives the same outputs from the definitions in 64 bits.
Lengths are part of a case; values come from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one small round of the fp32 validation workload (4 requests, gamma 4): latency
        dict(name="attn_f32_r4", op="attention", dtype="f32", R=4, chunk_lo=1, chunk=5, kv_lo=33, kv=300,
             Hq=8, Hkv=2, D=64, page=16, layout="thd", lens=1),
        # plain decoding, one token for each of 16 users: latency of a memory-bound call
        dict(name="attn_decode_r16", op="attention", dtype="bf16", R=16, chunk_lo=1, chunk=1, kv_lo=200, kv=2048,
             Hq=32, Hkv=8, D=128, page=16, layout="thd", lens=2),
        # the target's pass of a verify round: anchor + up to 16 drafted tokens for 64 requests
        dict(name="attn_verify_r64", op="attention", dtype="bf16", R=64, chunk_lo=1, chunk=17, kv_lo=500, kv=8192,
             Hq=32, Hkv=8, D=128, page=64, layout="htd", lens=3),
        # the same over long documents: few requests, the work lies along the cache; 5 query heads a K/V head
        dict(name="attn_long_r4", op="attention", dtype="bf16", R=4, chunk_lo=17, chunk=17, kv_lo=100001, kv=131072,
             Hq=40, Hkv=8, D=128, page=32, layout="thd", lens=4),
        # a prompt's chunk behind what is cached already: compute-bound
        dict(name="attn_prefill_r2", op="attention", dtype="bf16", R=2, chunk_lo=2901, chunk=4096, kv_lo=5000, kv=8192,
             Hq=32, Hkv=8, D=128, page=64, layout="thd", lens=5),
        # new K and V of one verify round of 512 requests
        dict(name="append_r512", op="append", dtype="bf16", R=512, chunk_lo=1, chunk=17, kv_lo=17, kv=1024,
             Hkv=8, D=128, page=16, layout="thd", lens=6),
        # new K and V of two long prompts, heads-first cache
        dict(name="append_prompt_r2", op="append", dtype="bf16", R=2, chunk_lo=8191, chunk=16384, kv_lo=8191, kv=16384,
             Hkv=8, D=128, page=64, layout="htd", lens=7),
        # the bookkeeping of a round of 512 requests: rejected suffixes freed, the next chunk's pages taken
        dict(name="resize_r512", op="resize", dtype="bf16", R=512, kv_lo=100, kv=1024, n_pages=40000, Hkv=4, D=64,
             page=16, layers=1, layout="thd", lens=8),
        # 64 prompts each continued a second time: shared full pages, the last one copied in all layers
        dict(name="fork_r64", op="fork", dtype="bf16", R=128, forks=64, kv_lo=100, kv=1024, n_pages=3000, Hkv=8, D=128,
             page=16, layers=8, layout="thd", lens=9),
        # a pool half in use and scattered, moved together in all layers
        dict(name="compact_2k", op="compact", dtype="bf16", R=64, kv_lo=100, kv=300, n_pages=2000, moves=500, Hkv=8,
             D=128, page=16, layers=8, layout="thd", lens=10),
        # log-probabilities of the small fp32 round's tokens: latency
        dict(name="logprobs_f32_r4", op="logprobs", dtype="f32", R=4, gamma=4, V=1024, top=5, T=1.0, lens=11),
        # answers of a round of 512 requests, gamma 16: about a third of the target rows emitted a token
        dict(name="logprobs_r512", op="logprobs", dtype="bf16", R=512, gamma=16, V=151936, top=20, T=1.0, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "resize", "fork", "compact", "logprobs",
                     "logprobs"])
    c = dict(op=op, dtype="bf16", lens=rng.randrange(1 << 20))
    if op == "logprobs":
        if rng.random() < 0.2:
            c["dtype"] = "f32"
        c.update(R=_log_int(rng, 1, 512), gamma=rng.randint(1, 16), V=8 * _log_int(rng, 128, 18992),
                 top=rng.choice([1, 5, 20, 32]), T=rng.choice([1.0, 0.7]))
        return c
    c.update(Hkv=rng.choice([1, 2, 4, 8]), page=rng.choice([16, 32, 64, 128]), layout=rng.choice(["thd", "htd"]))
    c["D"] = rng.choice([64, 128]) if op != "attention" else rng.choice([64, 128, 128, 128, 80, 96])
    if op == "attention":
        kind = rng.choice(["decode", "verify", "verify", "prefill"])
        if kind != "prefill" and rng.random() < 0.15:
            c["dtype"] = "f32"
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 4, 5, 7, 8])
        small = c["dtype"] == "f32"
        c["chunk"] = {"decode": 1, "verify": rng.randint(2, 17), "prefill": _log_int(rng, 100, 4096)}[kind]
        c["chunk_lo"] = 1 if kind != "prefill" else max(1, c["chunk"] // 2)
        c["kv"] = max(c["chunk"], _log_int(rng, 20, 4096 if small else 131072 if kind != "prefill" else 8192))
        c["kv_lo"] = max(c["chunk"], c["kv"] // rng.choice([1, 2, 10]))
        c["R"] = _log_int(rng, 1, 16 if small else 256 if kind != "prefill" else 4)
        while c["R"] > 1 and c["R"] * c["kv"] > 400000 // (8 if small else 1):
            c["R"] = (c["R"] + 1) // 2
        while c["R"] > 1 and c["R"] * c["chunk"] * c["kv"] * c["Hq"] > 2 * 4096 * 8192 * 32:
            c["R"] -= 1
        while c["chunk"] * c["kv"] * c["Hq"] > 2 * 4096 * 8192 * 32 and c["Hq"] > c["Hkv"]:
            c["Hq"] -= c["Hkv"]
        return c
    if op == "append":
        c["chunk"] = _log_int(rng, 1, 4096)
        c["chunk_lo"] = max(1, c["chunk"] // 8)
        c["R"] = max(1, min(512, _log_int(rng, 1, 512), 24000 // c["chunk"]))
        c["kv"] = c["chunk"] + _log_int(rng, 1, 2048)
        c["kv_lo"] = c["chunk"]
        return c
    c.update(kv=_log_int(rng, 40, 2000), layers=rng.choice([1, 2, 4, 8]))
    c["kv_lo"] = max(1, c["kv"] // 8)
    per = 2 + c["kv"] // c["page"]  # pages of one request at most
    page_bytes = c["layers"] * c["page"] * c["Hkv"] * c["D"] * 4
    most = min(40000, (1 << 30) // page_bytes)  # a pool of 1 GiB at most
    c["R"] = max(2, min(_log_int(rng, 2, 512), most // (4 * per)))
    if op == "resize":
        c["n_pages"] = c["R"] * (per + 4) + rng.randint(0, 2 * c["R"])
    elif op == "fork":
        c["forks"] = max(1, c["R"] // 2)
        c["n_pages"] = c["R"] * (per + 1) + rng.randint(0, 2 * c["R"])
    else:
        held = sum(-(-n // c["page"]) for n in _lens(c))
        c["n_pages"] = 2 * held + rng.randint(1, 100)
        c["moves"] = max(1, held // rng.choice([2, 4]))
    return c


def _lens(c):
    """kv_len of each request, from the case alone."""
    r = random.Random("len %d %d" % (c["lens"], c["kv"]))
    return [c["kv"]] + [r.randint(c["kv_lo"], c["kv"]) for _ in range(c["R"] - 1)]


def _chunks(c):
    """New tokens of each request, from the case alone."""
    r = random.Random("chunk %d %d" % (c["lens"], c["chunk"]))
    return [min(n, c["chunk"] if i == 0 else r.randint(c["chunk_lo"], c["chunk"])) for i, n in enumerate(_lens(c))]


def _new_lens(c):
    """Lengths after a round: most requests grow by the next chunk's net tokens,
    some are cut into their last page, a few end, some stay."""
    r = random.Random("new %d" % c["lens"])
    out = []
    for n in _lens(c):
        u = r.random()
        out.append(0 if u < 0.03 else max(0, n - r.randint(1, 40)) if u < 0.35 else n if u < 0.4 else n + r.randint(1, 17))
    return out


def _emits(c):
    """Emitted tokens of each request: a geometric accepted prefix and one more."""
    r = random.Random("emit %d" % c["lens"])
    out = []
    for _ in range(c["R"]):
        n = 1
        while n <= c["gamma"] and r.random() < 0.8:
            n += 1
        out.append(n)
    return out


def _max_pages(c):
    return -(-(c["kv"] + 32) // c["page"])


# ---------------------------------------------------------------------------- inputs
def _cache(c, g, layers, n_pages):
    """K and V pools seen as [layers, pages, tokens, heads, D]; "htd" stores heads before tokens."""
    shape = ([layers, n_pages, c["page"], c["Hkv"], c["D"]] if c["layout"] == "thd"
             else [layers, n_pages, c["Hkv"], c["page"], c["D"]])
    out = []
    for _ in range(2):
        t = torch.empty(shape, dtype=DTYPES[c["dtype"]], device=DEV).normal_(generator=g)
        out.append(t if c["layout"] == "thd" else t.transpose(2, 3))
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = dict(c=c)
    if c["op"] == "logprobs":
        n, V = c["R"] * (c["gamma"] + 1), c["V"]
        # target logits as the workloads have them: N(0, 3^2) and a Zipf(1.1) offset
        zipf = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
        Z = torch.empty(n, V, dtype=dt, device=DEV)
        for a in range(0, n, 512):
            b = min(n, a + 512)
            Z[a:b] = torch.randn(b - a, V, device=DEV, generator=g) * 3 + zipf
        s["Z"] = Z.view(c["R"], c["gamma"] + 1, V)
        # drawn tokens lie mostly among the frequent ids
        tok = (torch.rand(c["R"], c["gamma"] + 1, generator=cpu) ** 4 * V).int()
        tok[torch.arange(c["gamma"] + 1)[None] >= torch.tensor(_emits(c))[:, None]] = -1
        s["tokens"] = tok.to(DEV)
        return s
    lens = _lens(c)
    P = _max_pages(c)
    held = [-(-n // c["page"]) for n in lens]
    s["kv_len"] = _i32(lens)
    if c["op"] in ("attention", "append"):
        ch = _chunks(c)
        n_pages = sum(held) + 3
        perm = torch.randperm(n_pages, generator=cpu)
        T = sum(ch)
        s["T"] = T
        s["q_offsets"] = _i32([sum(ch[:i]) for i in range(len(ch))] + [T])
        s["k"], s["v"] = _cache(c, g, 1, n_pages)
        if c["op"] == "attention":
            s["q"] = torch.empty(T, c["Hq"], c["D"], dtype=dt, device=DEV).normal_(generator=g)
            s["scale"] = 1.0 / math.sqrt(c["D"])
        else:  # the new K and V are parts of one projection's output, as a model gives them
            qkv = torch.empty(T, 4 * c["Hkv"], c["D"], dtype=dt, device=DEV).normal_(generator=g)
            s["k_new"], s["v_new"] = qkv[:, 2 * c["Hkv"]:3 * c["Hkv"]], qkv[:, 3 * c["Hkv"]:]
        s["page_table"] = _table(lens, held, P, perm)
        return s
    n_pages = c["n_pages"]
    if c["op"] == "compact":  # exactly `moves` live pages lie at or above the number of live pages
        n_live, m = sum(held), c["moves"]
        low = torch.randperm(n_live, generator=cpu)[: n_live - m]
        high = n_live + torch.randperm(n_pages - n_live, generator=cpu)[:m]
        perm = torch.cat([low, high])[torch.randperm(n_live, generator=cpu)]
    else:
        perm = torch.randperm(n_pages, generator=cpu)
    if c["op"] == "fork":  # the second half of the requests is empty: the children
        for r in range(c["R"] - c["forks"], c["R"]):
            lens[r] = held[r] = 0
        s["kv_len"] = _i32(lens)
        s["parent"] = torch.randint(0, c["R"] - c["forks"], (c["forks"],), generator=cpu).int().to(DEV)
        s["child"] = (c["R"] - c["forks"] + torch.randperm(c["forks"], generator=cpu)).int().to(DEV)
    table = _table(lens, held, P, perm)
    rc = torch.zeros(n_pages, dtype=torch.int32)
    if c["op"] == "resize":
        # neighbours 4i and 4i+1 share the start of a prompt; of every fourth such pair the shorter one was cut
        # back into a shared page, which growing it has to copy first
        tab = table.cpu()
        for r in range(0, c["R"] - 1, 4):
            n = min(held[r], held[r + 1])
            n = n if r % 16 == 0 else n // 2
            tab[r + 1, :n] = tab[r, :n]
        table = tab.to(DEV)
        s["new_len"] = _i32(_new_lens(c))
    tab = table.cpu()
    rc.scatter_add_(0, tab[tab >= 0].long(), torch.ones(int((tab >= 0).sum()), dtype=torch.int32))
    s["page_table"], s["refcount"] = table, rc.to(DEV)
    s["k"], s["v"] = _cache(c, g, c["layers"], n_pages)
    return s


def _table(lens, held, P, perm):
    tab = torch.full((len(lens), P), -1, dtype=torch.int32)
    at = 0
    for r, h in enumerate(held):
        tab[r, :h] = perm[at: at + h].int()
        at += h
    return tab.to(DEV)


# ---------------------------------------------------------------------------- plain forms
def _attention_plain(s):
    c, q = s["c"], s["q"]
    kv, mq, page = c["kv"], c["chunk"], c["page"]
    off = s["q_offsets"].long()
    n, L = off[1:] - off[:-1], s["kv_len"].long()
    P = -(-kv // page)
    pages = s["page_table"][:, :P].long().clamp(min=0)
    j = torch.arange(P * page, device=DEV)
    has = (j < L[:, None])[:, :, None, None]
    K = torch.where(has, s["k"][0][pages].flatten(1, 2).float(), 0.0)  # [R, kv, Hkv, D]
    V = torch.where(has, s["v"][0][pages].flatten(1, 2).float(), 0.0)
    i = torch.arange(mq, device=DEV)
    qp = q[(off[:-1, None] + i).clamp(max=s["T"] - 1)].float()
    R, G = c["R"], c["Hq"] // c["Hkv"]
    qp = qp.view(R, mq, c["Hkv"], G, c["D"]).permute(0, 2, 3, 1, 4).reshape(R, c["Hkv"], G * mq, c["D"])
    S = (qp @ K.permute(0, 2, 3, 1)) * s["scale"]  # [R, Hkv, G mq, kv]
    pos = (L - n)[:, None] + i
    see = (j[None, None] <= pos[:, :, None])[:, None, None]  # [R, 1, 1, mq, kv]
    S = torch.where(see, S.view(R, c["Hkv"], G, mq, -1), -math.inf)
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(S - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(R, c["Hkv"], G * mq, -1) @ V.transpose(1, 2)).view(R, c["Hkv"], G, mq, c["D"])
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + torch.log(l))[..., 0]
    t = torch.arange(s["T"], device=DEV)
    r = torch.searchsorted(off, t, right=True) - 1
    at = t - off[r]
    return dict(out=o[r, :, :, at].reshape(s["T"], c["Hq"], c["D"]).to(q.dtype),
                lse=lse[r, :, :, at].reshape(s["T"], c["Hq"]))


def _append_plain(s):
    off, L = s["q_offsets"].long(), s["kv_len"].long()
    t = torch.arange(s["T"], device=DEV)
    r = torch.searchsorted(off, t, right=True) - 1
    pos = L[r] - off[r + 1] + t
    page, slot = s["page_table"].long()[r, pos // s["c"]["page"]], pos % s["c"]["page"]
    s["k"][0][page, slot] = s["k_new"]
    s["v"][0][page, slot] = s["v_new"]
    return dict(k=s["k"], v=s["v"])


def _copy_plain(s, src, dst):
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]


def _resize_plain(s):
    S = s["c"]["page"]
    tab, L, N, rc = (s[k].long() for k in ("page_table", "kv_len", "new_len", "refcount"))
    R, P = tab.shape
    old, new = (L + S - 1) // S, (N + S - 1) // S
    col = torch.arange(P, device=DEV)
    freed = (col >= new[:, None]) & (col < old[:, None])
    rc = rc.scatter_add(0, torch.where(freed, tab, 0).flatten(), -freed.long().flatten())
    free = rc == 0
    order = torch.argsort((~free).long(), stable=True)
    n_free = free.sum()
    row = torch.arange(R, device=DEV)
    at = (L // S).clamp(max=P - 1)
    last = tab[row, at].clamp(min=0)
    cow = (N > L) & (L % S != 0) & (rc[last] > 1)
    need = cow.long() + (new - old).clamp(min=0)
    start = need.cumsum(0) - need
    cow_done = cow & (start < n_free)
    grown = torch.minimum((n_free - start).clamp(min=0), need) - cow_done.long()
    held = torch.where(new > old, old + grown, torch.minimum(old, new))
    out_len = torch.where(N > L, torch.where(cow & ~cow_done, L, torch.minimum(N, held * S)), N)
    got = order[(start + cow)[:, None].add(col - old[:, None]).clamp(0, len(rc) - 1)]
    fresh = (col >= old[:, None]) & (col < held[:, None])
    out = torch.where(fresh, got, torch.where(col < held[:, None], tab, -1))
    own_page = order[start.clamp(max=len(rc) - 1)]
    out[row, at] = torch.where(cow_done, own_page, out[row, at])
    rc = rc.scatter_add(0, torch.where(cow_done, last, 0), -cow_done.long())
    rc = rc.scatter_add(0, torch.where(cow_done, own_page, 0), cow_done.long())
    rc = rc.scatter_add(0, torch.where(fresh, got, 0).flatten(), fresh.long().flatten())
    _copy_plain(s, last[cow_done], own_page[cow_done])
    return dict(page_table=out.int(), kv_len=out_len.int(), refcount=rc.int(), free_pages=(rc == 0).sum().int()[None],
                k=s["k"], v=s["v"])


def _fork_plain(s):
    S = s["c"]["page"]
    tab, L, rc, parent, child = (s[k].long() for k in ("page_table", "kv_len", "refcount", "parent", "child"))
    R, P = tab.shape
    free = rc == 0
    order = torch.argsort((~free).long(), stable=True)
    n_free = free.sum()
    n = L[parent]
    full, part = n // S, n % S != 0
    start = part.long().cumsum(0) - part.long()
    done = part & (start < n_free)
    col = torch.arange(P, device=DEV)
    shared = col < full[:, None]
    rows = torch.where(shared, tab[parent], -1)
    rc = rc.scatter_add(0, torch.where(shared, rows, 0).flatten(), shared.long().flatten())
    fresh = order[start.clamp(max=len(rc) - 1)]
    rc = rc.scatter_add(0, torch.where(done, fresh, 0), done.long())
    at = full.clamp(max=P - 1)
    i = torch.arange(len(parent), device=DEV)
    src = tab[parent, at].clamp(min=0)
    rows[i, at] = torch.where(done, fresh, rows[i, at])
    out, out_len = tab.clone(), L.clone()
    out[child] = rows
    out_len[child] = torch.where(part & ~done, full * S, n)
    _copy_plain(s, src[done], fresh[done])
    return dict(page_table=out.int(), kv_len=out_len.int(), refcount=rc.int(), free_pages=(rc == 0).sum().int()[None],
                k=s["k"], v=s["v"])


def _compact_plain(s):
    S = s["c"]["page"]
    tab, L, rc = (s[k].long() for k in ("page_table", "kv_len", "refcount"))
    ids = torch.arange(len(rc), device=DEV)
    live = rc > 0
    n_live = live.sum()
    high, low = live & (ids >= n_live), ~live & (ids < n_live)
    slots = torch.argsort((~low).long(), stable=True)
    to = torch.where(high, slots[(high.cumsum(0) - 1).clamp(min=0)], torch.where(live, ids, -1))
    used = torch.arange(tab.shape[1], device=DEV) < ((L + S - 1) // S)[:, None]
    out = torch.where(used, to[tab.clamp(min=0)], tab)
    src = torch.nonzero(high)[:, 0]
    dst = to[src]
    rc = rc.clone()
    rc[dst] = rc[src]
    rc[src] = 0
    _copy_plain(s, src, dst)
    return dict(page_table=out.int(), refcount=rc.int(), page_map=to.int(), n_live=n_live.int()[None], k=s["k"],
                v=s["v"])


def _logprobs_plain(s):
    c = s["c"]
    n, V, top = c["R"] * (c["gamma"] + 1), c["V"], c["top"]
    tok = s["tokens"].flatten().long()
    rows = torch.nonzero(tok >= 0)[:, 0]
    z = s["Z"].view(n, V)[rows].float()
    x = z * (1.0 / c["T"])
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    lse = m + torch.log(l)
    ent = lse[:, 0] - (e * x).sum(-1) / l[:, 0]
    # one 64-bit key for (logit descending, id ascending)
    bits = z.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) - torch.arange(V, device=DEV)
    ids = torch.topk(key, top, dim=-1).indices
    nan = torch.full((n,), math.nan, device=DEV)
    out = dict(logp=nan.clone(), entropy=nan.clone(), lse=nan.clone(),
               top_ids=torch.full((n, top), -1, dtype=torch.int32, device=DEV),
               top_logp=torch.full((n, top), math.nan, device=DEV))
    out["logp"][rows] = (x.gather(1, tok[rows, None]) - lse)[:, 0]
    out["entropy"][rows] = ent
    out["lse"][rows] = lse[:, 0]
    out["top_ids"][rows] = ids.int()
    out["top_logp"][rows] = x.gather(1, ids) - lse
    return {k: v.view(c["R"], c["gamma"] + 1, *v.shape[1:]) for k, v in out.items()}


_PLAIN = dict(attention=_attention_plain, append=_append_plain, resize=_resize_plain, fork=_fork_plain,
              compact=_compact_plain, logprobs=_logprobs_plain)


# ---------------------------------------------------------------------------- the package's calls
def _run_own(s):
    import speculative_decoding_draft_05_gb300 as pkg

    op = s["c"]["op"]
    ws = s.get("workspace")  # kept between calls, as a serving loop keeps it
    if op == "logprobs":
        r = pkg.dspark_logprobs(s["Z"], s["tokens"], s["c"]["T"], s["c"]["top"], workspace=ws)
        s["workspace"] = r["workspace"]
        return {k: r[k] for k in ("logp", "entropy", "lse", "top_ids", "top_logp")}
    if "cache" not in s:
        s["cache"] = pkg.PagedCache(s["k"], s["v"])
    cache = s["cache"]
    if op == "attention":
        r = pkg.dspark_paged_attention(s["q"], cache, 0, s["q_offsets"], s["kv_len"], s["page_table"], s["scale"],
                                       workspace=ws)
        s["workspace"] = r["workspace"]
        return dict(out=r["out"], lse=r["lse"])
    if op == "append":
        r = pkg.dspark_cache_append(cache, 0, s["k_new"], s["v_new"], s["q_offsets"], s["kv_len"], s["page_table"],
                                    workspace=ws)
        s["workspace"] = r["workspace"]
        return dict(k=s["k"], v=s["v"])
    if op == "resize":
        r = pkg.dspark_pages_resize(cache, s["page_table"], s["kv_len"], s["new_len"], s["refcount"], workspace=ws)
        keys = ("page_table", "kv_len", "refcount", "free_pages")
    elif op == "fork":
        r = pkg.dspark_pages_fork(cache, s["page_table"], s["kv_len"], s["parent"], s["child"], s["refcount"],
                                  workspace=ws)
        keys = ("page_table", "kv_len", "refcount", "free_pages")
    else:
        r = pkg.dspark_pages_compact(cache, s["page_table"], s["kv_len"], s["refcount"], workspace=ws)
        keys = ("page_table", "refcount", "page_map", "n_live")
    s["workspace"] = r["workspace"]
    return dict({k: r[k] for k in keys}, k=s["k"], v=s["v"])


def run(state):
    return _run_own(state) if own else _PLAIN[state["c"]["op"]](state)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "logprobs":
        n, rows = sum(_emits(c)), c["R"] * (c["gamma"] + 1)
        return dict(bytes=n * c["V"] * e + rows * (4 + 12 + 8 * c["top"]), flops=5 * n * c["V"])
    lens = _lens(c)
    if c["op"] == "attention":
        ch = _chunks(c)
        row = c["D"] * e
        b = sum(lens) * c["Hkv"] * row * 2 + sum(ch) * c["Hq"] * (2 * row + 4)
        seen = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, ch))
        return dict(bytes=b + 4 * sum(-(-n // c["page"]) for n in lens) + 8 * c["R"], flops=4 * c["D"] * c["Hq"] * seen)
    if c["op"] == "append":
        return dict(bytes=4 * sum(_chunks(c)) * c["Hkv"] * c["D"] * e + 8 * c["R"], flops=0)
    page = 2 * c["layers"] * c["page"] * c["Hkv"] * c["D"] * e  # K and V of a page in all layers
    meta = 8 * c["R"] * _max_pages(c) + 8 * c["n_pages"] + 12 * c["R"]
    if c["op"] == "resize":
        return dict(bytes=meta, flops=0)
    if c["op"] == "fork":  # nearly every parent's length ends inside a page
        return dict(bytes=meta + 2 * page * c["forks"], flops=0)
    return dict(bytes=meta + 2 * page * c["moves"], flops=0)


# ---------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    return dict(attention=_attention_exact, append=_append_exact, resize=_resize_exact, fork=_fork_exact,
                compact=_compact_exact, logprobs=_logprobs_exact)[c["op"]](c, s)


def _attention_exact(c, s):
    out = torch.zeros(s["T"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    off, G = s["q_offsets"].tolist(), c["Hq"] // c["Hkv"]
    for r, L in enumerate(s["kv_len"].tolist()):
        n = off[r + 1] - off[r]
        pg = s["page_table"][r, : -(-L // c["page"])].long()
        for h in range(c["Hkv"]):
            K = s["k"][0][pg][:, :, h].reshape(-1, c["D"])[:L].double()
            V = s["v"][0][pg][:, :, h].reshape(-1, c["D"])[:L].double()
            for a in range(0, n, 512):
                b = min(n, a + 512)
                q = s["q"][off[r] + a: off[r] + b, h * G: (h + 1) * G].double().reshape(-1, c["D"])
                pos = torch.arange(L - n + a, L - n + b, device=DEV).repeat_interleave(G)
                end = L - n + b  # no row of these sees a later key
                sc = s["scale"] * (q @ K[:end].T)
                sc[torch.arange(end, device=DEV)[None] > pos[:, None]] = -math.inf
                lg = torch.logsumexp(sc, 1)
                o = torch.exp(sc - lg[:, None]) @ V[:end]
                out[off[r] + a: off[r] + b, h * G: (h + 1) * G] = o.view(b - a, G, -1)
                lse[off[r] + a: off[r] + b, h * G: (h + 1) * G] = lg.view(b - a, G)
    return dict(out=out, lse=lse)


def _append_exact(c, s):
    off = s["q_offsets"].tolist()
    tab = s["page_table"].tolist()
    page, slot = [], []
    for r, L in enumerate(s["kv_len"].tolist()):
        for p in range(L - (off[r + 1] - off[r]), L):
            page.append(tab[r][p // c["page"]])
            slot.append(p % c["page"])
    page, slot = (torch.tensor(x, device=DEV) for x in (page, slot))
    k, v = s["k"].double(), s["v"].double()
    k[0].index_put_((page, slot), s["k_new"].double())
    v[0].index_put_((page, slot), s["v_new"].double())
    return dict(k=k, v=v)


def _moved(s, pairs):
    k, v = s["k"], s["v"]
    if pairs:
        src, dst = (torch.tensor(x, device=DEV) for x in zip(*pairs))
        kc, vc = k.index_select(1, src), v.index_select(1, src)
        k.index_copy_(1, dst, kc)
        v.index_copy_(1, dst, vc)
    return k.double(), v.double()


def _resize_exact(c, s):
    S, P = c["page"], s["page_table"].shape[1]
    tab, L, N, rc = (s[k].tolist() for k in ("page_table", "kv_len", "new_len", "refcount"))
    for r in range(len(L)):
        for j in range(-(-N[r] // S), -(-L[r] // S)):
            rc[tab[r][j]] -= 1
            tab[r][j] = -1
    free = [p for p, n in enumerate(rc) if n == 0]
    before, pairs, at = list(rc), [], 0
    for r in range(len(L)):
        if N[r] <= L[r]:
            L[r] = N[r]
            continue
        if L[r] % S and before[tab[r][L[r] // S]] > 1:
            if at >= len(free):
                continue
            old = tab[r][L[r] // S]
            pairs.append((old, free[at]))
            rc[old] -= 1
            rc[free[at]] = 1
            tab[r][L[r] // S] = free[at]
            at += 1
        held = -(-L[r] // S)
        while held < -(-N[r] // S) and at < len(free):
            tab[r][held] = free[at]
            rc[free[at]] = 1
            held, at = held + 1, at + 1
        L[r] = min(N[r], held * S)
    k, v = _moved(s, pairs)
    return dict(page_table=_i32(tab), kv_len=_i32(L), refcount=_i32(rc), free_pages=_i32([rc.count(0)]), k=k, v=v)


def _fork_exact(c, s):
    S = c["page"]
    tab, L, rc = (s[k].tolist() for k in ("page_table", "kv_len", "refcount"))
    free = [p for p, n in enumerate(rc) if n == 0]
    pairs, at = [], 0
    for a, b in zip(s["parent"].tolist(), s["child"].tolist()):
        full = L[a] // S
        tab[b] = tab[a][:full] + [-1] * (len(tab[a]) - full)
        for p in tab[b][:full]:
            rc[p] += 1
        L[b] = full * S
        if L[a] % S and at < len(free):
            pairs.append((tab[a][full], free[at]))
            tab[b][full] = free[at]
            rc[free[at]] = 1
            L[b] = L[a]
            at += 1
    k, v = _moved(s, pairs)
    return dict(page_table=_i32(tab), kv_len=_i32(L), refcount=_i32(rc), free_pages=_i32([rc.count(0)]), k=k, v=v)


def _compact_exact(c, s):
    S = c["page"]
    tab, L, rc = (s[k].tolist() for k in ("page_table", "kv_len", "refcount"))
    n_live = sum(n > 0 for n in rc)
    to = [p if n > 0 else -1 for p, n in enumerate(rc)]
    slots = iter([p for p in range(n_live) if rc[p] == 0])
    pairs = [(p, next(slots)) for p in range(n_live, len(rc)) if rc[p] > 0]
    for a, b in pairs:
        to[a], rc[b], rc[a] = b, rc[a], 0
    for r in range(len(L)):
        for j in range(-(-L[r] // S)):
            tab[r][j] = to[tab[r][j]]
    k, v = _moved(s, pairs)
    return dict(page_table=_i32(tab), refcount=_i32(rc), page_map=_i32(to), n_live=_i32([n_live]), k=k, v=v)


def _logprobs_exact(c, s):
    n, V, top = c["R"] * (c["gamma"] + 1), c["V"], c["top"]
    f = dict(dtype=torch.float64, device=DEV)
    out = dict(logp=torch.full((n,), math.nan, **f), entropy=torch.full((n,), math.nan, **f),
               lse=torch.full((n,), math.nan, **f), top_ids=torch.full((n, top), -1, dtype=torch.int32, device=DEV),
               top_logp=torch.full((n, top), math.nan, **f))
    tok = s["tokens"].flatten().long()
    rows = [i for i, t in enumerate(tok.tolist()) if t >= 0]
    for a in range(0, len(rows), 128):
        r = torch.tensor(rows[a: a + 128], device=DEV)
        lp = torch.log_softmax(s["Z"].view(n, V)[r].double() / c["T"], -1)
        out["logp"][r] = lp.gather(1, tok[r, None])[:, 0]
        out["entropy"][r] = -(lp.exp() * lp).sum(-1)
        out["lse"][r] = s["Z"].view(n, V)[r, 0].double() / c["T"] - lp[:, 0]
        best, ids = torch.sort(s["Z"].view(n, V)[r].float(), dim=-1, descending=True, stable=True)
        out["top_ids"][r] = ids[:, :top].int()
        out["top_logp"][r] = lp.gather(1, ids[:, :top])
    return {k: v.view(c["R"], c["gamma"] + 1, *v.shape[1:]) for k, v in out.items()}
