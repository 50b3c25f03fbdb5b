"""Measured cases of a 4-bit paged K/V cache and of the position rotation: attention over
the 4-bit cache, writing a chunk with K and Q rotated on the way (bf16, fp32 and 4-bit
caches), and reading positions back as values.

``run`` computes an operator either in its plain form (``own`` false: elementary torch
operations in 32 bits, in 64 where 4-bit codes are chosen) or through the package's public
calls (``own`` true).  ``exact`` gives the same outputs from the definitions in 64 bits.
Lengths are part of a case; values come from the seed.

The 4-bit cache: uint8 [layers, pages, heads, page / 16, 9 D].  A block holds 16 positions of a
head: [16, D / 2] bytes of e2m1 codes, the even element in the low four bits, then [16, D / 16]
e4m3 scales, one for 16 elements.  A value is code x scale x factor, one factor for K and one for V.
A group's scale is the e4m3 nearest to amax / (6 factor), a code the e2m1 nearest to
x / (scale factor), ties to the even one, at most 6.
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
        # a small round in fp32 over the 4-bit cache (4 requests, gamma 4): latency
        dict(name="attn4_f32_r4", op="attention", dtype="f32", cache="fp4", R=4, chunk_lo=1, chunk=5, kv_lo=33, kv=300,
             Hq=8, Hkv=2, D=64, page=16, lens=1),
        # plain decoding, one token for each of 16 users: latency of a memory-bound call
        dict(name="attn4_decode_r16", op="attention", dtype="bf16", cache="fp4", R=16, chunk_lo=1, chunk=1, kv_lo=200,
             kv=2048, Hq=32, Hkv=8, D=128, page=16, lens=2),
        # plain decoding of 64 users with long contexts, 8 query heads a K/V head
        dict(name="attn4_decode_r64", op="attention", dtype="bf16", cache="fp4", R=64, chunk_lo=1, chunk=1, kv_lo=1000,
             kv=16384, Hq=64, Hkv=8, D=128, page=32, lens=3),
        # the target's pass of a verify round: anchor + up to 16 drafted tokens for 64 requests
        dict(name="attn4_verify_r64", op="attention", dtype="bf16", cache="fp4", R=64, chunk_lo=1, chunk=17, kv_lo=500,
             kv=8192, Hq=32, Hkv=8, D=128, page=64, lens=4),
        # the same over long documents: few requests, the work lies along the cache; 5 query heads a K/V head
        dict(name="attn4_long_r4", op="attention", dtype="bf16", cache="fp4", R=4, chunk_lo=17, chunk=17, kv_lo=100001,
             kv=131072, Hq=40, Hkv=8, D=128, page=32, lens=5),
        # a prompt's chunk behind what is cached already: compute-bound
        dict(name="attn4_prefill_r2", op="attention", dtype="bf16", cache="fp4", R=2, chunk_lo=2901, chunk=4096,
             kv_lo=5000, kv=8192, Hq=32, Hkv=8, D=128, page=64, lens=6),
        # a small fp32 round, a part of each head rotated, neighbours as pairs: latency
        dict(name="rotary_f32_r4", op="append", dtype="f32", cache="f32", R=4, chunk_lo=1, chunk=5, kv_lo=33, kv=300,
             Hq=8, Hkv=2, D=64, rot=32, interleaved=True, page=16, layout="thd", lens=7),
        # one verify round of 512 requests into a bf16 cache
        dict(name="rotary_bf16_r512", op="append", dtype="bf16", cache="bf16", R=512, chunk_lo=1, chunk=17, kv_lo=17,
             kv=1024, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, page=16, layout="thd", lens=8),
        # the first answers' round of 512 short requests into a 4-bit cache, and the cache's positions as values
        dict(name="rotary_fp4_r512", op="append", dtype="bf16", cache="fp4", R=512, chunk_lo=1, chunk=17, kv_lo=17,
             kv=48, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, page=16, lens=9),
        # two long prompts into an empty 4-bit cache, and the cache's positions as values
        dict(name="rotary_fp4_prompt_r2", op="append", dtype="bf16", cache="fp4", R=2, chunk_lo=8191, chunk=16384,
             kv_lo=8191, kv=16384, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, page=64, lens=10),
        # the prefix of a request out of a bf16 cache (to be handed to another engine): latency
        dict(name="read_bf16_r1", op="read", dtype="bf16", cache="bf16", R=1, chunk_lo=700, chunk=700, kv_lo=700,
             kv=700, Hkv=8, D=128, page=16, layout="htd", lens=11),
        # 8 long prefixes out of the 4-bit cache, as bf16
        dict(name="read_fp4_r8", op="read", dtype="bf16", cache="fp4", R=8, chunk_lo=2000, chunk=8192, kv_lo=2000,
             kv=8192, Hkv=8, D=128, page=64, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "read"])
    c = dict(op=op, dtype="bf16", cache="fp4", lens=rng.randrange(1 << 20), Hkv=rng.choice([1, 2, 4, 8]),
             page=rng.choice([16, 32, 48, 64, 128]), D=rng.choice([64, 128, 128, 128, 96]))
    if op == "attention":
        kind = rng.choice(["decode", "decode", "verify", "verify", "prefill"])
        if kind != "prefill" and rng.random() < 0.15:
            c["dtype"] = "f32"
        small = c["dtype"] == "f32"
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 4, 5, 7, 8])
        c["chunk"] = {"decode": 1, "verify": rng.randint(2, 17), "prefill": _log_int(rng, 100, 4096)}[kind]
        c["chunk_lo"] = 1 if kind != "prefill" else max(1, c["chunk"] // 2)
        c["kv"] = max(c["chunk"], _log_int(rng, 20, 4096 if small else 131072 if kind != "prefill" else 8192))
        c["kv_lo"] = max(c["chunk"], c["kv"] // rng.choice([1, 2, 10]))
        c["R"] = _log_int(rng, 1, 16 if small else 256 if kind != "prefill" else 4)
        while c["R"] > 1 and c["R"] * c["kv"] > 500000 // (8 if small else 1):
            c["R"] = (c["R"] + 1) // 2
        while c["R"] > 1 and c["R"] * c["chunk"] * c["kv"] * c["Hq"] > 2 * 4096 * 8192 * 32:
            c["R"] -= 1
        while c["chunk"] * c["kv"] * c["Hq"] > 2 * 4096 * 8192 * 32 and c["Hq"] > c["Hkv"]:
            c["Hq"] -= c["Hkv"]
        return c
    if rng.random() < 0.4:
        c["cache"] = c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["layout"] = rng.choice(["thd", "htd"])
    c["chunk"] = _log_int(rng, 1, 8192)
    c["chunk_lo"] = max(1, c["chunk"] // 8)
    c["R"] = max(1, min(512, _log_int(rng, 1, 512), 24000 // c["chunk"]))
    # (a 4-bit case's outputs are all positions: not many more than the new ones)
    more = 2048 if c["cache"] != "fp4" else max(1, 24000 // c["R"] - c["chunk"])
    c["kv"] = c["chunk"] + _log_int(rng, 1, min(2048, more))
    c["kv_lo"] = c["chunk"]
    if op == "append":
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 4, 5, 8])
        c["rot"] = rng.choice([c["D"], c["D"], c["D"] // 2])
        c["interleaved"] = rng.random() < 0.3
    return c


def _lens(c):
    """kv_len of each request, from the case alone."""
    r = random.Random("len %d %d" % (c["lens"], c["kv"]))
    return [c["kv"]] + [r.randint(c["kv_lo"], c["kv"]) for _ in range(c["R"] - 1)]


def _chunks(c):
    """New tokens of each request, from the case alone."""
    r = random.Random("chunk %d %d" % (c["lens"], c["chunk"]))
    return [min(n, c["chunk"] if i == 0 else r.randint(c["chunk_lo"], c["chunk"])) for i, n in enumerate(_lens(c))]


# ---------------------------------------------------------------------------- the 4-bit format
def _scales(y):
    """e4m3 scales of groups y [..., 16] (already divided by the factor), and their values."""
    s = (y.abs().amax(-1) / 6).clamp(max=448).float().to(torch.float8_e4m3fn)
    return s, s.to(y.dtype)


def _encode(x, factor):
    """Codes [..., D / 2] and scales [..., D / 16], both bytes, of x [..., D]."""
    y = (x / factor).unflatten(-1, (-1, 16))
    s, sv = _scales(y)
    t = torch.where(sv[..., None] > 0, y.abs() / sv[..., None], 0.0)
    code = (t > 0.25).byte() + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5)
    code = (code + 8 * (y < 0).byte()).flatten(-2)
    return code[..., ::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _parts(pool, D):
    """The codes [..., 16, D / 2] and the scales [..., 16, D / 16] of blocks [..., 9 D], as views."""
    return pool[..., : 8 * D].unflatten(-1, (16, D // 2)), pool[..., 8 * D:].unflatten(-1, (16, D // 16))


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _decode(codes, scales, factor):
    """Values [..., D] in 32 bits."""
    lut = torch.tensor(_E2M1, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float() * factor
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


# ---------------------------------------------------------------------------- inputs
def _cache(c, g, n_pages):
    """K and V pools of one layer.  "htd" stores heads before tokens."""
    out = []
    for _ in range(2):
        if c["cache"] == "fp4":
            D = c["D"]
            t = torch.empty(1, n_pages, c["Hkv"], c["page"] // 16, 9 * D, dtype=torch.uint8, device=DEV)
            codes, scales = _parts(t[0], D)
            step = max(1, (1 << 26) // (c["Hkv"] * c["page"] * D))
            for a in range(0, n_pages, step):
                b = min(n_pages, a + step)
                x = torch.empty(b - a, c["Hkv"], c["page"] // 16, 16, D, device=DEV).normal_(generator=g)
                codes[a:b], scales[a:b] = _encode(x, 1.0)
            out.append(t)
            continue
        thd = c["layout"] == "thd"
        shape = [1, n_pages, c["page"], c["Hkv"], c["D"]] if thd else [1, n_pages, c["Hkv"], c["page"], c["D"]]
        t = torch.empty(shape, dtype=DTYPES[c["cache"]], device=DEV).normal_(generator=g)
        out.append(t if thd else t.transpose(2, 3))
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _sums(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    lens, ch = _lens(c), _chunks(c)
    held = [-(-n // c["page"]) for n in lens]
    T, n_pages = sum(ch), sum(held) + 3
    s = dict(c=c, T=T, N=sum(lens), kv_len=_i32(lens), q_offsets=_i32(_sums(ch)), all_offsets=_i32(_sums(lens)))
    perm = torch.randperm(n_pages, generator=cpu).int()
    table = torch.full((c["R"], max(held) + 1), -1, dtype=torch.int32)
    for r, h in enumerate(held):
        at = sum(held[:r])
        table[r, :h] = perm[at: at + h]
    s["page_table"] = table.to(DEV)
    s["k"], s["v"] = _cache(c, g, n_pages)
    # the second scales of calibrated caches are powers of two here, as a loader rounds them
    s["factors"] = (0.5, 0.25) if c["cache"] == "fp4" else (1.0, 1.0)
    if c["op"] == "attention":
        s["q"] = torch.empty(T, c["Hq"], c["D"], dtype=dt, device=DEV).normal_(generator=g)
        s["scale"] = 2.0 / math.sqrt(c["D"])  # (K's values are halved by its factor)
    elif c["op"] == "append":  # q, k, v: parts of one projection's output, as a model gives them
        qkv = torch.empty(T, c["Hq"] + 2 * c["Hkv"], c["D"], dtype=dt, device=DEV).normal_(generator=g)
        s["q"], s["k_new"], s["v_new"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
        inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        angle = torch.arange(c["kv"], dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    return s


# ---------------------------------------------------------------------------- plain forms
def _gathered(s, name, P):
    """One pool's pages of all requests as values [R, P page, Hkv, D] in 32 bits."""
    c = s["c"]
    pages = s["page_table"][:, :P].long().clamp(min=0)
    if c["cache"] != "fp4":
        return s[name][0][pages].flatten(1, 2).float()
    codes, scales = _parts(s[name][0][pages], c["D"])  # [R, P, Hkv, page / 16, 16, ..]
    x = _decode(codes, scales, s["factors"][name == "v"])
    return x.flatten(3, 4).transpose(2, 3).flatten(1, 2)


def _attention_plain(s):
    c, q = s["c"], s["q"]
    kv, mq, page = c["kv"], c["chunk"], c["page"]
    off = s["q_offsets"].long()
    n, L = off[1:] - off[:-1], s["kv_len"].long()
    P = -(-kv // page)
    j = torch.arange(P * page, device=DEV)
    has = (j < L[:, None])[:, :, None, None]
    K = torch.where(has, _gathered(s, "k", P), 0.0)  # [R, kv, Hkv, D]
    V = torch.where(has, _gathered(s, "v", P), 0.0)
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


def _places(s, offsets, n):
    """Position, page and place in the page of the rows of offsets."""
    off, L = offsets.long(), s["kv_len"].long()
    t = torch.arange(n, device=DEV)
    r = torch.searchsorted(off, t, right=True) - 1
    pos = L[r] - off[r + 1] + t
    return pos, s["page_table"].long()[r, pos // s["c"]["page"]], pos % s["c"]["page"]


def _rotated(c, x, cs):
    """x [T, H, D] with its first rot columns rotated; cs [T, rot]: cosines, sines."""
    rot = c["rot"]
    cos, sin = cs[:, None].chunk(2, -1)
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if c["interleaved"] else x[..., :rot].chunk(2, -1)
    ra, rb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ra, rb), -1).flatten(-2) if c["interleaved"] else torch.cat((ra, rb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _append_plain(s):
    c = s["c"]
    pos, page, slot = _places(s, s["q_offsets"], s["T"])
    cs = s["cos_sin"][pos]
    q = _rotated(c, s["q"].float(), cs).to(s["q"].dtype)
    if c["cache"] != "fp4":
        s["k"][0][page, slot] = _rotated(c, s["k_new"].float(), cs).to(s["k"].dtype)
        s["v"][0][page, slot] = s["v_new"]
        return dict(k=s["k"], v=s["v"], q=q)
    # 64 bits: values next to a border between two codes
    for name, x in (("k", _rotated(c, s["k_new"].double(), cs.double())), ("v", s["v_new"].double())):
        codes, scales = _parts(s[name][0], c["D"])
        codes[page, :, slot // 16, slot % 16], scales[page, :, slot // 16, slot % 16] = \
            _encode(x, s["factors"][name == "v"])
    return dict(_read_plain(s, s["all_offsets"], s["N"]), q=q)


def _read_plain(s, offsets, n):
    c, out = s["c"], {}
    _, page, slot = _places(s, offsets, n)
    for name in ("k", "v"):
        if c["cache"] != "fp4":
            out[name] = s[name][0][page, slot]
            continue
        codes, scales = _parts(s[name][0], c["D"])
        x = _decode(codes[page, :, slot // 16, slot % 16], scales[page, :, slot // 16, slot % 16],
                    s["factors"][name == "v"])
        out[name] = x.to(DTYPES[c["dtype"]])
    return out


# ---------------------------------------------------------------------------- the package's calls
def _run_own(s):
    import speculative_decoding_draft_05_gb300 as pkg

    c = s["c"]
    ws = s.get("workspace")  # kept between calls, as a serving loop keeps it
    if "own" not in s:
        s["own"] = pkg.PagedCacheFp4(s["k"], s["v"], *s["factors"]) if c["cache"] == "fp4" else \
            pkg.PagedCache(s["k"], s["v"])
    cache = s["own"]
    if c["op"] == "attention":
        r = pkg.dspark_paged_attention(s["q"], cache, 0, s["q_offsets"], s["kv_len"], s["page_table"], s["scale"],
                                       workspace=ws)
        s["workspace"] = r["workspace"]
        return dict(out=r["out"], lse=r["lse"])
    if c["op"] == "read":
        r = pkg.dspark_cache_read(cache, 0, s["q_offsets"], s["kv_len"], s["page_table"], s["T"], workspace=ws)
        s["workspace"] = r["workspace"]
        return dict(k=r["k"], v=r["v"])
    r = pkg.dspark_cache_append_rotary(cache, 0, s["k_new"], s["v_new"], s["q_offsets"], s["kv_len"],
                                       s["page_table"], s["cos_sin"], q=s["q"], interleaved=c["interleaved"],
                                       workspace=ws)
    s["workspace"] = r["workspace"]
    if c["cache"] != "fp4":
        return dict(k=s["k"], v=s["v"], q=r["q"])
    back = pkg.dspark_cache_read(cache, 0, s["all_offsets"], s["kv_len"], s["page_table"], s["N"],
                                 workspace=s["workspace"])
    return dict(k=back["k"], v=back["v"], q=r["q"])


def run(state):
    if own:
        return _run_own(state)
    op = state["c"]["op"]
    if op == "attention":
        return _attention_plain(state)
    return _append_plain(state) if op == "append" else _read_plain(state, state["q_offsets"], state["T"])


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    held = c["Hkv"] * c["D"] * 2 * (9 / 16 if c["cache"] == "fp4" else e)  # K and V of a position in the cache
    dense = c["Hkv"] * c["D"] * 2 * e  # and as rows
    lens, ch = _lens(c), _chunks(c)
    T = sum(ch)
    if c["op"] == "attention":
        b = sum(lens) * held + T * c["Hq"] * (2 * c["D"] * e + 4)
        seen = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, ch))
        return dict(bytes=b + 4 * sum(-(-n // c["page"]) for n in lens) + 8 * c["R"], flops=4 * c["D"] * c["Hq"] * seen)
    b = T * (held + dense) + 8 * c["R"]
    if c["op"] == "append":
        b += T * (2 * c["Hq"] * c["D"] * e + 4 * c["rot"])
        if c["cache"] == "fp4":  # and all positions as values
            b += sum(lens) * (held + dense)
    return dict(bytes=b, flops=0)


# ---------------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    return dict(attention=_attention_exact, append=_append_exact, read=_read_exact)[c["op"]](c, s)


def _values64(block_codes, block_scales, factor):
    """From the bits: (-1)^s 2^(e - 1) (1 + m / 2), for e = 0 m / 2; e4m3 with bias 7."""
    n = torch.stack((block_codes & 15, block_codes >> 4), -1).flatten(-2).long()
    sign, e, m = n >> 3, (n >> 1) & 3, n & 1
    v = torch.where(e > 0, torch.exp2((e - 1).double()) * (1 + m / 2), m.double() / 2) * (1 - 2 * sign)
    b = block_scales.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m / 512)
    return v * (sc * factor).repeat_interleave(16, -1)


def _request64(c, s, r, L, name, h):
    """Positions 0 .. L - 1 of request r and head h, [L, D]."""
    pg = s["page_table"][r, : -(-L // c["page"])].long()
    D = c["D"]
    if c["cache"] != "fp4":
        return s[name][0][pg][:, :, h].reshape(-1, D)[:L].double()
    x = s[name][0][pg, h]  # [P, page / 16, 9 D]
    codes = x[..., : 8 * D].reshape(-1, D // 2)[:L]
    scales = x[..., 8 * D:].reshape(-1, D // 16)[:L]
    return _values64(codes, scales, s["factors"][0 if name == "k" else 1])


def _attention_exact(c, s):
    out = torch.zeros(s["T"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    off, G = s["q_offsets"].tolist(), c["Hq"] // c["Hkv"]
    for r, L in enumerate(s["kv_len"].tolist()):
        n = off[r + 1] - off[r]
        for h in range(c["Hkv"]):
            K, V = _request64(c, s, r, L, "k", h), _request64(c, s, r, L, "v", h)
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


def _rotate64(c, x, cs):
    """Each pair as a complex number, times e^(i angle)."""
    rot, half = c["rot"], c["rot"] // 2
    i = torch.arange(half, device=DEV)
    a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    z = torch.complex(x[..., a], x[..., b]) * torch.complex(cs[:, :half], cs[:, half:])[:, None]
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _nearest64(x, values):
    """Index of the nearest of the ascending `values`, the even index where two are equally near."""
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _stored64(x, factor):
    """x [T, H, D] as a 4-bit cache gives it back."""
    e4m3 = torch.tensor([m / 512 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8) for e in range(16) for m in range(8)][:127],
                        dtype=torch.float64, device=DEV)
    e2m1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    y = (x / factor).unflatten(-1, (-1, 16))
    sc = e4m3[_nearest64(y.abs().amax(-1) / 6, e4m3)][..., None]
    t = torch.where(sc > 0, y.abs() / sc, 0)
    return (torch.sign(y) * e2m1[_nearest64(t, e2m1)] * sc * factor).flatten(-2)


def _append_exact(c, s):
    off, tab = s["q_offsets"].tolist(), s["page_table"].tolist()
    page, slot, pos, row = [], [], [], []
    for r, L in enumerate(s["kv_len"].tolist()):
        n = off[r + 1] - off[r]
        base = sum(_lens(c)[:r])
        for p in range(L - n, L):
            page.append(tab[r][p // c["page"]])
            slot.append(p % c["page"])
            pos.append(p)
            row.append(base + p)
    page, slot, pos, row = (torch.tensor(x, device=DEV) for x in (page, slot, pos, row))
    cs = s["cos_sin"].double()[pos]
    q, k = _rotate64(c, s["q"].double(), cs), _rotate64(c, s["k_new"].double(), cs)
    if c["cache"] != "fp4":
        K, V = s["k"].double(), s["v"].double()
        K[0].index_put_((page, slot), k)
        V[0].index_put_((page, slot), s["v_new"].double())
        return dict(k=K, v=V, q=q)
    out = _read_exact(c, s, whole=True)
    out["k"][row] = _stored64(k, s["factors"][0])
    out["v"][row] = _stored64(s["v_new"].double(), s["factors"][1])
    return dict(out, q=q)


def _read_exact(c, s, whole=False):
    out = dict(k=[], v=[])
    for r, L in enumerate(s["kv_len"].tolist()):
        n = L if whole else int(s["q_offsets"][r + 1] - s["q_offsets"][r])
        for name in out:
            out[name].append(torch.stack([_request64(c, s, r, L, name, h)[L - n:] for h in range(c["Hkv"])], 1))
    return {name: torch.cat(x) for name, x in out.items()}
