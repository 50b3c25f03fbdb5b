"""The 4-bit cache's format in 64 bits, from its definition, and inputs for tests of what reads and writes it.

A block of 16 positions of a head is 9 D bytes: [16, D / 2] e2m1 codes (the even element in the low four
bits), [16, D / 16] e4m3 scales.  A value is code x scale x factor.
"""
import math

import numpy as np
import torch

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
E4M3 = torch.tensor([m / 512 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8) for e in range(16) for m in range(8)],
                    dtype=torch.float64)
E4M3[127] = math.nan


def nearest(x, values):
    """Index of the nearest of the ascending values, the even index of two equally near; past the last: the last."""
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def encode(x, factor):
    """x [..., D] in 64 bits -> codes uint8 [..., D / 2], scales uint8 [..., D / 16]."""
    dev = x.device
    y = (x.double() / factor).unflatten(-1, (-1, 16))
    fine = y.isfinite().all(-1)
    amax = torch.where(fine, y.abs().amax(-1).nan_to_num(), 0)
    s = nearest(amax / 6, E4M3[:127].to(dev))
    sv = E4M3.to(dev)[s][..., None]
    ok = fine[..., None] & (sv > 0)
    t = torch.where(ok, y.abs().nan_to_num() / torch.where(ok, sv, 1), 0)
    c = (nearest(t, E2M1.to(dev)) + 8 * (ok & (y < 0))).to(torch.uint8).flatten(-2)
    return c[..., ::2] | (c[..., 1::2] << 4), torch.where(fine, s, 127).to(torch.uint8)


def decode(codes, scales, factor):
    """Values [..., D] in 64 bits."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = E2M1.to(codes.device)[n & 7] * (1 - 2 * (n >> 3))
    s = E4M3.to(codes.device)[(scales & 127).long()] * (1 - 2 * (scales >> 7).double()) * factor
    return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def parts(pool):
    """Views of a pool [..., 9 D]: codes [..., 16, D / 2] and scales [..., 16, D / 16]."""
    D = pool.shape[-1] // 9
    return pool[..., :8 * D].unflatten(-1, (16, D // 2)), pool[..., 8 * D:].unflatten(-1, (16, D // 16))


def values(pool, factor):
    """[layers, pages, heads, blocks, 9 D] -> [layers, pages, page_size, heads, D] in 64 bits."""
    codes, scales = parts(pool)
    return decode(codes, scales, factor).flatten(3, 4).transpose(2, 3)


def tables(lens, page, spare, g):
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + spare
    perm = torch.randperm(n_pages, generator=g).int()
    table = torch.full((len(lens), max(held + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = perm[at:at + h]
        at += h
    return table, n_pages


def pool_of(shape, g, strided):
    """Blocks of random codes and NaN scales: what unused slots may hold."""
    L, n, H, B, W = shape
    wide = [L, n, H, B + 2, W] if strided else list(shape)
    t = torch.randint(0, 256, wide, generator=g, dtype=torch.uint8)
    t[..., W // 9 * 8:] = 0x7f
    return t.cuda()[:, :, :, :B]


def make(dtype, chunks, lens, Hq, Hkv, D, page, seed=0, layers=1, spare=2, strided=False, factors=(0.5, 0.25)):
    """Random inputs of attention over a 4-bit cache; unused slots and pages hold NaN."""
    g = torch.Generator().manual_seed(seed)
    table, n_pages = tables(lens, page, spare, g)
    shape = [layers, n_pages, Hkv, page // 16, 9 * D]
    k, v = pool_of(shape, g, strided), pool_of(shape, g, strided)
    for r, n in enumerate(lens):
        pos = torch.arange(n)
        pg, slot = table[r, pos // page].long(), pos % page
        for pool, f in ((k, factors[0]), (v, factors[1])):
            codes, scales = parts(pool)
            c, s = encode(torch.randn(layers, n, Hkv, D, generator=g).cuda(), f)
            for layer in range(layers):
                codes[layer, pg, :, slot // 16, slot % 16] = c[layer]
                scales[layer, pg, :, slot // 16, slot % 16] = s[layer]
    T = sum(chunks)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    off = torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32).cuda()
    return dict(k=k, v=v, factors=factors, qkv=qkv, q=qkv[:, :Hq], off=off,
                lens=torch.tensor(lens, dtype=torch.int32).cuda(), table=table.cuda(), scale=1 / math.sqrt(D),
                chunks=chunks, L=lens, Hq=Hq, Hkv=Hkv, D=D, page=page)


def reference(i, layer=0):
    """out, lse and their tolerances, a request at a time in 64 bits on the GPU (what only goes into tolerances: 32)."""
    Hq, D, G, scale = i["Hq"], i["D"], i["Hq"] // i["Hkv"], i["scale"]
    bf = i["q"].dtype == BF16
    table, res, t = i["table"].long(), [], 0
    kf, vf = (values(i[x][layer:layer + 1], f)[0] for x, f in zip("kv", i["factors"]))
    for r, (n, L) in enumerate(zip(i["chunks"], i["L"])):
        pg = table[r, : -(-L // i["page"])]
        K, V = (x[pg].reshape(-1, i["Hkv"], D)[:L].repeat_interleave(G, 1) for x in (kf, vf))
        q = i["q"][t:t + n].double()
        t += n
        if n == 0:
            continue
        if L == 0:  # nothing to see
            z = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
            res.append((z, z[..., 0] - math.inf, z, z[..., 0]))
            continue
        pos = torch.arange(L - n, L, device="cuda")
        see = torch.arange(L, device="cuda") <= pos[:, None, None]  # [n, 1, L]
        s = torch.einsum("nhd,jhd->nhj", q, K) * scale
        sa = torch.einsum("nhd,jhd->nhj", q.float().abs(), K.float().abs()) * abs(scale)
        ds = (D + 3) * U * torch.where(see, sa, 0.0).amax(2) + 2 * U * torch.where(see, s.abs(), 0.0).amax(2)
        s = torch.where(see, s, -math.inf)
        lse = torch.logsumexp(s, 2)
        pr = torch.where(see, torch.exp(s - lse[..., None].nan_to_num(neginf=0.0)), 0.0)
        out = torch.einsum("nhj,jhd->nhd", pr, torch.nan_to_num(V) if see.all(2).any() else V)
        mix = torch.einsum("nhj,jhd->nhd", pr.float(), V.float().abs())
        # bf16: probabilities in fp16, 2^-11 relative, or, below 2^-14 of 2^7 at least, 2^-25 of it
        sums = ((2 * pos + 16) * U + ((pos + 1) * 2.0 ** -32 if bf else 0))[:, None]
        tol = (4 * ds + sums + (2.0 ** -11 if bf else 0))[..., None] * mix + (2.0 ** -8 * out.abs() if bf else 0)
        res.append((out, lse, tol, 2 * ds + sums + 4 * U * lse.abs()))
    return [torch.cat(x).cpu() for x in zip(*res)]
