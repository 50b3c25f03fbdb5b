"""Speculative serving rounds with a paged K/V cache, all on one GPU.

A small random target model (two attention layers) serves a few
requests with the library's calls in the order a serving loop makes them:

    dspark_draft_sample -> dspark_schedule            the drafted block, its length
    dspark_pages_resize                               pages for the chunk x_0, x_1 .. x_l
    per layer: dspark_cache_append, dspark_paged_attention
    dspark_verify -> dspark_logprobs                  accepted tokens, and what is
                                                      reported beside them
    dspark_pages_resize                               the rejected suffix is cut off

and, between rounds, dspark_pages_fork (one request continued twice) and
dspark_pages_compact.  The host reads nothing back inside a round: chunks are
laid out flat with offsets on the device, padded to R (gamma + 1) rows.

    python examples/paged_rounds.py
"""
from __future__ import annotations

import dataclasses
import math
import os
import sys
from typing import List

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_draft_05_gb300 as dspark  # noqa: E402


@dataclasses.dataclass
class Sizes:
    R: int = 6            # request slots
    gamma: int = 4        # drafted positions
    V: int = 1024
    layers: int = 2
    Hq: int = 8
    Hkv: int = 2
    D: int = 64
    r: int = 64           # rank of the draft's Markov head
    page: int = 16
    n_pages: int = 96
    max_pages: int = 12
    dtype: torch.dtype = torch.bfloat16


class Model:
    """Random weights of the toy target and of the draft head."""

    def __init__(self, s: Sizes, seed: int, dev):
        g = torch.Generator(device="cpu").manual_seed(seed)
        d = s.Hq * s.D

        def w(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(s.dtype).to(dev)

        self.embed = w(s.V, d, std=1.0)
        self.pos = w(s.page * s.max_pages, d, std=0.1)
        self.qkv = [w(d, (s.Hq + 2 * s.Hkv) * s.D, std=2.0 / math.sqrt(d)) for _ in range(s.layers)]
        self.out = [w(d, d, std=0.2 / math.sqrt(d)) for _ in range(s.layers)]
        # The output head has rank r, and the draft's Markov head W1 W2 is the
        # target without its attention: near enough that most drafts are accepted.
        a, self.W2 = w(d, s.r, std=1.0 / math.sqrt(d)), w(s.r, s.V, std=2.0 / math.sqrt(s.r))
        self.head = (a.float() @ self.W2.float()).to(s.dtype)
        self.W1 = (self.embed.float() @ a.float()).to(s.dtype).contiguous()


class Server:
    def __init__(self, s: Sizes = Sizes(), seed: int = 0, device="cuda:0"):
        self.s, self.seed, self.dev = s, seed, torch.device(device)
        self.m = Model(s, seed, self.dev)
        shape = (s.layers, s.n_pages, s.page, s.Hkv, s.D)
        # Uninitialised on purpose: positions past a request's length are never read.
        self.cache = dspark.PagedCache(*(torch.empty(shape, dtype=s.dtype, device=self.dev) for _ in range(2)))
        i32 = dict(dtype=torch.int32, device=self.dev)
        self.table = torch.full((s.R, s.max_pages), -1, **i32)
        self.len = torch.zeros(s.R, **i32)        # positions in the cache
        self.refcount = torch.zeros(s.n_pages, **i32)
        self.x0 = torch.zeros(s.R, **i32)         # the next chunk's first token
        self.live = torch.zeros(s.R, dtype=torch.bool, device=self.dev)
        B = s.R * (1 + s.gamma)
        self.sps = (1.0 / (1e-3 + 2e-5 * torch.arange(B + 1, dtype=torch.float64))).to(self.dev)
        self.rounds = 0
        self.ws = {}

    def _keep(self, name, result):
        self.ws[name] = result["workspace"]
        return result

    def _resize(self, new_len):
        r = self._keep("pages", dspark.dspark_pages_resize(
            self.cache, self.table, self.len, new_len, self.refcount, page_table_out=self.table, kv_len_out=self.len,
            refcount_out=self.refcount, workspace=self.ws.get("pages")))
        return r["free_pages"]

    def _forward(self, tokens, q_offsets, position):
        """Target logits [T, V] of a flat chunk whose rows are appended to the cache."""
        s, m = self.s, self.m
        h = m.embed[tokens.clamp(min=0).long()] + m.pos[position.clamp(0, m.pos.shape[0] - 1).long()]
        T = h.shape[0]
        for layer in range(s.layers):
            qkv = (h @ m.qkv[layer]).view(T, s.Hq + 2 * s.Hkv, s.D)
            q, k, v = qkv.split([s.Hq, s.Hkv, s.Hkv], dim=1)  # parts of one array: strided rows
            self._keep("append", dspark.dspark_cache_append(
                self.cache, layer, k, v, q_offsets, self.len, self.table, workspace=self.ws.get("append")))
            a = self._keep("attention", dspark.dspark_paged_attention(
                q, self.cache, layer, q_offsets, self.len, self.table, 1.0 / math.sqrt(s.D),
                workspace=self.ws.get("attention")))["out"]
            a = torch.where(position[:, None] >= 0, a.reshape(T, -1), 0)  # padding rows were not written
            h = h + a @ m.out[layer]
        return h @ m.head

    def prefill(self, slot: int, prompt: List[int]):
        """Put a prompt into an empty slot: all but its last token enter the cache."""
        n = len(prompt) - 1
        new_len = self.len.clone()
        new_len[slot] = n
        self._resize(new_len)
        counts = torch.zeros(self.s.R + 1, dtype=torch.int32)
        counts[slot + 1] = n
        tok = torch.tensor(prompt[:-1], dtype=torch.int32, device=self.dev)
        self._forward(tok, counts.cumsum(0).int().to(self.dev), torch.arange(n, device=self.dev))
        self.x0[slot] = prompt[-1]
        self.live[slot] = True

    def fork(self, parent: int, child: int):
        i = lambda x: torch.tensor([x], dtype=torch.int32, device=self.dev)  # noqa: E731
        self._keep("fork", dspark.dspark_pages_fork(
            self.cache, self.table, self.len, i(parent), i(child), self.refcount, page_table_out=self.table,
            kv_len_out=self.len, refcount_out=self.refcount, workspace=self.ws.get("fork")))
        self.x0[child] = self.x0[parent]
        self.live[child] = True

    def end(self, slot: int):
        new_len = self.len.clone()
        new_len[slot] = 0
        self.live[slot] = False
        return self._resize(new_len)

    def compact(self):
        r = self._keep("compact", dspark.dspark_pages_compact(
            self.cache, self.table, self.len, self.refcount, page_table_out=self.table,
            refcount_out=self.refcount, workspace=self.ws.get("compact")))
        return r["n_live"]

    def round(self) -> dict:
        s, m, R, g = self.s, self.m, self.s.R, self.s.gamma
        seed = (self.seed << 20) + self.rounds
        self.rounds += 1
        # The drafted block and how much of it the target verifies.
        U = torch.zeros(R, g, s.V, dtype=s.dtype, device=self.dev)
        d = dspark.dspark_draft_sample(U, m.W1, m.W2, self.x0, 1.0, seed)
        conf = torch.full((R, g), 0.8, device=self.dev)
        ell = torch.where(self.live, dspark.dspark_schedule(conf, self.sps)["ell"], 0).int()
        # The chunk x_0, x_1 .. x_l of every live request, flat.
        count = torch.where(self.live, ell + 1, 0).int()
        off = torch.zeros(R + 1, dtype=torch.int32, device=self.dev)
        off[1:] = count.cumsum(0)
        block = torch.cat([self.x0[:, None], d["x"]], 1)                    # [R, gamma + 1]
        j = torch.arange(g + 1, device=self.dev, dtype=torch.int32)
        used = j < count[:, None]
        T = R * (g + 1)
        place = torch.where(used, off[:-1, None] + j, T).long()             # T: a slot for the rest
        flat = torch.full((T + 1,), -1, dtype=torch.int32, device=self.dev)
        flat[place] = torch.where(used, block, -1)
        position = torch.full((T + 1,), -1, dtype=torch.int32, device=self.dev)
        position[place] = torch.where(used, self.len[:, None] + j, -1)
        before = self.len.clone()
        self._resize(before + count)
        Z = self._forward(flat[:T], off, position[:T]).contiguous()
        # A slot that is not live has no rows; verify still wants one: it reads row 0 and its result is dropped.
        rows = torch.where(off[1:] > off[:-1], off[:-1], 0)
        starts = torch.cat([rows, off[-1:]]).int()
        v = dspark.dspark_verify(d["x"], d["logp"], d["lse"], d["scores"],
                                 Z[torch.minimum(starts[:-1, None] + torch.minimum(j, ell[:, None]),
                                                 torch.tensor(T - 1, device=self.dev)).long()].contiguous(),
                                 ell, 1.0, seed)
        emitted = torch.where(self.live[:, None], v["tokens"], -1)          # [R, gamma + 1], -1 past the last
        n_emit = torch.where(self.live, v["n_emit"], 0)
        # What is reported beside them: row off[r] + j holds the logits of emitted token j.
        flat_tok = torch.full((T + 1,), -1, dtype=torch.int32, device=self.dev)
        flat_tok[place] = torch.where(used, emitted, -1)
        lp = self._keep("logprobs", dspark.dspark_logprobs(Z, flat_tok[:T].contiguous(), 1.0, 3,
                                                           workspace=self.ws.get("logprobs")))
        # The anchor and the accepted tokens stay; the last emitted token starts the next chunk.
        free = self._resize(torch.where(self.live, before + n_emit, self.len).int())
        last = emitted.gather(1, (n_emit - 1).clamp(min=0)[:, None].long())[:, 0]
        self.x0 = torch.where(self.live, last, self.x0).int().contiguous()
        return dict(tokens=emitted, n_emit=n_emit, logits=Z, offsets=off, chunk=flat[:T], logprobs=lp, free_pages=free)


def main():
    srv = Server()
    g = torch.Generator().manual_seed(1)
    for slot in range(4):
        srv.prefill(slot, torch.randint(0, srv.s.V, (5 + 9 * slot,), generator=g).tolist())
    for k in range(8):
        if k == 3:
            srv.fork(3, 5)
        if k == 5:
            srv.end(1)
            print("live pages:", srv.compact().item())
        r = srv.round()
        lp = r["logprobs"]["logp"]
        n = r["n_emit"].tolist()
        print(f"round {k}: emitted {n}, mean logp {lp[~lp.isnan()].mean().item():.2f}, "
              f"free pages {r['free_pages'].item()}, lengths {srv.len.tolist()}")


if __name__ == "__main__":
    main()
