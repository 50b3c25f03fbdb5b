"""The serving loop of examples/paged_rounds.py: whatever the pages went through
(chunks, rejected suffixes, a fork, a compaction), every round's target logits are
those of the same model run densely, in 64 bits, over each request's tokens."""
import importlib.util
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("paged_rounds", os.path.join(ROOT, "examples", "paged_rounds.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules["paged_rounds"] = mod
    spec.loader.exec_module(mod)
    return mod


def dense(srv, tokens):
    """Logits [n, V] of a token sequence by the definition."""
    s, m = srv.s, srv.m
    n = len(tokens)
    f = lambda t: t.double().cpu()  # noqa: E731
    h = f(m.embed)[tokens] + f(m.pos)[:n]
    mask = torch.ones(n, n).tril().bool()
    for layer in range(s.layers):
        q, k, v = (h @ f(m.qkv[layer])).view(n, -1, s.D).split([s.Hq, s.Hkv, s.Hkv], dim=1)
        k, v = (x.repeat_interleave(s.Hq // s.Hkv, 1) for x in (k, v))
        a = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(s.D)
        p = torch.softmax(a.masked_fill(~mask, -math.inf), -1)
        h = h + torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1) @ f(m.out[layer])
    return h @ f(m.head)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rounds_over_pages_match_the_dense_model(dtype):
    ex = load()
    srv = ex.Server(ex.Sizes(dtype=dtype, n_pages=40), seed=3)
    g = torch.Generator().manual_seed(2)
    history = {}
    for slot, n in ((0, 3), (1, 17), (2, 40), (4, 2)):
        history[slot] = torch.randint(0, srv.s.V, (n,), generator=g).tolist()
        srv.prefill(slot, history[slot])
    # bf16: four products a layer round their results (2^-8 of values whose sums grow with two layers
    # of residuals); fp32: the same with 2^-24 and the sums' lengths.
    tol = 0.08 if dtype == torch.bfloat16 else 1e-4
    for k in range(9):
        if k == 3:
            srv.fork(2, 5)
            history[5] = list(history[2])
        if k == 5:
            srv.end(1)
            del history[1]
            srv.compact()
        r = srv.round()
        off, chunk = r["offsets"].tolist(), r["chunk"].tolist()
        lp = r["logprobs"]
        for slot in history:
            part = chunk[off[slot]: off[slot + 1]]
            assert part[0] == history[slot][-1]
            want = dense(srv, history[slot][:-1] + part)[-len(part):]
            got = r["logits"][off[slot]: off[slot + 1]].double().cpu()
            assert (got - want).norm() <= tol * want.norm(), (k, slot)
            new = [t for t in r["tokens"][slot].tolist() if t >= 0]
            assert len(new) == r["n_emit"][slot].item() >= 1
            # accepted tokens are the chunk's; each is reported with its own logits
            assert new[:-1] == part[1: len(new)]
            for j, t in enumerate(new):
                z = torch.log_softmax(got[j], -1)
                assert abs(lp["logp"][off[slot] + j].item() - z[t].item()) < 1e-4
                assert lp["top_ids"][off[slot] + j, 0].item() == int(got[j].argmax())
            history[slot] += new
            assert srv.len[slot].item() == len(history[slot]) - 1
        # no page is lost: the counts are what the tables hold
        held = torch.zeros(srv.s.n_pages, dtype=torch.int32)
        for row, n in zip(srv.table.tolist(), srv.len.tolist()):
            for p in row[: -(-n // srv.s.page)]:
                held[p] += 1
        assert torch.equal(held, srv.refcount.cpu())
        assert r["free_pages"].item() == int((held == 0).sum())
