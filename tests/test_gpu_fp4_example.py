"""The serving example with rotary positions and a 4-bit cache: its logits against the definition, with K and V as
the cache stores them, over rounds, a fork and a compaction.

Tolerances, as parts of the logits' norm.  What a layer stores depends on values that are rounded before, and one next
to a border between two codes may get the other code.  With fp32 that are 2e-6 of the elements, less than one
a sequence here: a single other code changes the logits by 0.0017 mostly and by 0.020 at most (150 tried on the
definition), so two of the worst are let through, and half of all comparisons have to be without any.  With bf16 a
hundredth of the codes are others: the definition with its products rounded to bf16 is 0.040 .. 0.055 off (three
seeds); twice that.  On the definition, positions one off change the logits by 0.08 or more (K's alone 0.17), a factor
of V of 1.25 by 0.146, another request's page by 0.33.
"""
import math

import pytest
import torch

import fp4
from test_gpu_rotary import BF16, F32, example, rotated

pytestmark = pytest.mark.gpu


def dense(srv, tokens):
    """Logits [n, V] of a token sequence, in 64 bits on the CPU."""
    s, m, n = srv.s, srv.m, len(tokens)
    f = lambda x: x.double().cpu()  # noqa: E731
    h, cs = f(m.embed)[tokens], f(m.cos_sin)[:n]
    later = torch.ones(n, n).triu(1).bool()
    for layer in range(s.layers):
        q, k, v = (h @ f(m.qkv[layer])).view(n, -1, s.D).split([s.Hq, s.Hkv, s.Hkv], dim=1)
        q, k = rotated(q, cs, False)[0], rotated(k, cs, False)[0]
        k, v = (fp4.decode(*fp4.encode(x, 1.0), 1.0).repeat_interleave(s.Hq // s.Hkv, 1) for x in (k, v))
        a = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(s.D)
        p = torch.softmax(a.masked_fill(later, -math.inf), -1)
        h = h + torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1) @ f(m.out[layer])
    return h @ f(m.head)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_logits_over_a_4_bit_cache(dtype):
    ex = example()
    srv = ex.Server(ex.Sizes(dtype=dtype, n_pages=40, rotary=True, fp4=True), seed=3)
    g = torch.Generator().manual_seed(2)
    history, off_by = {}, []
    for slot, n in ((0, 3), (1, 17), (2, 40), (4, 2)):
        history[slot] = torch.randint(0, srv.s.V, (n,), generator=g).tolist()
        srv.prefill(slot, history[slot])
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
            want = dense(srv, history[slot][:-1] + part)[-len(part):]
            off_by.append(((got - want).norm() / want.norm()).item())
            assert off_by[-1] <= (0.04 if dtype == F32 else 0.11), (k, slot)
            history[slot] += [x for x in r["tokens"][slot].tolist() if x >= 0]
    if dtype == F32:
        assert sorted(off_by)[len(off_by) // 2] <= 1e-4
