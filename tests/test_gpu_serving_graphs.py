"""The serving calls inside a CUDA graph: a replay gives what the calls give on their own."""
import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,page", [(torch.bfloat16, 128, 16), (torch.float32, 64, 8)], ids=["bf16", "f32"])
def test_a_replayed_round_is_the_same(dtype, D, page):
    g = torch.Generator().manual_seed(0)
    R, P, n_pages, Hq, Hkv, V = 9, 40, 300, 8, 2, 6000
    k, v = (torch.randn(2, n_pages, page, Hkv, D, generator=g).to(dtype).cuda() for _ in range(2))
    cache = dspark.PagedCache(k, v)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = [0, 17, 5, 130, 64, 1, 200, 33, 0]
    table, rc, at = torch.full((R, P), -1, dtype=torch.int32), torch.zeros(n_pages, dtype=torch.int32), 0
    for r, n in enumerate(lens):
        for j in range(-(-n // page)):
            table[r, j] = 2 * at  # every other page, so that compacting moves some
            rc[2 * at] = 1
            at += 1
    table, rc, lens = table.cuda(), rc.cuda(), i32(lens)
    chunk = i32([0, 3, 1, 5, 4, 2, 1, 6, 0])
    off = torch.cat([i32([0]), chunk.cumsum(0).int()])
    T = 25  # rows past the last request's are padding
    q, kn, vn = (torch.randn(T, h, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
    Z = (torch.randn(T, V, generator=g) * 3).to(dtype).cuda()
    tokens = torch.randint(-1, V, (T,), generator=g).int().cuda()
    new = lens + chunk

    def round_():
        st = dspark.dspark_pages_resize(cache, table, lens, new, rc)
        for layer in range(2):
            dspark.dspark_cache_append(cache, layer, kn, vn, off, st["kv_len"], st["page_table"])
        at = [dspark.dspark_paged_attention(q, cache, layer, off, st["kv_len"], st["page_table"], 0.1)
              for layer in range(2)]
        lp = dspark.dspark_logprobs(Z, tokens, 1.0, 5)
        fk = dspark.dspark_pages_fork(cache, st["page_table"], st["kv_len"], i32_pair[0], i32_pair[1], st["refcount"])
        cp = dspark.dspark_pages_compact(cache, fk["page_table"], fk["kv_len"], fk["refcount"])
        n = 22  # rows in use
        return [st["kv_len"], st["page_table"], *(x[key][:n] for x in at for key in ("out", "lse")),
                *(lp[key] for key in ("logp", "entropy", "lse", "top_ids", "top_logp")), fk["page_table"],
                fk["refcount"], fk["free_pages"], cp["page_table"], cp["refcount"], cp["page_map"], cp["n_live"]], \
            [st["workspace"], lp["workspace"], fk["workspace"], cp["workspace"], *(x["workspace"] for x in at)]

    i32_pair = i32([3, 7]), i32([0, 8])
    k0, v0 = k.clone(), v.clone()
    want, spaces = round_()
    assert [dspark.dspark_read_device_status(ws) for ws in spaces] == [0] * len(spaces)
    want = [x.clone() for x in want]
    k1, v1 = k.clone(), v.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, spaces = round_()
    for _ in range(2):
        k.copy_(k0)
        v.copy_(v0)
        graph.replay()
        for ws in spaces:
            assert dspark.dspark_read_device_status(ws) == 0
        for a, b in zip(want, got):
            assert torch.equal(a.nan_to_num(9.0) if a.is_floating_point() else a,
                               b.nan_to_num(9.0) if b.is_floating_point() else b)
        assert torch.equal(k, k1) and torch.equal(v, v1)
