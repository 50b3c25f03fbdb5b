"""The serving operators' C entries refuse bad host-side arguments before they touch a GPU (CPU only)."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_05_gb300 import binding, build

    build.build()
    return binding.load()


def cache(**kw):
    from speculative_decoding_draft_05_gb300.serving import _CacheStruct

    a = dict(k=256, v=256, dtype=1, layers=2, n_pages=10, page_size=16, heads=2, head_dim=64, layer_stride=20480,
             page_stride=2048, token_stride=128, head_stride=64)
    a.update(kw)
    return ctypes.byref(_CacheStruct(**a))


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(dtype=3), 1), (dict(layers=0), 1), (dict(n_pages=0), 1),
              (dict(page_size=0), 1), (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(page_stride=0), 1),
              (dict(token_stride=-1), 1), (dict(head_stride=0), 1), (dict(k=257), 1), (dict(head_dim=264), 2),
              (dict(heads=1025), 2), (dict(page_size=65537), 2), (dict(page_size=65536, heads=1024, head_dim=64), 2)]
WS = 1 << 30


def attention(lib, c=None, **kw):
    a = dict(q=256, ts=512, hs=64, Hq=4, layer=0, off=16, kv=16, tab=16, R=2, T=3, P=4, scale=0.1, out=256, lse=16,
             ws=256, wsb=WS)
    a.update(kw)
    return lib.dspark_paged_attention(a["q"], a["ts"], a["hs"], a["Hq"], c or cache(), a["layer"], a["off"], a["kv"],
                                      a["tab"], a["R"], a["T"], a["P"], a["scale"], a["out"], a["lse"], a["ws"],
                                      a["wsb"], None)


def test_attention(lib):
    for kw, st in BAD_CACHES:
        assert attention(lib, cache(**kw)) == st, kw
    for kw in (dict(q=None), dict(off=None), dict(kv=None), dict(tab=None), dict(out=None), dict(lse=None), dict(R=0),
               dict(T=-1), dict(P=0), dict(Hq=0), dict(Hq=3), dict(layer=2), dict(layer=-1), dict(scale=math.nan),
               dict(scale=math.inf), dict(q=257), dict(out=8), dict(ts=-1)):
        assert attention(lib, **kw) == 1, kw
    for kw in (dict(R=65536), dict(P=1 << 30, R=4), dict(T=1 << 30)):
        assert attention(lib, **kw) == 2, kw
    for kw in (dict(ws=None), dict(wsb=256), dict(ws=128)):
        assert attention(lib, **kw) == 3, kw
    assert lib.dspark_paged_attention_workspace_bytes(cache()) > 256
    assert lib.dspark_paged_attention_workspace_bytes(cache(head_dim=512)) == 0
    assert lib.dspark_paged_attention_workspace_bytes(None) == 0


def test_append(lib):
    def call(c=None, **kw):
        a = dict(layer=0, k=256, v=256, ts=128, hs=64, off=16, kv=16, tab=16, R=2, T=3, P=4, ws=256, wsb=WS)
        a.update(kw)
        return lib.dspark_cache_append(c or cache(), a["layer"], a["k"], a["v"], a["ts"], a["hs"], a["off"], a["kv"],
                                       a["tab"], a["R"], a["T"], a["P"], a["ws"], a["wsb"], None)

    for kw, st in BAD_CACHES:
        assert call(cache(**kw)) == st, kw
    for kw in (dict(k=None), dict(v=None), dict(off=None), dict(kv=None), dict(tab=None), dict(T=-1), dict(ts=-1),
               dict(k=257), dict(R=0), dict(P=0), dict(layer=2)):
        assert call(**kw) == 1, kw
    assert call(R=65536) == 2
    assert call(ws=None) == 3 and call(wsb=8) == 3 and call(ws=8) == 3


def test_pages(lib):
    def resize(c=None, **kw):
        a = dict(tab=16, kv=16, new=16, rc=16, R=2, P=4, to=16, ko=16, ro=16, free=16, ws=256, wsb=WS)
        a.update(kw)
        return lib.dspark_pages_resize(c or cache(), a["tab"], a["kv"], a["new"], a["rc"], a["R"], a["P"], a["to"],
                                       a["ko"], a["ro"], a["free"], a["ws"], a["wsb"], None)

    def fork(c=None, **kw):
        a = dict(tab=16, kv=16, rc=16, pa=16, ch=16, n=1, R=2, P=4, to=16, ko=16, ro=16, free=16, ws=256, wsb=WS)
        a.update(kw)
        return lib.dspark_pages_fork(c or cache(), a["tab"], a["kv"], a["rc"], a["pa"], a["ch"], a["n"], a["R"],
                                     a["P"], a["to"], a["ko"], a["ro"], a["free"], a["ws"], a["wsb"], None)

    def compact(c=None, **kw):
        a = dict(tab=16, kv=16, rc=16, R=2, P=4, to=16, ro=16, map=16, live=16, ws=256, wsb=WS)
        a.update(kw)
        return lib.dspark_pages_compact(c or cache(), a["tab"], a["kv"], a["rc"], a["R"], a["P"], a["to"], a["ro"],
                                        a["map"], a["live"], a["ws"], a["wsb"], None)

    for call in (resize, fork, compact):
        for kw, st in BAD_CACHES:
            assert call(cache(**kw)) == st, (call, kw)
        for kw in (dict(tab=None), dict(kv=None), dict(rc=None), dict(to=None), dict(ro=None), dict(R=0), dict(P=0)):
            assert call(**kw) == 1, (call, kw)
        assert call(R=65536) == 2 and call(R=4, P=1 << 30) == 2
        assert call(ws=None) == 3 and call(wsb=256) == 3 and call(ws=16) == 3
    assert resize(new=None) == 1 and resize(ko=None) == 1 and resize(free=None) == 1
    assert fork(pa=None) == 1 and fork(ch=None) == 1 and fork(free=None) == 1 and fork(n=-1) == 1 and fork(n=3) == 1
    assert compact(map=None) == 1 and compact(live=None) == 1
    assert lib.dspark_pages_copy(cache(), None, 16, 1, 256, 256, None) == 1
    assert lib.dspark_pages_copy(cache(), 16, 16, -1, 256, 256, None) == 1
    assert lib.dspark_pages_copy(cache(), 16, 16, 1, 256, 8, None) == 3
    assert lib.dspark_pages_workspace_bytes(0, 5) == 0 and lib.dspark_pages_workspace_bytes(5, 100) >= 256


def test_logprobs(lib):
    def call(**kw):
        a = dict(Z=256, dt=1, step=1024, tok=16, n=4, V=1024, T=1.0, top=5, lp=16, en=16, lse=16, ids=16, tl=16, ws=256,
                 wsb=WS)
        a.update(kw)
        return lib.dspark_logprobs(a["Z"], a["dt"], a["step"], a["tok"], a["n"], a["V"], a["T"], a["top"], a["lp"],
                                   a["en"], a["lse"], a["ids"], a["tl"], a["ws"], a["wsb"], None)

    for kw in (dict(Z=None), dict(tok=None), dict(lp=None), dict(en=None), dict(lse=None), dict(ids=None),
               dict(tl=None), dict(n=0), dict(V=0), dict(step=1000), dict(T=0.0), dict(T=-1.0), dict(T=math.nan),
               dict(T=math.inf), dict(dt=2), dict(top=-1), dict(Z=264), dict(step=1028)):
        assert call(**kw) == 1, kw
    for kw in (dict(V=1020), dict(top=33), dict(V=8, top=9), dict(V=(1 << 30) + 8, step=(1 << 30) + 8)):
        assert call(**kw) == 2, kw
    for kw in (dict(ws=None), dict(ws=64), dict(wsb=256)):
        assert call(**kw) == 3, kw
    assert lib.dspark_logprobs_workspace_bytes(0, 8) == 0 and lib.dspark_logprobs_workspace_bytes(1, 8) >= 256


def test_factors_past_the_largest_float(lib):
    # log2(e) scale, or log2(e) / T: every result would be NaN
    assert attention(lib, scale=3e38) == 1 and attention(lib, scale=-2.5e38) == 1
    for T in (1e-45, 1e-39, 4e-39):
        assert lib.dspark_logprobs(256, 1, 1024, 16, 4, 1024, T, 5, 16, 16, 16, 16, 16, 256, WS, None) == 1, T


def test_another_device_than_the_current_one_is_refused(monkeypatch):
    # a launch goes to the current device, whatever the stream and the tensors
    import torch

    from speculative_decoding_draft_05_gb300 import serving

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7 + index)
    assert serving._stream(torch.device("cuda", 0), None) == 7
    with pytest.raises(ValueError, match="current device"):
        serving._stream(torch.device("cuda", 1), None)
    with pytest.raises(ValueError, match="current device"):
        serving._stream(torch.device("cuda", 1), type("Stream", (), dict(cuda_stream=9))())


def test_attention_workspace_holds_the_launched_ctas_pieces(lib):
    # two pieces a CTA: rows of head_dim floats, a maximum and a sum; 152 CTAs of 256 rows, or 304 of 64
    def floor(D, bf16):
        simt, tc = 304 * 2 * 64 * (4 * D + 8), 152 * 2 * 256 * (4 * D + 8)
        return max(simt, tc) if bf16 and D <= 128 else simt

    for D in (16, 64, 128, 256):
        for dtype in (0, 1):
            n = lib.dspark_paged_attention_workspace_bytes(cache(dtype=dtype, head_dim=D))
            assert floor(D, dtype == 1) <= n <= floor(D, dtype == 1) + (1 << 15), (D, dtype, n)


def test_counts_that_a_step_past_the_end_would_overflow(lib):
    assert attention(lib, Hq=2, T=0x3fff8001) == 2   # 2^31 - 2^16 + 2 rows
    assert lib.dspark_cache_append(cache(), 0, 256, 256, 128, 64, 16, 16, 16, 2, 0x7fff0001, 4, 256, WS, None) == 2
    n = (1 << 30) + 1
    assert lib.dspark_logprobs(256, 1, 8, 16, n, 8, 1.0, 5, 16, 16, 16, 16, 16, 256, 1 << 60, None) == 2


def test_rows_that_step_evenly():
    import torch

    from speculative_decoding_draft_05_gb300.serving import _row_step

    Z = torch.empty(5, 7, 16)
    V = 16
    assert _row_step(Z) == V and _row_step(Z[0]) == V and _row_step(Z[0, 0]) == V
    assert _row_step(Z[:, :1]) == 7 * V and _row_step(Z[:, 3:4]) == 7 * V   # a dimension of one: its stride says nothing
    assert _row_step(Z[1:2]) == V and _row_step(Z[:1, ::2]) == 2 * V
    assert _row_step(Z[:, 0]) == 7 * V and _row_step(Z[2:3, 1:2]) == V
    assert _row_step(Z.view(5, 1, 7, 16)[:, :, :1]) == 7 * V
    assert _row_step(torch.empty(5, 7, 24)[..., :16]) == 24
    assert _row_step(Z[:, :6]) is None and _row_step(Z.transpose(0, 1)) is None
    assert _row_step(torch.empty(2, 3, 4, 16)[:, :, :2]) is None
    assert _row_step(torch.empty(2, 3, 4, 16)[:, ::3, ::4]) == 3 * 4 * V


def test_serving_kernels_read_nothing_by_the_non_coherent_path():
    # They may start while the kernel before them still writes what they read.
    import os
    import re

    from speculative_decoding_draft_05_gb300 import build

    for name in ("attention.cu", "attention.cuh", "attention_tc.cu", "logprobs.cu", "pages.cu"):
        with open(os.path.join(build.CSRC, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert "griddepcontrol" in code or "wait_for_previous" in code or name.endswith(".cuh"), name
        for word in ("__ldg", "__restrict__", "ld.global.nc"):
            assert word not in code, (name, word)


def test_a_pool_of_more_pages_than_their_numbers_can_be_rounded(lib):
    assert attention(lib, cache(n_pages=0x7fff0001)) == 2
