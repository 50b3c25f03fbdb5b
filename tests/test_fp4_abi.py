"""The 4-bit cache's and the rotation's C entries refuse bad host-side arguments before they touch a GPU (CPU only)."""
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

    a = dict(k=256, v=256, dtype=2, layers=2, n_pages=10, page_size=32, heads=2, head_dim=64, layer_stride=23040,
             page_stride=2304, token_stride=576, head_stride=1152)
    a.update(kw)
    return ctypes.byref(_CacheStruct(**a))


def rows(**kw):
    return cache(**dict(dict(dtype=1, page_size=16, layer_stride=20480, page_stride=2048, token_stride=128,
                             head_stride=64), **kw))


BAD = [(dict(k=None), 1), (dict(v=None), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(layers=0), 1),
       (dict(n_pages=0), 1), (dict(page_size=0), 1), (dict(heads=0), 1), (dict(head_dim=0), 1), (dict(page_stride=0), 1),
       (dict(head_stride=0), 1), (dict(k=264), 1), (dict(v=258), 1), (dict(token_stride=64), 1),
       (dict(page_stride=2312), 1), (dict(head_stride=1160), 1), (dict(layer_stride=8), 1),
       (dict(page_size=24), 2), (dict(head_dim=80, token_stride=720), 2), (dict(head_dim=288, token_stride=2592), 2),
       (dict(heads=1025), 2), (dict(page_size=65552), 2)]
WS = 1 << 30


def attention(lib, c=None, **kw):
    a = dict(q=256, ts=512, hs=64, Hq=4, dt=1, layer=0, kf=1.0, vf=1.0, off=16, kv=16, tab=16, R=2, T=3, P=4, scale=0.1,
             out=256, lse=16, ws=256, wsb=WS)
    a.update(kw)
    return lib.dspark_paged_attention_fp4(a["q"], a["ts"], a["hs"], a["Hq"], a["dt"], c or cache(), a["layer"], a["kf"],
                                          a["vf"], a["off"], a["kv"], a["tab"], a["R"], a["T"], a["P"], a["scale"],
                                          a["out"], a["lse"], a["ws"], a["wsb"], None)


FACTORS = (0.0, -1.0, math.nan, math.inf, 2.0 ** -61, 2.0 ** 61)


def test_attention(lib):
    for kw, st in BAD:
        assert attention(lib, cache(**kw)) == st, kw
    assert attention(lib, rows()) == 1
    for kw in (dict(q=None), dict(off=None), dict(kv=None), dict(tab=None), dict(out=None), dict(lse=None), dict(R=0),
               dict(T=-1), dict(P=0), dict(Hq=0), dict(Hq=3), dict(layer=2), dict(layer=-1), dict(scale=math.nan),
               dict(scale=math.inf), dict(q=257), dict(out=8), dict(ts=-1), dict(hs=-1), dict(dt=2), dict(dt=-1),
               dict(q=258, dt=0), dict(scale=3e38, kf=4.0), dict(scale=1e30, kf=2.0 ** 60)):
        assert attention(lib, **kw) == 1, kw
    for f in FACTORS:
        assert attention(lib, kf=f) == 1 and attention(lib, vf=f) == 1, f
    for kw in (dict(R=65536), dict(P=1 << 30, R=4), dict(T=1 << 30)):
        assert attention(lib, **kw) == 2, kw
    for kw in (dict(ws=None), dict(wsb=256), dict(ws=128)):
        assert attention(lib, **kw) == 3, kw
    # the calls for caches of rows do not take it
    assert lib.dspark_paged_attention(256, 512, 64, 4, cache(), 0, 16, 16, 16, 2, 3, 4, 0.1, 256, 16, 256, WS, None) == 1
    assert lib.dspark_cache_append(cache(), 0, 256, 256, 128, 64, 16, 16, 16, 2, 3, 4, 256, WS, None) == 1
    assert lib.dspark_paged_attention_workspace_bytes(cache()) == 0


def test_attention_workspace(lib):
    size = lib.dspark_paged_attention_fp4_workspace_bytes
    for D in (32, 64, 128, 256):
        for dt in (0, 1):
            assert size(cache(head_dim=D, token_stride=9 * D), dt) >= 304 * 2 * 64 * (4 * D + 8)
    assert size(rows(), 1) == 0 and size(None, 1) == 0 and size(cache(), 2) == 0
    assert size(cache(head_dim=288), 1) == 0 and size(cache(head_dim=0), 1) == 0


class Rotary(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("n_positions", ctypes.c_int),
                ("dim", ctypes.c_int), ("interleaved", ctypes.c_int)]


def append(lib, c=None, rot=None, **kw):
    a = dict(layer=0, kf=1.0, vf=1.0, dt=1, k=256, v=256, ts=128, hs=64, q=256, qts=256, qhs=64, Hq=4, qo=512, ots=256,
             ohs=64, off=16, kv=16, tab=16, R=2, T=3, P=4, ws=256, wsb=WS)
    a.update(kw)
    return lib.dspark_cache_append_rotary(c or cache(), a["layer"], a["kf"], a["vf"],
                                          None if rot is None else ctypes.byref(Rotary(**rot)), a["dt"], a["k"], a["v"],
                                          a["ts"], a["hs"], a["q"], a["qts"], a["qhs"], a["Hq"], a["qo"], a["ots"],
                                          a["ohs"], a["off"], a["kv"], a["tab"], a["R"], a["T"], a["P"], a["ws"],
                                          a["wsb"], None)


def test_append(lib):
    good = dict(cos_sin=256, positions=None, n_positions=100, dim=64, interleaved=0)
    for kw, st in BAD:
        assert append(lib, cache(**kw), good) == st, kw
    assert append(lib, rows(head_dim=264), good) == 2 and append(lib, rows(k=257), good) == 1
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(qo=None), dict(off=None), dict(kv=None), dict(tab=None),
               dict(T=-1), dict(ts=-1), dict(hs=-1), dict(qts=-1), dict(qhs=-1), dict(ots=-1), dict(ohs=-1), dict(Hq=-1),
               dict(k=257), dict(q=257), dict(qo=257), dict(dt=2), dict(R=0), dict(P=0), dict(layer=2),
               dict(q=512, ots=300), dict(q=512, ohs=80), dict(ots=0), dict(ots=63), dict(ohs=0), dict(ohs=63)):
        assert append(lib, None, good, **kw) == 1, kw
    for f in FACTORS:
        assert append(lib, None, good, kf=f) == 1 and append(lib, None, good, vf=f) == 1, f
    assert append(lib, rows(), good, dt=0) == 1 and append(lib, rows(dtype=0), good) == 1  # the cache's type
    for kw in (dict(cos_sin=None), dict(cos_sin=258), dict(n_positions=0), dict(dim=0), dict(dim=-2), dict(dim=3),
               dict(dim=66)):
        assert append(lib, None, dict(good, **kw)) == 1, kw
    for kw in (dict(R=65536), dict(T=0x7fff0001), dict(T=1 << 29)):
        assert append(lib, None, good, **kw) == 2, kw
    for kw in (dict(ws=None), dict(wsb=8), dict(ws=8)):
        assert append(lib, None, good, **kw) == 3, kw


def test_read(lib):
    def call(c=None, **kw):
        a = dict(layer=0, kf=1.0, vf=1.0, dt=1, off=16, kv=16, tab=16, R=2, T=3, P=4, k=256, v=256, ws=256, wsb=WS)
        a.update(kw)
        return lib.dspark_cache_read(c or cache(), a["layer"], a["kf"], a["vf"], a["dt"], a["off"], a["kv"], a["tab"],
                                     a["R"], a["T"], a["P"], a["k"], a["v"], a["ws"], a["wsb"], None)

    for kw, st in BAD:
        assert call(cache(**kw)) == st, kw
    for kw in (dict(k=None), dict(v=None), dict(k=264), dict(v=260), dict(off=None), dict(kv=None), dict(tab=None),
               dict(T=-1), dict(R=0), dict(P=0), dict(layer=-1), dict(dt=2)):
        assert call(**kw) == 1, kw
    for f in FACTORS:
        assert call(kf=f) == 1 and call(vf=f) == 1, f
    assert call(rows(), dt=0) == 1
    assert call(R=65536) == 2 and call(T=0x7fff0001) == 2
    assert call(ws=None) == 3 and call(wsb=8) == 3 and call(ws=8) == 3


def test_pages_take_a_4_bit_cache(lib):
    def resize(c, **kw):
        a = dict(tab=16, kv=16, new=16, rc=16, R=2, P=4, to=16, ko=16, ro=16, free=16, ws=256, wsb=256)
        a.update(kw)
        return lib.dspark_pages_resize(c, a["tab"], a["kv"], a["new"], a["rc"], a["R"], a["P"], a["to"], a["ko"],
                                       a["ro"], a["free"], a["ws"], a["wsb"], None)

    assert resize(cache()) == 3  # (past the checks of the cache: the workspace is too small)
    for kw, st in BAD:
        assert resize(cache(**kw)) == st, kw
    assert lib.dspark_pages_copy(cache(), 16, 16, 1, 256, 8, None) == 3


def test_the_binding_refuses(monkeypatch):
    import torch

    import speculative_decoding_draft_05_gb300 as dspark

    with pytest.raises(TypeError, match="CUDA"):
        dspark.PagedCacheFp4(torch.zeros(1, 1, 1, 1, 576, dtype=torch.uint8), None)
    with pytest.raises(TypeError, match="cache"):
        dspark.dspark_cache_read(None, 0, None, None, None, 1)
    with pytest.raises(ValueError, match="multiple"):
        dspark.PagedCacheFp4.zeros(1, 1, 24, 1, 64)
    with pytest.raises(ValueError, match="multiple"):
        dspark.PagedCacheFp4.zeros(1, 1, 16, 1, 80)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)  # (host tensors that pass for others: nothing is launched)
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    good = z(1, 4, 2, 2, 576)
    C = dspark.PagedCacheFp4
    for k, v, what in ((z(1, 4, 2, 2, 576, dt=torch.int8), good, TypeError), (good[0], good[0], ValueError),
                       (z(1, 4, 2, 2, 144), z(1, 4, 2, 2, 144), ValueError), (good, z(1, 4, 2, 2, 288), ValueError),
                       (good[:, :, :, :, ::2], good[:, :, :, :, ::2], ValueError),
                       (z(1, 4, 2, 4, 576)[:, :, :, ::2], z(1, 4, 2, 4, 576)[:, :, :, ::2], ValueError),
                       (good, z(1, 4, 4, 2, 576)[:, :, ::2], ValueError)):
        with pytest.raises(what):
            C(k, v)
    for f in FACTORS:
        with pytest.raises(ValueError, match="factor"):
            C(good, good, f)
        with pytest.raises(ValueError, match="factor"):
            C(good, good, 1.0, f)
    c = C(good, good)
    i32 = dict(dt=torch.int32)
    args = (z(3, **i32), z(2, **i32), z(2, 4, **i32))
    kv = z(5, 2, 64, dt=torch.bfloat16)
    call = dspark.dspark_cache_append_rotary
    for what, match, a, kw in (
            (TypeError, "k_new", (z(5, 2, 64, dt=torch.float16), kv), {}),
            (TypeError, "v_new", (kv, kv.float()), {}),
            (ValueError, "v_new", (kv, kv[:4]), {}),
            (ValueError, "k_new", (z(5, 3, 64, dt=torch.bfloat16), kv), {}),
            (ValueError, "cos_sin", (kv, kv), dict(cos_sin=z(64, dt=torch.float32))),
            (TypeError, "cos_sin", (kv, kv), dict(cos_sin=z(9, 64, dt=torch.float64))),
            (ValueError, "positions", (kv, kv), dict(positions=z(5, **i32))),
            (ValueError, "positions", (kv, kv), dict(cos_sin=z(9, 64, dt=torch.float32), positions=z(4, **i32))),
            (ValueError, "q must", (kv, kv), dict(q=kv[:4])),
            (TypeError, "q must", (kv, kv), dict(q=kv.float())),
            (ValueError, "q_out", (kv, kv), dict(q_out=kv)),
            (ValueError, "q_out", (kv, kv), dict(q=kv, q_out=kv[:4])),
            (ValueError, "q_out", (kv, kv), dict(q=kv, q_out=z(5, 3, 64, dt=torch.bfloat16)))):
        with pytest.raises(what, match=match):
            call(c, 0, *a, *args, **kw)
    with pytest.raises(TypeError, match="dtype"):
        dspark.dspark_cache_read(c, 0, *args, 5, dtype=torch.float16)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        dspark.dspark_paged_attention(z(5, 4, 64, dt=torch.float16), c, 0, *args, 0.1)


def test_kernels_read_nothing_by_the_non_coherent_path():
    # They may start while the kernel before them still writes what they read.
    import os
    import re

    from speculative_decoding_draft_05_gb300 import build

    for name in sorted(os.listdir(build.CSRC)):
        if not (name.startswith(("attention", "fp4", "rows", "append"))):
            continue
        with open(os.path.join(build.CSRC, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        for word in ("__ldg", "__restrict__", "ld.global.nc"):
            assert word not in code, (name, word)
