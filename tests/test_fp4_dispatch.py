"""Which kernel attention over a 4-bit cache takes, by the rows there are (CPU only: a stand-in for the CUDA runtime
writes the launches down)."""
import pytest

import fakecuda

FEW8, FEW16, MANY = "attention_fp4_kernelILi128ELi1", "attention_fp4_kernelILi128ELi2", "attention_tc_kernelILi128ELb1"
SIMT, TILES = "attention_fp4_simt_kernel", "attention_simt_kernel"


def kernels(calls, where):
    out = []
    for c, r in zip(calls, fakecuda.run([dict(c, op="attention") for c in calls], where)):
        assert r["status"] == 0, c
        assert "attention_combine" in r["launches"][-1]["kernel"]
        out.append(r["launches"][0]["kernel"])
    return out


def test_rows_of_bf16_queries(tmp_path):
    # requests, tokens, query heads of a K/V head
    want = [((32, 32, 4), FEW8), ((32, 32, 8), FEW8), ((32, 64, 4), FEW8), ((32, 256, 1), FEW8),   # chunks alike
            ((32, 96, 4), FEW16), ((32, 128, 4), FEW16), ((32, 64, 8), FEW16), ((32, 32, 16), FEW16),
            ((32, 512, 1), FEW16), ((32, 160, 4), MANY), ((32, 544, 1), MANY), ((32, 32, 17), MANY),
            ((1, 2, 4), FEW8), ((1, 4, 4), FEW16), ((1, 5, 4), MANY),                              # one request
            ((32, 5, 4), FEW8),                                                                    # some without tokens
            ((32, 33, 4), FEW8), ((32, 61, 4), FEW16), ((32, 95, 4), FEW16), ((32, 97, 4), MANY),  # uneven
            ((128, 467, 4), MANY), ((128, 357, 4), FEW16)]
    got = kernels([dict(R=R, T=T, G=G) for (R, T, G), _ in want], tmp_path)
    for (c, w), g in zip(want, got):
        assert w in g, (c, w, g)


@pytest.mark.parametrize("dtype, D", [("f32", 32), ("f32", 64), ("f32", 96), ("f32", 128), ("f32", 256), ("bf16", 160),
                                      ("bf16", 256)])
def test_rows_on_cuda_cores(tmp_path, dtype, D):
    narrow = D <= 64
    want = [((16, 16, 4), SIMT), ((16, 64, 4), SIMT), ((16, 80, 4), SIMT), ((16, 16, 20), SIMT),      # chunks alike
            ((16, 208, 4), TILES), ((16, 16, 49), TILES), ((1, 49, 1), TILES)]
    for T, G in ((96, 4), (128, 4), (192, 4), (16, 21), (16, 48)):
        want.append(((16, T, G), TILES if narrow else SIMT))
    want += [((16, 143, 4), SIMT), ((16, 239, 4), SIMT), ((16, 241, 4), TILES if narrow else SIMT),   # uneven
             ((16, 479, 4), TILES if narrow else SIMT), ((16, 481, 4), TILES)]
    got = kernels([dict(R=R, T=T, G=G, dtype=dtype, D=D) for (R, T, G), _ in want], tmp_path)
    for (c, w), g in zip(want, got):
        assert w in g, (c, w, g)


def test_calls_without_tokens(tmp_path):
    """They check their offsets in a kernel that other calls run too."""
    calls = [dict(R=4, T=0, G=G, D=D) for G in (1, 40) for D in (32, 64, 96, 128)]
    for c, k in zip(calls, kernels(calls, tmp_path)):
        assert f"attention_fp4_kernelILi{c['D']}" in k, (c, k)
    calls = [dict(R=4, T=0, G=4, D=D, dtype=t) for D, t in ((64, "f32"), (128, "f32"), (256, "f32"), (160, "bf16"))]
    for c, k in zip(calls, kernels(calls, tmp_path)):
        assert TILES in k, (c, k)
