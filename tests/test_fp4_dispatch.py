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
