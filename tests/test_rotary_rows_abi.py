"""dspark_cache_append_rotary refuses a q_out whose rows lie one over the other, and no other (CPU only: calls that
pass the checks of their arguments are stopped by a missing workspace)."""
import itertools

import pytest

from test_fp4_abi import append, lib, rows  # noqa: F401  (lib: a fixture)

INVALID, WORKSPACE = 1, 3
ROT = dict(cos_sin=256, positions=None, n_positions=100, dim=64, interleaved=0)


def status(lib, **kw):  # noqa: F811
    got = {append(lib, c, ROT, ws=None, **kw) for c in (None, rows())}
    assert len(got) == 1
    return got.pop()


def overlap(T, Hq, ts, hs, D):
    at = sorted(t * ts + h * hs for t in range(T) for h in range(Hq))
    return any(b - a < D for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("T, Hq, ts, hs, st", [
    (3, 4, 64, 64, INVALID),     # head 1 of a token is head 0 of the next
    (3, 4, 128, 64, INVALID),
    (3, 4, 255, 64, INVALID),
    (3, 4, 256, 64, WORKSPACE),
    (3, 4, 64, 191, INVALID),    # heads first
    (3, 4, 64, 192, WORKSPACE),
    (1, 4, 64, 64, WORKSPACE),   # strides of dimensions of one carry no meaning
    (3, 1, 64, 64, WORKSPACE),
    (1, 4, 0, 64, WORKSPACE),
    (3, 1, 64, 0, WORKSPACE),
    (0, 4, 0, 0, WORKSPACE),
    (3, 3, 192, 128, WORKSPACE),  # rows in one another's gaps
    (4, 4, 192, 128, INVALID),
    (0x7ffffff, 8, 512, 64, WORKSPACE),
    (0x7ffffff, 8, 511, 64, INVALID),
    (3, 4, 1 << 62, 1 << 61, INVALID),  # (2 heads on from a token: the next one)
    (3, 2, 1 << 62, 1 << 61, WORKSPACE),
])
def test_rows_over_one_another(lib, T, Hq, ts, hs, st):  # noqa: F811
    assert status(lib, T=T, Hq=Hq, ots=ts, ohs=hs) == st
    assert status(lib, T=T, Hq=Hq, ots=ts, ohs=hs, q=512, qts=ts, qhs=hs) == st  # in place


def test_all_small_layouts(lib):  # noqa: F811
    for T, Hq, ts, hs in itertools.product((1, 2, 3, 5), (1, 2, 3, 6), range(0, 400, 32), range(0, 400, 32)):
        want = INVALID if overlap(T, Hq, ts, hs, 64) else WORKSPACE
        assert status(lib, T=T, Hq=Hq, ots=ts, ohs=hs) == want, (T, Hq, ts, hs)
