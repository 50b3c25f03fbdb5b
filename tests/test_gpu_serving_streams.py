"""The serving calls on a stream that is not the current one: whose memory their results use."""
import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream whose blocks of the caching allocator hold t."""
    p = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= p < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


def calls():
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k, v = (torch.randn(1, 20, 16, 2, 64, device="cuda") for _ in range(2))
    cache = dspark.PagedCache(k, v)
    table, rc = i32([0, 1, -1], [2, -1, -1], [-1, -1, -1]), i32(*[1] * 3, *[0] * 17)
    lens, off = i32(20, 7, 0), i32(0, 1, 3, 3)
    q, new = torch.randn(3, 4, 64, device="cuda"), torch.randn(3, 2, 64, device="cuda")
    Z, tok = torch.randn(3, 5000, device="cuda"), i32(4, -1, 7)
    return {
        "append": lambda **kw: dspark.dspark_cache_append(cache, 0, new, new, off, lens, table, **kw),
        "attention": lambda **kw: dspark.dspark_paged_attention(q, cache, 0, off, lens, table, 0.1, **kw),
        "resize": lambda **kw: dspark.dspark_pages_resize(cache, table, lens, i32(3, 40, 1), rc, **kw),
        "fork": lambda **kw: dspark.dspark_pages_fork(cache, table, lens, i32(0), i32(2), rc, **kw),
        "compact": lambda **kw: dspark.dspark_pages_compact(cache, table, lens, rc, **kw),
        "copy": lambda **kw: dspark.dspark_pages_copy(cache, i32(2), i32(9), **kw),
        "logprobs": lambda **kw: dspark.dspark_logprobs(Z, tok, 1.0, 3, **kw),
        "logprobs of no rows": lambda **kw: dspark.dspark_logprobs(Z[:0], tok[:0], 1.0, 3, **kw),
    }


@pytest.mark.parametrize("name", ["append", "attention", "resize", "fork", "compact", "copy", "logprobs",
                                  "logprobs of no rows"])
def test_new_results_come_from_the_launch_stream(name):
    # A block of the current stream may still be read there by work that was
    # launched before the block was freed; only that stream may be handed it again.
    call, side = calls()[name], torch.cuda.Stream()
    want = call()
    torch.cuda.synchronize()
    free = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in [512] * 8 + [1 << 16, 1 << 21, 1 << 27]]
    del free  # (blocks of the current stream, to be taken if they may)
    got = call(stream=side)
    for key, t in got.items():
        if t.numel():
            assert owner(t) == side.cuda_stream, key
    assert dspark.dspark_read_device_status(got["workspace"], side) == 0
    for key, t in got.items():
        if key != "workspace":
            assert torch.equal(t.nan_to_num(9.0), want[key].nan_to_num(9.0)), key


def test_results_of_the_current_stream_given_by_name():
    call, cur = calls()["logprobs"], torch.cuda.current_stream()
    got = call(stream=cur)
    assert all(owner(t) == cur.cuda_stream for t in got.values())
