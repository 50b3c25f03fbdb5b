"""A process that uses two devices, one after the other: what the library finds out once, it finds out once a device
(CPU only: a stand-in for the CUDA runtime writes the launches down)."""
import fakecuda

CALLS = [dict(op="attention", cache="f32", dtype="f32", D=D) for D in (64, 128, 256)] + \
    [dict(op="attention", cache="bf16", D=D, T=T) for D in (64, 128, 256) for T in (4, 400)] + \
    [dict(op="attention", D=D, G=G, T=T) for D in (32, 64, 96, 128, 256) for G, T in ((4, 4), (16, 4), (4, 400))] + \
    [dict(op="attention", dtype="f32", D=D, G=G, T=T) for D in (64, 128, 256) for G, T in ((1, 4), (4, 4), (4, 16), (4, 400))] + \
    [dict(op=op, dtype=dt) for op in ("append", "read", "logprobs", "draft", "schedule", "verify") for dt in ("bf16", "f32")] + \
    [dict(op=op) for op in ("resize", "compact", "copy")] + \
    [dict(op=op, R=300, T=300) for op in ("draft", "verify")]


def test_every_call_runs_on_a_second_device(tmp_path):
    for c in CALLS:
        if c["op"] in ("append", "read") and c.get("dtype") == "f32":
            c["cache"] = "f32"
    got = fakecuda.run([dict(c, device=d) for d in (0, 1) for c in CALLS], tmp_path)
    first, second = got[:len(CALLS)], got[len(CALLS):]
    for c, a, b in zip(CALLS, first, second):
        assert a["status"] == 0 and a["launches"], c
        assert b["status"] == 0, c
        assert [(x["kernel"], x["smem"]) for x in a["launches"]] == [(x["kernel"], x["smem"]) for x in b["launches"]], c
        assert {x["device"] for x in b["launches"]} == {1}


def test_grids_follow_the_device(tmp_path):
    calls = [dict(op="attention", cache="bf16", T=400), dict(op="attention", T=400)]
    got = fakecuda.run([dict(c, device=d) for d in (1, 0, 2, 1) for c in calls], tmp_path)
    for n, sms in enumerate((132, 152, 112, 132)):
        for x in got[2 * n: 2 * n + 2]:
            assert x["status"] == 0 and x["launches"][0]["grid"] == sms and "attention_tc" in x["launches"][0]["kernel"]
