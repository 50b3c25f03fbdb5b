"""dspark_logprobs against the definition in 64 bits.

Tolerances.  With u = 2^-24: the scaled logit's rounding moves ln p by at most
4 u max|x|, the exponential's by 4 u, and the positive sums over a lane's 128
terms and the 5 + 5 + log2(chunks) merges by (160) u; so lse and logp are
within 200 u + 4 u max|x|, and the entropy, a difference of ln s and t / s whose
parts are each relative to the same sums, within 400 u (1 + ln V).
"""
import math

import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def reference(Z, tokens, T, top):
    V = Z.shape[-1]
    z = Z.reshape(-1, V).cpu().double()
    tok = tokens.reshape(-1).cpu().long()
    n = len(tok)
    out = dict(logp=torch.full((n,), math.nan, dtype=torch.float64),
               entropy=torch.full((n,), math.nan, dtype=torch.float64),
               lse=torch.full((n,), math.nan, dtype=torch.float64), ids=torch.full((n, top), -1, dtype=torch.int64),
               top=torch.full((n, top), math.nan, dtype=torch.float64))
    for i in range(n):
        if tok[i] < 0:
            continue
        x = z[i] / T
        m = x.max()
        lse = torch.logsumexp(x, 0)
        lp = (x - m) - torch.log(torch.exp(x - m).sum())  # (x - lse loses everything at |x| = 3e38)
        p = lp.exp()
        out["lse"][i] = lse
        out["logp"][i] = lp[tok[i]] if tok[i] < V else math.nan
        out["entropy"][i] = -torch.where(p > 0, p * lp, 0.0 * p).sum()
        rank = torch.where(z[i].isnan(), -math.inf, z[i])
        out["ids"][i] = torch.sort(rank, descending=True, stable=True).indices[:top]
        out["top"][i] = lp[out["ids"][i]]
    return out


def close(got, want, tol, what):
    got = got.reshape(want.shape).cpu().double()
    assert (got.isnan() == want.isnan()).all(), f"{what}: NaN pattern"
    fine = want.isfinite()
    same = want.isinf()
    assert (got[same] == want[same]).all(), what
    err = (got - want).abs()[fine]
    assert err.numel() == 0 or err.max() <= tol, f"{what}: {err.max():.3g} > {tol:.3g}"


@pytest.mark.parametrize("V", [1024, 9000])
def test_one_row_of_each_request(V):
    # [R, 1, V] of a wider array: the rows step evenly, the stride of the dimension of one says nothing
    Z = torch.randn(6, 4, V, generator=torch.Generator().manual_seed(41)).cuda()
    tok = torch.tensor([[3], [-1], [7], [0], [V - 1], [9]], dtype=torch.int32, device="cuda")
    a, b = run(Z[:, 2:3], tok, top=3), run(Z[:, 2:3].contiguous(), tok, top=3)
    for key in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(a[key].nan_to_num(9.0), b[key].nan_to_num(9.0)), key
    with pytest.raises(ValueError):
        run(Z[:, :2], torch.zeros(6, 2, dtype=torch.int32, device="cuda"))


def run(Z, tokens, T=1.0, top=0, status=0, **kw):
    r = dspark.dspark_logprobs(Z, tokens, T, top, **kw)
    assert dspark.dspark_read_device_status(r["workspace"], kw.get("stream")) == status
    w = reference(Z, tokens, T, top)
    z = Z.float()
    big = float(z[z.isfinite()].abs().max()) / T if z.isfinite().any() else 0.0
    tol = 200 * U + 4 * U * big
    close(r["lse"], w["lse"], tol, "lse")
    close(r["logp"], w["logp"], tol, "logp")
    close(r["entropy"], w["entropy"], 400 * U * (1 + math.log(Z.shape[-1])), "entropy")
    assert torch.equal(r["top_ids"].reshape(w["ids"].shape).cpu().long(), w["ids"])
    close(r["top_logp"], w["top"], tol, "top_logp")
    return r


def logits(shape, dtype, seed=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(shape, generator=g) * std
    z -= 1.1 * torch.log(torch.arange(1, shape[-1] + 1).float())
    return z.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [8, 16, 248, 256, 264, 1024, 4096, 4104, 32000, 151936])
@pytest.mark.parametrize("T,top", [(1.0, 5), (0.7, 1), (1.3, 32), (1.0, 0)])
def test_matches_the_definition(dtype, V, T, top):
    n = 7 if V < 100000 else 3
    top = min(top, V)
    Z = logits((n, V), dtype, seed=V)
    tokens = torch.randint(0, V, (n,), generator=torch.Generator().manual_seed(1)).int()
    tokens[0], tokens[1] = 0, V - 1
    run(Z, tokens.cuda(), T, top)


def test_verify_layout_and_skipped_rows():
    R, g, V = 5, 4, 1000
    Z = logits((R, g + 1, V), BF16, seed=2)
    tokens = torch.randint(0, V, (R, g + 1)).int()
    for r in range(R):
        tokens[r, r:] = -1  # request 0 emits nothing
    Z[0] = math.nan  # rows that are not read
    r = run(Z, tokens.cuda(), 1.0, 7)
    assert r["logp"].shape == (R, g + 1) and r["top_ids"].shape == (R, g + 1, 7)
    assert (r["top_ids"][0] == -1).all() and r["logp"][0].isnan().all()
    r = run(Z, torch.full_like(tokens, -1).cuda(), 1.0, 3)  # nothing wanted


@pytest.mark.parametrize("n,V", [(30000, 24), (13000, 264), (5000, 4096)])
def test_many_rows(n, V):
    Z = logits((n, V), BF16, seed=n)
    tokens = torch.randint(0, V, (n,), generator=torch.Generator().manual_seed(n)).int()
    keep = torch.zeros(n, dtype=torch.bool)
    keep[::97] = True  # few, but everywhere
    keep[4000:4100] = keep[-3:] = True
    if n == 30000:
        keep[12288:24576] = False
    tokens[~keep] = -1
    run(Z, tokens.cuda(), 1.0, 4)


def test_no_rows():
    Z = logits((2, 64), F32)[:0]
    r = dspark.dspark_logprobs(Z, torch.empty(0, dtype=torch.int32, device="cuda"), 1.0, 3,
                               workspace=torch.full((512,), 255, dtype=torch.uint8, device="cuda"))
    assert dspark.dspark_read_device_status(r["workspace"]) == 0 and r["top_ids"].shape == (0, 3)


def test_ties_go_to_the_lowest_id():
    V = 2048
    Z = torch.zeros(3, V, dtype=BF16, device="cuda")
    Z[1, ::3] = 1.0
    Z[2, 5] = -0.0
    Z[2, 1500:1540] = 2.0
    run(Z, torch.tensor([3, 0, 1501], dtype=torch.int32, device="cuda"), 1.0, 32)


@pytest.mark.parametrize("V", [16384, 40000, 262144])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_alternatives_of_long_rows(V, dtype):
    Z = logits((9, V), dtype, seed=V)
    Z[0] = 0.0                              # all tie
    Z[1, : V // 2] = -math.inf              # the frequent half masked
    Z[2] = -math.inf                        # fewer left than wanted
    Z[2, [5, V - 1, V // 3]] = 1.0
    Z[3] = Z[3].flip(0)                     # the best ids at the end
    Z[4] = 1.0                              # a few above many that tie
    Z[4, 7::997] = 2.0
    Z[5] = torch.finfo(dtype).min
    Z[5, V // 2 : V // 2 + 40] = 0.5
    Z[6, ::5] = math.nan
    Z[7, 1000] = math.inf
    tok = torch.tensor([3, V - 2, 5, V - 1, 7, V // 2, 1, 2, 0], dtype=torch.int32, device="cuda")
    for top in (1, 13, 32):
        r = dspark.dspark_logprobs(Z, tok, 1.0, top)
        w = reference(Z, tok, 1.0, top)
        assert torch.equal(r["top_ids"].cpu().long(), w["ids"])
        fine = [0, 1, 2, 3, 4, 8]
        tol = 200 * U + 4 * U * float(Z[fine].float()[Z[fine].isfinite()].abs().max())
        for name, key in (("lse", "lse"), ("logp", "logp"), ("top_logp", "top")):
            close(r[name][fine], w[key][fine], tol, name)
        close(r["lse"][5:6], w["lse"][5:6], tol, "lse over lowest values")
        close(r["entropy"][:6], w["entropy"][:6], 400 * U * (1 + math.log(V)), "entropy")
        assert r["lse"][6:8].isnan().all() and r["lse"][8].isfinite()


def test_masked_ids():
    V = 1024
    for dtype in (F32, BF16):
        Z = logits((6, V), dtype, seed=3)
        Z[0, 100:] = -math.inf
        Z[1, :] = -math.inf
        Z[1, 777] = 1.5                      # one id left: entropy 0
        Z[2, :] = -math.inf                  # none left
        Z[3, ::2] = torch.finfo(dtype).min   # masks of the type's lowest value
        Z[4, :] = torch.finfo(dtype).min
        Z[5, 3] = -math.inf
        tok = torch.tensor([5, 777, 0, 0, 9, 3], dtype=torch.int32, device="cuda")
        r = dspark.dspark_logprobs(Z, tok, 1.0, 8)
        w = reference(Z, tok, 1.0, 8)
        assert torch.equal(r["top_ids"].cpu().long(), w["ids"])
        tol = 200 * U + 4 * U * 20
        for name, key in (("lse", "lse"), ("logp", "logp"), ("top_logp", "top")):
            keep = [0, 1, 2, 5]
            close(r[name][keep], w[key][keep], tol, name)
        # row 2: lse = -inf, and nothing else is defined
        assert r["lse"][2] == -math.inf and r["entropy"][2].isnan() and r["logp"][2].isnan()
        close(r["entropy"][[0, 1, 3, 5]], w["entropy"][[0, 1, 3, 5]], 400 * U * (1 + math.log(V)), "entropy")
        close(r["logp"][3:4], w["logp"][3:4], 4 * U * float(torch.finfo(dtype).max), "a masked token")
        # row 4: a flat distribution, whatever its level
        close(r["logp"][4:5], w["logp"][4:5], 200 * U, "flat")
        close(r["entropy"][4:5], w["entropy"][4:5], 400 * U * (1 + math.log(V)), "flat entropy")


def test_nan_and_infinite_logits():
    V = 512
    Z = logits((4, V), F32, seed=4)
    Z[0, 17] = math.nan
    Z[1, 17] = math.inf
    Z[2, :] = math.nan
    tok = torch.tensor([3, 4, 5, 6], dtype=torch.int32, device="cuda")
    r = dspark.dspark_logprobs(Z, tok, 1.0, 6)
    w = reference(Z, tok, 1.0, 6)
    assert torch.equal(r["top_ids"].cpu().long(), w["ids"])
    for k in ("lse", "logp", "entropy"):
        assert r[k][:3].isnan().all() and r[k][3].isfinite()


def test_strided_rows_out_of_range_tokens_and_streams():
    V = 640
    wide = logits((9, 2 * V), BF16, seed=5)
    tok = torch.arange(9, dtype=torch.int32, device="cuda")
    run(wide[:, V:], tok, 1.0, 4)
    run(wide[::2, :V], tok[:5].contiguous(), 1.0, 4)
    three = logits((3, 4, 2 * V), BF16, seed=6)
    run(three[:, :, :V], torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4), 1.0, 4)
    with pytest.raises(ValueError):
        dspark.dspark_logprobs(three[:, :3, :V], tok.view(3, 3), 1.0)
    tok2 = tok.clone()
    tok2[4] = V
    run(wide[:, :V], tok2, 1.0, 4, status=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = dspark.dspark_logprobs(wide[:, :V], tok, 1.0, 4, stream=s)
    s.synchronize()
    assert torch.equal(r["logp"], dspark.dspark_logprobs(wide[:, :V], tok, 1.0, 4)["logp"])


def test_a_used_workspace_changes_nothing():
    Z = logits((50, 5000), BF16, seed=7)
    tok = torch.randint(-1, 5000, (50,)).int().cuda()
    a = dspark.dspark_logprobs(Z, tok, 1.0, 20)
    ws = torch.randint(0, 255, (a["workspace"].numel(),), dtype=torch.uint8, device="cuda")
    b = dspark.dspark_logprobs(Z, tok, 1.0, 20, workspace=ws)
    for k in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(a[k].nan_to_num(9), b[k].nan_to_num(9)), k


def test_rows_past_32_bit_offsets():
    V, n = 262144, 8300  # 2.18 G logits
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * V * n * 2:
        pytest.skip("not enough free device memory")
    Z = torch.empty(n, V, dtype=BF16, device="cuda")
    Z[-2:] = logits((2, V), BF16, seed=8)
    tok = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    tok[-2:] = torch.tensor([11, V - 1], dtype=torch.int32)
    r = dspark.dspark_logprobs(Z, tok, 1.0, 9)
    w = reference(Z[-2:], tok[-2:], 1.0, 9)
    close(r["logp"][-2:], w["logp"], 200 * U + 4 * U * 40, "logp")
    assert torch.equal(r["top_ids"][-2:].cpu().long(), w["ids"])


def test_refusals():
    Z, tok = logits((4, 1024), BF16), torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        dspark.dspark_logprobs(Z.half(), tok)
    with pytest.raises(TypeError):
        dspark.dspark_logprobs(Z.cpu(), tok)
    with pytest.raises(TypeError):
        dspark.dspark_logprobs(Z, tok.long())
    with pytest.raises(ValueError):
        dspark.dspark_logprobs(Z, tok[:3])
    with pytest.raises(ValueError):
        dspark.dspark_logprobs(Z, tok, 1.0, 3, top_ids=torch.empty(4, 2, dtype=torch.int32, device="cuda"))
    for kw in (dict(top=33), dict(top=-1)):
        with pytest.raises((dspark.DSparkError, RuntimeError)):
            dspark.dspark_logprobs(Z, tok, 1.0, **kw)
    for T in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(dspark.DSparkError):
            dspark.dspark_logprobs(Z, tok, T)
    with pytest.raises(dspark.DSparkError):
        dspark.dspark_logprobs(Z[:, :1020].contiguous(), tok)     # V % 8 != 0
    with pytest.raises(dspark.DSparkError):
        dspark.dspark_logprobs(Z[:, 4:1020], tok)                 # rows off 16 bytes
    with pytest.raises(ValueError):
        dspark.dspark_logprobs(Z, tok, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
