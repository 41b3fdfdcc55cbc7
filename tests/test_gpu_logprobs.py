"""Token log probabilities, entropy and alternatives against fp64, exact ids with ties to the lower id."""
import math

import pytest
import torch

import shared_routed_expert_b200 as m
from shared_routed_expert_b200 import build
from tests.serve_util import F32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def run(x, targets, n):
    T = x.shape[0]
    lp, ent = torch.full((T,), 7.0, device=DEV), torch.full((T,), 7.0, device=DEV)
    ids = torch.full((T, n), -5, dtype=torch.int32, device=DEV) if n else None
    top = torch.full((T, n), 7.0, device=DEV) if n else None
    m.moe_token_logprobs(x, targets, lp, ent, ids, top)
    torch.cuda.synchronize()
    return lp, ent, ids, top


def check(x, targets, n, got):
    """fp64 references. Errors allowed: M - x is a rounded fp32 difference and its base-2 exponent d another
    rounding (2 * 2^-24 |d| of a term, |d| < 24 where a term matters beside the largest), exp2 is good to
    2^-22, a term of t has two roundings more; sums of positive terms lose 2^-24 per addition in a row (at
    most 32 in a group, V / 8192 groups of a thread, 9 levels of warps and blocks: under 75 for V up to
    2^18). In all (48 + 4 + 2 + 75) 2^-24 < 2^-16.9 of l and t: relative 2^-16."""
    lp, ent, ids, top = got
    d = x.double()
    M = d.amax(1, keepdim=True)
    e = torch.exp(d - M)
    z = e.sum(1, keepdim=True)
    first = torch.zeros_like(d).scatter_(1, d.argmax(1, keepdim=True), 1.0)
    l = (e * (1 - first)).sum(1)                             # without the largest term: keeps relative accuracy
    ln1 = torch.log1p(l)
    t = torch.where(e > 0, e * (M - d), torch.zeros_like(e)).sum(1)
    want_ent = ln1 + t / z[:, 0]
    rel = 2.0 ** -16
    assert float(((ent.double() - want_ent).abs() - rel * want_ent - 1e-37).max()) <= 0
    ok = (targets >= 0) & (targets < x.shape[1])
    xt = d.gather(1, targets.long().clamp(0, x.shape[1] - 1)[:, None])[:, 0]
    want = torch.where(ok, xt - M[:, 0] - ln1, torch.full_like(xt, math.nan))
    assert torch.equal(torch.isnan(lp), torch.isnan(want))
    fin = torch.isfinite(want)
    assert torch.equal(lp.double()[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)])
    tol = 4 * F32 * (xt - M[:, 0]).abs() + rel * ln1
    assert float(((lp.double() - want).abs() - tol)[fin].max()) <= 0 if bool(fin.any()) else True
    if n:
        f = (x.float() + 0.0).view(torch.int32).long()
        f = torch.where(f < 0, -(f & 0x7FFFFFFF), f)
        key = f * (1 << 32) + (x.shape[1] - 1 - torch.arange(x.shape[1], device=DEV))
        want_ids = torch.topk(key, n, dim=1).indices
        assert torch.equal(ids.long(), want_ids)
        dd = d.gather(1, want_ids) - M
        w = dd - ln1[:, None]
        fin = torch.isfinite(w)
        assert torch.equal(torch.isfinite(top), fin)
        assert float((((top.double() - w).abs() - 4 * F32 * dd.abs() - rel * ln1[:, None])[fin]).max()) <= 0


CASES = [(1, 1, 1), (1, 7, 7), (3, 33, 32), (2, 1000, 5), (5, 4096, 1), (1, 131072, 20), (300, 5003, 8), (33, 65537, 32),
         (1, 200003, 32), (7, 100003, 0), (150, 20000, 3)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,n", CASES)
def test_matches_fp64(T, V, n, dt):
    g = torch.Generator(device=DEV)
    g.manual_seed(T * 1000 + V)
    x = torch.randn(T, V, generator=g, device=DEV) * 3
    x = x.to(torch.bfloat16) if dt == "bf16" else x
    targets = torch.randint(0, V, (T,), generator=g, device=DEV).int()
    check(x, targets, n, run(x, targets, n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_peaked_rows_keep_their_relative_accuracy(dt):
    x = torch.randn(64, 30000, device=DEV)
    peak = torch.randint(0, 30000, (64,), device=DEV)
    x[torch.arange(64, device=DEV), peak] = torch.linspace(5, 60, 64, device=DEV)
    x = x.to(torch.bfloat16) if dt == "bf16" else x
    got = run(x, peak.int(), 4)
    check(x, peak.int(), 4, got)
    assert float(got[1].max()) > 1 and 0 < float(got[1].min()) < 1e-15


@pytest.mark.parametrize("off,stride", [(0, 50001), (1, 50001), (3, 50008), (7, 60013)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_at_any_alignment(off, stride, dt):
    V, T = 50001, 6
    buf = torch.randn(T * stride + 16, device=DEV)
    buf = buf.to(torch.bfloat16) if dt == "bf16" else buf
    x = buf.as_strided((T, V), (stride, 1), off)
    targets = torch.randint(0, V, (T,), device=DEV).int()
    check(x, targets, 10, run(x, targets, 10))


@pytest.mark.parametrize("T,V", [(2, 100), (1, 150000), (200, 9000)])
def test_ties_go_to_the_lower_id(T, V):
    x = torch.zeros(T, V, device=DEV)
    t = torch.zeros(T, dtype=torch.int32, device=DEV)
    check(x, t, 32, run(x, t, 32))                          # nothing but ties
    x = (torch.randint(0, 5, (T, V), device=DEV).float() - 2) * 0.5   # many ties, zeros of both signs
    x = torch.where((x == 0) & (torch.rand_like(x) < 0.5), -x, x).to(torch.bfloat16)
    check(x, t, 32, run(x, t, 32))
    x = torch.full((T, V), -3.0, device=DEV)
    x[:, V // 2] = 1.0
    check(x, t, 3, run(x, t, 3))
    x = torch.arange(V, device=DEV).float().expand(T, V).contiguous()   # ascending
    check(x, t, 32, run(x, t, 32))


def test_infinities_nan_and_targets_outside():
    V = 40000
    x = torch.randn(9, V, device=DEV)
    x[0, 5:] = -math.inf                                    # five tokens possible
    x[1] = -math.inf                                        # none
    x[2, 777] = math.nan
    x[3, 31000] = math.inf
    x[4, 100:] = -math.inf
    x[4, 200] = math.nan
    x[4, 39999] = math.nan
    x[6] = -math.inf
    x[6, 12345] = 2.0                                       # one
    t = torch.tensor([3, 0, 0, 0, 0, -1, 12345, V, 0], dtype=torch.int32, device=DEV)
    lp, ent, ids, top = run(x, t, 8)
    good = [0, 5, 6, 7, 8]
    check(x[good], t[good], 5, (lp[good], ent[good], ids[good][:, :5], top[good][:, :5]))
    for r in (1, 2, 3, 4):
        assert math.isnan(lp[r]) and math.isnan(ent[r]) and bool(torch.isnan(top[r]).all())
    assert ids[0, 5:].tolist() == [5, 6, 7] and bool((top[0, 5:] == -math.inf).all())
    assert ids[1].tolist() == list(range(8))
    assert int(ids[2, 0]) == 777 and int(ids[3, 0]) == 31000 and ids[4, :2].tolist() == [200, 39999]
    assert float(lp[6]) == 0 and float(ent[6]) == 0
    x = torch.randn(3, V, device=DEV)
    lp, _, _, _ = run(x, torch.tensor([3, -100, 4], dtype=torch.int32, device=DEV), 0)
    assert torch.isnan(lp).tolist() == [False, True, False]


def test_only_alternatives_and_only_entropy():
    x = torch.randn(4, 9999, device=DEV)
    ids, top = torch.empty(4, 3, dtype=torch.int32, device=DEV), torch.empty(4, 3, device=DEV)
    ent = torch.empty(4, device=DEV)
    m.moe_token_logprobs(x, None, None, None, ids, top)
    m.moe_token_logprobs(x, None, None, ent)
    t = torch.zeros(4, dtype=torch.int32, device=DEV)
    lp, ent2, ids2, top2 = run(x, t, 3)
    assert torch.equal(ids, ids2) and torch.equal(top, top2) and torch.equal(ent, ent2)


def test_offsets_past_32_bits():
    V, T = 1000, 3
    stride = 1 << 31
    buf = torch.zeros(2 * stride + V, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((T, V), (stride, 1))
    x.copy_(torch.randn(T, V, device=DEV))
    t = torch.tensor([5, 6, 999], dtype=torch.int32, device=DEV)
    check(x.contiguous(), t, 4, run(x, t, 4))


def test_graph_replay_and_repeat_bit_for_bit():
    x = torch.randn(5, 131072, device=DEV).to(torch.bfloat16)
    t = torch.arange(5, dtype=torch.int32, device=DEV)
    lp, ent = torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    ids, top = torch.empty(5, 20, dtype=torch.int32, device=DEV), torch.empty(5, 20, device=DEV)
    m.moe_token_logprobs(x, t, lp, ent, ids, top)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_token_logprobs(x, t, lp, ent, ids, top)
    x.copy_(torch.randn(5, 131072, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    check(x, t, 20, (lp, ent, ids, top))
    a = run(x, t, 20)
    for u, v in zip(a, (lp, ent, ids, top)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,n", [(12, 32003, 32), (160, 16385, 1), (222, 17011, 5), (9, 8193, 1), (1, 4097, 7)])
def test_rows_over_several_blocks(T, V, n, dt):
    """Slices down to 4096 elements, and the single alternative."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T + V)
    x = (torch.randn(T, V, generator=g, device=DEV) * 3).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    targets = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    check(x, targets, n, run(x, targets, n))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hidden", ["lowest", -1e38, -1e34, -1e30, -3e4])
@pytest.mark.parametrize("T,V,n", [(16, 40000, 8), (300, 5003, 3), (8, 131072, 20), (16, 100, 0)])
def test_rows_masked_with_large_negative_numbers(T, V, n, hidden, dt):
    """Masks that are numbers: whole threads, slices and groups hold nothing else, in front of the tokens that
    are left, behind them, or on both sides. (A masked token's term is below 2^-1000, its logarithm's error as
    everywhere: the tolerances of `check`, where only terms with |d| < 24 count.)"""
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator(device=DEV)
    g.manual_seed(V)
    x = (torch.randn(T, V, generator=g, device=DEV) * 3).to(t)
    low = torch.finfo(t).min if hidden == "lowest" else hidden
    i = torch.arange(V, device=DEV)
    keep = [i < 5, i >= V - 5, i == V // 2, (i > V // 3) & (i < V // 3 + 1000), i % 97 == 3, i < V // 2, i >= V // 2, i < 0]
    for r in range(T):
        x[r, ~keep[r % 8]] = low
    if hidden == "lowest":
        x[0, ~keep[0]] = 0.45 * low                         # a difference that overflows in base 2 alone
        x[0, V - 1] = -0.45 * low
    targets = torch.randint(0, V, (T,), generator=g, device=DEV).int()
    targets[::2] = x[::2].argmax(1).int()
    check(x, targets, n, run(x, targets, n))
