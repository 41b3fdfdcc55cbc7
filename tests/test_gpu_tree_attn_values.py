"""Attention over the paged cache at values that a long context or a broken sequence brings: weights far
below the largest over E4M3 caches, and values without a number that every row sees."""
import math

import pytest
import torch

import shared_routed_expert_b200 as m
from shared_routed_expert_b200 import _lib, build
from tests.serve_util import Paged, attention_ref, mask_tensor, tree_sets
from tests.test_gpu_tree_attn import make_q, run

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


# B sequences of n new tokens, n n_q / n_kv rows of a kv head: up to 16 and up to 32 (warp-level products), more (tiles)
TAILS = [(80, 1, 12, 4, 128, 700), (80, 2, 48, 4, 64, 700), (40, 4, 24, 2, 128, 1400), (40, 30, 24, 2, 64, 1400),
         (80, 2, 8, 2, 256, 700), (80, 5, 8, 2, 256, 700), (40, 12, 8, 2, 256, 1400)]


@pytest.mark.parametrize("bits", [25.3, 23.5, 20.0])
@pytest.mark.parametrize("B,n,n_q,n_kv,d,ctx", TAILS)
def test_small_weights_over_e4m3_caches_count(B, n, n_q, n_kv, d, ctx, bits):
    """One key whose value is 0 outweighs each of the others by 2^bits; theirs are 1, so that the result is
    the others' share. Error allowed: a weight is rounded to fp16 beside a largest one of 2^7 or more, where
    its smallest step is 2^-24: 2^-25 2^-7 of the largest at most, for each key; and what attention_ref
    allows. As many items as blocks, so that few are cut."""
    P = Paged([n] * B, [ctx] * B, n_kv, d, 64, "e4m3", seed=40, k_scale=1.0, v_scale=1.0)
    one = 0x38                                              # 1.0
    P.k.fill_(0)
    P.v.fill_(one)
    for b in range(B):
        pg, sl = P.slots(b, 1)
        P.k[pg, :, sl] = one
        P.v[pg, :, sl] = 0
    q = torch.ones(P.T, n_q * d, dtype=torch.bfloat16, device=DEV)
    scale = bits * math.log(2) / d
    out, lse, st = run(P, q, n_q, scale=scale)
    assert st == _lib.MOE_OK
    ref, rl, to, tl = attention_ref(P, q, n_q, scale=scale)
    assert float(ref.max()) < 0.01 and float(ref.min()) > 0
    keys = ctx + n
    assert float(((out.view(P.T, n_q, d).double() - ref).abs() - to).max()) <= keys * 2.0 ** -32
    assert float(((lse.double() - rl).abs() - tl).max()) <= 0


def milliseconds(f):
    f()
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,ctx,n_q,n_kv,d,tree", [([1] * 64, [4000] * 64, 16, 2, 128, False), ([3] * 40, [3000] * 40, 8, 1, 64, True),
                                                   ([40, 40], [6000, 5000], 24, 2, 128, True), ([300], [4000], 12, 1, 64, False),
                                                   ([30] * 4, [5000] * 4, 8, 2, 256, False), ([60] * 4, [3000] * 4, 8, 2, 256, True)])
def test_a_cached_value_without_a_number_costs_no_second_look(n, ctx, n_q, n_kv, d, tree, kv):
    """A NaN among the cached values, which every row sees: it is in the rows' result, in its dimension alone,
    and the call takes no longer for it (the rows have nothing to be computed again for)."""
    P = Paged(n, ctx, n_kv, d, 64, kv, seed=41)
    sets = [w for a in n for w in tree_sets(a, 15)] if tree else None
    q = make_q(P, n_q)
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    out, lse = torch.empty_like(q), torch.empty(P.T, n_q, device=DEV)
    mask = mask_tensor(sets, 1) if tree else None

    def call():
        m.moe_tree_attention(cache, batch, n_q, q, out, ws, tree_mask=mask, lse=lse)

    clean = milliseconds(call)
    pg, sl = P.slots(0)
    P.v[pg[3], 0, sl[3], 5] = 0x7F if P.f8 else math.nan
    P.v[pg[ctx[0] - 1], 0, sl[ctx[0] - 1], d - 1] = 0x7F if P.f8 else math.nan
    spoiled = milliseconds(call)
    assert m.moe_get_status(ws) == _lib.MOE_OK
    ref, rl, to, tl = attention_ref(P, q, n_q, sets)
    got = out.view(P.T, n_q, d).double()
    assert bool(torch.isnan(ref).any()) and torch.equal(torch.isnan(got), torch.isnan(ref))
    assert float(torch.nan_to_num((got - ref).abs() - to, nan=0.0).max()) <= 0
    assert float(((lse.double() - rl).abs() - tl).max()) <= 0
    over = q.clone()
    m.moe_tree_attention(cache, batch, n_q, over, over, ws, tree_mask=mask)
    assert torch.equal(over.view(torch.int16), out.view(torch.int16))
    assert spoiled < 2 * clean + 0.05, (clean, spoiled)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,ctx,n_q,n_kv,d,tree", [([14, 3], [90, 700], 8, 2, 128, True), ([40, 9], [300, 64], 12, 1, 128, True),
                                                   ([100], [37], 4, 1, 64, False), ([50, 2], [500, 0], 2, 1, 256, True)])
def test_cached_and_unseen_values_without_a_number(n, ctx, n_q, n_kv, d, tree, kv):
    """NaN in a cached value and in a new token's that not every row sees, into a buffer and over the queries:
    each row has NaN in the dimensions of the values it sees, and in no other."""
    P = Paged(n, ctx, n_kv, d, 16, kv, seed=42)
    sets = [w for a in n for w in tree_sets(a, 16)] if tree else None
    pg, sl = P.slots(0)
    nan = 0x7F if P.f8 else math.nan
    P.v[pg[7], 0, sl[7], 5] = nan
    at = ctx[0] + 4
    P.v[pg[at], 0, sl[at], 9] = nan
    q = make_q(P, n_q)
    out, lse, st = run(P, q, n_q, sets)
    assert st == _lib.MOE_OK
    ref, rl, to, tl = attention_ref(P, q, n_q, sets)
    got = out.view(P.T, n_q, d).double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert bool(torch.isnan(ref[:n[0], 0, 5]).all()) and 0 < int(torch.isnan(ref[:n[0], 0, 9]).sum()) < n[0]
    assert float(torch.nan_to_num((got - ref).abs() - to, nan=0.0).max()) <= 0
    assert float(((lse.double() - rl).abs() - tl).max()) <= 0
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    over = q.clone()
    m.moe_tree_attention(cache, batch, n_q, over, over, ws, tree_mask=mask_tensor(sets, 2) if tree else None)
    assert torch.equal(over.view(torch.int16), out.view(torch.int16))


def test_rows_that_are_computed_again_behind_a_long_context():
    """A drafted token's NaN behind 524288 cached keys: the rows that do not see it take the warps that compute
    them again 10 s; the other warps wait for them, and the call ends well. (All cached pages are one
    page; as many sequences as blocks, so that the rows' keys are in one block's share.)"""
    B, n, n_q, d, page, ctx = 150, 32, 4, 256, 256, 524288
    i32 = dict(dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(43)
    k = torch.randn(B + 1, 1, page, d, generator=g, device=DEV).to(torch.bfloat16)
    v = torch.randn(B + 1, 1, page, d, generator=g, device=DEV).to(torch.bfloat16)
    v[1, 0, 5, 3] = math.nan                                # sequence 0, new token 5
    table = torch.zeros(B, ctx // page + 1, **i32)
    table[:, -1] = torch.arange(1, B + 1, **i32)
    cache = m.make_kv_cache(k, v)
    batch = m.make_kv_batch(torch.arange(B + 1, **i32) * n, torch.full((B,), ctx, **i32), table, n)
    q = torch.randn(B * n, n_q * d, generator=g, device=DEV).to(torch.bfloat16)
    out, ws = torch.empty_like(q), m.alloc_tree_attention_workspace(cache, n_q, B * n)
    mask = torch.tensor([[1 << i] for i in range(n)], dtype=torch.int64, device=DEV).repeat(B, 1)
    m.moe_tree_attention(cache, batch, n_q, q, out, ws, tree_mask=mask)       # (a token sees the cached ones and itself)
    assert m.moe_get_status(ws) == _lib.MOE_OK
    got = out.view(B, n, n_q, d).double()
    # each key of the page counts ctx / page times
    K, V = k[0, 0].double(), torch.nan_to_num(v[0, 0].double())
    for b in (0, 1, B - 1):
        for t in (0, 4, 6, n - 1):
            x = q.view(B, n, n_q, d)[b, t].double() @ torch.cat([K, k[b + 1, 0, t:t + 1].double()]).T / math.sqrt(d)
            w = torch.cat([torch.full((page,), ctx / page, device=DEV), torch.ones(1, device=DEV)]).double()
            p = w * torch.exp(x - x.amax(1, keepdim=True))
            p = p / p.sum(1, keepdim=True)
            vals = torch.cat([V, v[b + 1, 0, t:t + 1].double()])
            e = (d + 4) * 2.0 ** -24 / math.sqrt(d) * (q.view(B, n, n_q, d)[b, t].double().abs() @ K.abs().T).amax(1)
            # the roundings of attention_ref, and 2^-24 for each of a lane's additions in a row
            tol = 2.0 ** -8 * (p @ vals).abs() + (2.0 ** -8 + 4 * e + 2.0 ** -18 + (ctx + n) * 2.0 ** -24)[:, None] * (p @ vals.abs())
            assert bool(((got[b, t] - p @ vals).abs() <= tol).all()), (b, t)
    assert bool(torch.isnan(got[0, 5, :, 3]).all()) and int(torch.isnan(got).sum()) == n_q
