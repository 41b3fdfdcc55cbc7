"""Attention over the paged cache against fp64: head layouts, cache types and layouts, chains and
trees, lengths from zero, rows that see nothing, and infinities and NaN where a row does not look."""
import math

import pytest
import torch

from shared_routed_expert_b200 import _lib, build
import shared_routed_expert_b200 as m
from tests.serve_util import Paged, attention_ref, mask_tensor, tree_sets

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def make_q(P, n_q, seed=1, std=2.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(P.T, n_q * P.d, generator=g, device=DEV) * std).to(torch.bfloat16)


def run(P, q, n_q, sets=None, words=None, scale=None, lse=True, max_new=None):
    cache, batch = P.handles(m, max_new)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    out = torch.full((P.T, n_q * P.d), 7.5, dtype=torch.bfloat16, device=DEV)
    l = torch.full((P.T, n_q), 7.5, device=DEV) if lse else None
    mask = None
    if sets is not None:
        words = words or max(1, -(-max(P.n) // 64))
        full = sets + [0] * (P.T - len(sets))
        mask = mask_tensor(full, words)
    m.moe_tree_attention(cache, batch, n_q, q, out, ws, tree_mask=mask, lse=l, scale=scale)
    return out, l, m.moe_get_status(ws)


def check(P, q, n_q, out, lse, sets=None, scale=None, hide=None):
    ref, rl, to, tl = attention_ref(P, q, n_q, sets, scale, hide)
    T = P.starts[-1]
    got = out.view(P.T, n_q, P.d).double()
    assert torch.equal(torch.isnan(got[:T]), torch.isnan(ref[:T]))
    err = torch.nan_to_num((got[:T] - ref[:T]).abs() - to[:T], nan=0.0)
    assert float(err.max()) <= 0, float(err.max())
    if lse is not None:
        assert torch.equal(torch.isinf(lse[:T]), torch.isinf(rl[:T]))
        e = torch.where(torch.isinf(rl[:T]), torch.zeros_like(rl[:T]), (lse[:T].double() - rl[:T]).abs() - tl[:T])
        assert float(e.max()) <= 0, float(e.max())
    # rows behind the last sequence are left as they were
    assert bool((out[T:] == 7.5).all())
    if lse is not None:
        assert bool((lse[T:] == 7.5).all())


SHAPES = [
    # n, ctx, n_q, n_kv, d, page, layout
    ([1], [0], 1, 1, 64, 16, "hnd"),                       # one token, nothing cached
    ([1], [1], 12, 1, 128, 16, "hnd"),
    ([1, 1, 1, 1], [15, 16, 17, 300], 8, 2, 128, 16, "nhd"),
    ([1, 1, 1], [127, 128, 511], 96, 8, 128, 64, "hnd"),
    ([1], [5000], 12, 1, 128, 64, "hnd"),                  # one long context, split over the SMs
    ([4, 3, 1, 0, 2], [31, 0, 200, 50, 1000], 10, 5, 64, 32, "interleaved"),
    ([5, 2], [77, 640], 16, 1, 256, 64, "hnd"),
    ([1, 7], [2000, 33], 4, 4, 256, 128, "nhd"),           # no sharing of heads
    ([33, 65, 1], [100, 0, 63], 12, 1, 128, 16, "nhd"),
    ([130], [250], 8, 2, 64, 256, "hnd"),
    ([257, 19], [0, 513], 24, 2, 128, 64, "hnd"),
    ([300], [77], 2, 1, 256, 32, "interleaved"),
    ([700, 1, 40], [1111, 900, 0], 16, 2, 128, 128, "hnd"),
    ([1, 2, 1], [700, 0, 255], 12, 1, 128, 256, "hnd"),    # pages longer than a chunk of keys
    ([3], [100], 12, 1, 64, 16, "hnd"),                    # 36 rows: both halves of a tile on the same rows
    ([10, 11, 22], [5, 64, 200], 12, 1, 128, 32, "hnd"),   # 120, 132 and 264 rows
    ([2, 1], [4000, 130], 1024, 16, 64, 64, "hnd"),        # 64 query heads to a kv head
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"n{s[0][0]}_c{s[1][0]}_q{s[2]}_k{s[3]}_d{s[4]}_p{s[5]}_{s[6]}" for s in SHAPES])
def test_chain_matches_fp64(shape, kv):
    n, ctx, n_q, n_kv, d, page, layout = shape
    P = Paged(n, ctx, n_kv, d, page, kv, layout, seed=3, rows=sum(n) + 3)
    q = make_q(P, n_q)
    out, lse, st = run(P, q, n_q)
    assert st == _lib.MOE_OK
    check(P, q, n_q, out, lse)


TREES = [
    ([5], [40], 12, 1, 128, 16, 1),
    ([61, 17, 1, 64], [200, 0, 64, 127], 24, 2, 128, 64, 1),
    ([100, 3], [300, 5], 8, 2, 64, 32, 2),
    ([150], [33], 4, 1, 256, 64, 5),                       # more words than nodes need
    ([12, 9, 30], [1500, 17, 0], 96, 8, 128, 64, 1),
    ([200], [900], 12, 1, 128, 256, 4),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", TREES, ids=[f"n{s[0][0]}_c{s[1][0]}_q{s[2]}_d{s[4]}" for s in TREES])
def test_tree_matches_fp64(shape, kv):
    n, ctx, n_q, n_kv, d, page, words = shape
    P = Paged(n, ctx, n_kv, d, page, kv, "hnd", seed=4, rows=sum(n) + 2)
    sets = [w for b, a in enumerate(n) for w in tree_sets(a, 50 + b)]
    q = make_q(P, n_q)
    out, lse, st = run(P, q, n_q, sets, words)
    assert st == _lib.MOE_OK
    check(P, q, n_q, out, lse, sets)


@pytest.mark.parametrize("n_q,n_kv", [(4, 2), (96, 8)])
def test_rows_that_see_nothing_and_bits_behind_the_tree(n_q, n_kv):
    """Empty masks without a cached prefix give zeros and -infinity; bits of nodes the sequence
    does not have are ignored."""
    P = Paged([6, 9, 20], [0, 0, 3], n_kv, 128, 16, "bf16", seed=5)
    sets = tree_sets(6, 1) + tree_sets(9, 2) + tree_sets(20, 3)
    sets[2] = 0
    sets[7] = 0
    sets[8] = 1 << 30 | 1 << 63                            # only nodes that do not exist
    sets[20] = 0                                           # sees the prefix only
    q = make_q(P, n_q)
    out, lse, st = run(P, q, n_q, sets, 1)
    assert st == _lib.MOE_OK
    for r in (2, 7, 8):
        assert bool((out[r] == 0).all()) and bool((lse[r] == -math.inf).all())
    n = [6, 9, 20]
    cut = [w & ((1 << n[b]) - 1) for b in range(3) for w in sets[P.starts[b]:P.starts[b + 1]]]
    check(P, q, n_q, out, lse, cut)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_q,n_kv,d,n", [(8, 2, 128, 14), (12, 1, 128, 40), (4, 1, 64, 100), (2, 1, 256, 50)])
def test_what_a_row_does_not_see_does_not_reach_it(n_q, n_kv, d, n, kv):
    """A drafted node whose value (and key) holds NaN or infinity spoils the rows that see it
    and no other."""
    P = Paged([n, 3], [70, 20], n_kv, d, 16, kv, seed=6)
    sets = tree_sets(n, 9) + tree_sets(3, 10)
    pg, sl = P.slots(0)
    node = 70 + 5
    if kv == "e4m3":
        P.v[pg[node], 0, sl[node], 3] = 0x7F
    else:
        P.v[pg[node], 0, sl[node], 3] = math.inf
        P.v[pg[node], 0, sl[node], 4] = math.nan
    q = make_q(P, n_q)
    out, lse, st = run(P, q, n_q, sets)
    ref, rl, to, tl = attention_ref(P, q, n_q, sets)
    got = out.view(P.T, n_q, d).double()
    G = n_q // n_kv
    sees = torch.tensor([w >> 5 & 1 for w in sets[:n]] + [0, 0, 0], dtype=torch.bool, device=DEV)
    assert bool(sees.any()) and not bool(sees[:n].all())
    clean = ~sees
    assert bool(torch.isfinite(got[clean]).all())
    err = (got - ref).abs() - to
    assert float(err[clean].max()) <= 0
    assert not bool(torch.isfinite(got[sees][:, :G, 3]).any())
    assert bool(torch.isfinite(got[sees][:, :, 10]).all())          # other columns of those rows stay
    # a NaN key spoils the rows that see it, and only those
    P.k[pg[node], 0, sl[node], 1] = 0x7F if kv == "e4m3" else math.nan
    out, lse, st = run(P, q, n_q, sets)
    got = out.view(P.T, n_q, d).double()
    assert bool(torch.isnan(got[sees][:, :G]).all()) and bool(torch.isfinite(got[clean]).all())
    err = (got - ref).abs() - to
    assert float(err[clean].max()) <= 0


@pytest.mark.parametrize("n,n_q", [(3, 8), (90, 8)])
def test_later_tokens_of_a_chain_do_not_reach_earlier_ones(n, n_q):
    P = Paged([n], [45], 1, 128, 32, "bf16", seed=16)
    pg, sl = P.slots(0)
    at = 45 + n - 2
    P.v[pg[at], 0, sl[at], 7] = math.nan
    q = make_q(P, n_q)
    out, lse, st = run(P, q, n_q)
    ref, rl, to, tl = attention_ref(P, q, n_q)
    got = out.view(n, n_q, 128).double()
    assert float(((got - ref).abs() - to)[:n - 2].max()) <= 0
    assert bool(torch.isnan(got[n - 2:, :, 7]).all())


def test_extreme_scores():
    """Scores of thousands, all scores equal, scores of -infinity, negative and zero scales."""
    P = Paged([3, 2], [400, 9], 2, 128, 16, "bf16", seed=7)
    q = make_q(P, 8, std=200.0)
    out, lse, _ = run(P, q, 8)
    check(P, q, 8, out, lse)
    for scale in (0.0, -0.25):
        q = make_q(P, 8)
        out, lse, _ = run(P, q, 8, scale=scale)
        check(P, q, 8, out, lse, scale=scale)
    P.k.fill_(0)
    pg, sl = P.slots(1)
    P.k[pg, :, sl, 0] = -math.inf                          # every score of sequence 1 is -infinity
    q = q.abs()
    out, lse, _ = run(P, q, 8)
    assert bool((out[3:] == 0).all()) and bool((lse[3:] == -math.inf).all())
    assert bool(torch.isfinite(lse[:3]).all())


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_count_as_not_seen_and_are_reported(n):
    P = Paged([n, n], [100, 60], 1, 128, 16, "bf16", seed=8)
    P.table[0, 2] = P.pages
    P.table[0, 4] = -1
    q = make_q(P, 8)
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, 8, P.T)
    out, lse = torch.empty(P.T, 8 * 128, dtype=torch.bfloat16, device=DEV), torch.empty(P.T, 8, device=DEV)
    m.moe_tree_attention(cache, batch, 8, q, out, ws, lse=lse)
    assert m.moe_get_status(ws) == _lib.MOE_ERR_DEVICE
    assert m.moe_get_status(ws) == _lib.MOE_OK             # reading clears it
    i0, i1 = torch.arange(100 + n, device=DEV), torch.arange(60 + n, device=DEV)
    hide = [(i0 // 16 == 2) | (i0 // 16 == 4), i1 < 0]
    P.table[0, 2] = P.table[0, 4] = 0                      # (any page: hidden in the reference)
    check(P, q, 8, out, lse, hide=hide)


@pytest.mark.parametrize("n", [2, 30])
def test_bad_lengths_leave_a_sequence_alone(n):
    n_q = 8
    for what in ("ctx negative", "ctx too long", "too many rows", "rows outside"):
        P = Paged([n, n], [40, 33], 1, 128, 16, "bf16", seed=9)
        max_new = n
        if what == "ctx negative":
            P.ctx_len[1] = -1
        elif what == "ctx too long":
            P.ctx_len[1] = 16 * P.width - n + 1
        elif what == "too many rows":
            P.q_start[1] = n - 1                           # sequence 1 has n + 1 rows
            P.n[0] = n - 1
            P.starts[1] = n - 1
        else:
            P.q_start[2] = P.T + 1
            max_new = n + 1
        q = make_q(P, n_q)
        out, lse, st = run(P, q, n_q, max_new=max_new)
        assert st == _lib.MOE_ERR_DEVICE, what
        r, P.n[1] = P.starts[1], 0
        assert bool((out[r:] == 7.5).all()) and bool((lse[r:] == 7.5).all()), what
        ref, rl, to, tl = attention_ref(P, q, n_q)
        assert float(((out.view(P.T, n_q, 128).double() - ref).abs() - to)[:r].max()) <= 0


def test_strided_rows_and_no_lse():
    P = Paged([5, 33], [64, 10], 2, 64, 16, "bf16", seed=11)
    n_q = 6
    wide = torch.randn(P.T, (n_q + 4) * 64, device=DEV).to(torch.bfloat16)
    q = wide[:, :n_q * 64]                                 # the q heads of a fused qkv row
    outw = torch.full((P.T, n_q * 64 + 24), 3.0, dtype=torch.bfloat16, device=DEV)
    out = outw[:, 8:8 + n_q * 64]
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    m.moe_tree_attention(cache, batch, n_q, q, out, ws)
    check(P, q.contiguous(), n_q, out.contiguous(), None)
    assert bool((outw[:, :8] == 3).all()) and bool((outw[:, 8 + n_q * 64:] == 3).all())


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kv):
    """Pages more than 2^32 bytes (and 2^31 elements) apart."""
    stride = (1 << 31) + 4096 if kv == "bf16" else (1 << 32) + 4096
    d, page = 128, 16
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    big = torch.zeros(2 * stride + 8192, dtype=dt, device=DEV)
    k = big.as_strided((3, 1, page, d), (stride, page * d, d, 1), 0)
    v = big.as_strided((3, 1, page, d), (stride, page * d, d, 1), page * d)
    P2 = Paged([2, 30], [5, 0], 1, d, page, kv, seed=12)
    # three pages: sequence 0 in the last one, sequence 1 over the others
    P2.table = torch.tensor([[2, -1], [1, 0]], dtype=torch.int32, device=DEV)
    P2.pages = 3
    src = torch.randn(3, 1, page, d, device=DEV)
    conv = (lambda x: (x / 0.05).to(torch.float8_e4m3fn).view(torch.uint8)) if kv == "e4m3" else (lambda x: x.to(dt))
    k.copy_(conv(src))
    v.copy_(conv(src.flip(3)))
    P2.k, P2.v = k, v
    q = make_q(P2, 8)
    out, lse, st = run(P2, q, 8)
    assert st == _lib.MOE_OK
    check(P2, q, 8, out, lse)
    del big, k, v


@pytest.mark.parametrize("shape", [([1] * 8, [900] * 8, 96, 8), ([48, 20], [600, 50], 12, 1)])
def test_runs_repeat_bit_for_bit(shape):
    n, ctx, n_q, n_kv = shape
    P = Paged(n, ctx, n_kv, 128, 64, "bf16", seed=13)
    q = make_q(P, n_q)
    a, la, _ = run(P, q, n_q)
    b, lb, _ = run(P, q, n_q)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


@pytest.mark.parametrize("n", [1, 24])
def test_graph_replays_read_lengths_and_pages_of_the_time(n):
    """A captured call, replayed after the sequences have grown and changed pages; two graphs
    share one workspace."""
    n_q = 12
    P = Paged([n] * 3, [300, 120, 250], 1, 128, 16, "bf16", seed=14, extra_pages=20)
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    q = make_q(P, n_q)
    outs = [torch.full((P.T, n_q * 128), 7.5, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    lses = [torch.full((P.T, n_q), 7.5, device=DEV) for _ in range(2)]
    m.moe_tree_attention(cache, batch, n_q, q, outs[0], ws, lse=lses[0])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_tree_attention(cache, batch, n_q, q, outs[i], ws, lse=lses[i])
        graphs.append(g)
    for ctx in ([300, 120, 250], [17, 120, 0], [1, 300 - n, 64]):
        P.ctx = ctx
        P.ctx_len.copy_(torch.tensor(ctx, dtype=torch.int32))
        if ctx[1] > 120:                                    # sequence 1 grows into sequence 0's old pages
            P.table[1, :300 // 16 + 2] = P.table[0, :300 // 16 + 2]
        for i in range(2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            check(P, q, n_q, outs[i], lses[i])
    assert m.moe_get_status(ws) == _lib.MOE_OK


def test_other_stream_and_two_workspaces_at_once():
    P = Paged([1] * 16, [777] * 16, 2, 128, 64, "bf16", seed=15)
    n_q = 16
    q = make_q(P, n_q)
    cache, batch = P.handles(m)
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    torch.cuda.synchronize()
    for s in streams:
        ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
        out = torch.full((P.T, n_q * 128), 7.5, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((P.T, n_q), 7.5, device=DEV)
        res.append((ws, out, lse))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (ws, out, lse) in zip(streams, res):
            m.moe_tree_attention(cache, batch, n_q, q, out, ws, lse=lse, stream=s)
    torch.cuda.synchronize()
    for ws, out, lse in res:
        check(P, q, n_q, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_of", [lambda b: (b * 7) % 3, lambda b: 1 + (b * 5) % 40])
def test_more_sequences_than_threads(n_of, kv):
    """700 sequences (several to a thread of the kernels' scan), empty ones among them."""
    n = [n_of(b) for b in range(700)]
    ctx = [(b * 37) % 90 for b in range(700)]
    P = Paged(n, ctx, 1, 64, 16, kv, seed=21, rows=sum(n) + 1)
    q = make_q(P, 2)
    out, lse, st = run(P, q, 2)
    assert st == _lib.MOE_OK
    check(P, q, 2, out, lse)


def test_one_workspace_serves_every_kind_of_call():
    """Decoding, drafts and chunks in turn on one workspace, at several head widths."""
    ws = None
    for rounds in range(2):
        for n, ctx, n_q, n_kv, d, kv in (([1, 1], [3000, 50], 12, 1, 128, "bf16"), ([40, 3], [700, 0], 12, 1, 128, "e4m3"),
                                         ([2], [5000], 8, 1, 256, "bf16"), ([1], [900], 8, 2, 64, "e4m3"),
                                         ([300], [600], 12, 1, 128, "bf16"), ([30], [2000], 4, 2, 256, "e4m3")):
            P = Paged(n, ctx, n_kv, d, 64, kv, seed=22 + rounds)
            cache, batch = P.handles(m)
            if ws is None:
                wide = Paged([1], [1], 1, 256, 16, "bf16").handles(m)[0]
                ws = m.alloc_tree_attention_workspace(wide, 4, 512)
            q = make_q(P, n_q)
            out, lse = torch.full_like(q, 7.5), torch.full((P.T, n_q), 7.5, device=DEV)
            m.moe_tree_attention(cache, batch, n_q, q, out, ws, lse=lse)
            assert m.moe_get_status(ws) == _lib.MOE_OK
            check(P, q, n_q, out, lse)


@pytest.mark.parametrize("n,ctx", [([1] * 5, [3000] * 5), ([50, 9], [1500, 70])])
def test_output_over_the_queries(n, ctx):
    P = Paged(n, ctx, 1, 128, 64, "bf16", seed=24)
    q = make_q(P, 12)
    out, lse, _ = run(P, q, 12)
    q2 = q.clone()
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, 12, P.T)
    m.moe_tree_attention(cache, batch, 12, q2, q2, ws)
    assert torch.equal(q2.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,n_q,d", [(14, 1, 128), (40, 12, 128), (12, 8, 64), (40, 1, 256)])
def test_output_over_the_queries_beside_values_without_a_number(n, n_q, d, kv):
    """In place: rows that are computed again because a value they do not see holds NaN still find
    their queries."""
    P = Paged([n], [30], 1, d, 16, kv, seed=26)
    sets = tree_sets(n, 11)
    pg, sl = P.slots(0)
    P.v[pg[30 + 2], 0, sl[30 + 2], d - 1] = 0x7F if kv == "e4m3" else math.nan
    q = make_q(P, n_q)
    mask = mask_tensor(sets, 1)
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    got = q.clone()
    m.moe_tree_attention(cache, batch, n_q, got, got, ws, tree_mask=mask)
    ref, _, to, _ = attention_ref(P, q, n_q, sets)
    clean = torch.tensor([not w >> 2 & 1 for w in sets], dtype=torch.bool, device=DEV)
    assert bool(clean[3:].any()) and not bool(clean.all())
    err = (got.view(P.T, n_q, d).double() - ref).abs() - to
    assert float(err[clean].max()) <= 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,ctx,n_q,n_kv,page", [([600, 33], [1700, 0], 4, 1, 16), ([9, 9, 1], [3000, 129, 640], 16, 2, 64),
                                                 ([257, 64], [127, 128], 2, 2, 256), ([40], [1], 12, 12, 32)])
def test_many_rows_of_wide_heads(n, ctx, n_q, n_kv, page, kv):
    """Heads of 256 dimensions: several tiles, cut items, scores whose maximum keeps rising (keys that
    grow along the sequence, so that sums are rescaled), chains and trees."""
    P = Paged(n, ctx, n_kv, 256, page, kv, seed=27, rows=sum(n) + 2)
    q = make_q(P, n_q, std=0.7)
    for b in range(len(n)):
        pg, sl = P.slots(b)
        i = torch.arange(ctx[b] + n[b], device=DEV)
        ramp = ((i // 100 + 1).float() * 4).clamp(max=64)
        for h in range(n_kv):                              # one dimension rises by steps
            row = ramp if not P.f8 else ramp.to(torch.float8_e4m3fn).view(torch.uint8)
            P.k[pg, h, sl, 5] = row.to(P.k.dtype) if not P.f8 else row
    q.view(P.T, n_q, 256)[:, :, 5] = q.view(P.T, n_q, 256)[:, :, 5].abs() + 1
    for sets in (None, [w for a in n for w in tree_sets(a, 12)] if max(n) <= 300 else None):
        out, lse, st = run(P, q, n_q, sets)
        assert st == _lib.MOE_OK
        check(P, q, n_q, out, lse, sets)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_extreme_scores_bad_pages_and_waits_of_wide_heads(kv):
    n_q = 4
    P = Paged([40, 12], [400, 9], 1, 256, 16, kv, seed=28)
    q = make_q(P, n_q, std=60.0)
    out, lse, _ = run(P, q, n_q)
    check(P, q, n_q, out, lse)
    for scale in (0.0, -0.125):
        q = make_q(P, n_q)
        out, lse, _ = run(P, q, n_q, scale=scale)
        check(P, q, n_q, out, lse, scale=scale)
    sets = [0] * 20 + tree_sets(40, 13)[20:] + tree_sets(12, 14)     # rows that see the prefix alone
    out, lse, _ = run(P, q, n_q, sets)
    check(P, q, n_q, out, lse, sets)
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, n_q, P.T)
    _lib.moe_inject_attention_timeout(1)
    m.moe_tree_attention(cache, batch, n_q, q, out, ws, lse=lse)
    assert m.moe_get_status(ws) == _lib.MOE_ERR_TIMEOUT
    ws.zero_()
    P.table[0, 3] = P.pages
    m.moe_tree_attention(cache, batch, n_q, q, out, ws, lse=lse)
    assert m.moe_get_status(ws) == _lib.MOE_ERR_DEVICE
    i0, i1 = torch.arange(440, device=DEV), torch.arange(21, device=DEV)
    P.table[0, 3] = 0                                      # (any page: hidden in the reference)
    ref, _, to, _ = attention_ref(P, q, n_q, None, None, [i0 // 16 == 3, i1 < 0])
    assert float(((out.view(P.T, n_q, 256).double() - ref).abs() - to).max()) <= 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,d", [(1, 128), (3, 256), (30, 128), (5, 64)])
def test_waits_that_run_out_are_reported(n, d, kv):
    """Loads that never come: the bounded waits run out, the kernels return and say so, and a
    zeroed workspace works again."""
    P = Paged([n, n], [900, 40], 1, d, 16, kv, seed=25)
    q = make_q(P, 12)
    cache, batch = P.handles(m)
    ws = m.alloc_tree_attention_workspace(cache, 12, P.T)
    out, lse = torch.empty_like(q), torch.empty(P.T, 12, device=DEV)
    _lib.moe_inject_attention_timeout(1)
    m.moe_tree_attention(cache, batch, 12, q, out, ws, lse=lse)
    assert m.moe_get_status(ws) == _lib.MOE_ERR_TIMEOUT
    ws.zero_()
    m.moe_tree_attention(cache, batch, 12, q, out, ws, lse=lse)
    assert m.moe_get_status(ws) == _lib.MOE_OK
    check(P, q, 12, out, lse)
