"""The append to the paged cache, the move of accepted drafts inside it, and a speculative decoding
step made of append, attention, log probabilities and move."""
import dataclasses
import math

import numpy as np
import pytest
import torch

import oracle
import shared_routed_expert_b200 as m
from shared_routed_expert_b200 import _lib, build, synth
from tests.serve_util import F32, HALF_BF16, HALF_E4M3, Paged, mask_tensor, tree_sets

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def attn_inputs(T, n_q, n_kv, d, rot, max_pos, seed):
    cfg = synth.AttnConfig("t", T=T, n_q=n_q, n_kv=n_kv, d=d, rot=rot, max_pos=max_pos, seed=seed, sequential=False)
    return cfg, synth.make_attn_inputs(cfg, DEV)


APPEND = [
    # n, ctx, n_q, n_kv, d, rot, page, layout
    ([1], [0], 1, 1, 64, 32, 16, "hnd"),
    ([1, 1, 1], [15, 16, 400], 96, 8, 128, 64, 64, "hnd"),
    ([3, 0, 30, 1], [10, 5, 0, 63], 10, 5, 128, 128, 32, "nhd"),
    ([7, 50], [200, 0], 4, 2, 256, 128, 16, "interleaved"),
    ([40, 1], [3, 255], 6, 3, 64, 0, 128, "hnd"),
    ([300], [11], 12, 1, 128, 64, 256, "nhd"),
    ([1] * 70, list(range(70)), 3, 3, 128, 64, 16, "hnd"),
    # rotations whose halves end inside a lane's dimensions
    ([9, 4], [2, 30], 5, 1, 128, 24, 16, "hnd"),
    ([9, 4], [2, 30], 5, 1, 64, 36, 16, "hnd"),
    ([9, 4], [2, 30], 4, 2, 64, 8, 16, "nhd"),
    ([9, 4], [2, 30], 4, 4, 64, 12, 16, "hnd"),
    ([700], [100], 24, 2, 128, 64, 64, "hnd"),              # more heads than the SMs hold at once
    ([600, 13], [3, 90], 13, 13, 64, 32, 16, "hnd"),
    ([400], [0], 30, 10, 256, 256, 32, "hnd"),
]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", APPEND, ids=[f"T{sum(s[0])}_q{s[2]}_d{s[4]}_r{s[5]}_{s[7]}" for s in APPEND])
def test_append_matches_fp64(shape, kv):
    n, ctx, n_q, n_kv, d, rot, page, layout = shape
    T = sum(n) + 2                                          # two padding rows
    P = Paged(n, ctx, n_kv, d, page, kv, layout, seed=1, rows=T, k_scale=0.02, v_scale=0.11)
    cfg, inp = attn_inputs(T, n_q, n_kv, d, rot, 512, 31)
    cache, batch = P.handles(m)
    k0, v0 = P.k.clone(), P.v.clone()
    qkv0 = inp["qkv"].clone()
    q_out = torch.full((T, n_q * d), 7.5, dtype=torch.bfloat16, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    inp["pos"][-1] = -5                                     # padding rows are not looked at
    m.moe_qk_norm_rope_append(cache, batch, n_q, rot, cfg.eps, inp["qkv"], inp["pos"], inp["q_w"], inp["k_w"],
                              inp["cos_sin"], q_out, bad)
    torch.cuda.synchronize()
    assert int(bad) == 0
    assert torch.equal(inp["qkv"].view(torch.int16), qkv0.view(torch.int16))
    assert bool((q_out[sum(n):] == 7.5).all())
    # q rows and bf16 keys: bit for bit those of moe_qk_norm_rope
    both = inp["qkv"][:sum(n)].clone()
    _lib.moe_qk_norm_rope(cfg, both, inp["pos"][:sum(n)].contiguous(), inp["q_w"], inp["k_w"], inp["cos_sin"])
    heads = both.view(sum(n), n_q + 2 * n_kv, d)
    assert torch.equal(q_out[:sum(n)].view(-1, n_q, d).view(torch.int16), heads[:, :n_q].contiguous().view(torch.int16))
    ref = torch.from_numpy(oracle.qk_norm_rope(_bits(qkv0[:sum(n)]), inp["pos"][:sum(n)].cpu().numpy(), _bits(inp["q_w"]),
                                               _bits(inp["k_w"]), inp["cos_sin"].cpu().numpy(), n_q, n_kv, d, rot,
                                               cfg.eps)).to(DEV).view(sum(n), n_q + n_kv, d)
    new = torch.zeros(P.pages, page, dtype=torch.bool, device=DEV)
    row = 0
    for b in range(len(n)):
        pg, sl = P.slots(b)
        pg, sl = pg[ctx[b]:], sl[ctx[b]:]
        new[pg, sl] = True
        vin = qkv0[row:row + n[b]].view(n[b], n_q + 2 * n_kv, d)[:, n_q + n_kv:]
        for h in range(n_kv):
            gk, gv = P.k[pg, h, sl], P.v[pg, h, sl]
            if kv == "bf16":
                assert torch.equal(gk.view(torch.int16), heads[row:row + n[b], n_q + h].contiguous().view(torch.int16))
                assert torch.equal(gv.view(torch.int16), vin[:, h].contiguous().view(torch.int16))
                continue
            want_v = (vin[:, h].float() / P.vs).clamp(-448, 448).to(torch.float8_e4m3fn)
            assert torch.equal(gv, want_v.view(torch.uint8))
            want = (ref[row:row + n[b], n_q + h] / P.ks).clamp(-448, 448)
            got = gk.view(torch.float8_e4m3fn).double()
            # one rounding to E4M3 (normal: 2^-4 of the value, below 2^-6: half of 2^-9) of an fp32 value
            # whose own error is at most (d + 16) 2^-24 of the head's largest value
            tol = torch.maximum(HALF_E4M3 * want.abs(), torch.full_like(want, 2.0 ** -10)) + \
                (d + 16) * F32 * want.abs().amax(1, keepdim=True)
            assert bool(((got - want).abs() <= tol).all())
        row += n[b]
    # every other slot is as it was, bit for bit
    for t, t0 in ((P.k, k0), (P.v, v0)):
        it = torch.uint8 if kv == "e4m3" else torch.int16
        a, b_ = t.permute(0, 2, 1, 3)[~new].contiguous().view(it), t0.permute(0, 2, 1, 3)[~new].contiguous().view(it)
        assert torch.equal(a, b_)


def test_append_in_place_without_norms_and_at_one_row():
    """q_out over the q heads of qkv itself; no norm weights: rotation alone; T = 1."""
    for T in (1, 9):
        P = Paged([T], [20], 2, 128, 16, "bf16", seed=2)
        cfg, inp = attn_inputs(T, 4, 2, 128, 64, 64, 5)
        cache, batch = P.handles(m)
        qkv = inp["qkv"].clone()
        m.moe_qk_norm_rope_append(cache, batch, 4, 64, cfg.eps, qkv, inp["pos"], None, None, inp["cos_sin"],
                                  qkv[:, :4 * 128])
        x = inp["qkv"].double().view(T, 8, 128)
        cs = inp["cos_sin"].double()[inp["pos"].long()][:, None]
        a, b = x[:, :6, :32], x[:, :6, 32:64]
        ref = torch.cat([a * cs[..., :32] - b * cs[..., 32:], b * cs[..., :32] + a * cs[..., 32:], x[:, :6, 64:]], -1)
        got = qkv.double().view(T, 8, 128)
        # one rounding, and the products' fp32 errors (2 * 2^-24 of each)
        tol = HALF_BF16 * ref.abs() + 4 * F32 * (x[:, :6].abs().amax(-1, keepdim=True) * 2)
        assert bool(((got[:, :4] - ref[:, :4]).abs() <= tol[:, :4]).all())
        assert torch.equal(qkv.view(torch.int16).view(T, 8, 128)[:, 4:], inp["qkv"].view(torch.int16).view(T, 8, 128)[:, 4:])
        pg, sl = P.slots(0)
        K = P.k[pg[20:], :, sl[20:]].double()
        assert bool(((K - ref[:, 4:]).abs() <= tol[:, 4:]).all())


def test_append_counts_bad_tokens_and_stores_nothing_of_them():
    n_q, n_kv, d = 4, 2, 128
    P = Paged([5, 6, 3], [14, 40, 2], n_kv, d, 16, "bf16", seed=3)
    cfg, inp = attn_inputs(14, n_q, n_kv, d, 64, 100, 6)
    cache, batch = P.handles(m)
    inp["pos"][2] = 100                                     # sequence 0, token 2: position out of range
    inp["pos"][3] = -1
    P.table[1, 2] = P.pages                                 # sequence 1: cache indexes 40..45 lie in its page 2
    P.ctx_len[2] = -1                                       # sequence 2: three tokens without a slot
    k0, v0 = P.k.clone(), P.v.clone()
    q_out = torch.full((14, n_q * d), 7.5, dtype=torch.bfloat16, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.moe_qk_norm_rope_append(cache, batch, n_q, 64, cfg.eps, inp["qkv"], inp["pos"], inp["q_w"], inp["k_w"],
                              inp["cos_sin"], q_out, bad)
    assert int(bad) == 2 + 6 + 3
    assert bool((q_out[2:4] == 7.5).all())
    assert not bool((q_out[4:] == 7.5).all(1).any()) and not bool((q_out[:2] == 7.5).all(1).any())
    changed = (P.k.view(torch.int16) != k0.view(torch.int16)).permute(0, 2, 1, 3).any(-1).any(-1)
    pg, sl = P.slots(0)
    want = torch.zeros_like(changed)
    for i in (14, 15, 18):
        want[pg[i], sl[i]] = True
    assert torch.equal(changed, want)
    assert torch.equal((P.v.view(torch.int16) != v0.view(torch.int16)).permute(0, 2, 1, 3).any(-1).any(-1), want)


def test_append_with_rows_out_of_order_stays_inside_the_cache():
    """q_start [5, 40, 60, 7, 8]: the search lands row 30 in the sequence of rows 40..59, in front
    of its first row; such tokens are counted and nothing of them is stored."""
    n_q, n_kv, d, T = 2, 1, 128, 64
    qkv = torch.randn(T, (n_q + 2 * n_kv) * d, device=DEV).to(torch.bfloat16)
    k = torch.full((12, n_kv, 16, d), 7.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(12, **i32).reshape(4, 3)
    batch = m.make_kv_batch(torch.tensor([5, 40, 60, 7, 8], **i32), torch.zeros(4, **i32), table, 40)
    bad = torch.zeros(1, **i32)
    q_out = torch.zeros(T, n_q * d, dtype=torch.bfloat16, device=DEV)
    m.moe_qk_norm_rope_append(m.make_kv_cache(k, v), batch, n_q, 0, 1e-5, qkv, None, None, None, None, q_out, bad)
    # the rows' sequences: the last entry of q_start that the search counts as reached
    want_k, want_v, want_bad = torch.full_like(k, 7.0), torch.full_like(v, 7.0), 0
    q_start = [5, 40, 60, 7, 8]
    for t in range(T):
        b = sum(s <= t for s in q_start[:4]) - 1
        if b < 0 or t >= q_start[b + 1]:
            continue
        n, i = q_start[b + 1] - q_start[b], t - q_start[b]
        if n < 0 or n > 40 or i < 0:
            want_bad += 1
            continue
        want_k[table[b, i // 16], 0, i % 16] = qkv[t, n_q * d:(n_q + 1) * d]
        want_v[table[b, i // 16], 0, i % 16] = qkv[t, (n_q + 1) * d:]
    assert want_bad > 0 and int(bad) == want_bad
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_append_e4m3_saturates_and_keeps_nan():
    P = Paged([1], [0], 1, 64, 16, "e4m3", seed=4, k_scale=0.5, v_scale=0.25)
    cache, batch = P.handles(m)
    qkv = torch.zeros(1, 3 * 64, dtype=torch.bfloat16, device=DEV)
    qkv[0, 128:134] = torch.tensor([1000.0, -1000.0, math.inf, -math.inf, math.nan, 112.0], device=DEV)
    q_out = torch.empty(1, 64, dtype=torch.bfloat16, device=DEV)
    m.moe_qk_norm_rope_append(cache, batch, 1, 0, 1e-5, qkv, None, None, None, None, q_out)
    pg, sl = P.slots(0)
    got = P.v[pg[0], 0, sl[0], :6].view(torch.float8_e4m3fn).float().tolist()
    assert got[:4] == [448.0, -448.0, 448.0, -448.0] and math.isnan(got[4]) and got[5] == 448.0


def _moved(P, src, dst, acc):
    """What the cache holds after the accepted tokens moved, from a copy."""
    for t in (P.k, P.v):
        c = t.clone()
        for b, a in enumerate(acc):
            pg, sl = P.slots(b)
            for i, j in enumerate(a):
                d, s = P.ctx[b] + i, P.ctx[b] + j
                if t.dim() == 4:
                    t[pg[d], :, sl[d]] = c[pg[s], :, sl[s]]
                else:
                    t[:, pg[d], :, sl[d]] = c[:, pg[s], :, sl[s]]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d,page,layout,layers", [(128, 16, "hnd", 1), (64, 32, "nhd", 1), (256, 16, "interleaved", 1),
                                                   (128, 64, "hnd", 5)])
def test_compact_moves_the_accepted_tokens(d, page, layout, layers, kv):
    n, ctx = [20, 61, 1, 7, 0, 40], [13, 0, 5, 64, 9, 30]
    acc = [[0, 2, 5, 6, 19], list(range(61)), [0], [], [], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 20, 39]]
    P = Paged(n, ctx, 3, d, page, kv, layout, seed=5, layers=None if layers == 1 else layers)
    width = 64
    lists = torch.full((6, width), -99, dtype=torch.int32, device=DEV)     # entries behind the count are not read
    for b, a in enumerate(acc):
        lists[b, :len(a)] = torch.tensor(a, dtype=torch.int32)
    count = torch.tensor([len(a) for a in acc], dtype=torch.int32, device=DEV)
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    k0, v0 = P.k.clone(), P.v.clone()
    ck, cv = (P.k, P.v) if layers == 1 else (P.k[0], P.v[0])
    cache = m.make_kv_cache(ck, cv, P.ks, P.vs)
    batch = m.make_kv_batch(P.q_start, P.ctx_len, P.table, 61)
    m.moe_kv_compact(cache, batch, lists, count, layers, P.k.stride(0) if layers > 1 else 0, bad)
    torch.cuda.synchronize()
    assert int(bad) == 0
    gk, gv = P.k.clone(), P.v.clone()
    P.k.copy_(k0)
    P.v.copy_(v0)
    _moved(P, None, None, acc)
    it = torch.uint8 if kv == "e4m3" else torch.int16
    assert torch.equal(gk.view(it), P.k.clone().view(it)) and torch.equal(gv.view(it), P.v.clone().view(it))


def test_compact_leaves_bad_sequences_alone():
    n = [8] * 9
    P = Paged(n, [10] * 9, 2, 64, 16, "bf16", seed=6)
    rows = [[0, 3, 3], [0, 5, 4], [0, 8, 9], [-1, 2, 3], [0, 2, 4], [0, 1, 7], [1, 2, 3], [1, 2, 5], [2, 4, 6]]
    lists = torch.tensor(rows, dtype=torch.int32, device=DEV)
    count = torch.tensor([3, 3, 2, 3, 4, 3, -1, 3, 3], dtype=torch.int32, device=DEV)
    P.table[5, 1] = -1                                      # sequence 5 reaches a bad page
    P.ctx_len[8] = 1 << 30
    k0 = P.k.clone()
    bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache, batch = P.handles(m)
    m.moe_kv_compact(cache, batch, lists, count, bad_seqs=bad)
    assert int(bad) == 8
    gk = P.k.clone()
    P.k.copy_(k0)
    v0 = P.v.clone()
    P.v.copy_(v0)
    _moved(P, None, None, [[], [], [], [], [], [], [], [1, 2, 5], []])
    assert torch.equal(gk.view(torch.int16), P.k.view(torch.int16))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_speculative_step_equals_plain_decoding(kv):
    """Prefill a prompt, append and attend to a drafted tree, accept one path and move it, then decode
    one more token: that token's output equals attention over a cache that was filled with the prompt
    and the accepted tokens in order, bit for bit where the cache is."""
    n_q, n_kv, d, rot, page = 8, 2, 128, 64, 16
    B, prompt, tree = 3, [37, 5, 64], [9, 12, 20]
    paths = [[0, 2, 5], [0, 1], [0, 3, 4, 11]]
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    cfg, inp = attn_inputs(1, n_q, n_kv, d, rot, 256, 8)
    table = torch.arange(B * 8, dtype=torch.int32, device=DEV).flip(0).reshape(B, 8).contiguous()
    width = (n_q + 2 * n_kv) * d

    def new_cache():
        dt = torch.bfloat16 if kv == "bf16" else torch.uint8
        ks, vs = (1.0, 1.0) if kv == "bf16" else (0.05, 0.05)
        return m.make_kv_cache(*[torch.full((B * 8, n_kv, page, d), 0x7F, dtype=dt, device=DEV) for _ in range(2)], ks, vs)

    def rows(counts):
        return [torch.randn(c, width, generator=g, device=DEV).to(torch.bfloat16) for c in counts]

    def step(cache, ctx, qkvs, poss, mask=None):
        counts = [x.shape[0] for x in qkvs]
        starts = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
        batch = m.make_kv_batch(starts, torch.tensor(ctx, dtype=torch.int32, device=DEV), table, max(counts))
        qkv = torch.cat(qkvs)
        T = qkv.shape[0]
        q = torch.empty(T, n_q * d, dtype=torch.bfloat16, device=DEV)
        bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        m.moe_qk_norm_rope_append(cache, batch, n_q, rot, cfg.eps, qkv, torch.tensor(sum(poss, []), dtype=torch.int32, device=DEV),
                                  inp["q_w"], inp["k_w"], inp["cos_sin"], q, bad)
        out, lse = torch.empty_like(q), torch.empty(T, n_q, device=DEV)
        ws = m.alloc_tree_attention_workspace(cache, n_q, T)
        m.moe_tree_attention(cache, batch, n_q, q, out, ws, tree_mask=mask, lse=lse)
        assert int(bad) == 0 and m.moe_get_status(ws) == _lib.MOE_OK
        return batch, out, lse

    prompts, drafts, last = rows(prompt), rows(tree), rows([1] * B)
    sets = [tree_sets(tree[b], 70 + b) for b in range(B)]
    for b, p in enumerate(paths):                           # the accepted path is a path of the tree
        for i, j in enumerate(p):
            sets[b][j] = sum(1 << k for k in p[:i + 1])
    depth = [[bin(w).count("1") - 1 for w in s] for s in sets]

    spec = new_cache()
    step(spec, [0] * B, prompts, [list(range(c)) for c in prompt])
    batch, out_tree, _ = step(spec, prompt, drafts, [[prompt[b] + x for x in depth[b]] for b in range(B)],
                              mask_tensor(sum(sets, []), 1))
    accepted = torch.zeros(B, 4, dtype=torch.int32, device=DEV)
    for b, p in enumerate(paths):
        accepted[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    n_acc = [len(p) for p in paths]
    m.moe_kv_compact(spec, batch, accepted, torch.tensor(n_acc, dtype=torch.int32, device=DEV))
    ctx = [prompt[b] + n_acc[b] for b in range(B)]
    _, out_spec, lse_spec = step(spec, ctx, last, [[c] for c in ctx])

    plain = new_cache()
    step(plain, [0] * B, prompts, [list(range(c)) for c in prompt])
    _, out_chain, _ = step(plain, prompt, [drafts[b][paths[b]] for b in range(B)],
                           [[prompt[b] + i for i in range(n_acc[b])] for b in range(B)])
    _, out_plain, lse_plain = step(plain, ctx, last, [[c] for c in ctx])
    for a, b_ in zip(spec.tensors, plain.tensors):
        it = torch.int16 if kv == "bf16" else torch.uint8
        for b in range(B):
            i = torch.arange(ctx[b] + 1, device=DEV)
            pg, sl = table[b].long()[i // page], i % page
            assert torch.equal(a[pg, :, sl].view(it), b_[pg, :, sl].view(it))
    assert torch.equal(out_spec.view(torch.int16), out_plain.view(torch.int16)) and torch.equal(lse_spec, lse_plain)
    # the tree's accepted rows are the chain's: each side is off by one rounding of the result and one
    # of each weight, which all in all weigh at most the largest value; 2^-12 of it for the fp32 sums
    at = [sum(tree[:b]) + j for b in range(B) for j in paths[b]]
    x, y = out_tree[at].double(), out_chain.double()
    v = plain.tensors[1]
    v = (v.view(torch.float8_e4m3fn).double() * 0.05) if kv == "e4m3" else v.double()
    big = float(torch.nan_to_num(v, nan=0.0).abs().max())
    assert bool(((x - y).abs() <= HALF_BF16 * (x.abs() + y.abs()) + 2 * (HALF_BF16 + 2.0 ** -12) * big).all())

    # score the drafts with log probabilities of a synthetic head
    logits = torch.randn(len(at), 5003, generator=g, device=DEV).to(torch.bfloat16)
    tok = torch.randint(0, 5003, (len(at),), generator=g, device=DEV).int()
    lp = torch.empty(len(at), device=DEV)
    m.moe_token_logprobs(logits, tok, lp)
    ref = torch.log_softmax(logits.double(), 1).gather(1, tok.long()[:, None])[:, 0]
    assert float((lp.double() - ref).abs().max()) <= 64 * F32 * float(ref.abs().max())


def test_append_and_compact_in_a_graph():
    P = Paged([4, 4], [10, 30], 2, 128, 16, "bf16", seed=21, extra_pages=0)
    cfg, inp = attn_inputs(8, 4, 2, 128, 64, 128, 9)
    cache, batch = P.handles(m)
    q_out = torch.empty(8, 4 * 128, dtype=torch.bfloat16, device=DEV)
    acc = torch.tensor([[0, 2], [1, 3]], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([2, 2], dtype=torch.int32, device=DEV)

    def go():
        m.moe_qk_norm_rope_append(cache, batch, 4, 64, cfg.eps, inp["qkv"], inp["pos"], inp["q_w"], inp["k_w"],
                                  inp["cos_sin"], q_out)
        m.moe_kv_compact(cache, batch, acc, cnt)

    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    P.ctx_len.copy_(torch.tensor([3, 7], dtype=torch.int32))
    k0, v0 = P.k.clone(), P.v.clone()
    g.replay()
    torch.cuda.synchronize()
    gk, gv = P.k.clone(), P.v.clone()
    P.k.copy_(k0)
    P.v.copy_(v0)
    go()
    torch.cuda.synchronize()
    assert torch.equal(gk.view(torch.int16), P.k.view(torch.int16)) and torch.equal(gv.view(torch.int16), P.v.view(torch.int16))
    assert not torch.equal(gk.view(torch.int16), k0.view(torch.int16))


@pytest.mark.parametrize("n_q", [4, 24, 33])
@pytest.mark.parametrize("T", [13, 700])
@pytest.mark.parametrize("d,rot", [(128, 24), (128, 64), (64, 36), (64, 12), (64, 8), (256, 128)])
def test_append_keeps_the_bits_of_the_norm_and_rotation_beside_infinities(d, rot, T, n_q):
    """q rows and bf16 keys equal moe_qk_norm_rope's bit for bit, whichever warp has the head: negative
    zeros, infinities and NaN in one dimension of a row, weights that are infinite or zero, and rows so small
    that the mean square vanishes (eps 0). Where a dimension does not rotate, an infinity stays one."""
    n_kv = 3 if n_q % 3 == 0 else 2
    for eps in (1e-5, 0.0):
        P = Paged([T], [5], n_kv, d, 16, "bf16", seed=30)
        cfg, inp = attn_inputs(T, n_q, n_kv, d, rot, 900, 12)
        cfg = dataclasses.replace(cfg, eps=eps)
        cache, batch = P.handles(m)
        x = inp["qkv"].view(T, n_q + 2 * n_kv, d)
        x[::2, :, 1::3] = -0.0
        x[1, :, d - 3], x[2, :, d - 6], x[3, :, rot // 2 + 1], x[4, :, 0] = math.inf, math.nan, -math.inf, math.inf
        x[5] = torch.where(x[5] == 0, x[5], 1e-30 * torch.sign(x[5]))
        for w in (inp["q_w"], inp["k_w"]):
            w[d - 2], w[1], w[d - 5] = math.inf, 0.0, -1.0
        both = inp["qkv"].clone()
        q_out = torch.empty(T, n_q * d, dtype=torch.bfloat16, device=DEV)
        m.moe_qk_norm_rope_append(cache, batch, n_q, rot, eps, inp["qkv"], inp["pos"], inp["q_w"], inp["k_w"],
                                  inp["cos_sin"], q_out)
        _lib.moe_qk_norm_rope(cfg, both, inp["pos"], inp["q_w"], inp["k_w"], inp["cos_sin"])
        want = both.view(T, n_q + 2 * n_kv, d)[:, :n_q + n_kv].clone()
        u = x[:, :n_q + n_kv].float()
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps)
        u = u * torch.cat([inp["q_w"].float().expand(n_q, d), inp["k_w"].float().expand(n_kv, d)])
        stays = torch.isinf(u) & (torch.arange(d, device=DEV) >= rot)
        assert bool(stays.any()) and bool(torch.isnan(want[stays]).all())
        want[stays] = u[stays].to(torch.bfloat16)
        pg, sl = P.slots(0)
        got = torch.cat([q_out.view(T, n_q, d), P.k[pg[5:], :, sl[5:]]], 1)
        assert bool(torch.isnan(want).any()) and bool((want == 0).any())
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(got.view(torch.int16)[fine], want.view(torch.int16)[fine])


def test_append_without_norms_passes_infinities_through():
    """Heads without a norm: dimensions that do not rotate keep their value, whatever it is."""
    P = Paged([9], [5], 2, 64, 16, "bf16", seed=31)
    cfg, inp = attn_inputs(9, 4, 2, 64, 12, 64, 13)
    cache, batch = P.handles(m)
    x = inp["qkv"].view(9, 8, 64)
    x[1, :, 20], x[2, :, 63], x[3, :, 40] = math.inf, -0.0, -math.inf
    q_out = torch.empty(9, 4 * 64, dtype=torch.bfloat16, device=DEV)
    m.moe_qk_norm_rope_append(cache, batch, 4, 12, cfg.eps, inp["qkv"], inp["pos"], None, None, inp["cos_sin"], q_out)
    pg, sl = P.slots(0)
    got = torch.cat([q_out.view(9, 4, 64), P.k[pg[5:], :, sl[5:]]], 1)[..., 12:].contiguous()
    assert torch.equal(got.view(torch.int16), x[:, :6, 12:].contiguous().view(torch.int16))


def test_steps_without_rows_or_sequences():
    """Tensors of no rows (whose address is NULL) through every call: nothing happens."""
    k = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16, device=DEV)
    cache = m.make_kv_cache(k, k.clone())
    i32 = dict(dtype=torch.int32, device=DEV)
    b16 = dict(dtype=torch.bfloat16, device=DEV)
    for B in (0, 2):
        batch = m.make_kv_batch(torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(B, 1, **i32), 0)
        ws = m.alloc_tree_attention_workspace(cache, 4, 0)
        q = torch.empty(0, 4 * 128, **b16)
        m.moe_qk_norm_rope_append(cache, batch, 4, 64, 1e-5, torch.empty(0, 6 * 128, **b16), torch.empty(0, **i32), None, None,
                                  torch.ones(4, 64, device=DEV), q)
        m.moe_tree_attention(cache, batch, 4, q, torch.empty_like(q), ws, lse=torch.empty(0, 4, device=DEV))
        m.moe_tree_attention(cache, batch, 4, q, q, ws, tree_mask=torch.empty(0, 1, dtype=torch.int64, device=DEV))
        m.moe_kv_compact(cache, batch, torch.zeros(B, 3, **i32), torch.zeros(B, **i32))
        assert m.moe_get_status(ws) == _lib.MOE_OK
    f = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    m.moe_token_logprobs(f(0, 50), torch.empty(0, **i32), f(0), f(0), torch.empty(0, 3, **i32), f(0, 3))
    m.moe_token_logprobs(f(0, 50), None, None, f(0))
    torch.cuda.synchronize()
    assert not bool(k.any())
