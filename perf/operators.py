"""Performance cases of the serving operators beside the fused QK-norm + RoPE step: appending keys and
values to a paged cache, attention of drafted token trees over that cache, moving the accepted nodes'
keys and values together, and the log probabilities that drafts and prompts are scored with.

A case is a dict; `prepare` makes its inputs on the GPU from a seed, `run` makes one pass and returns
every output. With `own` false a pass is the plain form (elementary torch operations, fp32 or fp64,
rounded once at the end), with `own` true the calls a user makes of the package. `exact` restates each
operator in fp64, one head or block of rows at a time.
"""
import math
import random

import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    heads = dict(n_q=96, n_kv=8, d=128, page=64)           # the attention heads of the qknorm_* workloads
    return [
        # one sequence decoding one token: a launch and its latency
        dict(name="append_1tok", op="append", B=1, n_min=1, n_max=1, ctx_min=777, ctx_max=777, rot=64, kv="bf16", **heads),
        # a decode batch into an 8-bit cache, each sequence at its own length
        dict(name="append_decode64_e4m3", op="append", B=64, n_min=1, n_max=1, ctx_min=1, ctx_max=1000, rot=64,
             kv="e4m3", **heads),
        # a prefill chunk of five prompts of odd lengths, some with a cached prefix that ends inside a page
        dict(name="append_prefill", op="append", B=5, n_min=37, n_max=1601, ctx_min=0, ctx_max=333, rot=64, kv="bf16",
             **heads),
        # one sequence decoding against a long context: the smallest attention call, bound by latency
        dict(name="attn_decode1", op="attn", B=1, n_min=1, n_max=1, ctx_min=4096, ctx_max=4096, tree=False, kv="bf16",
             **heads),
        # the decode batch over an 8-bit cache, ragged contexts: bound by reading the cache
        dict(name="attn_decode64_e4m3", op="attn", B=64, n_min=1, n_max=1, ctx_min=64, ctx_max=8191, tree=False,
             kv="e4m3", **heads),
        # four drafted tokens in a row for each of 32 sequences (a chain: every token sees those before it)
        dict(name="attn_chain4", op="attn", B=32, n_min=4, n_max=4, ctx_min=100, ctx_max=8100, tree=False, kv="bf16",
             **heads),
        # token trees of up to 61 nodes over ragged contexts: many query rows for each key read
        dict(name="attn_tree61", op="attn", B=12, n_min=23, n_max=61, ctx_min=500, ctx_max=9000, tree=True, kv="bf16",
             **heads),
        # the largest: a 4096-token prefill chunk behind 12288 cached tokens, bound by the tensor cores
        dict(name="attn_chunk4096", op="attn", B=1, n_min=4096, n_max=4096, ctx_min=12288, ctx_max=12288, tree=False,
             kv="bf16", **heads),
        # one row of logits with alternatives: what a single decoding sequence asks for after each token
        dict(name="logprobs_1row", op="logprobs", T=1, V=131072, top=20, dtype="bf16"),
        # scoring a prompt chunk or a large batch of drafts; an odd vocabulary, so rows start at any alignment
        dict(name="logprobs_2048", op="logprobs", T=2048, V=100003, top=5, dtype="f32"),
        # after one sequence's tree was verified: three accepted nodes, in all layers of a small model
        dict(name="compact_1seq", op="compact", layers=8, B=1, n_min=31, n_max=31, ctx_min=100, ctx_max=100, depth=3,
             kv="bf16", n_kv=8, d=128, page=64),
        # the same for a batch over an 8-bit cache of 92 layers
        dict(name="compact_92layers_e4m3", op="compact", layers=92, B=32, n_min=40, n_max=61, ctx_min=1, ctx_max=190,
             depth=6, kv="e4m3", n_kv=8, d=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "logprobs", "compact"])
    if op == "logprobs":
        V = _log_int(rng, 1000, 200000)
        return dict(op=op, T=_log_int(rng, 1, max(1, min(4096, 200_000_000 // V))), V=V, top=rng.choice([0, 1, 5, 20, 32]),
                    dtype=rng.choice(["bf16", "f32"]))
    n_kv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 128, 256])
    case = dict(op=op, n_kv=n_kv, d=d, page=rng.choice([16, 32, 64, 128, 256]), kv=rng.choice(["bf16", "e4m3"]))
    if op == "compact":
        n = rng.randint(12, 150)
        B, ctx = _log_int(rng, 1, 32), _log_int(rng, 1, 200)
        per = -(-(n + ctx) // case["page"]) * case["page"] * n_kv * d          # at most 700M numbers in all layers' keys
        case.update(layers=_log_int(rng, 1, max(1, min(92, 700_000_000 // (per * (B + 1))))), B=B, n_min=max(12, n // 2),
                    n_max=n, ctx_min=0, ctx_max=ctx, depth=rng.randint(2, 6))
        return case
    case.update(n_q=n_kv * rng.choice([1, 2, 4, 5, 8, 12, 16]))
    if op == "append":
        n = _log_int(rng, 1, 4096)
        case.update(B=_log_int(rng, 1, max(1, 8192 // n)), n_min=max(1, n // 3), n_max=n, ctx_min=0,
                    ctx_max=_log_int(rng, 1, 1000), rot=rng.choice([0, d // 2, d]))
        return case
    tree = rng.random() < 0.4
    n = _log_int(rng, 2, 200) if tree else _log_int(rng, 1, 4096)
    ctx = _log_int(rng, 1, 16384)
    # no more pairs of query rows and keys than the largest listed case, and a cache of at most 4M token heads
    B = _log_int(rng, 1, max(1, min(128, 2_000_000_000 // (n * (n + ctx) * case["n_q"]), 4_000_000 // ((n + ctx) * n_kv))))
    case.update(B=B, n_min=max(1, n // 3), n_max=n, ctx_min=ctx // 10, ctx_max=ctx, tree=tree)
    return case


# ---------------------------------------------------------------- shapes that follow from a case

def _spread(lo, hi, B, phase):
    """B whole numbers spread over lo..hi, the largest first, the others in no order."""
    return [hi if b == 0 else lo + int(((b * 0.6180339887 + phase) % 1.0) * (hi - lo + 1)) for b in range(B)]


def _lengths(case):
    n = _spread(case["n_min"], case["n_max"], case["B"], 0.37)
    ctx = _spread(case["ctx_min"], case["ctx_max"], case["B"], 0.81)
    return n, ctx


def work(case):
    if case["op"] == "logprobs":
        esz = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["T"] * (case["V"] * esz + 12 + 8 * case["top"]), "flops": 5 * case["T"] * case["V"]}
    n, ctx = _lengths(case)
    T, d, n_kv, csz = sum(n), case["d"], case["n_kv"], 2 if case["kv"] == "bf16" else 1
    if case["op"] == "compact":
        moved = case["layers"] * case["B"] * (case["depth"] - 1) * n_kv * d * csz * 2
        return {"bytes": 2 * moved, "flops": 0}
    n_q = case["n_q"]
    if case["op"] == "append":
        read = T * (n_q + 2 * n_kv) * d * 2 + T * case["rot"] * 4
        return {"bytes": read + T * n_q * d * 2 + T * 2 * n_kv * d * csz, "flops": T * (n_q + n_kv) * d * 8}
    keys = sum(a + c for a, c in zip(n, ctx))
    pairs = sum(a * c + (a * a if case["tree"] else a * (a + 1) // 2) for a, c in zip(n, ctx))
    return {"bytes": keys * n_kv * d * 2 * csz + T * n_q * (4 * d + 4), "flops": 4 * pairs * n_q * d}


# ---------------------------------------------------------------- inputs

def _codes(x, scale):
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _cache(case, g, pages, lead=()):
    """K and V of a paged cache [..., pages, n_kv, page, d], keys of unit size, values N(0, 1)."""
    shape = (*lead, pages, case["n_kv"], case["page"], case["d"])
    k = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if case["kv"] == "e4m3" else torch.bfloat16)
    v = torch.randn(shape, generator=g, device=DEV, dtype=k.dtype)
    ks, vs = (0.0625, 0.04) if case["kv"] == "e4m3" else (1.0, 1.0)
    if case["kv"] == "e4m3":
        k, v = _codes(k, ks), _codes(v, vs)
    return k, v, ks, vs


def _batch(case, g):
    n, ctx = _lengths(case)
    per = [-(-(a + c) // case["page"]) for a, c in zip(n, ctx)]
    width, pages = max(per), sum(per) + 1                          # one page that no sequence owns
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.zeros(case["B"], width, dtype=torch.int32, device=DEV)
    at = 0
    for b, p in enumerate(per):
        table[b, :p] = order[at:at + p]
        at += p
    starts = [0]
    for a in n:
        starts.append(starts[-1] + a)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    # the token rows laid out by sequence, as a plain form indexes them: row of token i of sequence b, or the last row
    rows = torch.tensor([[starts[b] + i if i < n[b] else starts[-1] for i in range(max(n))] for b in range(case["B"])],
                        device=DEV)
    return {"n": n, "ctx": ctx, "T": starts[-1], "pages": pages, "q_start": i32(starts), "ctx_len": i32(ctx), "table": table,
            "rows": rows, "n_t": i32(n), "max_new": max(n)}


def _tree(n, r):
    """Ancestor sets (as whole numbers, bit j: node j) and depths of a tree of n drafted tokens, parents before children."""
    sets, depth = [1], [0]
    for i in range(1, n):
        p = r.randrange(max(0, i - 9), i)
        sets.append(sets[p] | 1 << i)
        depth.append(depth[p] + 1)
    return sets, depth


def _signed(w):
    return w - (1 << 64) if w >= 1 << 63 else w


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = random.Random(seed)
    s = {"case": case}
    if case["op"] == "logprobs":
        T, V = case["T"], case["V"]
        # a language model's rows: a broad body and, row by row, a few likely tokens
        x = torch.randn(T, V, generator=g, device=DEV) * 2.0
        x.scatter_add_(1, torch.randint(0, V, (T, 8), generator=g, device=DEV),
                       torch.rand(T, 8, generator=g, device=DEV) * 8.0 + 6.0)
        s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["targets"] = torch.randint(0, V, (T,), generator=g, device=DEV).int()
        f = lambda *z, dt=torch.float32: torch.empty(z, dtype=dt, device=DEV)  # noqa: E731
        s.update(lp=f(T), ent=f(T), ids=f(T, case["top"], dt=torch.int32), top=f(T, case["top"]))
        return s
    bt = s["batch"] = _batch(case, g)
    T, n_kv, d = bt["T"], case["n_kv"], case["d"]
    lead = (case["layers"],) if case["op"] == "compact" else ()
    s["k"], s["v"], s["ks"], s["vs"] = _cache(case, g, bt["pages"], lead)
    if case["op"] == "compact":
        # the accepted path: the root, then nodes of the later branches (behind the places they move to)
        acc = [[0] + sorted(r.sample(range(case["depth"], bt["n"][b]), case["depth"] - 1)) for b in range(case["B"])]
        s["accepted"] = torch.tensor(acc, dtype=torch.int32, device=DEV)
        s["n_acc"] = torch.full((case["B"],), case["depth"], dtype=torch.int32, device=DEV)
    elif case["op"] == "append":
        n_q, rot = case["n_q"], case["rot"]
        qkv = torch.randn(T, n_q + 2 * n_kv, d, generator=g, device=DEV)
        qkv *= torch.pow(10.0, torch.rand(T, n_q + 2 * n_kv, 1, generator=g, device=DEV) - 0.5)
        s["qkv"] = qkv.reshape(T, -1).to(torch.bfloat16)
        s["max_pos"] = max(c + a for a, c in zip(bt["n"], bt["ctx"])) + 1
        s["pos"] = torch.cat([torch.arange(c, c + a, device=DEV) for a, c in zip(bt["n"], bt["ctx"])]).int()
        s["q_w"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
        s["k_w"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
        ang = torch.arange(s["max_pos"], device=DEV).double()[:, None] * torch.pow(
            1.0e6, -2.0 * torch.arange(rot // 2, device=DEV).double() / max(rot, 1))
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["q_out"] = torch.empty(T, n_q * d, dtype=torch.bfloat16, device=DEV)
        # the cache index of each token, as a plain form stores it
        s["at"] = s["pos"].long()
        s["seq"] = torch.repeat_interleave(torch.arange(case["B"], device=DEV), bt["n_t"].long())
    else:
        n_q = case["n_q"]
        s["q"] = (torch.randn(T, n_q * d, generator=g, device=DEV) * 2.0).to(torch.bfloat16)
        s["out"] = torch.empty(T, n_q * d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, n_q, dtype=torch.float32, device=DEV)
        s["mask"] = None
        if case["tree"]:
            words = -(-bt["max_new"] // 64)
            bits = [w for a in bt["n"] for w in _tree(a, r)[0]]
            s["mask"] = torch.tensor([[_signed(w >> 64 * j & (1 << 64) - 1) for j in range(words)] for w in bits],
                                     dtype=torch.int64, device=DEV)
    if own:
        import shared_routed_expert_b200 as m
        lk, lv = (s["k"][0], s["v"][0]) if lead else (s["k"], s["v"])
        s["cache"] = m.make_kv_cache(lk, lv, s["ks"], s["vs"])
        s["seqs"] = m.make_kv_batch(bt["q_start"], bt["ctx_len"], bt["table"], bt["max_new"])
        if case["op"] == "attn":
            s["ws"] = m.alloc_tree_attention_workspace(s["cache"], case["n_q"], T)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"append": _append, "attn": _attn, "compact": _compact, "logprobs": _logprobs}[s["case"]["op"]](s)


def _held(s):
    """The cache as the values it holds (8-bit caches: E4M3 numbers, times one scale for all)."""
    f8 = s["case"]["kv"] == "e4m3"
    return [t.view(torch.float8_e4m3fn) if f8 else t for t in (s["k"], s["v"])]


def _append(s):
    c, bt = s["case"], s["batch"]
    if own:
        import shared_routed_expert_b200 as m
        m.moe_qk_norm_rope_append(s["cache"], s["seqs"], c["n_q"], c["rot"], 1e-5, s["qkv"], s["pos"], s["q_w"], s["k_w"],
                                  s["cos_sin"], s["q_out"])
        return [s["q_out"], *_held(s)]
    T, n_q, n_kv, d, half = bt["T"], c["n_q"], c["n_kv"], c["d"], c["rot"] // 2
    x = s["qkv"].view(T, n_q + 2 * n_kv, d).float()
    u = x[:, :n_q + n_kv]
    u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-5)
    u = u * torch.cat([s["q_w"].float().expand(n_q, d), s["k_w"].float().expand(n_kv, d)])
    cs = s["cos_sin"][s["pos"].long()][:, None]
    co, si = cs[..., :half], cs[..., half:]
    a, b = u[..., :half], u[..., half:2 * half]
    u = torch.cat([a * co - b * si, b * co + a * si, u[..., 2 * half:]], -1)
    s["q_out"].copy_(u[:, :n_q].reshape(T, -1))
    k, v = u[:, n_q:], x[:, n_q + n_kv:]
    page = bt["table"][s["seq"], s["at"] // c["page"]].long()
    slot = s["at"] % c["page"]
    f8 = c["kv"] == "e4m3"
    s["k"][page, :, slot] = _codes(k, s["ks"]) if f8 else k.to(torch.bfloat16)
    s["v"][page, :, slot] = _codes(v, s["vs"]) if f8 else v.to(torch.bfloat16)
    return [s["q_out"], *_held(s)]


def _wide(t, scale, dt):
    return (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).to(dt) * scale


def _attn(s):
    c, bt = s["case"], s["batch"]
    if own:
        import shared_routed_expert_b200 as m
        m.moe_tree_attention(s["cache"], s["seqs"], c["n_q"], s["q"], s["out"], s["ws"], tree_mask=s["mask"], lse=s["lse"])
        return [s["out"], s["lse"]]
    B, n, n_q, n_kv, d, P = c["B"], bt["max_new"], c["n_q"], c["n_kv"], c["d"], c["page"]
    G, T = n_q // n_kv, bt["T"]
    L = bt["table"].shape[1] * P
    at = bt["table"].long()

    def keys(t, scale):                                            # [B, n_kv, L, d]
        return _wide(t[at], scale, torch.float32).transpose(1, 2).reshape(B, n_kv, L, d)

    q = torch.cat([s["q"].float(), s["q"].new_zeros(1, n_q * d).float()])[bt["rows"]]
    q = q.view(B, n, n_kv, G, d).permute(0, 2, 1, 3, 4).reshape(B, n_kv, n * G, d)
    x = (q @ keys(s["k"], s["ks"]).transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(B, n_kv, n, G, L)
    j = torch.arange(L, device=DEV) - bt["ctx_len"][:, None]       # [B, L]: place among the new tokens, < 0 in the prefix
    i = torch.arange(n, device=DEV)
    inside = (j < bt["n_t"][:, None])[:, None]
    if s["mask"] is None:
        seen = (j[:, None] <= i[:, None]) & inside                 # [B, n, L]
    else:
        m = torch.cat([s["mask"], s["mask"].new_zeros(1, s["mask"].shape[1])])[bt["rows"]]
        jj = j.clamp(0, 64 * m.shape[2] - 1)[:, None].expand(B, n, L)
        bit = torch.gather(m, 2, jj // 64) >> (jj % 64) & 1
        seen = ((j < 0)[:, None] | (bit != 0)) & inside
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(B, n_kv, n * G, L) @ keys(s["v"], s["vs"])).view(B, n_kv, n, G, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    real = bt["rows"] < T
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, n, n_q * d)[real])
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(B, n, n_q)[real])
    return [s["out"], s["lse"]]


def _compact(s):
    c, bt = s["case"], s["batch"]
    if own:
        import shared_routed_expert_b200 as m
        m.moe_kv_compact(s["cache"], s["seqs"], s["accepted"], s["n_acc"], n_layers=c["layers"], layer_stride=s["k"].stride(0))
        return _held(s)
    ctx = bt["ctx_len"][:, None].long()
    src, dst = ctx + s["accepted"].long(), ctx + torch.arange(c["depth"], device=DEV)
    P, table = c["page"], bt["table"].long()
    sp, dp = torch.gather(table, 1, src // P), torch.gather(table, 1, dst // P)
    s["k"][:, dp, :, dst % P] = s["k"][:, sp, :, src % P]
    s["v"][:, dp, :, dst % P] = s["v"][:, sp, :, src % P]
    return _held(s)


def _logprobs(s):
    c = s["case"]
    if own:
        import shared_routed_expert_b200 as m
        m.moe_token_logprobs(s["logits"], s["targets"], s["lp"], s["ent"], s["ids"], s["top"])
        return [s["lp"], s["ent"], s["ids"], s["top"]]
    V, n = c["V"], c["top"]
    x = s["logits"].double()                                       # 64 bits: long sums, and rows with one likely token
    lp = x - torch.logsumexp(x, 1, keepdim=True)
    ent = -(lp.exp() * lp).sum(1)
    # ties go to the lowest id: the fp32 value's order in the high half of the key, the id's in the low half
    f = s["logits"].float().view(torch.int32).long()
    order = torch.where(f < 0, -(f & 0x7FFFFFFF), f)
    ids = torch.topk(order * (1 << 32) + (V - 1 - torch.arange(V, device=DEV)), n, dim=1).indices
    s["lp"].copy_(torch.gather(lp, 1, s["targets"].long()[:, None])[:, 0])
    s["ent"].copy_(ent)
    s["ids"].copy_(ids)
    s["top"].copy_(torch.gather(lp, 1, ids))
    return [s["lp"], s["ent"], s["ids"], s["top"]]


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["op"] == "compact":
        return None                                                # bits are moved, nothing is computed
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_append(s):
    c, bt = s["case"], s["batch"]
    n_q, n_kv, d, half = c["n_q"], c["n_kv"], c["d"], c["rot"] // 2
    out = torch.empty(bt["T"], n_q, d, dtype=torch.float64, device=DEV)
    f8 = c["kv"] == "e4m3"
    k64, v64 = [(t.view(torch.float8_e4m3fn) if f8 else t).double() for t in (s["k"], s["v"])]
    for h in range(n_q + 2 * n_kv):
        x = s["qkv"][:, h * d:(h + 1) * d].double()
        if h < n_q + n_kv:
            x = x / torch.sqrt((x * x).sum(1, keepdim=True) / d + 1e-5) * (s["q_w"] if h < n_q else s["k_w"]).double()
            co, si = s["cos_sin"].double()[s["pos"].long()].split(half, 1) if half else (x[:, :0], x[:, :0])
            x = torch.cat([x[:, :half] * co - x[:, half:2 * half] * si, x[:, half:2 * half] * co + x[:, :half] * si,
                           x[:, 2 * half:]], 1)
        if h < n_q:
            out[:, h] = x
            continue
        to, scale, hh = (k64, s["ks"], h - n_q) if h < n_q + n_kv else (v64, s["vs"], h - n_q - n_kv)
        x = (x / scale).clamp(-448.0, 448.0) if f8 else x
        row = 0
        for b, (n, ctx) in enumerate(zip(bt["n"], bt["ctx"])):
            slots = torch.arange(ctx, ctx + n, device=DEV)
            to[bt["table"][b].long()[slots // c["page"]], hh, slots % c["page"]] = x[row:row + n]
            row += n
    return [out.view(bt["T"], -1), k64, v64]


def _exact_attn(s):
    c, bt = s["case"], s["batch"]
    n_q, n_kv, d, P = c["n_q"], c["n_kv"], c["d"], c["page"]
    out = torch.zeros(bt["T"], n_q, d, dtype=torch.float64, device=DEV)
    lse = torch.full((bt["T"], n_q), -math.inf, dtype=torch.float64, device=DEV)
    row = 0
    for b, (n, ctx) in enumerate(zip(bt["n"], bt["ctx"])):
        slots = torch.arange(ctx + n, device=DEV)
        page, off = bt["table"][b].long()[slots // P], slots % P
        seen = torch.ones(n, ctx + n, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            seen[:, ctx:] = torch.tril(torch.ones(n, n, dtype=torch.bool, device=DEV))
        else:
            m = s["mask"][row:row + n]
            for j in range(n):
                seen[:, ctx + j] = (m[:, j // 64] >> (j % 64)) & 1 != 0
        for h in range(n_kv):
            K, V = _wide(s["k"][page, h, off], 1.0, torch.float64) * s["ks"], _wide(s["v"][page, h, off], 1.0, torch.float64) * s["vs"]
            for qh in range(h * n_q // n_kv, (h + 1) * n_q // n_kv):
                x = s["q"][row:row + n, qh * d:(qh + 1) * d].double() @ K.T / math.sqrt(d)
                x[~seen] = -math.inf
                z = torch.logsumexp(x, 1)
                out[row:row + n, qh] = torch.nan_to_num(torch.exp(x - z[:, None])) @ V
                lse[row:row + n, qh] = z
        row += n
    return [out.view(bt["T"], -1), lse]


def _exact_logprobs(s):
    lp = torch.empty_like(s["lp"], dtype=torch.float64)
    ent = torch.empty_like(lp)
    for t0 in range(0, lp.numel(), 64):
        x = s["logits"][t0:t0 + 64].double()
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(1)
        ent[t0:t0 + 64] = torch.log(z) + (e * (m - x)).sum(1) / z
        lp[t0:t0 + 64] = x.gather(1, s["targets"][t0:t0 + 64].long()[:, None])[:, 0] - m[:, 0] - torch.log(z)
    return [lp, ent, None, None]
