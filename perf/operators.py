"""Cases of the batched-request operators: block tables from request lengths
(wf_batch_tables), the cache write through them (wf_batch_append) and the
attention of a batch whose requests share a prefix (wf_batch_attn).

`run` computes a case in plain torch operations where `own` is false and
through the library's calls where it is true.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of requests between two decoding steps: nothing but latency
        dict(name="tables_few", kind="tables", page=16, batch=5, lens=1, cached=700, fresh=1, prefix=300),
        # a full decoding batch, one new token each
        dict(name="tables_decode", kind="tables", page=16, batch=1024, lens=2, cached=4000, fresh=1, prefix=4680),
        # requests that enter with ragged prompts: about 65000 new tokens
        dict(name="tables_prompts", kind="tables", page=32, batch=61, lens=3, cached=130, fresh=2200, prefix=0),
        # one decoding step's rows, 40 query heads on 8 key heads
        dict(name="append_decode", kind="append", heads=40, kv_heads=8, dim=128, page=16, batch=32, lens=4,
             cached=900, fresh=1, prefix=1000),
        # two branches of a 4-chunk round of the 1.3B shape: 37440 tokens, 12 heads
        dict(name="append_round", kind="append", heads=12, kv_heads=12, dim=128, page=64, batch=2, lens=0,
             cached=0, fresh=18720, prefix=32760),
        # one request, one token, a short history: latency
        dict(name="attn_one", kind="attn", heads=12, kv_heads=12, dim=128, page=16, batch=1, lens=0, cached=33,
             fresh=1, prefix=300, block=1),
        # an ordinary decoding step on a common prefix
        dict(name="attn_decode", kind="attn", heads=32, kv_heads=8, dim=128, page=16, batch=64, lens=5, cached=1000,
             fresh=1, prefix=8192, block=1),
        # many candidates of one long history, one key head per query head
        dict(name="attn_decode_long", kind="attn", heads=12, kv_heads=12, dim=128, page=64, batch=96, lens=6,
             cached=4000, fresh=1, prefix=32760, block=1),
        # a few proposed tokens per request, groups of five heads, 64-wide heads
        dict(name="attn_proposed", kind="attn", heads=40, kv_heads=8, dim=64, page=32, batch=33, lens=7, cached=600,
             fresh=5, prefix=4680, block=1),
        # ragged prompts after a common instruction, token-causal
        dict(name="attn_prompts", kind="attn", heads=24, kv_heads=4, dim=128, page=16, batch=7, lens=8, cached=0,
             fresh=2600, prefix=1000, block=1),
        # two branches denoise one chunk each after seven shared chunks and one of their own (1.3B shape)
        dict(name="attn_round", kind="attn", heads=12, kv_heads=12, dim=128, page=128, batch=2, lens=0, cached=4680,
             fresh=4680, prefix=32760, block=4680),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: tables and appends of 1 to 65000 new tokens, attention of decoding steps, short proposals,
    ragged prompts and chunk rounds, with up to 32760 shared tokens."""
    kind = rng.choice(("tables", "append", "attn", "attn", "attn"))
    page = rng.choice((16, 32, 64, 128))
    lens = rng.randrange(1, 1 << 20)
    if kind == "tables":
        batch = _log(rng, 1, 1024)
        return dict(kind=kind, page=page, batch=batch, lens=lens, cached=_log(rng, 1, 4000),
                    fresh=rng.choice((1, _log(rng, 2, max(2, 60000 // batch)))), prefix=rng.choice((0, _log(rng, 1, 32760))))
    heads, kv_heads = rng.choice(((12, 12), (40, 40), (40, 8), (32, 8), (24, 4), (16, 1), (28, 4), (3, 3)))
    dim = rng.choice((64, 128))
    case = dict(kind=kind, heads=heads, kv_heads=kv_heads, dim=dim, page=page, lens=lens)
    if kind == "append":
        batch = _log(rng, 1, 256)
        fresh = rng.choice((1, _log(rng, 1, max(1, 12000 // batch))))
        return dict(case, batch=batch, cached=_log(rng, 1, 2000), fresh=fresh, prefix=_log(rng, 1, 32760))
    form = rng.choice(("decode", "decode", "proposed", "prompts", "round"))
    if form == "decode":
        case.update(batch=_log(rng, 1, 96), cached=_log(rng, 1, 4000), fresh=1, prefix=rng.choice((0, _log(rng, 1, 32760))),
                    block=1)
    elif form == "proposed":
        case.update(batch=_log(rng, 1, 48), cached=_log(rng, 1, 1500), fresh=_log(rng, 2, 24), prefix=_log(rng, 1, 9000),
                    block=1)
    elif form == "prompts":
        case.update(batch=_log(rng, 1, 7), cached=rng.choice((0, _log(rng, 1, 1000))), fresh=_log(rng, 30, 2600),
                    prefix=rng.choice((0, _log(rng, 1, 4680))), block=1)
    else:
        block = _log(rng, 20, 2340)
        case.update(batch=rng.choice((1, 2, 3)), lens=0, cached=block * rng.choice((0, 1, 2)),
                    fresh=block * rng.choice((1, 2)), prefix=rng.choice((0, _log(rng, 1, 16380))), block=block)
    return case


def _lengths(case):
    """(cached, fresh) of every request.  lens 0: all alike; otherwise cached spread over 0 .. the case's number and
    fresh over 1 .. the case's number."""
    n = case["batch"]
    if case["lens"] == 0:
        return [case["cached"]] * n, [case["fresh"]] * n
    r = random.Random(case["lens"])
    return [r.randint(0, case["cached"]) for _ in range(n)], [r.randint(1, case["fresh"]) for _ in range(n)]


def _pages(tokens, page):
    return -(-tokens // page)


def _visible(case, cached, fresh):
    """Own keys that each new token of a request sees."""
    g = case["block"]
    return [min(cached + fresh, ((cached + i) // g + 1) * g) for i in range(fresh)]


def work(case):
    cached, fresh = _lengths(case)
    page, new = case["page"], sum(fresh)
    if case["kind"] == "tables":
        pages = sum(_pages(c + f, page) - _pages(c, page) for c, f in zip(cached, fresh))
        # lengths in; free pages in and table entries out; token starts; slot and position of every new token
        return {"bytes": 8 * case["batch"] + 8 * pages + 4 * (case["batch"] + 1) + 8 * new, "flops": 0}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if case["kind"] == "append":
        row = 2 * (heads + 2 * kv_heads) * dim * 2  # Q, K, V read; Q', K', V written
        return {"bytes": new * (row + 4 * dim + 4), "flops": new * 3 * (heads + kv_heads) * dim}
    pairs = sum(sum(_visible(case, c, f)) + f * case["prefix"] for c, f in zip(cached, fresh))
    keys = case["prefix"] + sum(cached) + new
    return {"bytes": 2 * new * heads * dim * 2 + 4 * new * heads + 2 * keys * kv_heads * dim * 2,
            "flops": 4 * dim * heads * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    cached, fresh = _lengths(case)
    page, batch, prefix, new = case["page"], case["batch"], case["prefix"], sum(fresh)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    have = [_pages(c, page) for c in cached]
    need = [_pages(c + f, page) for c, f in zip(cached, fresh)]
    cols = max(need)
    prefix_pages = _pages(prefix, page)
    spare = 7
    pool_pages = prefix_pages + sum(need) + spare
    order = torch.randperm(pool_pages, generator=g, device="cuda").to(torch.int32)
    s = dict(case=case, new=new)
    s["cached"] = torch.tensor(cached, dtype=torch.int32, device="cuda")
    s["fresh"] = torch.tensor(fresh, dtype=torch.int32, device="cuda")
    s["prefix_len"] = torch.tensor([prefix], dtype=torch.int32, device="cuda")
    s["prefix_table"] = order[:max(prefix_pages, 1)].contiguous()
    # the pages that the requests hold already, request by request, then the free ones
    held = order[prefix_pages:prefix_pages + sum(have)]
    haves = torch.tensor(have, device="cuda")
    table = torch.zeros(batch, cols, dtype=torch.int32, device="cuda")
    col = torch.arange(cols, device="cuda").expand(batch, cols)
    table[col < haves[:, None]] = held
    s["table"] = table
    s["free_head"] = torch.tensor([3], dtype=torch.int32, device="cuda")  # three were taken before
    s["free_pages"] = torch.cat([order[:3], order[prefix_pages + sum(have):]]).contiguous()
    if own:
        from chunk_causal_attention_block_b200 import wf
        s["desc"] = wf.make_batch_desc(case.get("heads", 1), case.get("kv_heads", 1), case.get("dim", 128), page,
                                       pool_pages, max_requests=batch, max_tokens=new, max_request_pages=cols,
                                       max_prefix_pages=prefix_pages, block_tokens=case.get("block", 1))
        s["plan"] = torch.zeros(wf.wf_batch_plan_bytes(s["desc"]), dtype=torch.uint8, device="cuda")
    for name, n in (("token_start", batch + 1), ("slot_map", new), ("positions", new), ("free_head_out", 1)):
        s[name] = torch.zeros(n, dtype=torch.int32, device="cuda")
    if case["kind"] == "tables":
        return s
    (_tables_own if own else _tables)(s)  # once a step, for all layers
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(BF16)  # noqa: E731
    s["q"] = rand(new, heads, dim)
    if case["kind"] == "append":
        s["k"], s["v"] = rand(new, kv_heads, dim), rand(new, kv_heads, dim)
        s["q_rot"] = torch.empty_like(s["q"])
        rate = 10000.0 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float64) / (dim // 2))
        angle = s["positions"].double()[:, None] * rate
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        s["k_pool"] = torch.zeros(pool_pages * page, kv_heads, dim, dtype=BF16, device="cuda")
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        return s
    s["k_pool"], s["v_pool"] = rand(pool_pages * page, kv_heads, dim), rand(pool_pages * page, kv_heads, dim)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(heads, new, dtype=torch.float32, device="cuda")
    if own:
        s["workspace"] = torch.zeros(wf.wf_batch_workspace_bytes(s["desc"]), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"tables": _tables_own, "append": _append_own, "attn": _attn_own}[kind](s)
    return {"tables": _tables, "append": _append, "attn": _attn}[kind](s)


def _tables_own(s):
    from chunk_causal_attention_block_b200 import wf
    wf.wf_batch_tables(s["desc"], s["cached"], s["fresh"], s["prefix_len"], s["free_pages"], s["free_head"],
                       s["free_head_out"], s["table"], s["token_start"], s["slot_map"], s["positions"], s["plan"],
                       stream=torch.cuda.current_stream())
    return s["table"], s["token_start"], s["slot_map"], s["positions"], s["free_head_out"]


def _append_own(s):
    from chunk_causal_attention_block_b200 import wf
    wf.wf_batch_append(s["desc"], s["plan"], s["slot_map"], s["k"], s["v"], s["k_pool"], s["v_pool"], q=s["q"],
                       rope=s["rope"], q_rot=s["q_rot"], stream=torch.cuda.current_stream())
    return s["q_rot"], s["k_pool"], s["v_pool"]


def _attn_own(s):
    from chunk_causal_attention_block_b200 import wf
    wf.wf_batch_attn(s["desc"], s["plan"], s["table"], s["prefix_table"], s["q"], s["k_pool"], s["v_pool"], s["out"],
                     s["lse"], workspace=s["workspace"], stream=torch.cuda.current_stream())
    return s["out"], s["lse"]


def _tables(s):
    page, new = s["case"]["page"], s["new"]
    cached, fresh, table = s["cached"].long(), s["fresh"].long(), s["table"]
    start = torch.cat([torch.zeros_like(fresh[:1]), fresh.cumsum(0)])
    have, need = (cached + page - 1) // page, (cached + fresh + page - 1) // page
    first = s["free_head"].long() + (need - have).cumsum(0) - (need - have)
    col = torch.arange(table.shape[1], device="cuda")
    is_new = (col >= have[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free_pages"].numel() - 1)
    table.copy_(torch.where(is_new, s["free_pages"][at], table))
    token = torch.arange(new, device="cuda")
    request = torch.searchsorted(start, token, right=True) - 1
    local = cached[request] + token - start[request]
    slot = table[request, local // page].long() * page + local % page
    s["token_start"].copy_(start)
    s["slot_map"].copy_(slot)
    s["positions"].copy_(s["prefix_len"].long() + local)
    s["free_head_out"].copy_(s["free_head"] + (need - have).sum())
    return table, s["token_start"], s["slot_map"], s["positions"], s["free_head_out"]


def _rotate(x, rope):
    even, odd = x.float()[..., 0::2], x.float()[..., 1::2]
    c, n = rope[:, None, :, 0], rope[:, None, :, 1]
    return torch.stack([even * c - odd * n, even * n + odd * c], -1).flatten(-2)


def _append(s):
    slot = s["slot_map"].long()
    s["k_pool"][slot] = _rotate(s["k"], s["rope"]).to(BF16)
    s["v_pool"][slot] = s["v"]
    s["q_rot"].copy_(_rotate(s["q"], s["rope"]))
    return s["q_rot"], s["k_pool"], s["v_pool"]


def _attn(s):
    """All requests at once, padded to the longest; the prefix is multiplied once for all of them."""
    case = s["case"]
    page, batch, prefix, block = case["page"], case["batch"], case["prefix"], case["block"]
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    group, rows = heads // kv_heads, max(_lengths(case)[1])
    cached, fresh, start = s["cached"].long(), s["fresh"].long(), s["token_start"].long()
    length = cached + fresh
    key = torch.arange(s["table"].shape[1] * page, device="cuda")
    k_own = s["k_pool"].view(-1, page, kv_heads, dim)[s["table"].long()].view(batch, -1, kv_heads, dim)
    v_own = s["v_pool"].view(-1, page, kv_heads, dim)[s["table"].long()].view(batch, -1, kv_heads, dim)
    here = (key < length[:, None])[:, :, None, None]
    k_own, v_own = k_own.float() * here, v_own.float() * here
    at = torch.arange(prefix, device="cuda")
    slots = s["prefix_table"].long()[at // page] * page + at % page
    k_pre, v_pre = s["k_pool"][slots].float(), s["v_pool"][slots].float()
    row = torch.arange(rows, device="cuda")
    token = (start[:-1, None] + row).clamp(max=s["new"] - 1)
    q = (s["q"].float() / math.sqrt(dim))[token].view(batch, rows, kv_heads, group, dim)
    p_pre = torch.einsum("bnkgd,pkd->kgbnp", q, k_pre)
    p_own = torch.einsum("bnkgd,blkd->kgbnl", q, k_own)
    seen = torch.minimum(length[:, None], ((cached[:, None] + row) // block + 1) * block)
    p_own.masked_fill_(key >= seen[:, :, None], -math.inf)
    top = p_own.amax(-1, keepdim=True)
    if prefix:
        top = torch.maximum(top, p_pre.amax(-1, keepdim=True))
    p_pre.sub_(top).exp_()
    p_own.sub_(top).exp_()
    total = p_pre.sum(-1) + p_own.sum(-1)
    o = torch.einsum("kgbnp,pkd->bnkgd", p_pre, v_pre) + torch.einsum("kgbnl,blkd->bnkgd", p_own, v_own)
    o = (o / total.permute(2, 3, 0, 1)[..., None]).reshape(batch * rows, heads, dim)
    lse = (top[..., 0] + total.log()).reshape(heads, batch * rows)
    live = (row < fresh[:, None]).reshape(-1)
    at = torch.arange(batch * rows, device="cuda")[live]
    s["out"].copy_(o[at])
    s["lse"].copy_(lse[:, at])
    return s["out"], s["lse"]


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    if case["kind"] == "tables":
        return None
    s = prepare(case, seed)
    cached, fresh = _lengths(case)
    page, prefix = case["page"], case["prefix"]
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    table = s["table"].tolist()
    if case["kind"] == "append":
        position = torch.tensor([prefix + c + i for c, f in zip(cached, fresh) for i in range(f)], device="cuda")
        slot = torch.tensor([table[b][(c + i) // page] * page + (c + i) % page
                             for b, (c, f) in enumerate(zip(cached, fresh)) for i in range(f)], device="cuda")
        rate = 10000.0 ** (-torch.arange(dim // 2, device="cuda", dtype=torch.float64) * 2 / dim)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), position.double()[:, None] * rate)
        spin = lambda x: torch.view_as_real(torch.view_as_complex(  # noqa: E731
            x.double().unflatten(-1, (dim // 2, 2))) * turn[:, None, :]).flatten(-2)
        k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
        k_pool[slot], v_pool[slot] = spin(s["k"]), s["v"].double()
        return spin(s["q"]), k_pool, v_pool
    group = heads // kv_heads
    tokens = lambda pages, n: torch.tensor([pages[i // page] * page + i % page for i in range(n)],  # noqa: E731
                                           device="cuda", dtype=torch.long)
    pre = tokens(s["prefix_table"].tolist(), prefix)
    k_pre, v_pre = s["k_pool"][pre].double(), s["v_pool"][pre].double()
    out = torch.empty(s["new"], heads, dim, dtype=torch.float64, device="cuda")
    lse = torch.empty(heads, s["new"], dtype=torch.float64, device="cuda")
    first = 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        mine = tokens(table[b], c + f)
        hide = torch.arange(prefix + c + f, device="cuda") >= prefix + torch.tensor(_visible(case, c, f), device="cuda")[:, None]
        for kv in range(kv_heads):
            keys = torch.cat([k_pre[:, kv], s["k_pool"][mine, kv].double()])
            values = torch.cat([v_pre[:, kv], s["v_pool"][mine, kv].double()])
            for h in range(kv * group, (kv + 1) * group):
                score = (s["q"][first:first + f, h].double() @ keys.T / math.sqrt(dim)).masked_fill(hide, -math.inf)
                lse[h, first:first + f] = score.logsumexp(-1)
                out[first:first + f, h] = score.softmax(-1) @ values
        first += f
    return out, lse
