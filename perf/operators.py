"""What the serving operators are measured on: page tables from request
lengths, the append of new keys and values to a paged cache, and the
attention of a batch of requests over one shared, long prefix (read once for
all of them) and their own tokens behind it.

The setting is a group of rollouts: one long prompt, many continuations.  The
prompt's keys lie in pages that every request reads; what a request adds lies
in pages of its own.  A serving step builds the page tables of the new
tokens, writes their keys and values to the cache, and attends.  Head counts,
head dimensions and lengths are those of the package's workloads
(``long_context_sparse_gb300.synth.WORKLOADS``): 8 heads of 128, 16 or 64
heads of 512 (one key and one value shared by all heads), 1k to 1M tokens.

``own = False`` runs the plain form (elementary torch operations in fp32),
``own = True`` the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step of a 64-rollout group: latency of one small launch
        dict(name="tables_decode", op="tables", batch=64, page=64, new_lo=1, new_hi=1,
             cached_hi=2048, pad=0, lens=1),
        # admission of many ragged prompts at once, some requests idle
        dict(name="tables_prompts", op="tables", batch=2047, page=16, new_lo=0, new_hi=1023,
             cached_hi=777, pad=37, lens=2),
        # one decode step's keys (one latent tensor: K = V)
        dict(name="append_decode", op="append", tokens=64, page=64, dim=512, kv=1, pad=0),
        # a whole 128k prompt written to the cache, keys and values apart
        dict(name="append_prompt", op="append", tokens=131071, page=64, dim=512, kv=2, pad=1),
        # one request, one token, a short prompt of odd length: the smallest call
        dict(name="attn_single", op="attn", batch=1, heads=16, dim=512, kv=1, page=64,
             prefix=1021, q_lo=1, q_hi=1, own_hi=7, pad=0, lens=3),
        # the small configuration: 8 heads of 128, keys and values apart
        dict(name="attn_tiny", op="attn", batch=5, heads=8, dim=128, kv=2, page=16,
             prefix=1000, q_lo=1, q_hi=1, own_hi=300, pad=3, lens=4),
        # an ordinary decode step of a small group behind a 16k prompt
        dict(name="attn_group16", op="attn", batch=16, heads=64, dim=512, kv=1, page=64,
             prefix=16384, q_lo=1, q_hi=1, own_hi=1024, pad=0, lens=5),
        # several draft tokens a request (speculative decoding), ragged, d = 256
        dict(name="attn_drafts", op="attn", batch=24, heads=16, dim=256, kv=2, page=32,
             prefix=65535, q_lo=1, q_hi=8, own_hi=513, pad=5, lens=6),
        # a 1M-token prompt, few rollouts: bound by reading the prompt once
        dict(name="attn_long", op="attn", batch=8, heads=16, dim=512, kv=1, page=128,
             prefix=1048576, q_lo=1, q_hi=1, own_hi=4096, pad=0, lens=7),
        # ragged prompts' ends behind a shared 16k prompt: many query tokens
        dict(name="attn_prompts", op="attn", batch=4, heads=16, dim=512, kv=2, page=64,
             prefix=16384, q_lo=100, q_hi=700, own_hi=700, pad=0, lens=8),
        # a 64-rollout group behind a 128k prompt, 64 heads: the largest
        dict(name="attn_group64", op="attn", batch=64, heads=64, dim=512, kv=1, page=64,
             prefix=131072, q_lo=1, q_hi=1, own_hi=2048, pad=0, lens=9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1 << 30)
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    if op == "tables":
        batch = _log(rng, 1, 2047)
        lo = rng.choice([0, 1])
        return dict(op=op, batch=batch, page=page, new_lo=lo, new_hi=_log(rng, 1, 1023),
                    cached_hi=_log(rng, 1, 4096), pad=pad, lens=lens)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 131071), page=page, dim=rng.choice([128, 256, 512]),
                    kv=rng.choice([1, 2]), pad=pad)
    heads = rng.choice([1, 5, 8, 16, 16, 24, 64, 64, 128])
    dim = rng.choice([128, 256, 512, 512])
    batch = _log(rng, 1, 64)
    q_hi = rng.choice([1, 1, _log(rng, 1, 512)])
    q_hi = max(1, min(q_hi, 32768 // (batch * heads)))
    rows = batch * q_hi * heads
    prefix = _log(rng, 1, max(2, min(1 << 20, (1 << 29) // rows)))
    return dict(op=op, batch=batch, heads=heads, dim=dim, kv=rng.choice([1, 2]), page=page,
                prefix=prefix, q_lo=rng.choice([0, 1]) if q_hi > 1 else 1, q_hi=q_hi,
                own_hi=max(q_hi, _log(rng, 1, 4096)), pad=pad, lens=lens)


def _lens(case):
    """The requests' lengths, before the seed shuffles their order: for tables
    (cached, new) and for attn (new, all own tokens) of each request."""
    r = random.Random(case["lens"])
    if case["op"] == "tables":
        return [(r.randrange(case["cached_hi"] + 1), r.randint(case["new_lo"], case["new_hi"]))
                for _ in range(case["batch"])]
    out = []
    for _ in range(case["batch"]):
        q = r.randint(case["q_lo"], case["q_hi"])
        out.append((q, r.randint(q, max(q, case["own_hi"]))))
    return out


def _pages(n, page):
    return -(-n // page)


# ----------------------------------------------------------------- states


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"tables": _prepare_tables, "append": _prepare_append,
            "attn": _prepare_attn}[case["op"]](case, seed, gen)


def _prepare_tables(case, seed, gen):
    page = case["page"]
    lens = _lens(case)
    random.Random(seed).shuffle(lens)
    have = [_pages(c, page) for c, _ in lens]
    need = [_pages(c + n, page) for c, n in lens]
    new_pages = sum(need) - sum(have)
    tokens = sum(n for _, n in lens)
    n_pages = sum(need) + 7
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    width = max(1, max(need))
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
    # the pages that the requests hold already
    h = torch.tensor(have, device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < h[:, None]
    table[held] = perm[: sum(have)]
    s = dict(op="tables", page=page, batch=case["batch"], tokens=tokens, new_pages=new_pages,
             cached=_i32([c for c, _ in lens]), new=_i32([n for _, n in lens]),
             free=perm[sum(have):].contiguous(), table=table,
             slots=torch.empty(max(1, tokens + case["pad"]), dtype=torch.int32, device=DEV))
    if own:
        import long_context_sparse_gb300 as dsa
        s["cfg"] = dsa.ServeConfig(n_pages=n_pages, page_size=page, batch=case["batch"],
                                   max_blocks=width, max_tokens=s["slots"].numel())
        s["ws"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_TABLES, DEV)
        s["out"] = dsa.PageTables(
            block_table=table, slot_map=s["slots"],
            cu_tokens=torch.empty(case["batch"] + 1, dtype=torch.int32, device=DEV),
            seq_lens=torch.empty(case["batch"], dtype=torch.int32, device=DEV),
            pages_taken=torch.empty(1, dtype=torch.int32, device=DEV))
    return s


def _prepare_append(case, seed, gen):
    page, dim, tokens = case["page"], case["dim"], case["tokens"]
    n_pages = _pages(tokens, page) + 3
    slots = torch.randperm(n_pages, generator=gen, device=DEV)
    slots = (slots[:, None] * page + torch.arange(page, device=DEV)[None, :]).reshape(-1)
    slots = torch.cat([slots[:tokens], slots.new_full((case["pad"],), -1)]).to(torch.int32)

    def rows(n):
        return torch.randn((n, dim), generator=gen, device=DEV).to(torch.bfloat16)

    s = dict(op="append", tokens=tokens, kv=case["kv"], dim=dim, slots=slots.contiguous(),
             new=[rows(tokens + case["pad"]) for _ in range(case["kv"])],
             pages=[rows(n_pages * page).view(n_pages, page, dim) for _ in range(case["kv"])])
    if own:
        import long_context_sparse_gb300 as dsa
        s["cfg"] = dsa.ServeConfig(n_pages=n_pages, page_size=page, batch=1, max_blocks=n_pages,
                                   max_tokens=slots.numel(), d_qk=dim, d_v=dim)
        s["ws"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_APPEND, DEV)
    return s


def _prepare_attn(case, seed, gen):
    page, dim, heads, prefix = case["page"], case["dim"], case["heads"], case["prefix"]
    lens = _lens(case)
    random.Random(seed).shuffle(lens)
    batch = case["batch"]
    tokens = sum(q for q, _ in lens)
    total = max(1, tokens + case["pad"])
    n_prefix = _pages(prefix, page)
    width = max(1, max(_pages(n, page) for _, n in lens))
    n_own = [_pages(n, page) for _, n in lens]
    n_pages = n_prefix + sum(n_own) + 3
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < torch.tensor(n_own, device=DEV)[:, None]
    table[held] = perm[n_prefix:n_prefix + sum(n_own)]

    def cache():
        return torch.randn((n_pages, page, dim), generator=gen, device=DEV,
                           dtype=torch.bfloat16)

    k = cache()
    v = k if case["kv"] == 1 else cache()
    # scores of standard deviation 2 at the default scale 1/sqrt(dim)
    q = (2 * torch.randn((total, heads, dim), generator=gen, device=DEV)).to(torch.bfloat16)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    s = dict(op="attn", page=page, dim=dim, heads=heads, prefix=prefix, batch=batch,
             tokens=tokens, kv=case["kv"], q=q, k=k, v=v, lens=lens, q_max=max(1, max(x for x, _ in lens)),
             own_max=max(1, max(n for _, n in lens)), n_pages=n_pages,
             prefix_table=perm[:n_prefix].contiguous(), table=table,
             seq_lens=_i32([n for _, n in lens]), cu=_i32(cu),
             o=torch.zeros((total, heads, dim), dtype=torch.bfloat16, device=DEV),
             lse=torch.zeros((total, heads), dtype=torch.float32, device=DEV))
    if own:
        import long_context_sparse_gb300 as dsa
        s["cfg"] = dsa.ServeConfig(n_pages=n_pages, page_size=page, batch=batch, max_blocks=width,
                                   max_tokens=total, attn_heads=heads, d_qk=dim, d_v=dim)
        s["ws"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_PREFIX, DEV)
    return s


# -------------------------------------------------------------------- run


def run(state):
    return {"tables": _run_tables, "append": _run_append, "attn": _run_attn}[state["op"]](state)


def _run_tables(s):
    if own:
        import long_context_sparse_gb300 as dsa
        r = dsa.build_page_tables(s["cfg"], s["cached"], s["new"], s["free"], s["table"],
                                  out=s["out"], ws=s["ws"])
        return dict(block_table=r.block_table, slot_map=r.slot_map, cu_tokens=r.cu_tokens,
                    seq_lens=r.seq_lens, pages_taken=r.pages_taken)
    page, batch, tokens = s["page"], s["batch"], s["tokens"]
    cached, new = s["cached"].long(), s["new"].long()
    ids = torch.arange(batch, device=DEV)
    have = (cached + page - 1) // page
    add = (cached + new + page - 1) // page - have
    end = torch.cumsum(add, 0)
    # pages from the free list, in the order of the requests
    req = torch.repeat_interleave(ids, add, output_size=s["new_pages"])
    j = torch.arange(s["new_pages"], device=DEV)
    s["table"][req, have[req] + j - (end - add)[req]] = s["free"][: s["new_pages"]]
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    req = torch.repeat_interleave(ids, new, output_size=tokens)
    pos = cached[req] + torch.arange(tokens, device=DEV) - cu[req]
    s["slots"][:tokens] = s["table"][req, pos // page] * page + (pos % page).to(torch.int32)
    s["slots"][tokens:] = -1
    return dict(block_table=s["table"], slot_map=s["slots"], cu_tokens=cu.to(torch.int32),
                seq_lens=(cached + new).to(torch.int32), pages_taken=end[-1:].to(torch.int32))


def _run_append(s):
    if own:
        import long_context_sparse_gb300 as dsa
        dsa.append_cache(s["cfg"], s["slots"], s["new"][0], s["pages"][0],
                         v_new=s["new"][1] if s["kv"] == 2 else None,
                         v_pages=s["pages"][1] if s["kv"] == 2 else None, ws=s["ws"])
        return s["pages"]
    at = s["slots"][: s["tokens"]].long()
    for new, pages in zip(s["new"], s["pages"]):
        pages.view(-1, s["dim"])[at] = new[: s["tokens"]]
    return s["pages"]


def _run_attn(s):
    if own:
        import long_context_sparse_gb300 as dsa
        o, lse = dsa.prefix_attn(s["cfg"], s["q"], s["k"], s["prefix_table"], s["prefix"],
                                 s["table"], s["seq_lens"], s["cu"],
                                 v_pages=s["v"] if s["kv"] == 2 else None,
                                 o=s["o"], lse=s["lse"], ws=s["ws"])
        return [o, lse]
    page, dim, heads, tokens, batch = s["page"], s["dim"], s["heads"], s["tokens"], s["batch"]
    if tokens == 0:
        return [s["o"], s["lse"]]
    scale = 1.0 / math.sqrt(dim)
    k, v = s["k"].view(-1, dim), s["v"].view(-1, dim)
    # the prefix: every row against the same keys
    pos = torch.arange(s["prefix"], device=DEV)
    at = s["prefix_table"].long()[pos // page] * page + pos % page
    kp = k[at].float()
    vp = kp if s["kv"] == 1 else v[at].float()
    q = s["q"][:tokens].float() * scale
    sp = q.view(tokens * heads, dim) @ kp.T
    # the requests' own tokens, padded to the longest; token i of a request
    # sees the own positions up to its own
    cu, n = s["cu"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    req = torch.repeat_interleave(torch.arange(batch, device=DEV), new, output_size=tokens)
    row = torch.arange(tokens, device=DEV) - cu[req]
    qb = q.new_zeros((batch, s["q_max"], heads, dim))
    qb[req, row] = q
    pos = torch.arange(s["own_max"], device=DEV)
    at = s["table"].long()[:, pos // page].clamp(min=0) * page + pos % page
    ko = k[at].float()
    vo = ko if s["kv"] == 1 else v[at].float()
    so = torch.bmm(qb.view(batch, -1, dim), ko.transpose(1, 2))
    so = so.view(batch, s["q_max"], heads, -1)[req, row]
    seen = pos[None, :] <= ((n - new)[req] + row)[:, None]
    so = so.masked_fill(~seen[:, None, :], float("-inf")).view(tokens * heads, -1)
    m = torch.maximum(sp.amax(1), so.amax(1))[:, None]
    sp = (sp - m).exp_()
    so = (so - m).exp_()
    total = sp.sum(1) + so.sum(1)
    pb = so.new_zeros((batch, s["q_max"], heads, so.shape[1]))
    pb[req, row] = so.view(tokens, heads, -1)
    ob = torch.bmm(pb.view(batch, -1, so.shape[1]), vo).view(batch, s["q_max"], heads, dim)
    o = (sp @ vp).view(tokens, heads, dim) + ob[req, row]
    s["o"][:tokens] = (o / total.view(tokens, heads, 1)).to(torch.bfloat16)
    s["lse"][:tokens] = (m[:, 0] + total.log()).view(tokens, heads)
    return [s["o"], s["lse"]]


# ------------------------------------------------------------------- work


def work(case):
    if case["op"] == "tables":
        lens, page = _lens(case), case["page"]
        new_pages = sum(_pages(c + n, page) - _pages(c, page) for c, n in lens)
        tokens = sum(n for _, n in lens) + case["pad"]
        # lengths in; table entries, slots, offsets and lengths out
        return dict(bytes=4 * (4 * case["batch"] + 2 * new_pages + tokens + 2), flops=0)
    if case["op"] == "append":
        return dict(bytes=case["tokens"] * (4 + 4 * case["kv"] * case["dim"]) + 4 * case["pad"],
                    flops=0)
    lens = _lens(case)
    tokens = sum(q for q, _ in lens)
    keys = case["prefix"] + sum(n for q, n in lens if q)
    rows = case["heads"] * tokens
    seen = case["heads"] * sum(q * case["prefix"] + sum(range(n - q + 1, n + 1)) for q, n in lens)
    return dict(bytes=rows * (4 * case["dim"] + 4) + 2 * case["kv"] * case["dim"] * keys,
                flops=4 * seen * case["dim"])


# ------------------------------------------------------------------ exact


def exact(case, seed):
    """The definitions in 64 bits, one request or one token at a time."""
    s = prepare(case, seed)
    if case["op"] == "tables":
        cached, new, free = (s[n].tolist() for n in ("cached", "new", "free"))
        table, slots, cu = s["table"].tolist(), [], [0]
        taken = 0
        for b in range(s["batch"]):
            for i in range(cached[b], cached[b] + new[b]):
                p, r = divmod(i, s["page"])
                if r == 0:
                    table[b][p] = free[taken]
                    taken += 1
                slots.append(table[b][p] * s["page"] + r)
            cu.append(len(slots))
        slots += [-1] * (s["slots"].numel() - len(slots))
        return dict(block_table=torch.tensor(table), slot_map=torch.tensor(slots),
                    cu_tokens=torch.tensor(cu),
                    seq_lens=torch.tensor([c + n for c, n in zip(cached, new)]),
                    pages_taken=torch.tensor([taken]))
    if case["op"] == "append":
        if s["slots"].numel() > 4096:  # a copy, one token at a time
            return None
        for i, at in enumerate(s["slots"].tolist()):
            for new, pages in zip(s["new"], s["pages"]):
                if at >= 0:
                    pages[at // case["page"], at % case["page"]] = new[i]
        return [p.double() for p in s["pages"]]
    if work(case)["flops"] > 4e12:  # double-precision products: over 20 s
        return None
    o, lse = s["o"].double(), s["lse"].double()
    first = 0
    pages = s["table"].tolist()
    for b, (n_new, n_own) in enumerate(s["lens"]):
        for i in range(n_new):
            see = n_own - n_new + i + 1
            q = s["q"][first + i].double() / math.sqrt(s["dim"])
            own_pages = torch.tensor(pages[b][: _pages(see, s["page"])], device=DEV, dtype=torch.long)
            ks = [(s["k"], s["v"], own_pages, see),
                  (s["k"], s["v"], s["prefix_table"].long(), s["prefix"])]
            m = torch.full((s["heads"], 1), -math.inf, dtype=torch.float64, device=DEV)
            t = torch.zeros_like(m)
            acc = torch.zeros((s["heads"], s["dim"]), dtype=torch.float64, device=DEV)
            for kk, vv, ids, length in ks:
                step = 65536 // s["page"]
                for p in range(0, ids.numel(), step):
                    left = length - p * s["page"]
                    a = kk[ids[p:p + step]].reshape(-1, s["dim"])[:left].double()
                    c = a if kk is vv else vv[ids[p:p + step]].reshape(-1, s["dim"])[:left].double()
                    x = q @ a.T
                    top = torch.maximum(m, x.amax(1, keepdim=True))
                    e = torch.exp(x - top)
                    f = torch.exp(m - top)
                    acc = acc * f + e @ c
                    t = t * f + e.sum(1, keepdim=True)
                    m = top
            o[first + i] = acc / t
            lse[first + i] = (m + torch.log(t))[:, 0]
        first += n_new
    return [o, lse]
