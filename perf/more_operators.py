"""What the operators for drafting, scoring and forgetting are measured on.

A group of rollouts continues one long prompt over a paged cache.  Each step
may draft a tree of tokens for every request: the tree's mask is built once
(``build_tree``) and the rows attend the prompt, their request's own tokens
and their ancestors (``tree_attn``).  What each cached token received of the
attention is accumulated (``key_weights``), the tokens that received least are
dropped when a request passes its budget (``evict_cache``, ``release_pages``),
and the tokens' log probabilities, the entropies and the best alternatives
come from the logits (``token_logprobs``), with the gradient for the trainer
(``token_logprobs_bwd``).

Head counts, head dimensions and lengths are those of the package's workloads
and of the serving cases: 8 heads of 128, 16 or 64 heads of 512 (one key and
one value shared by all heads).  Vocabularies are generic.

``own = False`` runs the plain form (elementary torch operations in fp32),
``own = True`` the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one request drafts a small tree behind a short prompt: latency
        dict(name="tree_single", op="tree", batch=1, heads=16, dim=512, kv=1, page=64, prefix=1021,
             q_lo=7, q_hi=7, own_hi=40, pad=0, lens=1),
        # a group of 16 behind a 16k prompt, ragged trees of up to 31 tokens
        dict(name="tree_group16", op="tree", batch=16, heads=64, dim=512, kv=1, page=64,
             prefix=16384, q_lo=8, q_hi=31, own_hi=1024, pad=0, lens=2),
        # wide trees, keys and values apart, d = 256, an odd prompt, some padding
        dict(name="tree_wide", op="tree", batch=24, heads=16, dim=256, kv=2, page=32, prefix=65535,
             q_lo=33, q_hi=64, own_hi=2048, pad=5, lens=3),
        # the small configuration: weights of a handful of short requests
        dict(name="weights_tiny", op="weights", batch=5, heads=8, dim=128, page=16, q_lo=0, q_hi=7,
             own_hi=300, tree=True, pad=3, lens=4),
        # a decode step of a 64-rollout group: bound by reading the keys once
        dict(name="weights_decode", op="weights", batch=64, heads=64, dim=512, page=64, q_lo=1,
             q_hi=1, own_hi=8192, tree=False, pad=0, lens=5),
        # the last window of each of a few long prompts looks back at all of them
        dict(name="weights_window", op="weights", batch=6, heads=64, dim=512, page=128, q_lo=20,
             q_hi=64, own_hi=20000, tree=False, pad=0, lens=6),
        # a group of 64 back to a budget of 2048 tokens, half of its cache
        dict(name="evict_group", op="evict", batch=64, dim=512, kv=1, page=64, own_lo=1500,
             own_hi=4096, keep=2048, first=4, last=256, lens=7),
        # one long request, keys and values apart, back to a 32k budget
        dict(name="evict_long", op="evict", batch=1, dim=512, kv=2, page=64, own_lo=131071,
             own_hi=131071, keep=32768, first=16, last=1024, lens=8),
        # the sampled tokens of a 64-rollout step, with their alternatives
        dict(name="logp_decode", op="logp", rows=64, vocab=131072, dtype="bf16", n_top=20, pad=0,
             masked=0),
        # every token of a rollout, for the trainer; odd vocabulary, fp32
        dict(name="logp_rollout", op="logp", rows=4095, vocab=100277, dtype="fp32", n_top=5,
             pad=11, masked=0),
        # gradients of a short odd batch in half precision, padded rows
        dict(name="grad_short", op="grad", rows=301, vocab=50257, dtype="fp16", n_top=0, pad=0,
             masked=7),
        # gradients of a rollout's tokens: bound by reading and writing the logits
        dict(name="grad_rollout", op="grad", rows=8192, vocab=131072, dtype="bf16", n_top=0,
             pad=0, masked=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "weights", "evict", "logp", "grad"])
    page = rng.choice([16, 32, 64, 128])
    lens = rng.randrange(1 << 30)
    pad = rng.choice([0, 0, rng.randrange(1, 64)])
    if op in ("logp", "grad"):
        vocab = _log(rng, 1000, 200000)
        rows = _log(rng, 1, max(1, min(8192, (1 << 29) // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    n_top=rng.choice([0, 1, 5, 20, 64]) if op == "logp" else 0,
                    pad=rng.choice([0, rng.randrange(1, 128)]), masked=rng.choice([0, 3, 7]))
    dim = rng.choice([128, 256, 512, 512])
    if op == "evict":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 16, min(200000, 400000 // batch))
        return dict(op=op, batch=batch, dim=dim, kv=rng.choice([1, 2]), page=page,
                    own_lo=rng.choice([0, hi // 2]), own_hi=hi,
                    keep=max(1, int(hi * rng.choice([0.1, 0.25, 0.5, 0.75]))),
                    first=rng.choice([0, 1, 4]), last=rng.choice([0, 1, hi // 16]), lens=lens)
    heads = rng.choice([1, 5, 8, 16, 16, 24, 64, 64, 128])
    batch = _log(rng, 1, 64)
    q_hi = rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 64)])
    q_hi = max(1, min(q_hi, 32768 // (batch * heads)))
    q_lo = rng.choice([0, 1]) if q_hi > 1 else 1
    if op == "weights":
        most = max(q_hi, min(32768, 500000 // batch, (1 << 29) // (batch * q_hi * heads)))
        return dict(op=op, batch=batch, heads=heads, dim=dim, page=page, q_lo=q_lo, q_hi=q_hi,
                    own_hi=max(q_hi, _log(rng, 1, most)), tree=rng.choice([False, True]), pad=pad,
                    lens=lens)
    rows = batch * q_hi * heads
    prefix = rng.choice([0, 1, 1, 1]) * _log(rng, 1, max(2, min(1 << 19, (1 << 29) // rows)))
    return dict(op=op, batch=batch, heads=heads, dim=dim, kv=rng.choice([1, 2]), page=page,
                prefix=prefix, q_lo=q_lo, q_hi=q_hi, own_hi=max(q_hi, _log(rng, 1, 4096)), pad=pad,
                lens=lens)


def _lens(case):
    """The requests' lengths, before the seed shuffles their order: (new, all
    own tokens) of each, for evict (0, own tokens)."""
    r = random.Random(case["lens"])
    if case["op"] == "evict":
        return [(0, r.randint(case["own_lo"], case["own_hi"])) for _ in range(case["batch"])]
    out = []
    for _ in range(case["batch"]):
        q = r.randint(case["q_lo"], case["q_hi"])
        out.append((q, r.randint(q, max(q, case["own_hi"]))))
    return out


def _pages(n, page):
    return -(-n // page)


def _words(case):
    return _pages(case["q_hi"], 32)


# ----------------------------------------------------------------- states


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"tree": _prepare_tree, "weights": _prepare_weights, "evict": _prepare_evict,
            "logp": _prepare_logits, "grad": _prepare_logits}[case["op"]](case, seed, gen)


def _batch(case, seed, gen, n_prefix=0):
    """Requests over a shuffled cache: lengths, offsets, tables, parents."""
    page, batch = case["page"], case["batch"]
    lens = _lens(case)
    rnd = random.Random(seed)
    rnd.shuffle(lens)
    n_own = [_pages(n, page) for _, n in lens]
    width = max(1, max(n_own))
    n_pages = n_prefix + sum(n_own) + 3
    perm = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(width, device=DEV)[None, :] < torch.tensor(n_own, device=DEV)[:, None]
    table[held] = perm[n_prefix:n_prefix + sum(n_own)]
    tokens = sum(q for q, _ in lens)
    total = max(1, tokens + case.get("pad", 0))
    cu = [0]
    parents = []
    for q, _ in lens:
        cu.append(cu[-1] + q)
        # most drafted tokens follow one of the last few, some start anew
        parents += [i - 1 - min(i, int(rnd.expovariate(0.5))) for i in range(q)]
    parents += [-1] * (total - tokens)
    return dict(page=page, batch=batch, lens=lens, n_pages=n_pages, width=width, table=table,
                prefix_table=perm[:n_prefix].contiguous(), tokens=tokens, total=total,
                cu=_i32(cu), seq_lens=_i32([n for _, n in lens]), parents=_i32(parents),
                q_max=max(1, max(q for q, _ in lens)), own_max=max(1, max(n for _, n in lens)))


def _config(case, s):
    import long_context_sparse_gb300 as dsa
    return dsa.ServeConfig(n_pages=s["n_pages"], page_size=s["page"], batch=s["batch"],
                           max_blocks=s["width"], max_tokens=s["total"],
                           attn_heads=case.get("heads", 1), d_qk=case["dim"], d_v=case["dim"])


def _cache(s, dim, gen):
    return torch.randn((s["n_pages"], s["page"], dim), generator=gen, device=DEV,
                       dtype=torch.bfloat16)


def _queries(case, s, gen):
    # scores of standard deviation 2 at the default scale 1/sqrt(dim)
    return (2 * torch.randn((s["total"], case["heads"], case["dim"]), generator=gen,
                            device=DEV)).to(torch.bfloat16)


def _prepare_tree(case, seed, gen):
    n_prefix = _pages(case["prefix"], case["page"])
    s = _batch(case, seed, gen, n_prefix)
    s.update(op="tree", dim=case["dim"], heads=case["heads"], kv=case["kv"],
             prefix=case["prefix"], words=_words(case), k=_cache(s, case["dim"], gen))
    s["v"] = s["k"] if case["kv"] == 1 else _cache(s, case["dim"], gen)
    s["q"] = _queries(case, s, gen)
    s["bits"] = torch.zeros((s["total"], s["words"]), dtype=torch.int32, device=DEV)
    s["o"] = torch.zeros((s["total"], case["heads"], case["dim"]), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((s["total"], case["heads"]), dtype=torch.float32, device=DEV)
    if own:
        import long_context_sparse_gb300 as dsa
        s["cfg"] = _config(case, s)
        s["ws_tree"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_TREE, DEV)
        s["ws"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_PREFIX, DEV)
    return s


def _prepare_weights(case, seed, gen):
    s = _batch(case, seed, gen)
    s.update(op="weights", dim=case["dim"], heads=case["heads"], decay=0.875,
             k=_cache(s, case["dim"], gen))
    s["q"] = _queries(case, s, gen)
    s["w"] = torch.empty((s["n_pages"], s["page"]), device=DEV).exponential_(1.0, generator=gen)
    s["w_out"] = torch.zeros_like(s["w"])
    s["bits"] = _plain_bits(s, _words(case)) if case["tree"] else None
    # the row sums, as the step's attention leaves them
    s["lse"] = torch.zeros((s["total"], case["heads"]), dtype=torch.float32, device=DEV)
    k = s["k"].view(-1, case["dim"])
    pages = s["table"].tolist()
    first = 0
    for b, (q, n) in enumerate(s["lens"]):
        if q:
            at = torch.arange(n, device=DEV)
            ids = torch.tensor(pages[b], device=DEV)
            x = (s["q"][first:first + q].reshape(-1, case["dim"]).float()
                 @ k[ids[at // s["page"]] * s["page"] + at % s["page"]].float().T)
            x = (x / math.sqrt(case["dim"])).view(q, case["heads"], n)
            x = x.masked_fill(~_seen(s, b, first, q, n)[:, None, :], -math.inf)
            s["lse"][first:first + q] = torch.logsumexp(x, 2)
        first += q
    if own:
        import long_context_sparse_gb300 as dsa
        s["cfg"] = _config(case, s)
        s["ws"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_WEIGHTS, DEV)
    return s


def _seen(s, b, first, q, n):
    """[q, n]: which own tokens the rows of one request see."""
    pos = torch.arange(n, device=DEV)
    i = torch.arange(q, device=DEV)
    if s["bits"] is None:
        return pos[None, :] <= (n - q + i)[:, None]
    node = pos - (n - q)
    bit = (s["bits"][first:first + q][:, node.clamp(min=0) // 32] >> (node % 32)) & 1
    return (node < 0)[None, :] | (bit != 0)


def _prepare_evict(case, seed, gen):
    s = _batch(case, seed, gen)
    s.update(op="evict", dim=case["dim"], kv=case["kv"], first=case["first"], last=case["last"],
             k=_cache(s, case["dim"], gen))
    s["v"] = s["k"] if case["kv"] == 1 else _cache(s, case["dim"], gen)
    # some tokens never received anything to speak of: ties at zero
    w = torch.empty((s["n_pages"], s["page"]), device=DEV).exponential_(1.0, generator=gen)
    s["w"] = torch.where(w < 0.2, torch.zeros_like(w), w)
    s["w_out"] = torch.zeros_like(w)
    s["keep"] = _i32([case["keep"]] * s["batch"])
    left = [min(n, case["keep"]) for _, n in s["lens"]]
    s["kept"] = sum(left)
    s["released"] = sum(_pages(n, s["page"]) - _pages(m, s["page"])
                        for (_, n), m in zip(s["lens"], left))
    s["pages_out"] = torch.full((s["n_pages"],), -1, dtype=torch.int32, device=DEV)
    if own:
        import long_context_sparse_gb300 as dsa
        s["cfg"] = _config(case, s)
        s["ws"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_EVICT, DEV)
        s["ws_release"] = dsa.serve_workspace(s["cfg"], dsa.SERVE_WS_TABLES, DEV)
        s["out"] = dsa.ReleasedPages(
            new_lens=torch.empty(s["batch"], dtype=torch.int32, device=DEV), pages=s["pages_out"],
            n_released=torch.empty(1, dtype=torch.int32, device=DEV))
    return s


def _prepare_logits(case, seed, gen):
    rows, vocab = case["rows"], case["vocab"]
    dtype = DTYPES[case["dtype"]]
    full = torch.empty((rows, vocab + case["pad"]), dtype=dtype, device=DEV)
    ids = torch.empty(rows, dtype=torch.int64, device=DEV)
    for r in range(0, rows, 512):
        # a few likely tokens above a wide bulk
        x = torch.randn(full[r:r + 512].shape, generator=gen, device=DEV) * 2
        x += 12 * (torch.rand(x.shape, generator=gen, device=DEV) < 30 / vocab)
        if case["masked"]:
            x[:, ::case["masked"]] = -math.inf
        full[r:r + 512] = x.to(dtype)
        x = torch.exp(full[r:r + 512, :vocab].float() - full[r:r + 512, :vocab].amax(1, True).float())
        u = torch.rand((x.shape[0], 1), generator=gen, device=DEV) * x.sum(1, keepdim=True)
        ids[r:r + 512] = (torch.cumsum(x, 1) < u).sum(1).clamp(max=vocab - 1)
    if case["masked"] and vocab > 1:  # a token that was drawn is not a masked one
        ids = torch.where(ids % case["masked"] == 0, (ids + 1) % vocab, ids)
        ids = torch.where(ids % case["masked"] == 0, torch.ones_like(ids), ids)
    s = dict(op=case["op"], logits=full[:, :vocab], tokens=ids.to(torch.int32), scale=0.8,
             n_top=case["n_top"])
    if case["op"] == "grad":
        s["g_logp"] = torch.randn(rows, generator=gen, device=DEV)
        s["g_entropy"] = torch.randn(rows, generator=gen, device=DEV) * 0.1
        s["lse"], s["entropy"] = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        for r in range(0, rows, 512):
            x = s["logits"][r:r + 512].double() * s["scale"]
            lse = torch.logsumexp(x, 1, keepdim=True)
            p = torch.exp(x - lse)
            s["lse"][r:r + 512] = lse[:, 0].float()
            s["entropy"][r:r + 512] = -torch.where(p > 0, p * (x - lse), 0.0).sum(1).float()
    if own:
        import long_context_sparse_gb300 as dsa
        s["ws"] = dsa.logprobs_workspace(DEV)
    return s


# -------------------------------------------------------------------- run


def run(state):
    return {"tree": _run_tree, "weights": _run_weights, "evict": _run_evict, "logp": _run_logp,
            "grad": _run_grad}[state["op"]](state)


def _request_of(s):
    """Each row's request and its number in it."""
    cu = s["cu"].long()
    req = torch.repeat_interleave(torch.arange(s["batch"], device=DEV), cu[1:] - cu[:-1],
                                  output_size=s["tokens"])
    return req, torch.arange(s["tokens"], device=DEV) - cu[req]


def _reach(s, n):
    """[batch, n, n]: node j is i or an ancestor of it."""
    req, row = _request_of(s)
    up = s["parents"][: s["tokens"]].long()
    a = torch.zeros((s["batch"], n, n + 1), device=DEV)
    a[req, row, torch.where(up < 0, torch.full_like(up, n), up)] = 1.0
    a = a[:, :, :n] + torch.eye(n, device=DEV)
    for _ in range(max(1, (n - 1).bit_length())):
        a = (a @ a).clamp(max=1.0)
    return a > 0


def _plain_bits(s, words):
    reach = _reach(s, 32 * words)
    req, row = _request_of(s)
    bits = torch.zeros((s["total"], words), dtype=torch.int32, device=DEV)
    x = reach[req, row].view(-1, words, 32).long() << torch.arange(32, device=DEV)
    x = x.sum(2)
    bits[: s["tokens"]] = torch.where(x >= 1 << 31, x - (1 << 32), x).to(torch.int32)
    return bits


def _padded(s, x):
    """Rows of x [tokens, ..] by request, padded to the longest."""
    req, row = _request_of(s)
    out = x.new_zeros((s["batch"], s["q_max"]) + x.shape[1:])
    out[req, row] = x
    return out


def _own_slots(s):
    pos = torch.arange(s["own_max"], device=DEV)
    return s["table"].long()[:, pos // s["page"]].clamp(min=0) * s["page"] + pos % s["page"]


def _visible(s, bits):
    """[tokens, own_max]: which own tokens each row sees."""
    req, row = _request_of(s)
    cu, n = s["cu"].long(), s["seq_lens"].long()
    base = (n - (cu[1:] - cu[:-1]))[req]
    pos = torch.arange(s["own_max"], device=DEV)
    if bits is None:
        return pos[None, :] <= (base + row)[:, None]
    node = pos[None, :] - base[:, None]
    word = torch.gather(bits[: s["tokens"]], 1, (node // 32).clamp(0, bits.shape[1] - 1))
    bit = (word >> (node % 32).to(torch.int32)) & 1
    return (node < 0) | ((bit != 0) & (node < (cu[1:] - cu[:-1])[req][:, None]))


def _run_tree(s):
    if own:
        import long_context_sparse_gb300 as dsa
        bits = dsa.build_tree(s["cfg"], s["parents"], s["cu"], out=s["bits"], ws=s["ws_tree"])
        o, lse = dsa.tree_attn(s["cfg"], s["q"], s["k"], s["prefix_table"], s["prefix"], s["table"],
                               s["seq_lens"], s["cu"], bits,
                               v_pages=s["v"] if s["kv"] == 2 else None, o=s["o"], lse=s["lse"],
                               ws=s["ws"])
        return [bits, o, lse]
    page, dim, heads, tokens, batch = s["page"], s["dim"], s["heads"], s["tokens"], s["batch"]
    if tokens == 0:
        return [s["bits"], s["o"], s["lse"]]
    bits = _plain_bits(s, s["words"])
    k, v = s["k"].view(-1, dim), s["v"].view(-1, dim)
    q = s["q"][:tokens].float() / math.sqrt(dim)
    req, row = _request_of(s)
    # each request's own tokens, padded to the longest
    at = _own_slots(s)
    ko = k[at].float()
    vo = ko if s["kv"] == 1 else v[at].float()
    so = torch.bmm(_padded(s, q).view(batch, -1, dim), ko.transpose(1, 2))
    so = so.view(batch, s["q_max"], heads, -1)[req, row]
    so = so.masked_fill(~_visible(s, bits)[:, None, :], -math.inf).view(tokens * heads, -1)
    m = so.amax(1)
    # the prefix: every row against the same keys
    if s["prefix"]:
        pos = torch.arange(s["prefix"], device=DEV)
        at = s["prefix_table"].long()[pos // page] * page + pos % page
        kp = k[at].float()
        vp = kp if s["kv"] == 1 else v[at].float()
        sp = q.view(tokens * heads, dim) @ kp.T
        m = torch.maximum(m, sp.amax(1))
        sp = (sp - m[:, None]).exp_()
    so = (so - m[:, None]).exp_()
    total = so.sum(1)
    o = torch.bmm(_padded(s, so.view(tokens, heads, -1)).view(batch, -1, so.shape[1]), vo)
    o = o.view(batch, s["q_max"], heads, dim)[req, row]
    if s["prefix"]:
        total = total + sp.sum(1)
        o = o + (sp @ vp).view(tokens, heads, dim)
    s["o"][:tokens] = (o / total.view(tokens, heads, 1)).to(torch.bfloat16)
    s["lse"][:tokens] = (m + total.log()).view(tokens, heads)
    return [bits, s["o"], s["lse"]]


def _run_weights(s):
    if own:
        import long_context_sparse_gb300 as dsa
        return dsa.key_weights(s["cfg"], s["q"], s["lse"], s["k"], s["table"], s["seq_lens"],
                               s["cu"], s["w"], tree_bits=s["bits"], decay=s["decay"],
                               w_out=s["w_out"], ws=s["ws"])
    if s["tokens"] == 0:
        return s["w_out"]
    dim, heads, tokens, batch = s["dim"], s["heads"], s["tokens"], s["batch"]
    q = s["q"][:tokens].float() / math.sqrt(dim)
    req, row = _request_of(s)
    at = _own_slots(s)
    x = torch.bmm(_padded(s, q).view(batch, -1, dim),
                  s["k"].view(-1, dim)[at].float().transpose(1, 2))
    x = x.view(batch, s["q_max"], heads, -1)
    lse = _padded(s, s["lse"][:tokens])
    seen = _padded(s, _visible(s, s["bits"]))
    p = torch.where(seen[:, :, None, :], (x - lse[..., None]).exp_(), 0.0)
    add = p.sum((1, 2))
    # tokens of this step start from nothing, requests without rows stay
    cu, n = s["cu"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    pos = torch.arange(s["own_max"], device=DEV)[None, :]
    old = torch.where(pos < (n - new)[:, None], s["w"].view(-1)[at] * s["decay"], 0.0)
    live = (pos < n[:, None]) & (new > 0)[:, None]
    out = torch.cat([s["w_out"].view(-1), s["w_out"].new_zeros(1)])
    out[torch.where(live, at, torch.full_like(at, out.numel() - 1))] = old + add
    s["w_out"].view(-1)[:] = out[:-1]
    return s["w_out"]


def _run_evict(s):
    if own:
        import long_context_sparse_gb300 as dsa
        dsa.evict_cache(s["cfg"], s["w"], s["table"], s["seq_lens"], s["keep"], s["k"],
                        v_pages=s["v"] if s["kv"] == 2 else None, n_first=s["first"],
                        n_last=s["last"], w_out=s["w_out"], ws=s["ws"])
        r = dsa.release_pages(s["cfg"], s["seq_lens"], s["keep"], s["table"], out=s["out"],
                              ws=s["ws_release"])
        return [s["k"], s["v"], s["w_out"], r.new_lens, r.pages, r.n_released]
    page, dim, batch = s["page"], s["dim"], s["batch"]
    n = s["seq_lens"].long()[:, None]
    keep = torch.minimum(n, s["keep"].long()[:, None])
    at = _own_slots(s)
    pos = torch.arange(s["own_max"], device=DEV)[None, :].expand(batch, -1)
    w = s["w"].view(-1)[at]
    rank = torch.where((pos < s["first"]) | (pos >= n - s["last"]), math.inf, w)
    rank = torch.where(pos < n, rank, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True)[1]
    kept = torch.zeros_like(pos, dtype=torch.bool).scatter_(1, order, pos < keep)
    # the i-th place that is freed below the budget takes the i-th token kept above it
    hole = (pos < keep) & ~kept
    mover = (pos >= keep) & kept
    place = torch.where(mover, torch.cumsum(mover, 1) - 1, s["own_max"])
    movers = pos.new_zeros((batch, s["own_max"] + 1)).scatter_(1, place, pos)
    src = torch.where(hole, torch.gather(movers, 1, (torch.cumsum(hole, 1) - 1).clamp(min=0)), pos)
    left = keep[:, 0]
    req = torch.repeat_interleave(torch.arange(batch, device=DEV), left, output_size=s["kept"])
    dst = torch.arange(s["kept"], device=DEV) - (torch.cumsum(left, 0) - left)[req]
    to, take = at[req, dst], at[req, src[req, dst]]
    for c in [s["k"]] if s["kv"] == 1 else [s["k"], s["v"]]:
        c.view(-1, dim)[to] = c.view(-1, dim)[take]
    s["w_out"].view(-1)[to] = s["w"].view(-1)[take]
    have, need = (n[:, 0] + page - 1) // page, (left + page - 1) // page
    gone = have - need
    end = torch.cumsum(gone, 0)
    req = torch.repeat_interleave(torch.arange(batch, device=DEV), gone, output_size=s["released"])
    j = torch.arange(s["released"], device=DEV)
    s["pages_out"][: s["released"]] = s["table"][req, need[req] + j - (end - gone)[req]]
    return [s["k"], s["v"], s["w_out"], left.to(torch.int32), s["pages_out"],
            end[-1:].to(torch.int32)]


def _order(x):
    """fp32 as integers in the same order, the two zeros alike."""
    i = (x + 0.0).view(torch.int32).long()
    return torch.where(i < 0, -1 - (i & 0x7FFFFFFF), i)


def _run_logp(s):
    if own:
        import long_context_sparse_gb300 as dsa
        r = dsa.token_logprobs(s["logits"], s["tokens"], n_top=s["n_top"], scale=s["scale"],
                               ws=s["ws"])
        return [r.logp, r.lse, r.entropy, r.top_ids, r.top_logp]
    x = s["logits"].float()
    vocab = x.shape[1]
    if s["n_top"]:
        key = _order(x) * (1 << 20) + (vocab - 1 - torch.arange(vocab, device=DEV))
        ids = vocab - 1 - (torch.topk(key, s["n_top"], dim=1)[0] & ((1 << 20) - 1))
        del key
    else:
        ids = torch.zeros((x.shape[0], 0), dtype=torch.int64, device=DEV)
    x = x * s["scale"]
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    lse = m + total.log()
    entropy = total.log()[:, 0] - torch.where(e > 0, e * (x - m), 0.0).sum(1) / total[:, 0]
    logp = torch.gather(x, 1, s["tokens"].long()[:, None]) - lse
    return [logp[:, 0], lse[:, 0], entropy, ids.to(torch.int32), torch.gather(x, 1, ids) - lse]


def _run_grad(s):
    if own:
        import long_context_sparse_gb300 as dsa
        return dsa.token_logprobs_bwd(s["logits"], s["tokens"], s["lse"], s["entropy"],
                                      s["g_logp"], g_entropy=s["g_entropy"], scale=s["scale"],
                                      ws=s["ws"])
    logp = s["logits"].float() * s["scale"] - s["lse"][:, None]
    p = logp.exp()
    g, h = s["g_logp"][:, None], s["g_entropy"][:, None]
    d = torch.where(p > 0, -p * (g + h * (logp + s["entropy"][:, None])), 0.0)
    d[torch.arange(d.shape[0], device=DEV), s["tokens"].long()] += s["g_logp"]
    return (d * s["scale"]).to(s["logits"].dtype)


# ------------------------------------------------------------------- work


def work(case):
    if case["op"] in ("logp", "grad"):
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["rows"] * case["vocab"]
        if case["op"] == "logp":
            return dict(bytes=n * size + case["rows"] * (16 + 8 * case["n_top"]), flops=0)
        return dict(bytes=2 * n * size + 20 * case["rows"], flops=0)
    lens, dim = _lens(case), case["dim"]
    if case["op"] == "evict":
        moved = kept = 0
        pages = 0
        for _, n in lens:
            k = min(n, case["keep"])
            fixed = min(k, case["first"] + case["last"])
            # kept tokens behind the budget: the last ones, and the others' share
            if n > k:
                behind = max(0, n - max(k, n - case["last"]))
                rest = max(0, n - k - behind)
                moved += behind + rest * (k - fixed) / max(1, n - fixed)
            kept += k
            pages += _pages(n, case["page"]) - _pages(k, case["page"])
        return dict(bytes=int(moved * (4 * case["kv"] * dim) + 4 * sum(n for _, n in lens)
                              + 4 * kept + 8 * pages + 12 * case["batch"]), flops=0)
    tokens = sum(q for q, _ in lens)
    rows = case["heads"] * tokens
    own_keys = sum(n for q, n in lens if q)
    if case["op"] == "weights":
        seen = case["heads"] * sum(q * (n - q) + (q * (q + 1)) // 2 for q, n in lens)
        return dict(bytes=rows * (2 * dim + 4) + own_keys * (2 * dim + 8), flops=2 * seen * dim)
    seen = case["heads"] * sum(q * (case["prefix"] + n - q) + (q * (q + 1)) // 2 for q, n in lens)
    return dict(bytes=rows * (4 * dim + 4) + 2 * case["kv"] * dim * (case["prefix"] + own_keys)
                + tokens * (4 + 4 * _words(case)), flops=4 * seen * dim)


# ------------------------------------------------------------------ exact


def exact(case, seed):
    """The definitions in 64 bits, one request or one block of rows at a time."""
    if work(case)["flops"] > 4e12:  # double-precision products: over 20 s
        return None
    s = prepare(case, seed)
    return {"tree": _exact_tree, "weights": _exact_weights, "evict": _exact_evict,
            "logp": _exact_logp, "grad": _exact_grad}[case["op"]](case, s)


def _ancestors(s):
    """For each row its node and its ancestors, by walking up."""
    up, out, first = s["parents"].tolist(), [], 0
    for q, _ in s["lens"]:
        for i in range(q):
            line, at = [], i
            while at >= 0:
                line.append(at)
                at = up[first + at]
            out.append(line)
        first += q
    return out


def _exact_tree(case, s):
    dim, heads = s["dim"], s["heads"]
    lines = _ancestors(s)
    bits = [[0] * s["words"] for _ in range(s["total"])]
    for t, line in enumerate(lines):
        for j in line:
            bits[t][j // 32] |= 1 << (j % 32)
    bits = [[x - (1 << 32) if x >= 1 << 31 else x for x in row] for row in bits]
    o, lse = s["o"].double(), s["lse"].double()
    pages, first = s["table"].tolist(), 0
    prefix = s["prefix_table"].long()
    for b, (q, n) in enumerate(s["lens"]):
        if q == 0:
            continue
        x = s["q"][first:first + q].double().reshape(q * heads, dim) / math.sqrt(dim)
        m = torch.full((q * heads, 1), -math.inf, dtype=torch.float64, device=DEV)
        t, acc = torch.zeros_like(m), torch.zeros_like(x)
        mask = torch.zeros((q, n), dtype=torch.bool)
        mask[:, : n - q] = True
        for i in range(q):
            mask[i, [n - q + j for j in lines[first + i]]] = True
        mask = mask.to(DEV).repeat_interleave(heads, 0)
        own_pages = torch.tensor(pages[b][: _pages(n, s["page"])], device=DEV, dtype=torch.long)
        for ids, length, see in ((own_pages, n, mask), (prefix, case["prefix"], None)):
            step = max(1, (1 << 27) // (q * heads) // s["page"])
            for p in range(0, ids.numel(), step):
                left = length - p * s["page"]
                a = s["k"][ids[p:p + step]].reshape(-1, dim)[:left].double()
                c = s["v"][ids[p:p + step]].reshape(-1, dim)[:left].double()
                y = x @ a.T
                if see is not None:
                    lo = p * s["page"]
                    y[~see[:, lo:lo + a.shape[0]]] = -math.inf
                top = torch.maximum(m, y.amax(1, keepdim=True))
                safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
                e, f = torch.exp(y - safe), torch.exp(m - safe)
                acc, t, m = acc * f + e @ c, t * f + e.sum(1, keepdim=True), top
        o[first:first + q] = (acc / t).view(q, heads, dim)
        lse[first:first + q] = (m + torch.log(t)).view(q, heads)
        first += q
    return [torch.tensor(bits, dtype=torch.int32), o, lse]


def _exact_weights(case, s):
    dim, heads = s["dim"], s["heads"]
    lines = _ancestors(s)
    out = s["w_out"].double().view(-1)
    pages, first = s["table"].tolist(), 0
    for b, (q, n) in enumerate(s["lens"]):
        if q == 0:
            continue
        x = s["q"][first:first + q].double().reshape(q * heads, dim) / math.sqrt(dim)
        lse = s["lse"][first:first + q].double().reshape(q * heads, 1)
        for p, page in enumerate(pages[b][: _pages(n, s["page"])]):
            lo = p * s["page"]
            hi = min(n, lo + s["page"])
            e = torch.exp(x @ s["k"][page, : hi - lo].double().T - lse).view(q, heads, -1).sum(1)
            if hi > n - q:  # the step's own tokens among them
                see = torch.tensor([[j < n - q or (j - (n - q) in lines[first + i] if case["tree"]
                                                   else j <= n - q + i) for j in range(lo, hi)]
                                    for i in range(q)], device=DEV)
                e = torch.where(see, e, 0.0)
            old = s["w"][page, : hi - lo].double() * s["decay"]
            old[max(0, n - q - lo):] = 0.0
            out[page * s["page"]: page * s["page"] + hi - lo] = old + e.sum(0)
        first += q
    return out.view_as(s["w_out"])


def _exact_evict(case, s):
    page = s["page"]
    k, v = s["k"].clone(), s["v"].clone()
    w, w_out = s["w"].cpu().view(-1).tolist(), s["w_out"].cpu().view(-1).tolist()
    released, lens = [], []
    moves = []
    for (_, n), table in zip(s["lens"], s["table"].tolist()):
        slots = [table[j // page] * page + j % page for j in range(n)]
        left = min(n, case["keep"])
        ranked = sorted(range(n), key=lambda j: (not (j < case["first"] or j >= n - case["last"]),
                                                 0.0 if j < case["first"] or j >= n - case["last"]
                                                 else -w[slots[j]], j))
        kept = set(ranked[:left])
        freed = [j for j in range(left) if j not in kept]
        late = sorted(j for j in kept if j >= left)
        source = dict(zip(freed, late))
        for j in range(left):
            w_out[slots[j]] = w[slots[source.get(j, j)]]
        moves += [(slots[a], slots[b]) for a, b in source.items()]
        released += table[_pages(left, page): _pages(n, page)]
        lens.append(left)
    if moves:
        to, take = torch.tensor(moves, device=DEV).T
        for c in [k] if case["kv"] == 1 else [k, v]:
            c.view(-1, case["dim"])[to] = c.view(-1, case["dim"])[take]
    if case["kv"] == 1:
        v = k
    out = s["pages_out"].tolist()
    out[: len(released)] = released
    return [k.double(), v.double(), torch.tensor(w_out, dtype=torch.float64).view(s["w"].shape),
            torch.tensor(lens), torch.tensor(out), torch.tensor([len(released)])]


def _exact_logp(case, s):
    outs = []
    for r in range(0, case["rows"], 256):
        x = s["logits"][r:r + 256].double()
        order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, : case["n_top"]]
        x = x * s["scale"]
        lse = torch.logsumexp(x, 1)
        y = x - lse[:, None]
        p = torch.exp(y)
        tok = s["tokens"][r:r + 256].long()
        outs.append([y[torch.arange(y.shape[0], device=DEV), tok], lse,
                     -torch.where(p > 0, p * y, 0.0).sum(1), order,
                     torch.stack([z[i] for z, i in zip(y, order)])])
    return [torch.cat(x) for x in zip(*outs)]


def _exact_grad(case, s):
    out = torch.empty(s["logits"].shape, dtype=torch.float64, device=DEV)
    for r in range(0, case["rows"], 256):
        x = s["logits"][r:r + 256].double() * s["scale"]
        y = x - s["lse"][r:r + 256].double()[:, None]
        p = torch.exp(y)
        n = torch.arange(x.shape[0], device=DEV)
        one = torch.zeros_like(x)
        one[n, s["tokens"][r:r + 256].long()] = 1.0
        g = s["g_logp"][r:r + 256].double()[:, None]
        h = s["g_entropy"][r:r + 256].double()[:, None]
        y = torch.where(p > 0, y, 0.0)
        out[r:r + 256] = s["scale"] * (g * (one - p)
                                       - h * p * (y + s["entropy"][r:r + 256].double()[:, None]))
    return out
