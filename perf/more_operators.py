"""Timed cases of the operators of a round over a paged key/value cache, with trees of drafted tokens.

Each case is one call as an engine makes it.  With `own` false, `run` computes the call in its
plain form (elementary torch operations in binary32, rounded once at the end); with `own` true it
makes the library's call on the same state.  `exact` evaluates the definitions in binary64.

  append  spec_cache_append: a round's keys and values written to the paged cache and its queries
          to a buffer, queries and keys rotated by their tokens' positions
  attend  spec_tree_attention: attention of a round's rows over the cached context and over each
          row's own ancestors among the drafted tokens
  accept  spec_tree_accept: the walk down a tree of drafts with the tokens sampled from the
          target's rows
  keep    spec_cache_keep: the accepted path's cache entries moved behind the context

A request's rows are a root (the last emitted token) and its drafts; `branch` is how many of a
row's drafts may share a parent (0: a chain).
"""
import math

import torch

own = False


# ---- cases -------------------------------------------------------------------------------------

def _append(name, B, drafts, root, ctx, page, heads, kv_heads, D, rot, adjacent, dtype, branch,
            ragged):
    return {"name": name, "op": "append", "B": B, "drafts": drafts, "root": root, "ctx": ctx,
            "page": page, "heads": heads, "kv_heads": kv_heads, "D": D, "rot": rot,
            "adjacent": adjacent, "dtype": dtype, "branch": branch, "ragged": ragged}


def _attend(name, B, drafts, ctx_lo, ctx_hi, page, heads, kv_heads, D, branch, ragged, lse):
    return {"name": name, "op": "attend", "B": B, "drafts": drafts, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "page": page, "heads": heads, "kv_heads": kv_heads, "D": D,
            "branch": branch, "ragged": ragged, "lse": lse}


def _accept(name, B, drafts, branch, ragged):
    return {"name": name, "op": "accept", "B": B, "drafts": drafts, "branch": branch,
            "ragged": ragged}


def _keep(name, B, layers, drafts, depth, ctx, page, kv_heads, D):
    return {"name": name, "op": "keep", "B": B, "layers": layers, "drafts": drafts, "depth": depth,
            "ctx": ctx, "page": page, "kv_heads": kv_heads, "D": D}


def listed():
    return [
        # one request's round of 5 drafts, one layer: latency
        _append("append 1x6", 1, 5, True, 1000, 16, 32, 8, 128, 128, False, "bf16", 0, False),
        # 64 requests with trees of 15 drafts, half of a head rotated, projections left in 32 bits
        _append("append trees 64x16", 64, 15, True, 4000, 32, 64, 8, 128, 64, True, "f32", 3, True),
        # 8 prompts of up to 8192 tokens
        _append("append prompts 8x8192", 8, 8192, False, 0, 64, 32, 8, 128, 128, False, "bf16", 0,
                True),
        # one request's round of 5 drafts over a short context: latency
        _attend("attend 1x6, 1000", 1, 5, 1000, 1000, 16, 32, 8, 128, 0, False, False),
        # the token-level benchmark's round of 64 requests with contexts of every length
        _attend("attend 64x6, 16k ragged", 64, 5, 1, 16384, 64, 32, 8, 128, 0, False, False),
        # trees of 63 drafts, many query heads for each key: bound by products
        _attend("attend trees 32x64, 4k", 32, 63, 512, 4096, 64, 64, 8, 128, 4, False, True),
        # one request with a long context and a tree of 15 drafts
        _attend("attend tree 1x16, 128k", 1, 15, 131072, 131072, 128, 32, 8, 128, 2, False, False),
        # a small ragged batch of odd sizes, narrow heads, contexts from nothing
        _attend("attend odd 17x9, 3k", 17, 8, 0, 3001, 32, 28, 4, 64, 0, True, True),
        # one request's tree of 15 drafts
        _accept("accept 1x15", 1, 15, 2, False),
        # 512 trees of up to 63 drafts
        _accept("accept 512x63", 512, 63, 4, True),
        # one request, one layer
        _keep("keep 1 request", 1, 1, 15, 5, 1000, 16, 8, 128),
        # 64 requests, every layer of a model
        _keep("keep 64 requests, 32 layers", 64, 32, 63, 8, 250, 64, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "accept", "keep"))
    kv = rng.choice((1, 2, 4, 5, 8))
    D = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        heads = kv * rng.choice((1, 2, 3, 4, 7, 8))
        prompt = rng.random() < 0.4
        drafts = _log(rng, 16, 8192) if prompt else rng.randint(0, 63)
        most = max(1, int(3.0e4 / max(1, drafts) * 4096 / (heads * D)))
        c = _append("", min(_log(rng, 1, 256), most), max(drafts, 1) if prompt else drafts,
                    not prompt, 0 if prompt else _log(rng, 1, 4000), page, heads, kv, D,
                    rng.choice((D // 2, D)), rng.random() < 0.5, rng.choice(("bf16", "f32")),
                    0 if prompt else rng.choice((0, 2, 4)), rng.random() < 0.5)
    elif op == "attend":
        heads = kv * rng.choice((1, 2, 3, 4, 7, 8))
        drafts = rng.choice((0, rng.randint(1, 16), rng.randint(1, 63)))
        hi = _log(rng, 1, 131072)
        rows = (drafts + 1) * heads
        most = min(2.0e9 / (4 * kv * D * (hi + drafts)), 1.5e11 / (4 * rows * D * (hi + drafts)))
        c = _attend("", max(1, min(_log(rng, 1, 256), int(most))), drafts,
                    rng.choice((0, hi // 2, hi)), hi, page, heads, kv, D, rng.choice((0, 2, 4)),
                    rng.random() < 0.5, rng.random() < 0.5)
    elif op == "accept":
        c = _accept("", _log(rng, 1, 512), rng.randint(1, 63), rng.choice((0, 2, 4)),
                    rng.random() < 0.5)
    else:
        drafts = rng.randint(1, 63)
        ctx = _log(rng, 1, 1000)
        B = _log(rng, 1, 64)
        most = max(1, int(2.0e9 / (4 * kv * D * B * (ctx + drafts + page))))
        c = _keep("", B, min(_log(rng, 1, 64), most), drafts, rng.randint(1, min(8, drafts)), ctx,
                  page, kv, D)
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _int(lo, hi, n, g):
    """n int32 in lo .. hi."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _trees(B, R, branch, g):
    """parents int32 [B, R]: row i hangs from one of the rows that leave it at most about `branch`
    siblings, as a drafter that keeps its likeliest nodes makes them, or from a row nearby."""
    i = torch.arange(R, device="cuda")
    lo = torch.clamp((i - 1) // branch - 2, min=0)
    hi = torch.clamp(i - 1, min=0)
    u = torch.rand((B, R), generator=g, device="cuda") ** 2
    p = lo + torch.floor(u * (hi - lo + 1)).long().clamp(max=R)
    p = torch.minimum(p, hi)
    p[:, 0] = -1
    return p.to(torch.int32).contiguous()


def _lengths(c, g):
    """draft_len int32 [B]: all of the drafts, or ragged (a prompt has one token at least)."""
    if c["ragged"]:
        return _int(0 if c.get("root", True) else 1, c["drafts"], c["B"], g)
    return torch.full((c["B"],), c["drafts"], dtype=torch.int32, device="cuda")


def _pages(lengths, longest, page, g):
    """(page_table int32 [B, most], number of pages): every request's pages somewhere in a cache
    that could hold the longest of them all, no page twice, -1 behind a request's last."""
    need = (lengths.long() + page - 1) // page
    most = max(1, (longest + page - 1) // page)
    n = len(lengths) * most + 3
    order = torch.randperm(n, generator=g, device="cuda")
    at = torch.arange(most, device="cuda")[None]
    first = torch.cumsum(need, 0) - need
    table = order[(first[:, None] + at).clamp(max=n - 1)]
    return torch.where(at < need[:, None], table, -1).to(torch.int32).contiguous(), n


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _prepare_append(c, g):
    B, R = c["B"], c["drafts"] + int(c["root"])
    Hq, Hk, D = c["heads"], c["kv_heads"], c["D"]
    draft_len = _lengths(c, g)
    ctx = _int(c["ctx"] // 2, c["ctx"], B, g)
    table, n = _pages(ctx + draft_len + int(c["root"]), c["ctx"] + R, c["page"], g)
    # what a fused projection leaves: queries, keys and values of a row beside one another
    qkv = _normal((B * R, Hq + 2 * Hk, D), g, _DT[c["dtype"]])
    # cos and sin of every position, as a model keeps them
    h = c["rot"] // 2
    angle = (torch.arange(c["ctx"] + R, device="cuda", dtype=torch.float64)[:, None] *
             10000.0 ** (-torch.arange(h, device="cuda", dtype=torch.float64) / h))
    return {"q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "v": qkv[:, Hq + Hk:],
            "cos_sin": torch.cat((torch.cos(angle), torch.sin(angle)), 1).float(),
            "k_cache": _normal((n, c["page"], Hk, D), g),
            "v_cache": _normal((n, c["page"], Hk, D), g), "page_table": table, "ctx_len": ctx,
            "row0": torch.arange(B, device="cuda") * R, "draft_len": draft_len,
            "drafts": c["drafts"], "root": c["root"], "R": R, "adjacent": c["adjacent"],
            "parents": _trees(B, R, c["branch"], g).view(-1) if c["branch"] else None,
            "q_out": torch.zeros((B * R, Hq, D), dtype=torch.bfloat16, device="cuda"),
            "status": _status()}


def _prepare_attend(c, g):
    B, R, Hk, D = c["B"], c["drafts"] + 1, c["kv_heads"], c["D"]
    draft_len = _lengths(c, g)
    ctx = _int(c["ctx_lo"], c["ctx_hi"], B, g)
    table, n = _pages(ctx + draft_len + 1, c["ctx_hi"] + R, c["page"], g)
    q = _normal((B * R, c["heads"], D), g) * 2  # some keys stand out
    return {"q": q, "k_cache": _normal((n, c["page"], Hk, D), g),
            "v_cache": _normal((n, c["page"], Hk, D), g), "page_table": table, "ctx_len": ctx,
            "row0": torch.arange(B, device="cuda") * R, "draft_len": draft_len,
            "drafts": c["drafts"], "R": R, "scale": 1.0 / math.sqrt(D),
            "parents": _trees(B, R, c["branch"], g).view(-1) if c["branch"] else None,
            "out": torch.zeros_like(q),
            "lse": torch.zeros((B * R, c["heads"]), device="cuda") if c["lse"] else None,
            "status": _status()}


def _prepare_accept(c, g):
    B, R, N = c["B"], c["drafts"] + 1, c["drafts"]
    parents = _trees(B, R, c["branch"] or 1, g)
    if not c["branch"]:
        parents = (torch.arange(R, device="cuda", dtype=torch.int32) - 1).repeat(B, 1)
    # few tokens, so that some of the sampled ones were drafted, and siblings differ or not
    few = max(2, c["branch"])
    return {"sampled": _int(0, few, B * R, g), "draft_tokens": _int(0, few, B * N, g),
            "parents": parents.reshape(-1).contiguous(), "row0": torch.arange(B, device="cuda") * R,
            "draft_row0": torch.arange(B, device="cuda") * N, "draft_len": _lengths(c, g),
            "drafts": N, "B": B, "R": R,
            "accepted_len": torch.zeros(B, dtype=torch.int32, device="cuda"),
            "out_tokens": torch.zeros((B, R), dtype=torch.int32, device="cuda"),
            "path": torch.zeros((B, N), dtype=torch.int32, device="cuda"),
            "correction": torch.zeros(B, dtype=torch.int32, device="cuda"), "status": _status()}


def _prepare_keep(c, g):
    B, N, page = c["B"], c["drafts"], c["page"]
    ctx = _int((c["ctx"] + 1) // 2, c["ctx"], B, g)
    table, n = _pages(ctx + N + 1, c["ctx"] + N + 1, page, g)
    accepted = _int(0, c["depth"], B, g)
    # a path: ascending rows of the tree
    order = torch.rand((B, N), generator=g, device="cuda").argsort(1) + 1
    path = order[:, :c["depth"]].sort(1)[0]
    at = torch.arange(N, device="cuda")[None]
    full = torch.full((B, N), -1, dtype=torch.int64, device="cuda")
    full[:, :c["depth"]] = path
    # the first `accepted` of them, ascending: a path cut short keeps its first rows
    full = torch.where(at < accepted[:, None], full, -1)
    shape = (c["layers"], n, page, c["kv_heads"], c["D"])
    return {"k_cache": _normal(shape, g), "v_cache": _normal(shape, g), "page_table": table,
            "ctx_len": ctx, "accepted_len": accepted, "path": full.to(torch.int32).contiguous(),
            "new_len": torch.zeros(B, dtype=torch.int32, device="cuda"), "depth": c["depth"],
            "status": _status()}


def prepare(case, seed):
    return {"op": case["op"], **globals()["_prepare_" + case["op"]](case, _gen(seed))}


# ---- plain forms -------------------------------------------------------------------------------

def _ancestors(parents, B, R):
    """bool [B, R, R]: row j is row i or one of its ancestors.  With N the matrix of parents,
    (1 + N)^128 holds C(128, length of the way) there, at most 2.4e37, and 0 elsewhere."""
    p = parents.view(B, R, 1).long()
    step = (torch.arange(R, device=p.device) == p).float() + torch.eye(R, device=p.device)
    return torch.linalg.matrix_power(step, 128) > 0


def _depth(s, B, R):
    if s["parents"] is None:
        return torch.arange(R, device=s["q"].device).expand(B, R)
    return _ancestors(s["parents"], B, R).sum(-1) - 1


def _place(table, at, page):
    """Index of place `at` [B, n] of each request among all places of the cache."""
    return table.gather(1, at // page).long() * page + at % page


def _rotate(x, cos, sin, adjacent):
    """x [..., D] rotated in its first 2 h elements, h the width of cos and sin."""
    h = cos.shape[-1]
    if adjacent:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., 2 * h:]), -1)


def _plain_append(s):
    B, R = s["draft_len"].shape[0], s["R"]
    page = s["k_cache"].shape[1]
    # rows behind a request's last repeat that one, so that they write what it writes
    last = (s["draft_len"].long() + int(s["root"]) - 1)[:, None]
    i = torch.minimum(torch.arange(R, device=last.device)[None], last)
    row = (s["row0"][:, None] + i).view(-1)
    ctx = s["ctx_len"].long()[:, None]
    angle = s["cos_sin"][(ctx + _depth(s, B, R).gather(1, i)).view(-1)]
    h = angle.shape[1] // 2
    cos, sin = angle[:, None, :h], angle[:, None, h:]
    slot = _place(s["page_table"], ctx + i, page).view(-1)
    k_all, v_all = (s[n].view(-1, *s[n].shape[2:]) for n in ("k_cache", "v_cache"))
    k_all[slot] = _rotate(s["k"][row].float(), cos, sin, s["adjacent"]).to(k_all.dtype)
    v_all[slot] = s["v"][row].to(v_all.dtype)
    s["q_out"][row] = _rotate(s["q"][row].float(), cos, sin, s["adjacent"]).to(s["q_out"].dtype)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _visible(s, B, R, keys):
    """bool [B, R, keys]: place j belongs to the context, to row i or to an ancestor of row i."""
    ctx = s["ctx_len"].long()[:, None]
    at = torch.arange(keys, device=ctx.device)[None] - ctx
    if s["parents"] is None:
        own_ = torch.arange(R, device=ctx.device)[None, :, None] >= at[:, None, :]
    else:
        own_ = _ancestors(s["parents"], B, R).gather(
            2, at.clamp(0, R - 1)[:, None, :].expand(B, R, keys))
        own_ = own_ & (at < R)[:, None, :]
    return own_ | (at < 0)[:, None, :]


def _plain_attend(s):
    B, R = s["draft_len"].shape[0], s["R"]
    _, page, Hk, D = s["k_cache"].shape
    Hq = s["q"].shape[1]
    last = s["draft_len"].long()[:, None]
    i = torch.minimum(torch.arange(R, device=last.device)[None], last)
    row = s["row0"][:, None] + i
    table = s["page_table"].clamp_min(0).long()
    keys = table.shape[1] * page
    seen = _visible(s, B, R, keys).gather(1, i[:, :, None].expand(B, R, keys))
    k = s["k_cache"][table].view(B, keys, Hk, D).permute(0, 2, 3, 1).float()
    v = s["v_cache"][table].view(B, keys, Hk, D).permute(0, 2, 1, 3).float()
    # the query heads of one key head beside the rows
    q = s["q"][row].float().view(B, R, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    x = (q @ k) * s["scale"]
    x = x.view(B, Hk, Hq // Hk, R, keys).masked_fill_(~seen[:, None, None], -math.inf)
    x = x.view(B, Hk, -1, keys)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    y = (e @ v) / total
    y = y.view(B, Hk, Hq // Hk, R, D).permute(0, 3, 1, 2, 4).reshape(B, R, Hq, D)
    s["out"][row] = y.to(s["out"].dtype)
    if s["lse"] is None:
        return {"out": s["out"]}
    z = (top + torch.log(total)).view(B, Hk, Hq // Hk, R).permute(0, 3, 1, 2).reshape(B, R, Hq)
    s["lse"][row] = z
    return {"out": s["out"], "lse": s["lse"]}


def _plain_accept(s):
    """A row is accepted where it and all its ancestors were sampled from their parents' rows, each
    the first of its siblings with that token."""
    B, R, N = s["B"], s["R"], s["drafts"]
    dev = s["sampled"].device
    n = s["draft_len"].long()[:, None]
    i = torch.arange(R, device=dev)
    parent = s["parents"].view(B, R).long().clamp_min(0)
    token = torch.cat((torch.full((B, 1), -1, device=dev), s["draft_tokens"].view(B, N).long()), 1)
    sampled = s["sampled"].view(B, R).long()
    ok = (token == sampled.gather(1, parent)) & (i[None] <= n)
    same = (parent[:, :, None] == parent[:, None, :]) & ok[:, :, None] & ok[:, None, :]
    same = same & (i[:, None] > i[None, :]) & (i[None, :] > 0)  # a sibling before it
    ok = ok & ~same.any(-1)
    ok[:, 0] = True
    taken = (_ancestors(s["parents"], B, R).float() @ (~ok).float()[:, :, None])[:, :, 0] == 0
    taken[:, 0] = False
    count = taken.sum(1, keepdim=True)
    order = torch.where(taken, i[None], R).sort(1)[0]  # a child comes after its parent
    inside = i[None] < count
    path = torch.where(inside, order, 0)
    end = path.gather(1, (count - 1).clamp_min(0)) * (count > 0)
    correction = sampled.gather(1, end)
    out = torch.where(inside, token.gather(1, path),
                      torch.where(i[None] == count, correction, -1))
    s["accepted_len"].copy_(count[:, 0])
    s["out_tokens"].copy_(out)
    s["path"].copy_(torch.where(inside, path, -1)[:, :N])
    s["correction"].copy_(correction[:, 0])
    return {k: s[k] for k in ("accepted_len", "out_tokens", "path", "correction")}


def _plain_keep(s):
    page = s["k_cache"].shape[2]
    ctx, accepted = s["ctx_len"].long()[:, None], s["accepted_len"].long()[:, None]
    i = torch.arange(s["depth"], device=ctx.device)[None]
    inside = i < accepted
    # places behind the accepted ones repeat the root's, which stays where it is
    src = ctx + torch.where(inside, s["path"][:, :s["depth"]].long(), 0)
    dst = ctx + torch.where(inside, i + 1, 0)
    src, dst = (_place(s["page_table"], x, page).view(-1) for x in (src, dst))
    k, v = (s[n].view(s[n].shape[0], -1, *s[n].shape[3:]) for n in ("k_cache", "v_cache"))
    k[:, dst] = k[:, src]
    v[:, dst] = v[:, src]
    s["new_len"].copy_((ctx + 1 + accepted)[:, 0])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "ctx_len": s["new_len"]}


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    if not own:
        return _PLAIN[state["op"]](state)
    return _OWN[state["op"]](state)


def _own_append(s):
    import speculative_decoding_verification_token_gb300 as sv
    q = sv.spec_cache_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"],
                             s["ctx_len"], s["row0"], s["draft_len"], s["drafts"],
                             cos_sin=s["cos_sin"], adjacent=s["adjacent"], parents=s["parents"],
                             bonus_row=s["root"], q_out=s["q_out"], status=s["status"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import speculative_decoding_verification_token_gb300 as sv
    out = sv.spec_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"],
                                 s["row0"], s["draft_len"], s["drafts"], parents=s["parents"],
                                 scale=s["scale"], out=s["out"], lse=s["lse"], status=s["status"])
    return {"out": out} if s["lse"] is None else {"out": out, "lse": s["lse"]}


def _own_accept(s):
    import speculative_decoding_verification_token_gb300 as sv
    sv.spec_tree_accept(s["sampled"], s["draft_tokens"], s["parents"], s["row0"], s["draft_row0"],
                        s["draft_len"], s["drafts"], accepted_len=s["accepted_len"],
                        out_tokens=s["out_tokens"], path=s["path"], correction=s["correction"],
                        status=s["status"])
    return {k: s[k] for k in ("accepted_len", "out_tokens", "path", "correction")}


def _own_keep(s):
    import speculative_decoding_verification_token_gb300 as sv
    sv.spec_cache_keep(s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"],
                       s["accepted_len"], s["path"], new_len=s["new_len"], status=s["status"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "ctx_len": s["new_len"]}


_PLAIN = {"append": _plain_append, "attend": _plain_attend, "accept": _plain_accept,
          "keep": _plain_keep}
_OWN = {"append": _own_append, "attend": _own_attend, "accept": _own_accept, "keep": _own_keep}


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "append":
        e = 2 if c["dtype"] == "bf16" else 4
        drafts = (c["drafts"] + (0 if c["root"] else 1)) / 2 if c["ragged"] else c["drafts"]
        rows = c["B"] * (drafts + int(c["root"]))
        width = (c["heads"] + 2 * c["kv_heads"]) * c["D"]
        turned = (c["heads"] + c["kv_heads"]) * c["rot"]
        table = min(rows, c["ctx"] + c["drafts"] + 1) * c["rot"] * 4
        return {"bytes": rows * width * (e + 2) + table, "flops": 3 * rows * turned}
    if c["op"] == "attend":
        rows = (c["drafts"] / 2 if c["ragged"] else c["drafts"]) + 1
        keys = (c["ctx_lo"] + c["ctx_hi"]) / 2 + rows
        b = c["B"] * (keys * c["kv_heads"] * 4 + rows * c["heads"] * 4) * c["D"]
        if c["lse"]:
            b += c["B"] * rows * c["heads"] * 4
        return {"bytes": b, "flops": 4 * c["B"] * rows * c["heads"] * c["D"] * keys}
    if c["op"] == "accept":
        nodes = c["B"] * (c["drafts"] / 2 if c["ragged"] else c["drafts"])
        return {"bytes": nodes * 12 + c["B"] * (32 + 8 * c["drafts"]), "flops": nodes * 2}
    moved = c["B"] * c["depth"] / 2 * c["layers"]  # few rows of a path lie where they are kept
    return {"bytes": moved * c["kv_heads"] * c["D"] * 8 + c["B"] * 16, "flops": moved}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _way_up(parents, first, i):
    """Row i and its ancestors, from a list of parents."""
    way = []
    while i >= 0:
        way.append(i)
        i = i - 1 if parents is None else parents[first + i]
    return way


def _exact_append(s):
    page = s["k_cache"].shape[1]
    k_out, v_out, q_out = (s[n].double() for n in ("k_cache", "v_cache", "q_out"))
    parents = None if s["parents"] is None else s["parents"].tolist()
    table = s["page_table"].tolist()
    rows, slots, at = [], [], []
    for r, (first, n, ctx) in enumerate(zip(s["row0"].tolist(), s["draft_len"].tolist(),
                                            s["ctx_len"].tolist())):
        for i in range(n + int(s["root"])):
            rows.append(first + i)
            slots.append(table[r][(ctx + i) // page] * page + (ctx + i) % page)
            at.append(ctx + (i if parents is None else len(_way_up(parents, first, i)) - 1))
    rows, slots, at = (torch.tensor(x, device=k_out.device) for x in (rows, slots, at))
    rot = s["cos_sin"].shape[1]
    cs = s["cos_sin"].double()[at]
    # the rotation as a product of complex numbers
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None, :]

    def rotated(x):
        y = x[rows].double()
        head = y[:, :, :rot]
        if s["adjacent"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:2], -1, 2).contiguous()) * turn
            y[:, :, :rot] = torch.view_as_real(z).reshape(head.shape)
        else:
            z = torch.complex(head[..., :rot // 2].contiguous(),
                              head[..., rot // 2:].contiguous()) * turn
            y[:, :, :rot] = torch.cat((z.real, z.imag), -1)
        return y

    k_out.view(-1, *k_out.shape[2:])[slots] = rotated(s["k"])
    v_out.view(-1, *v_out.shape[2:])[slots] = s["v"][rows].double()
    q_out[rows] = rotated(s["q"])
    return {"q": q_out, "k_cache": k_out, "v_cache": v_out}


def _exact_attend(s):
    """Request by request, row by row over the keys that it sees."""
    page, Hk = s["k_cache"].shape[1:3]
    Hq, D = s["q"].shape[1:]
    out = s["out"].double()
    lse = None if s["lse"] is None else s["lse"].double()
    parents = None if s["parents"] is None else s["parents"].tolist()
    for r, (first, n, ctx) in enumerate(zip(s["row0"].tolist(), s["draft_len"].tolist(),
                                            s["ctx_len"].tolist())):
        places = torch.arange(ctx + n + 1, device=out.device)
        slot = s["page_table"][r].long()[places // page] * page + places % page
        k, v = (s[c].view(-1, Hk, D)[slot].double() for c in ("k_cache", "v_cache"))
        seen = torch.zeros((n + 1, ctx + n + 1), dtype=torch.bool, device=out.device)
        seen[:, :ctx] = True
        a = [(i, ctx + j) for i in range(n + 1) for j in _way_up(parents, first, i)]
        a = torch.tensor(a, device=out.device)
        seen[a[:, 0], a[:, 1]] = True
        q = s["q"][first:first + n + 1].double().view(n + 1, Hk, Hq // Hk, D)
        x = torch.einsum("ihgd,jhd->ihgj", q, k) * s["scale"]
        x[(~seen)[:, None, None, :].expand_as(x)] = -math.inf
        z = torch.logsumexp(x, -1)
        y = torch.einsum("ihgj,jhd->ihgd", torch.exp(x - z[..., None]), v)
        out[first:first + n + 1] = y.reshape(n + 1, Hq, D)
        if lse is not None:
            lse[first:first + n + 1] = z.reshape(n + 1, Hq)
    return {"out": out} if lse is None else {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] in ("accept", "keep"):
        return None  # whole numbers; copies
    return {"append": _exact_append, "attend": _exact_attend}[case["op"]](prepare(case, seed))
