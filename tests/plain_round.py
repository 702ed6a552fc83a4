"""Plain binary64 forms of the calls of a round over a paged cache, written from their definitions in
include/specverify.h for the tests, and inputs for them."""
import torch


def ancestors(parents, first, i):
    """Row i and its ancestors (parents None: a chain)."""
    way = []
    while i >= 0:
        way.append(i)
        i = i - 1 if parents is None else int(parents[first + i])
    return way


def place(table, r, j, page):
    return int(table[r, j // page]), j % page


def make_tree(n, g, shape="random"):
    """parents of n rows."""
    if shape == "chain":
        return torch.arange(n, dtype=torch.int32) - 1
    if shape == "star":
        return torch.tensor([-1] + [0] * (n - 1), dtype=torch.int32)[:n]
    if shape == "forest":  # every third row follows the context directly
        p = [-1 if i % 3 == 0 else int(torch.randint(0, i, (1,), generator=g)) for i in range(n)]
    else:
        p = [-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, n)]
    return torch.tensor(p[:n], dtype=torch.int32)


def make_round(ctx, draft_len, gmax, page, heads, kv, D, seed=0, bonus=1, tree=None, gap=2,
               spare_pages=3, q_scale=1.0, nan_elsewhere=True, device="cuda"):
    """Inputs of a round: rows of the requests with `gap` unused rows between them, pages in random
    order, NaN in every place that belongs to no request."""
    g = torch.Generator().manual_seed(seed)
    B = len(ctx)
    n = [d + bonus for d in draft_len]
    need = [(c + k + page - 1) // page for c, k in zip(ctx, n)]
    most = max(need + [1])
    pages = sum(need) + spare_pages
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, most + 1), -7, dtype=torch.int32)  # (entries that nothing may follow)
    at = 0
    for r in range(B):
        table[r, :need[r]] = order[at:at + need[r]].to(torch.int32)
        at += need[r]
    row0, at = [], 1
    for k in n:
        row0.append(at)
        at += k + gap
    rows = at
    kc = torch.randn((pages, page, kv, D), generator=g).to(torch.bfloat16)
    vc = torch.randn((pages, page, kv, D), generator=g).to(torch.bfloat16)
    if nan_elsewhere:
        used = torch.zeros((pages, page), dtype=torch.bool)
        for r in range(B):
            for j in range(ctx[r] + n[r]):
                used[place(table, r, j, page)] = True
        kc[~used] = float("nan")
        vc[~used] = float("nan")
    q = (torch.randn((rows, heads, D), generator=g) * q_scale).to(torch.bfloat16)
    parents = None
    if tree:
        parents = torch.full((rows,), -1, dtype=torch.int32)
        for r in range(B):
            parents[row0[r]:row0[r] + n[r]] = make_tree(n[r], g, tree)
    i32 = torch.int32
    s = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, ctx_len=torch.tensor(ctx, dtype=i32),
             row0=torch.tensor(row0), draft_len=torch.tensor(draft_len, dtype=i32), parents=parents)
    host = {k: v for k, v in s.items()}
    dev = {k: v.to(device) if v is not None else None for k, v in s.items()}
    dev.update(max_draft_len=gmax, bonus_row=bool(bonus))
    return host, dev, n, rows


def attention(s, n, scale):
    """{row: (out [heads, D], lse [heads], bound of out [heads, D], bound of lse [heads])}.

    The bounds count every rounding of the path.  A score's D products are exact in binary32 and
    their sum is off by at most D steps of 2^-23 of the sum of magnitudes (additions that truncate
    included); with the shift and the exponential (2^-20 covers a few units of ex2 and of scores up to
    a hundred) that moves e^x by a factor of d.  e^x is rounded to bf16 (2^-8), the products with v
    are summed in binary32 (2^-23 a key), the quotient is rounded to bf16 (2^-8)."""
    page, kv, D = s["k_cache"].shape[1:]
    heads = s["q"].shape[1]
    got = {}
    for r in range(len(n)):
        first, ctx = int(s["row0"][r]), int(s["ctx_len"][r])
        for i in range(n[r]):
            seen = list(range(ctx)) + sorted(ctx + j for j in ancestors(s["parents"], first, i))
            idx = [place(s["page_table"], r, j, page) for j in seen]
            pg, of = torch.tensor([a for a, _ in idx]), torch.tensor([b for _, b in idx])
            k = s["k_cache"][pg, of].double().repeat_interleave(heads // kv, 1)  # [keys, heads, D]
            v = s["v_cache"][pg, of].double().repeat_interleave(heads // kv, 1)
            q = s["q"][first + i].double()
            x = torch.einsum("hd,jhd->hj", q, k) * scale
            mag = torch.einsum("hd,jhd->hj", q.abs(), k.abs()) * abs(scale)
            lse = torch.logsumexp(x, 1)
            w = torch.exp(x - lse[:, None])
            out = torch.einsum("hj,jhd->hd", w, v)
            d = (mag * D * 2.0 ** -23 + 2.0 ** -20).amax(1)
            reach = torch.einsum("hj,jhd->hd", w, v.abs())
            err = reach * (2.0 ** -8 + 2.2 * d[:, None] + len(seen) * 2.0 ** -23)
            got[first + i] = (out, lse, (out.abs() + err) * 2.0 ** -8 + err,
                              d + len(seen) * 2.0 ** -23 + lse.abs() * 2.0 ** -22)
    return got


def accept(sampled, tokens, parents, row0, draft_row0, draft_len, r):
    """(path, emitted tokens) of request r, from lists."""
    first, dfirst, n = row0[r], draft_row0[r], draft_len[r]
    path, emitted, at = [], [], 0
    while True:
        t = sampled[first + at]
        emitted.append(t)
        kids = [i for i in range(1, n + 1)
                if (i - 1 if parents is None else parents[first + i]) == at
                and tokens[dfirst + i - 1] == t]
        if not kids:
            return path, emitted
        at = kids[0]
        path.append(at)


def keep(cache, table, ctx, accepted, path):
    """In place on cache [layers, pages, page, heads, D]."""
    page = cache.shape[2]
    old = cache.clone()
    for r in range(len(ctx)):
        for i in range(accepted[r]):
            a, b = place(table, r, ctx[r] + path[r][i], page)
            c, d = place(table, r, ctx[r] + 1 + i, page)
            cache[:, c, d] = old[:, a, b]
