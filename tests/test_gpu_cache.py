"""spec_cache_append, spec_tree_accept and spec_cache_keep against their plain forms, and a whole round
of all the calls together."""
import math

import pytest
import torch

import plain_round as pr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return sv


def status():
    return torch.full((1,), 9, dtype=torch.int32, device="cuda")


# ---- append ------------------------------------------------------------------------------------

def rotated(x, cs, adjacent):
    """(x [heads, D] turned by cs [rot] = cosines, sines; the sum of magnitudes that went in)."""
    x, cs = x.double(), cs.double()
    h = len(cs) // 2
    c, s = cs[:h], cs[h:]
    y, m = x.clone(), torch.zeros_like(x)
    ia = torch.arange(h) * 2 if adjacent else torch.arange(h)
    ib = ia + 1 if adjacent else ia + h
    a, b = x[:, ia], x[:, ib]
    y[:, ia], y[:, ib] = a * c - b * s, a * s + b * c
    m[:, ia], m[:, ib] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    return y, m


def near(got, want, mag):
    """One rounding to bf16 of a sum of two products with three binary32 roundings."""
    tol = want.abs() * 2.0 ** -8 + mag * 3 * 2.0 ** -24 * 1.01
    return ((got.double() - want).abs() <= tol).all()


APPEND = [  # contexts, drafts, most, bonus, page, heads, kv, D, rot, tree
    ([0], [0], 0, 1, 16, 1, 1, 16, 16, None),
    ([1000], [5], 5, 1, 16, 32, 8, 128, 128, None),
    ([7, 0, 31, 32], [5, 3, 0, 6], 6, 1, 16, 8, 2, 128, 64, "random"),
    ([100, 90], [127, 64], 127, 1, 32, 4, 2, 64, 64, "random"),
    ([0, 0, 5], [40, 700, 0], 700, 0, 64, 5, 1, 128, 32, None),
    ([3, 9], [9, 2], 9, 1, 1, 3, 3, 48, 32, "star"),       # pages of one place
    ([13], [4], 4, 1, 48, 8, 8, 256, 240, "forest"),       # pages of an odd size
    ([77], [6], 6, 0, 16, 0, 4, 80, 80, None),             # no queries
    ([20, 4], [3, 3], 3, 1, 16, 70, 35, 128, 0, None),     # no rotation
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("case", APPEND, ids=[str(i) for i in range(len(APPEND))])
def test_append(sv, case, dtype, adjacent):
    ctx, drafts, gmax, bonus, page, heads, kv, D, rot, tree = case
    host, dev, n, rows = pr.make_round(ctx, drafts, gmax, page, max(heads, 1), kv, D, bonus=bonus,
                                       tree=tree, seed=D + page)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((rows, heads + 2 * kv, D), generator=g).to(dtype)
    if heads:
        qkv[2, 0, 0] = 3e38  # infinite in no step but the rounding, if that
    angle = torch.rand((max(ctx) + gmax + 1, max(rot // 2, 1)), generator=g) * 7 - 3
    cs = torch.cat((torch.cos(angle), torch.sin(angle)), 1) if rot else None
    d = qkv.cuda()
    kc, vc = dev["k_cache"].clone(), dev["v_cache"].clone()
    st = status()
    q_out = torch.full((rows, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sv.spec_cache_append(d[:, :heads] if heads else None, d[:, heads:heads + kv], d[:, heads + kv:],
                         kc, vc, dev["page_table"], dev["ctx_len"], dev["row0"], dev["draft_len"], gmax,
                         cos_sin=cs.cuda() if rot else None, adjacent=adjacent, parents=dev["parents"],
                         bonus_row=bool(bonus), q_out=q_out if heads else None, status=st)
    torch.cuda.synchronize()
    assert int(st) == sv.SV_OK
    kc, vc, q_out = kc.cpu(), vc.cpu(), q_out.cpu()
    want_k, want_v = host["k_cache"].clone(), host["v_cache"].clone()
    used = torch.zeros(rows, dtype=torch.bool)
    for r in range(len(ctx)):
        first = int(host["row0"][r])
        for i in range(n[r]):
            row = first + i
            used[row] = True
            pos = ctx[r] + len(pr.ancestors(host["parents"], first, i)) - 1
            at = pr.place(host["page_table"], r, ctx[r] + i, page)
            x = qkv[row]
            turn = (lambda y: rotated(y, cs[pos], adjacent)) if rot else (
                lambda y: (y.double(), torch.zeros_like(y).double()))
            for got, src in ((kc[at], x[heads:heads + kv]), (q_out[row], x[:heads])):
                y, mag = turn(src)
                fine = mag < 1e38
                assert near(torch.where(fine, got.float(), 0.0), torch.where(fine, y, 0.0), mag * fine)
            assert torch.equal(vc[at], x[heads + kv:].to(torch.bfloat16))
            want_k[at], want_v[at] = kc[at], vc[at]
    # nothing else was written
    assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))
    assert (q_out[~used] == 7).all()


def test_append_in_place_and_strided(sv):
    """Queries rotated where they lie; caches with heads outside the places; a cos_sin table wider than
    rot."""
    host, dev, n, rows = pr.make_round([50, 3], [5, 2], 5, 16, 8, 2, 64, seed=21, tree="random")
    g = torch.Generator("cuda").manual_seed(2)
    qkv = torch.randn((rows, 12, 64), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randn((64, 96), generator=g, device="cuda")[:, :64]
    kw = dict(parents=dev["parents"], cos_sin=table)
    a = [dev[k] for k in ("page_table", "ctx_len", "row0", "draft_len")] + [5]
    kc, vc = torch.zeros_like(dev["k_cache"]), torch.zeros_like(dev["v_cache"])
    want = sv.spec_cache_append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], kc, vc, *a, **kw)
    k2, v2 = (torch.zeros_like(c).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for c in (kc, vc))
    mine = qkv.clone()
    got = sv.spec_cache_append(mine[:, :8], mine[:, 8:10], mine[:, 10:], k2, v2, *a, q_out=mine[:, :8], **kw)
    assert got.data_ptr() == mine.data_ptr()
    for r in range(2):
        f = int(host["row0"][r])
        assert torch.equal(mine[f:f + n[r], :8], want[f:f + n[r]])
    assert torch.equal(mine[:, 8:], qkv[:, 8:])
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


@pytest.mark.parametrize("gmax", [5, 100])  # one cluster of CTAs; many CTAs
@pytest.mark.parametrize("what", ["length", "context", "table", "page", "row", "parent", "position"])
def test_append_bad_data(sv, what, gmax):
    host, dev, n, rows = pr.make_round([70, 90], [5, 5], gmax, 16, 4, 2, 64, seed=22, tree="random")
    qkv = torch.randn((rows, 8, 64), device="cuda")
    cs = torch.randn((100 if what != "position" else 92, 64), device="cuda")
    if what == "length":
        dev["draft_len"][1] = gmax + 1
    elif what == "context":
        dev["ctx_len"][1] = -3
    elif what == "table":
        dev["ctx_len"][1] = 2**31 - 2
    elif what == "page":
        dev["page_table"][1, 5] = -1
    elif what == "row":
        dev["row0"][1] = -1
    elif what == "parent":
        dev["parents"][int(host["row0"][1]) + 2] = 2
    else:
        dev["parents"] = None
    st = status()
    kc, vc = dev["k_cache"].clone(), dev["v_cache"].clone()
    sv.spec_cache_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], kc, vc, dev["page_table"], dev["ctx_len"],
                         dev["row0"], dev["draft_len"], gmax, cos_sin=cs, parents=dev["parents"], status=st)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    # the places of the first request are right all the same
    for i in range(6):
        at = pr.place(host["page_table"], 0, 70 + i, 16)
        assert torch.equal(vc[at].cpu(), qkv[int(host["row0"][0]) + i, 6:].to(torch.bfloat16).cpu())


# ---- accept ------------------------------------------------------------------------------------

@pytest.mark.parametrize("B,gmax,tokens,tree", [(1, 0, 2, None), (1, 15, 2, "random"), (5, 5, 2, None),
                                                (130, 63, 3, "random"), (40, 127, 2, "random"),
                                                (33, 127, 1, None), (9, 40, 1, "star"),
                                                (17, 31, 2, "forest"), (64, 1, 2, "random"), (256, 7, 2, "random"),
                                                (300, 9, 2, "random")])
@pytest.mark.parametrize("ragged", [False, True])
def test_accept(sv, B, gmax, tokens, tree, ragged):
    g = torch.Generator().manual_seed(B + gmax)
    n = torch.randint(0, gmax + 1, (B,), generator=g) if ragged else torch.full((B,), gmax)
    row0 = torch.randperm(B, generator=g) * (gmax + 2) + 1
    drow0 = torch.randperm(B, generator=g) * (gmax + 1)
    rows, drafts = B * (gmax + 2) + 1, B * (gmax + 1)
    sampled = torch.randint(0, tokens, (rows,), generator=g).to(torch.int32)
    tok = torch.randint(0, tokens, (drafts,), generator=g).to(torch.int32)
    parents = None
    if tree:
        parents = torch.full((rows,), 99, dtype=torch.int32)
        for r in range(B):
            parents[row0[r]:row0[r] + n[r] + 1] = pr.make_tree(int(n[r]) + 1, g, tree)
    wide = torch.full((B, gmax + 4), 55, dtype=torch.int32, device="cuda")
    st = status()
    out = sv.spec_tree_accept(sampled.cuda(), tok.cuda(), parents.cuda() if tree else None, row0.cuda(),
                              drow0.cuda(), n.to(torch.int32).cuda(), gmax, out_tokens=wide, status=st)
    assert int(st) == sv.SV_OK
    got = {k: v.cpu().tolist() for k, v in out.items()}
    for r in range(B):
        path, emitted = pr.accept(sampled.tolist(), tok.tolist(), parents.tolist() if tree else None,
                                  row0.tolist(), drow0.tolist(), n.tolist(), r)
        assert got["accepted_len"][r] == len(path)
        assert got["path"][r] == path + [-1] * (gmax - len(path))
        assert got["out_tokens"][r] == emitted + [-1] * (gmax - len(path)) + [55] * 3
        assert got["correction"][r] == emitted[-1]


@pytest.mark.parametrize("B", [3, 40, 400])
@pytest.mark.parametrize("what", ["length", "row", "draft row", "parent", "sample"])
def test_accept_bad_data(sv, what, B):
    i32 = dict(dtype=torch.int32, device="cuda")
    sampled, tok = torch.zeros(4 * B, **i32), torch.zeros(3 * B, **i32)
    parents = torch.tensor([-1, 0, 1, 2] * B, **i32)
    row0, drow0 = torch.arange(B, device="cuda") * 4, torch.arange(B, device="cuda") * 3
    n = torch.full((B,), 3, **i32)
    if what == "length":
        n[1] = 4
    elif what == "row":
        row0[1] = 4 * B - 3
    elif what == "draft row":
        drow0[1] = 3 * B - 2
    elif what == "parent":
        parents[5] = 1
    else:
        sampled[5] = -2
    st = status()
    out = sv.spec_tree_accept(sampled, tok, parents, row0, drow0, n, 3, status=st)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    assert (out["path"][torch.arange(B, device="cuda") != 1] == torch.tensor([1, 2, 3], **i32)).all()


# ---- keep --------------------------------------------------------------------------------------

@pytest.mark.parametrize("layers,B,N,depth,page,kv,D,ctx", [
    (1, 1, 1, 1, 16, 1, 8, 0), (2, 3, 9, 4, 16, 2, 64, 40), (3, 5, 63, 20, 8, 8, 128, 100),
    (1, 4, 127, 127, 16, 1, 128, 30), (0, 2, 5, 2, 16, 2, 64, 10), (5, 2, 30, 30, 1, 3, 24, 17),
    (2, 7, 40, 9, 24, 40, 256, 5)])
def test_keep(sv, layers, B, N, depth, page, kv, D, ctx):
    g = torch.Generator().manual_seed(N)
    lens = [ctx + r for r in range(B)]
    host, dev, n, _ = pr.make_round(lens, [N] * B, N, page, 1, kv, D, seed=N)
    pages = host["k_cache"].shape[0]
    k, v = (torch.randn((layers, pages, page, kv, D), generator=g).to(torch.bfloat16) for _ in "kv")
    accepted = [int(torch.randint(0, depth + 1, (1,), generator=g)) for _ in range(B)]
    accepted[0] = depth
    path = torch.full((B, N), -5, dtype=torch.int32)
    for r in range(B):
        rows = torch.randperm(N, generator=g)[:accepted[r]].sort()[0] + 1
        if r == B - 1:
            rows = torch.arange(accepted[r]) + 1  # a chain: nothing moves
        path[r, :accepted[r]] = rows.to(torch.int32)
    st = status()
    kd, vd = k.cuda(), v.cuda()
    new = sv.spec_cache_keep(kd, vd, dev["page_table"], dev["ctx_len"],
                             torch.tensor(accepted, dtype=torch.int32).cuda(), path.cuda(), status=st)
    assert int(st) == sv.SV_OK
    assert new.tolist() == [c + 1 + a for c, a in zip(lens, accepted)]
    pr.keep(k, host["page_table"], lens, accepted, path.tolist())
    pr.keep(v, host["page_table"], lens, accepted, path.tolist())
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_keep_one_layer_strided_and_chain(sv):
    host, dev, n, _ = pr.make_round([20, 30], [6, 6], 6, 16, 1, 2, 64, seed=31)
    both = torch.stack((dev["k_cache"].nan_to_num(0), dev["v_cache"].nan_to_num(0)), 1)
    want = both.clone()
    accepted = torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    new = sv.spec_cache_keep(both[:, 0], both[:, 1], dev["page_table"], dev["ctx_len"], accepted, None)
    assert new.tolist() == [23, 34] and torch.equal(both, want)
    path = torch.tensor([[1, 4, -1], [2, 3, 6]], dtype=torch.int32, device="cuda")
    sv.spec_cache_keep(both[:, 0], both[:, 1], dev["page_table"], dev["ctx_len"], accepted, path, new_len=new)
    for c in (0, 1):
        x = want[:, c].cpu()[None].clone()
        pr.keep(x, host["page_table"], [20, 30], [2, 3], path.tolist())
        assert torch.equal(both[:, c].cpu(), x[0])


@pytest.mark.parametrize("layers", [1, 5])
@pytest.mark.parametrize("what", ["accepted", "order", "zero", "context", "page", "far"])
def test_keep_bad_data(sv, what, layers):
    host, dev, n, _ = pr.make_round([20, 30, 40], [6] * 3, 6, 16, 1, 2, 64, seed=32, nan_elsewhere=False)
    accepted = torch.tensor([2, 2, 2], dtype=torch.int32, device="cuda")
    path = torch.tensor([[2, 4, 5]] * 3, dtype=torch.int32, device="cuda")
    if what == "accepted":
        accepted[1] = 4
    elif what == "order":
        path[1, 1] = 2
    elif what == "zero":
        path[1, 0] = 0
    elif what == "context":
        dev["ctx_len"][1] = -1
    elif what == "page":
        dev["page_table"][1, 2] = 10**6
        path[1, 1] = 6
        dev["ctx_len"][1] = 31
    else:
        path[1, 1] = 2**31 - 1
    st = status()
    k, v = (dev[c][None].repeat(layers, 1, 1, 1, 1) for c in ("k_cache", "v_cache"))
    sv.spec_cache_keep(k, v, dev["page_table"], dev["ctx_len"], accepted, path, status=st)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    want = host["k_cache"][None].repeat(layers, 1, 1, 1, 1)
    pr.keep(want, host["page_table"], [20, 30, 40], [2, 0, 2], path.tolist())
    assert torch.equal(k.cpu(), want)  # the others' entries moved, the bad request's did not


# ---- a round -----------------------------------------------------------------------------------

def test_round_of_all_calls(sv):
    """Two layers, trees of drafts: append and attention in each, projection, samples, accept, keep,
    history; then the next round finds the cache that decoding the emitted tokens one by one leaves."""
    torch.manual_seed(0)
    B, N, heads, kv, D, H, V, page, layers = 3, 9, 4, 2, 64, 128, 512, 16, 2
    ctx = [37, 0, 100]
    host, dev, n, rows = pr.make_round(ctx, [N, 4, N], N, page, heads, kv, D, seed=41, tree="random", gap=0,
                                       spare_pages=12, nan_elsewhere=False)
    pages = host["k_cache"].shape[0]
    # room for the rounds that follow
    table = torch.randperm(pages)[:3 * (pages // 3)].view(3, -1).to(torch.int32).cuda()
    k = torch.randn((layers, pages, page, kv, D), device="cuda").to(torch.bfloat16)
    v = torch.randn((layers, pages, page, kv, D), device="cuda").to(torch.bfloat16)
    start = k.clone(), v.clone()
    f = lambda *s: (torch.randn(s, device="cuda") / math.sqrt(s[-1])).to(torch.bfloat16)  # noqa: E731
    embed = f(V, H) * 8
    qkv_w = [f((heads + 2 * kv) * D, H) for _ in range(layers)]
    o_w = [f(H, heads * D) for _ in range(layers)]
    head = f(V, H) * 6
    cs = torch.rand((200, D), device="cuda") * 2 - 1

    def forward(tokens, lay, gmax, k, v):
        """Hidden rows of a round, its keys and values left in k, v."""
        h = embed[tokens.long()].float()
        st = [status() for _ in range(2 * layers)]
        for a in range(layers):
            x = (h.to(torch.bfloat16).float() @ qkv_w[a].float().t()).view(-1, heads + 2 * kv, D)
            q = sv.spec_cache_append(x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], k[a], v[a],
                                     table, lay["ctx_len"], lay["row0"], lay["draft_len"], gmax, cos_sin=cs,
                                     parents=lay["parents"], status=st[2 * a])
            y = torch.zeros_like(q)
            sv.spec_tree_attention(q, k[a], v[a], table, lay["ctx_len"], lay["row0"], lay["draft_len"], gmax,
                                   parents=lay["parents"], out=y, status=st[2 * a + 1])
            h = h + y.float().flatten(1) @ o_w[a].float().t()
        assert all(int(s) == 0 for s in st)
        return h.to(torch.bfloat16)

    i32 = torch.int32
    lay = {x: dev[x] for x in ("ctx_len", "row0", "draft_len", "parents")}
    draft_row0 = torch.arange(B, device="cuda") * N
    drafts = torch.randint(0, V, (B * N,), device="cuda", dtype=i32)

    def tokens_of(drafts):
        t = torch.zeros(rows, dtype=i32, device="cuda")
        for r in range(B):
            a = int(host["row0"][r])
            t[a] = 7 + r
            t[a + 1:a + n[r]] = drafts[r * N:r * N + n[r] - 1]
        return t

    # draft what the target itself would take, for some nodes: then some paths are long
    for _ in range(4):
        kk, vv = k.clone(), v.clone()
        logits = forward(tokens_of(drafts), lay, N, kk, vv).float() @ head.float().t()
        best = logits.argmax(1)
        for r in range(B):
            a = int(host["row0"][r])
            for i in range(1, n[r], 1 + r % 2):
                drafts[r * N + i - 1] = best[a + int(host["parents"][a + i])]
    tokens = tokens_of(drafts)
    hidden = forward(tokens, lay, N, k, v)
    logits = hidden.float() @ head.float().t()
    sampled = logits.argmax(1).to(i32)
    out = sv.spec_tree_accept(sampled, drafts, lay["parents"], lay["row0"], draft_row0, lay["draft_len"], N)
    new = sv.spec_cache_keep(k, v, table, lay["ctx_len"], out["accepted_len"], out["path"])
    assert int(out["status"]) == 0 and int(out["accepted_len"].max()) > 1
    counts = torch.zeros((B, V), dtype=i32, device="cuda")
    bits = [torch.zeros((B, V // 32), dtype=i32, device="cuda") for _ in range(2)]
    sv.spec_history_append(out["out_tokens"], counts, *bits)
    assert counts.sum(1).tolist() == (out["accepted_len"] + 1).tolist()

    # the same requests decoded one token at a time
    k1, v1 = start
    for r in range(B):
        emitted = [7 + r] + out["out_tokens"][r, :int(out["accepted_len"][r])].tolist()
        assert new[r] == ctx[r] + len(emitted)
        for i, t in enumerate(emitted):
            one = dict(ctx_len=torch.tensor([ctx[r] + i], dtype=i32, device="cuda"),
                       row0=torch.zeros(1, dtype=torch.int64, device="cuda"),
                       draft_len=torch.zeros(1, dtype=i32, device="cuda"), parents=None)
            saved, table = table, table[r:r + 1].contiguous()
            forward(torch.tensor([t], device="cuda"), one, 0, k1, v1)
            table = saved
    for r in range(B):
        for j in range(int(new[r])):
            at = pr.place(table.cpu(), r, j, page)
            # layer 0 sees the same inputs: equal to the bit; layer 1's come through an attention
            # whose sums may be cut otherwise: 2^-8 a rounding, and a few of them on the way
            assert torch.equal(k[0][at], k1[0][at]) and torch.equal(v[0][at], v1[0][at]), (r, j)
            for a, b in ((k[1][at], k1[1][at]), (v[1][at], v1[1][at])):
                assert (a.float() - b.float()).norm() <= 2.0 ** -5 * b.float().norm(), (r, j)
