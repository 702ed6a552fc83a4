"""spec_tree_attention against its binary64 form: contexts from nothing to long ones, chains, trees and
forests, head layouts, strides and page sizes, and what lies in places that a row does not see."""
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


def run(sv, dev, scale=None, **kw):
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    rows, heads, D = dev["q"].shape
    out = torch.full((rows, heads, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, heads), 77.0, device="cuda")
    args = dict(dev, **kw)
    sv.spec_tree_attention(args.pop("q"), scale=scale, out=out, lse=lse, status=st, **args)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(st)


def wide_table(dev, columns):
    """The same pages in a table of more columns (calls of few pages may take another way)."""
    t = torch.full((dev["page_table"].shape[0], columns), -7, dtype=torch.int32, device="cuda")
    t[:, :dev["page_table"].shape[1]] = dev["page_table"]
    return dict(dev, page_table=t)


def check(host, n, out, lse, scale):
    want = pr.attention(host, n, scale)
    for row in range(out.shape[0]):
        if row not in want:  # rows of no request stay as they were
            assert (out[row] == 77).all() and (lse[row] == 77).all(), row
            continue
        o, z, tol_o, tol_z = want[row]
        off = (lse[row].double() - z).abs()
        assert (off <= tol_z).all(), (row, float((off / tol_z).max()))
        off = (out[row].double() - o).abs()
        assert (off <= tol_o).all(), (row, float((off / tol_o).max()))


SHAPES = [  # contexts, drafts, most drafts, page, heads, kv heads, D, tree
    ([0], [0], 0, 16, 1, 1, 64, None),                      # a lone key
    ([1], [0], 0, 8, 8, 8, 128, None),
    ([127, 128, 129], [0, 0, 0], 3, 16, 8, 2, 128, None),   # ends around a tile's
    ([120, 122, 125], [5, 5, 5], 5, 32, 32, 8, 128, None),  # a round across a tile's end
    ([0, 1, 15, 16, 17, 300], [5, 0, 3, 5, 1, 4], 6, 16, 8, 2, 128, None),
    ([700, 33], [15, 15], 15, 64, 16, 4, 64, "random"),
    ([700, 33], [15, 2], 15, 64, 16, 4, 128, "random"),
    ([0, 250], [63, 40], 63, 128, 16, 2, 128, "random"),
    ([5, 200], [63, 63], 64, 256, 8, 1, 64, "star"),
    ([126, 1], [127, 100], 127, 32, 4, 4, 128, "random"),   # the largest trees
    ([126, 64], [126, 30], 127, 16, 14, 2, 64, "forest"),
    ([130], [20], 20, 512, 28, 4, 128, "chain"),            # pages longer than a tile
    ([40, 41], [5, 4], 5, 8, 7, 1, 64, "random"),
    ([77], [3], 3, 16, 128, 1, 128, "random"),              # as many heads a key head as can be
    ([90, 2], [1, 2], 2, 16, 100, 1, 64, None),
    ([64], [300], 300, 32, 8, 2, 128, None),                # a prompt's chunk
    ([0], [200], 200, 16, 4, 4, 64, None),
]


@pytest.mark.parametrize("case", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("q_scale,columns", [(1.0, 0), (6.0, 0), (1.0, 1100)])
def test_shapes(sv, case, q_scale, columns):
    ctx, drafts, gmax, page, heads, kv, D, tree = case
    host, dev, n, _ = pr.make_round(ctx, drafts, gmax, page, heads, kv, D, seed=len(ctx) + page,
                                    tree=tree, q_scale=q_scale)
    out, lse, st = run(sv, wide_table(dev, columns) if columns else dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("heads,kv", [(8, 8), (24, 2), (6, 2), (40, 4)])
@pytest.mark.parametrize("ctx,drafts", [([8100], [5]), ([1023, 4], [1, 3]), ([5000, 0, 900], [2, 1, 0])])
def test_few_requests_of_longer_contexts(sv, ctx, drafts, heads, kv):
    """The work of a call of few requests, in runs of tiles of any number."""
    host, dev, n, _ = pr.make_round(ctx, drafts, 5, 32, heads, kv, 128, seed=sum(ctx), tree="random")
    for d in (dev, wide_table(dev, 1100)):
        out, lse, st = run(sv, d)
        assert st == sv.SV_OK
        check(host, n, out, lse, 1 / math.sqrt(128))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv", [(8, 8), (32, 8), (64, 8)])
@pytest.mark.parametrize("ctx,drafts", [([900, 2000, 1], [5, 0, 3]), ([3900, 0, 128, 77], [7, 7, 1, 4])])
@pytest.mark.parametrize("tree", [None, "random"])
def test_some_requests(sv, ctx, drafts, heads, kv, D, tree):
    """Too many for the largest runs of SMs each, too few for the whole device: among them contexts of fewer tiles
    than a run has SMs, and none; the same rows from a table that takes the other way."""
    page = 16 if ctx[0] < 1000 else 64
    host, dev, n, _ = pr.make_round(ctx, drafts, 7, page, heads, kv, D, seed=len(ctx) + heads, tree=tree)
    for d in (dev, wide_table(dev, 1100)):
        out, lse, st = run(sv, d)
        assert st == sv.SV_OK
        check(host, n, out, lse, 1 / math.sqrt(D))
    dev["page_table"][1, 0] = dev["k_cache"].shape[0]
    out, lse, st = run(sv, dev)
    assert st == sv.SV_ERR_BAD_INPUT


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,kv", [(8, 2), (12, 12), (32, 2)])
def test_long_ragged_batch(sv, D, heads, kv):
    """Requests of very different lengths: their work is cut anywhere."""
    ctx = [3000, 0, 1, 517, 129, 2047, 64, 5, 900, 1500, 31, 257]
    drafts = [5, 0, 7, 3, 2, 7, 6, 1, 0, 4, 5, 7]
    host, dev, n, _ = pr.make_round(ctx, drafts, 7, 16, heads, kv, D, seed=5, tree="random")
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / math.sqrt(D))


def test_each_place_alone(sv):
    """A query that one key answers alone gets that key's value: every place of a tile's two, in turn."""
    D, page, ctx = 128, 16, 257
    host, dev, n, rows = pr.make_round([ctx], [ctx], ctx, page, 1, 1, D, seed=2, bonus=0)
    g = torch.Generator().manual_seed(3)
    sign = (torch.randint(0, 2, (ctx + ctx, D), generator=g) * 2 - 1).to(torch.bfloat16)
    for j in range(2 * ctx):
        host["k_cache"][pr.place(host["page_table"], 0, j, page)] = sign[j]
    first = int(host["row0"][0])
    # row i looks for place i: its score is D = 128 times 8, of another about +-11 times 8
    host["q"][first:first + ctx, 0] = sign[:ctx] * 8
    dev["k_cache"], dev["q"] = host["k_cache"].cuda(), host["q"].cuda()
    out, _, st = run(sv, dev, scale=1.0)
    assert st == sv.SV_OK
    for i in range(ctx):
        v = host["v_cache"][pr.place(host["page_table"], 0, i, page)][0].float()
        # (the weight is rounded to bf16, its sum is not; then the quotient is)
        assert ((out[first + i, 0].float() - v).abs() <= 2.0 ** -7 * v.abs() * 1.01).all(), i


@pytest.mark.parametrize("heads", [8, 40, 64])
def test_rising_scores(sv, heads):
    """Keys whose scores climb along the context, far beyond any first guess of the maximum, and
    fall again."""
    D = 128
    host, dev, n, _ = pr.make_round([2000], [5], 5, 32, heads, 2, D, seed=4)
    for j in range(2006):
        f = min(j, 2 * 1300 - j) / 60
        host["k_cache"][pr.place(host["page_table"], 0, j, 32)] = (
            f + 0.1 * torch.randn((2, D), generator=torch.Generator().manual_seed(j))).to(torch.bfloat16)
    host["q"] = host["q"].abs()
    dev["k_cache"], dev["q"] = host["k_cache"].cuda(), host["q"].cuda()
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
@pytest.mark.parametrize("heads", [8, 32, 80])
def test_scales(sv, scale, heads):
    host, dev, n, _ = pr.make_round([300, 9], [4, 2], 4, 16, heads, 2, 64, seed=6, tree="random")
    out, lse, st = run(sv, dev, scale=scale)
    assert st == sv.SV_OK
    check(host, n, out, lse, scale)


@pytest.mark.parametrize("tree", [None, "random"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx,heads", [(0, 8), (60, 8), (125, 8), (0, 16), (250, 16), (125, 64), (3, 64)])
def test_unseen_rows_do_not_reach(sv, tree, bad, ctx, heads):
    """What a drafted row left in the cache reaches only the rows that see it (up to 64 rows a key head,
    up to 128, more)."""
    D, kv, N = 128, 2, 9
    host, dev, n, _ = pr.make_round([ctx], [N], N, 16, heads, kv, D, seed=7, tree=tree)
    clean = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in host.items()}
    for j in (4, 7):
        for c in ("k_cache", "v_cache"):
            host[c][pr.place(host["page_table"], 0, ctx + j, 16)][0, 3:6] = bad  # head 0 of the cache
    dev["k_cache"], dev["v_cache"] = host["k_cache"].cuda(), host["v_cache"].cuda()
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    want = pr.attention(clean, n, 1 / math.sqrt(D))
    first = int(host["row0"][0])
    for i in range(n[0]):
        way = pr.ancestors(host["parents"], first, i)
        o, z, tol_o, tol_z = want[first + i]
        for h in range(heads):
            if h < heads // kv and (4 in way or 7 in way):
                continue
            assert ((out[first + i, h].double() - o[h]).abs() <= tol_o[h]).all(), (i, h)
            assert (lse[first + i, h].double() - z[h]).abs() <= tol_z[h], (i, h)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [2, 12, 40])
@pytest.mark.parametrize("tree", [None, "random"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite_reach_who_sees_them(sv, bad, tree, heads, D):
    """An infinite or NaN value of the context or of an ancestor makes that element of the result
    what the sum is; the other elements stay."""
    N, ctx = 6, 140
    for j in (3, ctx + 2):
        host, dev, n, _ = pr.make_round([ctx], [N], N, 16, heads, 1, D, seed=8, tree=tree, q_scale=0.1)
        clean = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in host.items()}
        host["v_cache"][pr.place(host["page_table"], 0, j, 16)][0, 5] = bad
        dev["v_cache"] = host["v_cache"].cuda()
        out, _, st = run(sv, dev)
        assert st == sv.SV_OK
        want = pr.attention(clean, n, 1 / math.sqrt(D))
        first = int(host["row0"][0])
        for i in range(n[0]):
            o, _, tol, _ = want[first + i]
            sees = j < ctx or j - ctx in pr.ancestors(host["parents"], first, i)
            off = (out[first + i].double() - o).abs() <= tol
            if sees:
                x = out[first + i, :, 5].float()
                assert (x != x).all() if bad != bad else (x == bad).all(), (j, i)
                off[:, 5] = True
            assert off.all(), (j, i)


@pytest.mark.parametrize("heads,kv,rows", [(2, 2, 230), (4, 1, 150), (3, 3, 100)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_of_long_chains_that_are_not_finite(sv, bad, heads, kv, rows):
    """... in rows far into a prompt, for the rows before them and those behind."""
    D, ctx = 128, 40
    host, dev, n, _ = pr.make_round([ctx, 300], [rows, 2], rows, 16, heads, kv, D, seed=18, bonus=0, q_scale=0.1)
    clean = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in host.items()}
    spots = [rows - 5, rows // 2 + 7, 3]
    for e, j in enumerate(spots):
        host["v_cache"][pr.place(host["page_table"], 0, ctx + j, 16)][0, 60 + 10 * e] = bad
    dev["v_cache"] = host["v_cache"].cuda()
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    want = pr.attention(clean, n, 1 / math.sqrt(D))
    first = int(host["row0"][0])
    for row, (o, z, tol, tol_z) in want.items():
        off = (out[row].double() - o).abs() <= tol
        assert ((lse[row].double() - z).abs() <= tol_z).all()
        for e, j in enumerate(spots):
            if first <= row < first + rows and row - first >= j:
                x = out[row, :heads // kv, 60 + 10 * e].float()
                assert (x != x).all() if bad != bad else (x == bad).all(), (row - first, j)
                off[:heads // kv, 60 + 10 * e] = True
        assert off.all(), row - first


@pytest.mark.parametrize("B", [33, 130, 700])
@pytest.mark.parametrize("heads", [2, 16])
def test_many_requests(sv, B, heads):
    """More requests than a warp has lanes, some without rows, some bad."""
    g = torch.Generator().manual_seed(B)
    ctx = torch.randint(0, 60, (B,), generator=g).tolist()
    drafts = torch.randint(0, 9, (B,), generator=g).tolist()
    drafts[-1] = 3
    host, dev, n, _ = pr.make_round(ctx, drafts, 8, 16, heads, 1, 64, seed=19, bonus=0, gap=0)
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / 8)
    bad = [0, B // 2, B - 2]
    dev["draft_len"][torch.tensor(bad, device="cuda")] = 9
    for r in bad:
        n[r] = 0
    out, lse, st = run(sv, dev)
    assert st == sv.SV_ERR_BAD_INPUT
    want = pr.attention(host, n, 1 / 8)
    for row, (o, z, tol, tol_z) in want.items():
        assert ((out[row].double() - o).abs() <= tol).all(), row


@pytest.mark.parametrize("kv", [1, 2, 8])
def test_bad_queries_stay_alone(sv, kv):
    host, dev, n, _ = pr.make_round([200], [5 if kv > 1 else 20], 20, 16, 8, kv, 128, seed=9)
    first = int(host["row0"][0])
    q = host["q"].clone()
    q[first + 2, 3] = float("nan")
    q[first + 4, 1] = float("inf")
    dev["q"] = q.cuda()
    out, lse, st = run(sv, dev)
    want = pr.attention(host, n, 1 / math.sqrt(128))
    for i in range(n[0]):
        for h in range(8):
            if (i, h) in ((2, 3), (4, 1)):
                assert out[first + i, h].isnan().all()
                continue
            o, z, tol_o, tol_z = want[first + i]
            assert ((out[first + i, h].double() - o[h]).abs() <= tol_o[h]).all(), (i, h)


@pytest.mark.parametrize("layout", ["heads first", "joint", "padded", "fused q"])
def test_layouts(sv, layout):
    """Caches with the heads outside the places, keys and values in one tensor, padded heads; queries
    beside other projections; results into a wider tensor."""
    D, kv, heads, page = 64, 2, 6, 16
    host, dev, n, rows = pr.make_round([150, 20], [4, 3], 5, page, heads, kv, D, seed=10, tree="random")
    kc, vc = dev["k_cache"], dev["v_cache"]
    if layout == "heads first":
        dev["k_cache"], dev["v_cache"] = (c.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
                                          for c in (kc, vc))
    elif layout == "joint":
        both = torch.stack((kc, vc), 1)
        dev["k_cache"], dev["v_cache"] = both[:, 0], both[:, 1]
    elif layout == "padded":
        both = torch.full((*kc.shape[:3], 2 * D + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
        both[..., :D], both[..., D + 8:2 * D + 8] = kc, vc
        dev["k_cache"], dev["v_cache"] = both[..., :D], both[..., D + 8:2 * D + 8]
    else:
        wide = torch.full((rows, heads + 3, D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 2:2 + heads, 8:] = dev["q"]
        dev["q"] = wide[:, 2:2 + heads, 8:]
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / math.sqrt(D))
    wide = torch.full((rows, heads + 2, D + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    args = dict(dev)
    sv.spec_tree_attention(args.pop("q"), out=wide[:, 1:1 + heads, 8:8 + D], **args)
    for r in range(2):
        first = int(host["row0"][r])
        assert torch.equal(wide[first:first + n[r], 1:1 + heads, 8:8 + D].cpu(), out[first:first + n[r]])
    assert (wide[:, 0] == 5).all() and (wide[:, -1] == 5).all()
    assert (wide[..., :8] == 5).all() and (wide[..., 8 + D:] == 5).all()


def test_shared_pages_and_heads_of_requests(sv):
    """Two requests whose contexts lie in the same pages."""
    D, page = 128, 32
    host, dev, n, _ = pr.make_round([96, 96], [3, 3], 3, page, 8, 2, D, seed=11, tree="random")
    host["page_table"][1, :3] = host["page_table"][0, :3]
    dev["page_table"] = host["page_table"].cuda()
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / math.sqrt(D))


def test_rows_do_not_depend_on_the_batch(sv):
    """A request alone, and the same one among others, to rounding; the same call twice, to the bit."""
    D = 128
    ctx, drafts = [500, 3000, 40, 900], [5, 3, 7, 0]
    host, dev, n, _ = pr.make_round(ctx, drafts, 7, 16, 16, 4, D, seed=12)
    a, b = run(sv, dev), run(sv, dev)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(host, n, a[0], a[1], 1 / math.sqrt(D))
    for r in range(4):
        one = dict(dev, row0=dev["row0"][r:r + 1], ctx_len=dev["ctx_len"][r:r + 1],
                   draft_len=dev["draft_len"][r:r + 1], page_table=dev["page_table"][r:r + 1])
        out, lse, _ = run(sv, one)
        sub = dict(host, row0=host["row0"][r:r + 1], ctx_len=host["ctx_len"][r:r + 1],
                   page_table=host["page_table"][r:r + 1])
        check(sub, [n[r]], out, lse, 1 / math.sqrt(D))


def test_cache_beyond_32_bits(sv):
    """Pages whose offsets pass 2^32 elements and 2^33 bytes."""
    D, kv, page = 128, 8, 128
    pages = (1 << 32) // (kv * D * page) + 40
    cache = torch.zeros((2, pages, page, kv, D), dtype=torch.bfloat16, device="cuda")
    host, dev, n, _ = pr.make_round([300, 130], [4, 2], 4, page, 16, kv, D, seed=13)
    far = pages - host["k_cache"].shape[0]
    cache[0, far:], cache[1, far:] = dev["k_cache"], dev["v_cache"]
    dev["page_table"] = torch.where(dev["page_table"] >= 0, dev["page_table"] + far, -7).to(torch.int32)
    dev["k_cache"], dev["v_cache"] = cache[0], cache[1]
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / math.sqrt(D))


def test_nothing_to_do(sv):
    host, dev, n, rows = pr.make_round([5, 9], [0, 0], 3, 16, 4, 2, 64, seed=14, bonus=0)
    out, lse, st = run(sv, dev)  # no rows at all
    assert st == sv.SV_OK and (out == 77).all() and (lse == 77).all()
    empty = dict(dev, row0=dev["row0"][:0], ctx_len=dev["ctx_len"][:0], draft_len=dev["draft_len"][:0],
                 page_table=dev["page_table"][:0])
    out, lse, st = run(sv, empty)
    assert st == sv.SV_OK and (out == 77).all()
    # some requests without rows
    host, dev, n, rows = pr.make_round([5, 90, 0], [0, 3, 0], 3, 16, 4, 2, 64, seed=15, bonus=0)
    out, lse, st = run(sv, dev)
    assert st == sv.SV_OK
    check(host, n, out, lse, 1 / 8)


@pytest.mark.parametrize("heads,columns", [(4, 0), (4, 1100), (64, 0)])
@pytest.mark.parametrize("what", ["length", "negative length", "context", "table", "page", "negative page",
                                  "row", "parent", "own parent"])
def test_bad_data_is_reported(sv, what, heads, columns):
    """... and leaves the other requests alone."""
    host, dev, n, rows = pr.make_round([70, 30, 90], [5, 5, 5], 5, 16, heads, 2, 64, seed=16, tree="random")
    if columns:
        dev = wide_table(dev, columns)
    first = int(host["row0"][1])
    if what == "length":
        dev["draft_len"][1] = 6
    elif what == "negative length":
        dev["draft_len"][1] = -1
    elif what == "context":
        dev["ctx_len"][1] = -1
    elif what == "table":
        dev["ctx_len"][1] = dev["page_table"].shape[1] * 16 - 5
    elif what == "page":
        dev["page_table"][1, 2] = dev["k_cache"].shape[0]
    elif what == "negative page":
        dev["page_table"][1, 0] = -1
    elif what == "row":
        dev["row0"][1] = rows - 5
    elif what == "parent":
        dev["parents"][first + 3] = -2
    else:
        dev["parents"][first + 3] = 3
    out, lse, st = run(sv, dev)
    assert st == sv.SV_ERR_BAD_INPUT
    want = pr.attention(host, n, 1 / 8)
    if what == "row":
        return  # (the last request's rows may be those that the bad one names)
    for r in (0, 2):
        for i in range(n[r]):
            row = int(host["row0"][r]) + i
            o, z, tol_o, tol_z = want[row]
            assert ((out[row].double() - o).abs() <= tol_o).all(), (r, i)


def test_other_stream_and_graph(sv):
    """On a side stream with tensors of the call's own; captured and replayed with new lengths."""
    host, dev, n, rows = pr.make_round([300, 20], [4, 2], 4, 16, 8, 2, 128, seed=17, tree="random")
    want = run(sv, dev)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = dict(dev)
    q = args.pop("q")
    got = sv.spec_tree_attention(q, stream=side, **args)
    side.synchronize()
    for r in range(2):
        first = int(host["row0"][r])
        assert torch.equal(got[first:first + n[r]].cpu(), want[first:first + n[r]])
    need = sv.spec_tree_attention_workspace_bytes(2, 4, True, 8, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_tree_attention(q, out=out, workspace=ws, status=st, **args)
    dev["ctx_len"].copy_(torch.tensor([120, 11], dtype=torch.int32))
    host["ctx_len"] = torch.tensor([120, 11], dtype=torch.int32)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert int(st) == sv.SV_OK
    want = pr.attention(host, n, 1 / math.sqrt(128))
    for row, (o, _, tol, _) in want.items():
        assert ((out[row].cpu().double() - o).abs() <= tol).all(), row
