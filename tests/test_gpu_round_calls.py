"""The calls of a round over a paged cache through the binding: with and without the marshalling module,
on other streams, in captured graphs that run at once, from two host threads."""
import threading

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
    sv.lib()
    assert sv._fast is not None
    return sv


def inputs(seed=3, ctx=(300, 20, 77), drafts=(5, 2, 4), heads=8, kv=2, D=64, columns=0):
    host, dev, n, rows = pr.make_round(list(ctx), list(drafts), max(drafts), 16, heads, kv, D, seed=seed,
                                       tree="random", nan_elsewhere=False)
    g = torch.Generator("cuda").manual_seed(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    B = len(ctx)
    dev.update(qkv=torch.randn((rows, heads + 2 * kv, D), generator=g, device="cuda"),
               cos_sin=torch.randn((1000, D), generator=g, device="cuda"),
               sampled=torch.randint(0, 2, (rows,), generator=g, **i32),
               tokens=torch.randint(0, 2, (B * max(drafts),), generator=g, **i32),
               draft_row0=torch.arange(B, device="cuda") * max(drafts))
    if columns:
        t = torch.full((B, columns), -7, **i32)
        t[:, :dev["page_table"].shape[1]] = dev["page_table"]
        dev["page_table"] = t
    return host, dev, n, rows


def calls(sv, s, given, stream=None):
    """Every call once, in the order of a round; returns the results."""
    rows, heads, D = s["q"].shape
    kv = s["k_cache"].shape[2]
    B, g = len(s["ctx_len"]), s["max_draft_len"]
    new = lambda *n, **kw: torch.zeros(n, device="cuda", **kw) if given else None  # noqa: E731
    i32 = dict(dtype=torch.int32)
    st = [new(1, **i32) for _ in range(4)]
    lay = dict(page_table=s["page_table"], ctx_len=s["ctx_len"], row0=s["row0"], draft_len=s["draft_len"],
               max_draft_len=g, parents=s["parents"], stream=stream)
    q = sv.spec_cache_append(s["qkv"][:, :heads], s["qkv"][:, heads:heads + kv], s["qkv"][:, heads + kv:],
                             s["k_cache"], s["v_cache"], cos_sin=s["cos_sin"],
                             q_out=new(rows, heads, D, dtype=torch.bfloat16), status=st[0], **lay)
    lse = torch.zeros((rows, heads), device="cuda") if given else None
    out = sv.spec_tree_attention(q, s["k_cache"], s["v_cache"], out=torch.zeros_like(q) if given else None,
                                 lse=lse, status=st[1], **lay)
    acc = sv.spec_tree_accept(s["sampled"], s["tokens"], s["parents"], s["row0"], s["draft_row0"],
                              s["draft_len"], g, accepted_len=new(B, **i32), out_tokens=new(B, g + 1, **i32),
                              path=new(B, g, **i32), correction=new(B, **i32), status=st[2], stream=stream)
    length = sv.spec_cache_keep(s["k_cache"], s["v_cache"], s["page_table"], s["ctx_len"],
                                acc["accepted_len"], acc["path"], new_len=new(B, **i32), status=st[3],
                                stream=stream)
    return dict(q=q, out=out, lse=lse, new_len=length, k=s["k_cache"], v=s["v_cache"], acc=acc, st=st)


def used(host, n, t):
    """The requests' rows of t."""
    return torch.cat([t[int(a):int(a) + k] for a, k in zip(host["row0"], n)])


def same(host, n, a, b):
    for k in ("q", "out"):
        assert torch.equal(used(host, n, a[k]), used(host, n, b[k])), k
    for k in ("new_len", "k", "v"):
        assert torch.equal(a[k], b[k]), k
    for k in ("accepted_len", "out_tokens", "path", "correction"):
        assert torch.equal(a["acc"][k], b["acc"][k]), k


@pytest.mark.parametrize("columns", [0, 1100])
@pytest.mark.parametrize("heads", [8, 64])
def test_same_with_and_without_the_module(sv, monkeypatch, heads, columns):
    codes = []

    class Spy:
        def __getattr__(self, name):
            real = getattr(sv._fastcall, name)
            return lambda *a: codes.append(real(*a)) or codes[-1]

    kw = dict(heads=heads, columns=columns)
    host, s, n, _ = inputs(**kw)
    calls(sv, s, True)  # (the workspace is there from here on)
    with monkeypatch.context() as m:
        m.setattr(sv, "_fast", Spy())
        quick = calls(sv, inputs(**kw)[1], True)
    assert codes == [0] * 4
    assert all(int(t) == 0 for t in quick["st"])
    monkeypatch.setattr(sv, "_fast", None)
    monkeypatch.setattr(sv, "_load_fast", lambda: None)
    slow = calls(sv, inputs(**kw)[1], True)
    same(host, n, quick, slow)
    assert torch.equal(used(host, n, quick["lse"]), used(host, n, slow["lse"]))
    same(host, n, quick, calls(sv, inputs(**kw)[1], False))


@pytest.mark.parametrize("given", [False, True])
def test_on_another_stream(sv, given):
    """With long work ahead on the side stream, and tensors of the calls' own or the caller's."""
    host, s, n, _ = inputs()
    want = calls(sv, s, True)
    s = inputs()[1]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = calls(sv, s, given, side)
    filler = [torch.full((k,), 7.0, device="cuda") for k in (64, 1000, 4000, 1 << 16, 1 << 20) for _ in range(8)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in filler)
    same(host, n, want, got)


def test_two_graphs_at_once(sv):
    """Captured without a workspace of the caller's, each graph has its own: replayed together on two
    streams they give what each gives alone.  (Long contexts, cut into many parts.)"""
    made = []
    for seed in (5, 6):
        host, s, n, _ = inputs(seed, (9000, 4000, 7000, 100), (5, 3, 6, 2), 16, 2, 128, 1100)
        a = dict(page_table=s["page_table"], ctx_len=s["ctx_len"], row0=s["row0"], draft_len=s["draft_len"],
                 max_draft_len=s["max_draft_len"], parents=s["parents"])
        out, st = torch.zeros_like(s["q"]), torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.spec_tree_attention(s["q"], s["k_cache"], s["v_cache"], out=out, status=st, **a)
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                sv.spec_tree_attention(s["q"], s["k_cache"], s["v_cache"], out=out, status=st, **a)
        made.append((graph, out, want, st, torch.cuda.Stream(), s))
    for _ in range(20):
        for graph, out, _, _, stream, _ in made:
            with torch.cuda.stream(stream):
                out.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, st, _, _ in made:
        assert int(st) == 0 and torch.equal(out, want)


def test_two_host_threads(sv):
    """Each on a stream of its own."""
    host, s, n, _ = inputs(7, (3000, 50), (4, 4), columns=1100)
    want = calls(sv, s, True)
    results = {}

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                t = inputs(7, (3000, 50), (4, 4), columns=1100)[1]
                results[i] = calls(sv, t, True)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(2):
        same(host, n, want, results[i])


@pytest.mark.parametrize("fast", [True, False])
def test_wrong_arguments(sv, monkeypatch, fast):
    """Shapes, types, layouts and devices that do not fit are refused by name, with and without the
    module."""
    if not fast:
        monkeypatch.setattr(sv, "_fast", None)
        monkeypatch.setattr(sv, "_load_fast", lambda: None)
    _, s, _, rows = inputs()
    i32 = dict(dtype=torch.int32, device="cuda")
    z = lambda *n: torch.zeros(n, **i32)  # noqa: E731
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    lay = {k: s[k] for k in ("page_table", "ctx_len", "row0", "draft_len", "max_draft_len", "parents")}
    append = dict(q=s["qkv"][:, :8], k=s["qkv"][:, 8:10], v=s["qkv"][:, 10:], k_cache=s["k_cache"],
                  v_cache=s["v_cache"], q_out=bf(rows, 8, 64), cos_sin=s["cos_sin"], status=z(1), **lay)
    attend = dict(q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], out=bf(rows, 8, 64), status=z(1),
                  lse=torch.zeros((rows, 8), device="cuda"), **lay)
    accept = dict(sampled=s["sampled"], draft_tokens=s["tokens"], parents=s["parents"], row0=s["row0"],
                  draft_row0=s["draft_row0"], draft_len=s["draft_len"], max_draft_len=5, accepted_len=z(3),
                  out_tokens=z(3, 6), path=z(3, 5), correction=z(3), status=z(1))
    keep = dict(k_cache=s["k_cache"], v_cache=s["v_cache"], page_table=s["page_table"], ctx_len=s["ctx_len"],
                accepted_len=z(3), path=z(3, 5) + 1, new_len=z(3), status=z(1))
    half, cpu = s["q"].half(), s["q"].cpu()
    kc = s["k_cache"]
    common = [("page_table", z(2, 40)), ("page_table", s["page_table"].long()), ("ctx_len", z(4)),
              ("ctx_len", z(3).float()), ("page_table", s["page_table"].t()), ("v_cache", kc[:, :, :1]),
              ("v_cache", kc.float()), ("k_cache", kc.cpu()), ("v_cache", kc.transpose(1, 2).contiguous().transpose(1, 2)),
              ("status", z(1).long())]
    lengths = [("row0", z(3)), ("row0", torch.zeros(4, dtype=torch.int64, device="cuda")), ("draft_len", z(3, 1)),
               ("draft_len", z(3).long()), ("parents", z(rows + 1)), ("parents", z(rows).long())]
    for call, good, bad in (
            (sv.spec_cache_append, append, common + lengths + [
                ("q", half), ("k", s["qkv"][:, 8:11]), ("v", s["qkv"][:, 9:10]), ("k", s["qkv"][:, 8:10].transpose(1, 2)),
                ("q_out", bf(rows, 7, 64)), ("q_out", s["qkv"][:, :8]), ("cos_sin", s["cos_sin"].double()), ("v", cpu)]),
            (sv.spec_tree_attention, attend, common + lengths + [
                ("q", half), ("q", cpu), ("q", s["q"].float()), ("q", bf(rows, 8, 32)), ("out", bf(rows, 8, 65)[:, :, :63]),
                ("lse", torch.zeros((rows, 7), device="cuda")), ("lse", bf(rows, 8)), ("q", None),
                ("workspace", z(4))]),
            (sv.spec_tree_accept, accept, lengths + [
                ("sampled", s["sampled"].long()), ("draft_tokens", s["tokens"].cpu()), ("out_tokens", z(3, 5)),
                ("path", z(3, 4)), ("accepted_len", z(2)), ("correction", z(3).long()), ("draft_row0", z(3))]),
            (sv.spec_cache_keep, keep, common + [("accepted_len", z(3).long()), ("path", z(2, 5)),
                                                 ("path", z(3, 5).long()), ("new_len", z(2))])):
        call(**good)
        for name, value in bad:
            with pytest.raises((TypeError, ValueError)):
                call(**{**good, name: value})
    # synchronous refusals of the library keep their codes
    for call, kw, code in ((sv.spec_tree_attention, dict(attend, scale=float("nan")), sv.SV_ERR_INVALID),
                           (sv.spec_cache_append, dict(append, max_draft_len=-1), sv.SV_ERR_INVALID),
                           (sv.spec_cache_keep, dict(keep, new_len=s["ctx_len"]), sv.SV_ERR_INVALID),
                           (sv.spec_tree_accept, dict(accept, max_draft_len=-1), sv.SV_ERR_INVALID),
                           (sv.spec_tree_attention, dict(attend, max_draft_len=128), sv.SV_ERR_UNSUPPORTED)):
        with pytest.raises(sv.SpecVerifyError) as e:
            call(**kw)
        assert e.value.code == code
    torch.cuda.synchronize()
