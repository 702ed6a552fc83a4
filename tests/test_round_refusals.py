"""The calls of a round over a paged cache refuse invalid arguments synchronously: nothing is launched,
so no GPU is needed."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    build.build()
    return sv


FAKE = C.c_void_p(4096)  # never dereferenced: validation fails first
ODD = C.c_void_p(4100)
OTHER = C.c_void_p(8192)


def test_append_refusals(sv):
    def call(q=FAKE, ldq=512, qh=64, k=FAKE, ldk=512, kh=64, v=FAKE, dtype=1, rows=12, heads=4, kv=2, D=64,
             cs=FAKE, ldcs=64, pos=100, rot=64, adj=0, row0=FAKE, g=5, bonus=1, parents=None, B=2, ldp=4,
             mp=4, qo=C.c_void_p(8192), ldqo=256, qoh=64, kc=FAKE, pages=9, page=16, ps=2048, ts=128, hs=64):
        return sv.lib().spec_cache_append(q, ldq, qh, k, ldk, kh, v, ldk, kh, dtype, rows, heads, kv, D, cs,
                                          ldcs, pos, rot, adj, row0, FAKE, g, bonus, parents, B, FAKE, FAKE,
                                          ldp, mp, qo, ldqo, qoh, kc, FAKE, pages, page, ps, ts, hs, None, None)
    bad, no = sv.SV_ERR_INVALID, sv.SV_ERR_UNSUPPORTED
    for kw in (dict(dtype=2), dict(g=-1), dict(bonus=2), dict(B=-1), dict(rows=-1), dict(mp=-1), dict(ldp=3),
               dict(pages=-1), dict(page=0), dict(heads=-1), dict(kv=0), dict(D=0), dict(adj=2), dict(rot=0),
               dict(rot=80), dict(ldcs=63), dict(pos=-1), dict(cs=None), dict(k=None), dict(v=None),
               dict(kc=None), dict(row0=None), dict(q=None), dict(qo=None),
               dict(qo=FAKE), dict(qo=FAKE, dtype=0)):
        assert call(**kw) == bad, kw
    for kw in (dict(D=72, rot=64), dict(D=272), dict(rot=24), dict(parents=FAKE, g=128), dict(q=ODD), dict(k=ODD),
               dict(kc=ODD), dict(ldq=508), dict(kh=60), dict(ps=2044), dict(ts=132), dict(hs=66), dict(ldqo=260),
               dict(ldcs=65), dict(B=2**20, g=2**20), dict(heads=2**30, kv=1)):
        assert call(**kw) == no, kw
    assert call(B=0) == sv.SV_OK and call(g=0, bonus=0) == sv.SV_OK and call(rows=0) == sv.SV_OK


def test_attention_refusals(sv):
    def call(q=FAKE, ldq=512, qh=64, rows=12, heads=4, kv=2, D=64, scale=0.1, row0=FAKE, g=5, bonus=1,
             parents=None, B=2, ldp=4, mp=4, kc=FAKE, pages=9, page=16, ps=2048, ts=128, hs=64, out=FAKE,
             ldo=256, lse=None, ldl=0, ws=FAKE, wb=1 << 40):
        return sv.lib().spec_tree_attention(q, ldq, qh, rows, heads, kv, D, scale, row0, FAKE, g, bonus, parents,
                                            B, FAKE, FAKE, ldp, mp, kc, FAKE, pages, page, ps, ts, hs, out, ldo,
                                            64, lse, ldl, None, ws, wb, None)
    bad, no = sv.SV_ERR_INVALID, sv.SV_ERR_UNSUPPORTED
    for kw in (dict(g=-1), dict(bonus=-1), dict(B=-1), dict(rows=-2), dict(ldp=3), dict(pages=-1), dict(page=0),
               dict(heads=0), dict(kv=0), dict(heads=5), dict(D=0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=3e38), dict(lse=FAKE, ldl=3), dict(q=None), dict(kc=None),
               dict(out=None),
               dict(row0=None), dict(ws=None), dict(wb=0)):
        assert call(**kw) == bad, kw
    for kw in (dict(D=32), dict(D=256), dict(heads=258), dict(page=4), dict(page=24), dict(parents=FAKE, g=128),
               dict(q=ODD), dict(out=ODD), dict(kc=ODD), dict(ldq=500), dict(ps=2052), dict(hs=63),
               dict(ws=C.c_void_p(4352 + 16))):
        assert call(**kw) == no, kw
    assert call(B=0) == sv.SV_OK and call(g=0, bonus=0) == sv.SV_OK and call(rows=0) == sv.SV_OK
    need = sv.spec_tree_attention_workspace_bytes
    assert need(2, 5, 1, 4, 2, 64) > 0
    assert need(2, 5, 1, 4, 3, 64) == need(-1, 5, 1, 4, 2, 64) == need(2, 5, 1, 4, 2, 32) == 0


def test_accept_refusals(sv):
    def call(sampled=FAKE, tok=FAKE, g=5, B=2, rows=12, drafts=10, acc=FAKE, out=FAKE, ldo=6, path=FAKE, ldp=5):
        return sv.lib().spec_tree_accept(sampled, tok, None, FAKE, FAKE, FAKE, g, B, rows, drafts, acc, out, ldo,
                                         None, path, ldp, None, None)
    bad = sv.SV_ERR_INVALID
    for kw in (dict(g=-1), dict(B=-1), dict(rows=-1), dict(drafts=-1), dict(ldo=5), dict(ldp=4), dict(sampled=None),
               dict(tok=None), dict(acc=None), dict(out=None)):
        assert call(**kw) == bad, kw
    assert call(g=128, ldo=200, ldp=200) == sv.SV_ERR_UNSUPPORTED
    assert call(B=0) == sv.SV_OK


def test_keep_refusals(sv):
    def call(acc=FAKE, path=FAKE, ldpath=5, n=5, B=2, ldp=4, mp=4, kc=FAKE, layers=2, ls=1 << 14, pages=9, page=16,
             ps=2048, ts=128, hs=64, kv=2, D=64, ctx=FAKE, new=None):
        return sv.lib().spec_cache_keep(acc, path, ldpath, n, B, ctx, FAKE, ldp, mp, kc, FAKE, layers, ls, pages,
                                        page, ps, ts, hs, kv, D, new, None, None)
    bad, no = sv.SV_ERR_INVALID, sv.SV_ERR_UNSUPPORTED
    for kw in (dict(acc=None), dict(ldpath=4), dict(n=-1), dict(B=-1), dict(ldp=3), dict(kc=None), dict(layers=-1),
               dict(pages=-1), dict(page=0), dict(kv=0), dict(D=0), dict(ctx=None), dict(new=FAKE)):
        assert call(**kw) == bad, kw
    # the lengths that a request's other layers still read
    assert call(acc=OTHER, new=OTHER) == bad
    for kw in (dict(n=128, ldpath=128), dict(D=12), dict(kc=ODD), dict(ls=4), dict(ps=2047), dict(ts=4),
               dict(B=2**20, layers=2**12)):
        assert call(**kw) == no, kw
    assert call(B=0) == sv.SV_OK


def test_host_tensors_and_wrong_types_are_refused(sv):
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    t = torch.zeros((1, 3), dtype=torch.int32)
    r = torch.zeros(1, dtype=torch.int64)
    for call in (lambda: sv.spec_cache_append(x, x, x, c, c, t, i, r, i, 1),
                 lambda: sv.spec_tree_attention(x, c, c, t, i, r, i, 1),
                 lambda: sv.spec_tree_accept(i, i, None, r, r, i, 1),
                 lambda: sv.spec_cache_keep(c, c, t, i, i, None)):
        with pytest.raises((ValueError, TypeError)):
            call()
