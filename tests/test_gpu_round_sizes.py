"""Draft lengths and bounds next to 2^31: a length that max_draft_len allows and the rows do not is bad data,
and the other requests are served."""
import math

import pytest
import torch

import plain_round as pr

pytestmark = pytest.mark.gpu

MOST = 2**31 - 1


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return sv


def one_bad(drafts, r, **kw):
    host, dev, n, rows = pr.make_round([70, 200, 3], [5, 5, 5], 5, 16, 8, 2, 64, seed=51, nan_elsewhere=False, **kw)
    dev["draft_len"][r] = drafts
    dev["max_draft_len"] = MOST
    return host, dev, n, rows


@pytest.mark.parametrize("bonus", [0, 1])
@pytest.mark.parametrize("r", [0, 1, 2])
@pytest.mark.parametrize("drafts", [MOST, MOST - 1, 2**30])
def test_attention(sv, drafts, r, bonus):
    host, dev, n, rows = one_bad(drafts, r, bonus=bonus)
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    out = torch.full((rows, 8, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    args = dict(dev)
    sv.spec_tree_attention(args.pop("q"), out=out, status=st, **args)
    torch.cuda.synchronize()
    assert int(st) == sv.SV_ERR_BAD_INPUT
    n[r] = 0
    want = pr.attention(host, n, 1 / math.sqrt(64))
    out = out.cpu()
    for row in range(rows):
        if row not in want:
            assert (out[row] == 77).all(), row
            continue
        o, _, tol, _ = want[row]
        assert ((out[row].double() - o).abs() <= tol).all(), row


def test_append(sv):
    host, dev, n, rows = one_bad(MOST, 1)
    x = torch.randn((rows, 12, 64), device="cuda")
    k, v = dev["k_cache"].clone(), dev["v_cache"].clone()
    q = torch.full((rows, 8, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    sv.spec_cache_append(x[:, :8], x[:, 8:10], x[:, 10:], k, v, dev["page_table"], dev["ctx_len"], dev["row0"],
                         dev["draft_len"], MOST, q_out=q, status=st)
    torch.cuda.synchronize()
    assert int(st) == sv.SV_ERR_BAD_INPUT
    want_k, want_v = host["k_cache"].clone(), host["v_cache"].clone()
    want_q = torch.full((rows, 8, 64), 77.0, dtype=torch.bfloat16)
    y = x.to(torch.bfloat16).cpu()
    for r in (0, 2):
        for i in range(n[r]):
            row = int(host["row0"][r]) + i
            at = pr.place(host["page_table"], r, int(host["ctx_len"][r]) + i, 16)
            want_q[row], want_k[at], want_v[at] = y[row, :8], y[row, 8:10], y[row, 10:]
    assert torch.equal(q.cpu(), want_q) and torch.equal(k.cpu(), want_k) and torch.equal(v.cpu(), want_v)
