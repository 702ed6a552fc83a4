"""A row whose position lies behind the cosines' last is left out whole by spec_cache_append: its query and its
place keep what they hold, whatever part of a head turns."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("tree", [None, "random"])
@pytest.mark.parametrize("D,rot", [(64, 32), (64, 64), (128, 16), (48, 32), (256, 240), (256, 16)])
def test_bad_position(sv, D, rot, tree, adjacent, dtype):
    heads, kv, ctx = 6, 2, [70, 90]
    host, dev, n, rows = pr.make_round(ctx, [5, 5], 5, 16, heads, kv, D, seed=71, tree=tree)
    g = torch.Generator().manual_seed(1)
    x = torch.randn((rows, heads + 2 * kv, D), generator=g).to(dtype).cuda()
    positions = 92  # of the second request's rows some are behind it
    q = torch.full((rows, heads, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kc, vc = dev["k_cache"].clone(), dev["v_cache"].clone()
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    call = lambda cs, q, kc, vc: sv.spec_cache_append(  # noqa: E731
        x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:], kc, vc, dev["page_table"], dev["ctx_len"],
        dev["row0"], dev["draft_len"], 5, cos_sin=cs, adjacent=adjacent, parents=dev["parents"], q_out=q, status=st)
    table = torch.rand((200, rot), generator=g).cuda()
    call(table[:positions], q, kc, vc)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    # where the table is long enough, and those rows as they were
    q2, k2, v2 = torch.full_like(q, 7.0), dev["k_cache"].clone(), dev["v_cache"].clone()
    call(table, q2, k2, v2)
    assert int(st) == sv.SV_OK
    left = 0
    for i in range(n[1]):
        if ctx[1] + len(pr.ancestors(host["parents"], int(host["row0"][1]), i)) - 1 < positions:
            continue
        left += 1
        at = pr.place(host["page_table"], 1, ctx[1] + i, 16)
        q2[int(host["row0"][1]) + i] = 7.0
        k2[at], v2[at] = dev["k_cache"][at], dev["v_cache"][at]
    assert left
    for a, b in ((q, q2), (kc, k2), (vc, v2)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
