"""spec_tree_attention under page tables so wide that the list of work is counted in 64 bits (from 2^22 units on, a
unit being a key tile of 128 places of a key head)."""
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


@pytest.mark.parametrize("B,heads,kv,D,tree", [
    (1, 32, 8, 128, "random"), (3, 8, 8, 64, None), (5, 40, 2, 128, "random"), (31, 16, 4, 128, None),
    (33, 8, 2, 64, "random"), (70, 64, 2, 64, None), (130, 8, 1, 128, "random"), (300, 20, 1, 64, None)])
def test_wide_tables(sv, B, heads, kv, D, tree):
    """Up to 32 requests, up to 128 and more, in the narrow kernel and (from 65 rows a key head on) the wide one; some
    requests without rows, one with a long context."""
    page, gmax = 256, 5
    g = torch.Generator().manual_seed(B)
    ctx = torch.randint(0, 300, (B,), generator=g).tolist()
    ctx[B // 2] = 2500
    drafts = torch.randint(0, gmax + 1, (B,), generator=g).tolist()
    drafts[0] = gmax
    host, dev, n, rows = pr.make_round(ctx, drafts, gmax, page, heads, kv, D, seed=B, bonus=int(B % 2), tree=tree)
    columns = -(-(1 << 22) * 128 // (B * kv * page))
    table = torch.full((B, columns), -7, dtype=torch.int32, device="cuda")
    table[:, :dev["page_table"].shape[1]] = dev["page_table"]
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    out = torch.full((rows, heads, D), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, heads), 77.0, device="cuda")
    args = dict(dev, page_table=table)
    sv.spec_tree_attention(args.pop("q"), out=out, lse=lse, status=st, **args)
    assert int(st) == sv.SV_OK
    out, lse = out.cpu(), lse.cpu()
    want = pr.attention(host, n, 1 / math.sqrt(D))
    for row in range(rows):
        if row not in want:
            assert (out[row] == 77).all() and (lse[row] == 77).all(), row
            continue
        o, z, tol_o, tol_z = want[row]
        assert ((lse[row].double() - z).abs() <= tol_z).all(), row
        assert ((out[row].double() - o).abs() <= tol_o).all(), row
    # a bad request among them
    args["draft_len"] = dev["draft_len"].clone()
    args["draft_len"][B // 2] = gmax + 1
    sv.spec_tree_attention(dev["q"], out=torch.zeros_like(dev["q"]), status=st, **args)
    assert int(st) == sv.SV_ERR_BAD_INPUT
