"""Scores of spec_tree_attention as large as its definition allows, 2^27 in magnitude, of either sign: keys whose
products with the query are whole numbers, so that the largest alone carry the weight."""
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


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D,heads,columns", [(64, 8, 0), (128, 8, 1100), (64, 64, 0), (128, 128, 0)])
@pytest.mark.parametrize("tree", [None, "random"])
def test_largest_scores(sv, D, heads, columns, tree, sign):
    """One cluster, the list, and the wide kernel.  Products of up to 2^10 D / 64, times a scale of 2^17 (2^16): exact in
    binary32, as their differences are.  m, such a score times log2(e), is rounded by up to half a step of 2^4, which
    all weights of a row share: equal products keep equal weights, and others, 2^16 or more below, none."""
    ctx, N, kv = [700, 130], 9, 2
    host, dev, n, rows = pr.make_round(ctx, [N, 4], N, 16, heads, kv, D, seed=81, tree=tree)
    g = torch.Generator().manual_seed(2)
    whole = lambda *s: torch.randint(1, 5, s, generator=g).to(torch.bfloat16)  # noqa: E731
    used = host["k_cache"].isfinite()
    host["k_cache"] = torch.where(used, sign * whole(*host["k_cache"].shape), host["k_cache"])
    host["q"] = whole(*host["q"].shape)
    scale = 2.0 ** 17 * 64 / D
    dev["k_cache"], dev["q"] = host["k_cache"].cuda(), host["q"].cuda()
    if columns:
        t = torch.full((2, columns), -7, dtype=torch.int32, device="cuda")
        t[:, :dev["page_table"].shape[1]] = dev["page_table"]
        dev["page_table"] = t
    out = torch.zeros_like(dev["q"])
    lse = torch.zeros((rows, heads), device="cuda")
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    args = dict(dev)
    sv.spec_tree_attention(args.pop("q"), scale=scale, out=out, lse=lse, status=st, **args)
    assert int(st) == sv.SV_OK
    out, lse = out.cpu().double(), lse.cpu().double()
    most = 0.0
    for r in range(2):
        first = int(host["row0"][r])
        for i in range(n[r]):
            seen = list(range(ctx[r])) + [ctx[r] + j for j in pr.ancestors(host["parents"], first, i)]
            idx = [pr.place(host["page_table"], r, j, 16) for j in seen]
            pg, of = torch.tensor([a for a, _ in idx]), torch.tensor([b for _, b in idx])
            k, v = (host[c][pg, of].double().repeat_interleave(heads // kv, 1) for c in ("k_cache", "v_cache"))
            x = torch.einsum("hd,jhd->hj", host["q"][first + i].double(), k) * scale
            most = max(most, float(x.abs().max()))
            w = torch.softmax(x, 1)
            want, z = torch.einsum("hj,jhd->hd", w, v), torch.logsumexp(x, 1)
            reach = torch.einsum("hj,jhd->hd", w, v.abs())
            # the weights (equal ones) and the result are rounded to bf16 (2^-8 each), sums to binary32
            tol = (reach + want.abs()) * 2.0 ** -8 * 1.01 + reach * 2.0 ** -20
            assert ((out[first + i] - want).abs() <= tol).all(), (r, i)
            # log2(e), its product with the scale, m plus the logarithm of the sum, ln(2) and the product with it
            # round by 2^-24 each (m's own rounding comes back in the sum)
            assert ((lse[first + i] - z).abs() <= z.abs() * 5.05 * 2.0 ** -24).all(), (r, i)
    assert 2.0 ** 25 < most <= 2.0 ** 27
