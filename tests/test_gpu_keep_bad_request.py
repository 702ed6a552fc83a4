"""new_len of a request that spec_cache_keep leaves out: its ctx_len, so that the next round finds it as it was."""
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


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("layers,B", [(1, 3), (5, 3), (40, 60)])
@pytest.mark.parametrize("what", ["accepted", "none accepted", "order", "zero", "context", "page", "far", "room"])
def test_length_of_a_bad_request(sv, what, layers, B, given):
    ctx = [20 + 3 * r for r in range(B)]
    host, dev, n, _ = pr.make_round(ctx, [6] * B, 6, 16, 1, 2, 64, seed=61, nan_elsewhere=False)
    i32 = dict(dtype=torch.int32, device="cuda")
    accepted = torch.full((B,), 2, **i32)
    path = torch.tensor([[2, 4, 5]] * B, **i32)
    if what == "accepted":
        accepted[1] = 4
    elif what == "none accepted":
        accepted[1] = -1
    elif what == "order":
        path[1, 1] = 2
    elif what == "zero":
        path[1, 0] = 0
    elif what == "context":
        dev["ctx_len"][1] = -7
    elif what == "page":
        dev["page_table"][1, 1] = 10**6
    elif what == "far":
        path[1, 1] = 2**31 - 1
    else:
        dev["ctx_len"][1] = dev["page_table"].shape[1] * 16 - 2
    lengths = dev["ctx_len"].tolist()
    st = torch.full((1,), 9, **i32)
    k, v = (dev[c][None].repeat(layers, 1, 1, 1, 1) for c in ("k_cache", "v_cache"))
    new = torch.full((B,), 55, **i32) if given else None
    new = sv.spec_cache_keep(k, v, dev["page_table"], dev["ctx_len"], accepted, path, new_len=new, status=st)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    assert new.tolist() == [c if r == 1 else c + 3 for r, c in enumerate(lengths)]
    assert dev["ctx_len"].tolist() == lengths
    want = host["k_cache"][None].repeat(layers, 1, 1, 1, 1)
    pr.keep(want, host["page_table"], ctx, [0 if r == 1 else 2 for r in range(B)], path.tolist())
    assert torch.equal(k.cpu(), want)


@pytest.mark.parametrize("what", ["accepted", "context"])
def test_length_of_a_bad_chain(sv, what):
    """Chains (no path) move nothing, and their lengths are told the same way."""
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, accepted = torch.tensor([20, 9, 3], **i32), torch.tensor([2, 1, 0], **i32)
    if what == "accepted":
        accepted[1] = -1
    else:
        ctx[1] = -2
    cache = torch.zeros((2, 6, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    st = torch.full((1,), 9, **i32)
    new = sv.spec_cache_keep(cache[0], cache[1], torch.arange(6, **i32).view(3, 2), ctx, accepted, None, status=st,
                             new_len=torch.full((3,), 55, **i32))
    assert int(st) == sv.SV_ERR_BAD_INPUT
    assert new.tolist() == [23, int(ctx[1]), 4]
