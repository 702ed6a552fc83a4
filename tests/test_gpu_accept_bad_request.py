"""What spec_tree_accept returns for a request whose data are bad: nothing is emitted, in buffers that held
something else, and the calls behind it leave that request as it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return sv


def inputs(B, what, bad):
    """Trees of three drafts, a chain each, whose rows all sample the token drafted behind them, then 5."""
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(sampled=torch.tensor([1, 2, 3, 5] * B, **i32), draft_tokens=torch.tensor([1, 2, 3] * B, **i32),
             parents=torch.tensor([-1, 0, 1, 2] * B, **i32), row0=torch.arange(B, device="cuda") * 4,
             draft_row0=torch.arange(B, device="cuda") * 3, draft_len=torch.full((B,), 3, **i32), max_draft_len=3)
    for r in bad:
        if what == "long":
            s["draft_len"][r] = 4
        elif what == "negative length":
            s["draft_len"][r] = -1
        elif what == "row":
            s["row0"][r] = 4 * B - 3
        elif what == "draft row":
            s["draft_row0"][r] = -1
        elif what == "first sample":
            s["sampled"][4 * r] = -2
        elif what == "later sample":
            s["sampled"][4 * r + 2] = -2**31
    return s


WHAT = ["long", "negative length", "row", "draft row", "first sample", "later sample"]


@pytest.mark.parametrize("parents", [True, False])
@pytest.mark.parametrize("B", [3, 40, 400])
@pytest.mark.parametrize("what", WHAT)
def test_outputs_of_a_bad_request(sv, what, B, parents):
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [1, B - 1]
    s = inputs(B, what, bad)
    if not parents:
        s["parents"] = None
    old = lambda *n: torch.full(n, 55, **i32)  # noqa: E731
    out = sv.spec_tree_accept(**s, accepted_len=old(B), out_tokens=old(B, 6), path=old(B, 5), correction=old(B),
                              status=old(1))
    assert int(out["status"]) == sv.SV_ERR_BAD_INPUT
    for r in range(B):
        got = [out[k][r].tolist() for k in ("accepted_len", "out_tokens", "path", "correction")]
        if r in bad:  # columns behind the last are not written
            assert got == [-1, [-1] * 4 + [55] * 2, [-1] * 3 + [55] * 2, -1], r
        else:
            assert got == [3, [1, 2, 3, 5, 55, 55], [1, 2, 3, 55, 55], 5], r


@pytest.mark.parametrize("what", WHAT)
def test_calls_behind_it(sv, what):
    """Neither the history nor the cache takes anything from the round before or from memory that nobody set."""
    B, page, kv, D = 3, 16, 2, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    out = sv.spec_tree_accept(**inputs(B, what, [1]))
    counts = torch.zeros((B, 32), **i32)
    bits = [torch.zeros((B, 1), **i32) for _ in range(2)]
    sv.spec_history_append(out["out_tokens"], counts, *bits)
    assert counts.sum(1).tolist() == [4, 0, 4]
    cache = torch.randn((2, 6, page, kv, D), device="cuda").to(torch.bfloat16)
    was = cache.clone()
    ctx = torch.tensor([20, 9, 3], **i32)
    st = torch.zeros(1, **i32)
    sv.spec_cache_keep(cache[0], cache[1], torch.arange(6, **i32).view(3, 2), ctx, out["accepted_len"], out["path"],
                       status=st)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    assert torch.equal(cache, was)  # chains lie in place
