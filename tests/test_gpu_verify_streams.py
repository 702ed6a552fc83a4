"""Verification, sampling and scheduling on streams other than the current one, with workspace,
status and outputs left to the binding."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_token_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return sv


def _inputs(B, gamma, V, seed):
    w = synth.scaled(synth.TOKEN_LARGE, B=B, gamma=gamma, V=V, seed=seed, gen_seed=seed)
    d = synth.token_inputs(w, device="cuda")
    g = np.random.default_rng(seed)
    K = gamma
    d["conf"] = torch.from_numpy(g.uniform(0.3, 1, (B, K)).astype(np.float32)).cuda()
    d["len"] = torch.full((B,), K, dtype=torch.int32, device="cuda")
    d["b_max"] = B * (K + 1)
    d["sps"] = torch.from_numpy(1.0 / (2e-3 + np.arange(d["b_max"] + 1) * 4e-6)).cuda()
    torch.cuda.synchronize()
    return d


def _round(sv, d, stream):
    """Drafts sampled, verified both ways, and the next round scheduled: every result, by name."""
    gm, rows = d["max_draft_len"], (d["target_row0"], d["draft_row0"], d["draft_len"])
    tok = sv.spec_sample_draft(d["draft"], *rows[1:], gm, d["seed"], stream=stream)
    a = sv.spec_verify_token(d["target"], d["draft"], *rows, gm, tok, d["seed"], stream=stream)
    b = sv.spec_verify_block(d["target"], d["draft"], *rows, gm, tok, d["seed"], stream=stream)
    c = sv.dspark_schedule(d["conf"], d["len"], d["sps"], d["b_max"], stream=stream)
    out = {"drafts": tok}
    for name, part in (("token", a), ("block", b), ("schedule", c)):
        out.update({name + "." + k: v for k, v in part.items() if v is not None})
    return out


def _same(got, want):
    torch.cuda.synchronize()
    assert got.keys() == want.keys()
    for k, v in want.items():
        assert torch.equal(got[k], v), k
        if k.endswith("status"):
            assert int(got[k]) == 0


def test_workspace_of_each_stream(sv):
    a = sv.workspace(1000)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = sv.workspace(1000)
        assert sv.workspace(500).data_ptr() == b.data_ptr()
    assert sv.workspace(1000).data_ptr() == a.data_ptr() != b.data_ptr()


def test_rounds_on_two_streams_at_once(sv):
    """Two rounds of unequal size from one host thread, neither waiting for the other."""
    ins = [_inputs(24, 5, 20000, 3), _inputs(9, 3, 33328, 4)]
    want = [_round(sv, d, None) for d in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # both queues fill before either runs
    got = [[_round(sv, d, s) for d, s in zip(ins, streams)] for _ in range(5)]
    for pair in got:
        for g, w in zip(pair, want):
            _same(g, w)


@pytest.mark.parametrize("busy", ["side", "current"])
def test_tensors_of_the_call_belong_to_its_stream(sv, busy):
    d = _inputs(8, 4, 5000, 9)
    want = _round(sv, d, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    if busy == "side":
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)  # some 20 ms
    else:
        torch.cuda._sleep(40_000_000)
        for n in (1, 2, 8, 40, 256, 4096, 1 << 18):  # freed, and still to be written
            for _ in range(8):
                torch.full((n,), 7, dtype=torch.int32, device="cuda")
    got = _round(sv, d, side)
    mine = [torch.full((n,), 7, dtype=torch.int32, device="cuda")
            for n in (1, 2, 8, 40, 256, 4096, 1 << 18) for _ in range(8)]
    _same(got, want)
    assert all((t == 7).all() for t in mine)


def test_stream_as_a_positional_argument(sv):
    g = torch.Generator("cuda").manual_seed(1)
    stats = torch.rand((2, 5, 4), generator=g, device="cuda") + 1
    tok = torch.rand((2, 5, 2), generator=g, device="cuda")
    want = sv.spec_verify_shard_merge(stats, tok)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sv.spec_verify_shard_merge(stats, tok, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = _inputs(3, 2, 504, 1)
    args = (d["conf"], d["len"], d["sps"], d["b_max"], True, None, None)
    want = sv.dspark_schedule(*args, None, sv.SV_STOP_ARGMAX)
    torch.cuda.synchronize()
    got = sv.dspark_schedule(*args, side, sv.SV_STOP_ARGMAX)
    _same(got, want)


def test_an_output_in_pinned_host_memory(sv):
    """What the caller gives may lie in host memory that the device can write."""
    N, K = 5, 3
    i32 = dict(dtype=torch.int32, device="cuda")
    sel, acc = torch.full((N,), K, **i32), torch.tensor([0, 1, 2, 3, 3], **i32)

    def update(out, stream):
        n = [torch.zeros(K, dtype=torch.float64, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        r = sv.dspark_acceptance_update(sel, acc, *n, cond_accept_out=out, stream=stream)
        torch.cuda.synchronize()
        assert int(r["status"]) == 0
        return r["cond_accept"]

    want = update(torch.zeros((N, K), device="cuda"), None)
    got = update(torch.zeros((N, K)).pin_memory(), torch.cuda.Stream())
    assert not got.is_cuda and torch.equal(got, want.cpu())
