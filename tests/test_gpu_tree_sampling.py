"""Tokens sampled from the target's rows for spec_tree_accept, as its definition names the call: up to 63 drafts a
request at once, larger trees with every row a request of its own."""
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


@pytest.mark.parametrize("gamma", [5, 63, 64, 127])
def test_sampled_then_accepted(sv, orc, gamma):
    B, V, seed = 5, 24, 77
    g = torch.Generator().manual_seed(gamma)
    n = [gamma, gamma // 2, 0, gamma, 3]
    row0 = torch.arange(B) * (gamma + 1)
    rows = B * (gamma + 1)
    draft_row0 = torch.arange(B) * gamma
    parents = torch.full((rows,), -1, dtype=torch.int32)
    for r in range(B):
        a = int(row0[r])
        parents[a:a + n[r] + 1] = pr.make_tree(n[r] + 1, g)
    logits = torch.randn((rows, V), generator=g) * 2
    tokens = torch.randint(0, V, (B * gamma,), generator=g).to(torch.int32)
    dl = torch.tensor(n, dtype=torch.int32)
    d = [t.cuda() for t in (logits, row0, dl, tokens, parents, draft_row0)]
    if gamma < 64:
        sampled = sv.spec_sample_draft(d[0], d[1], d[2] + 1, gamma + 1, seed)
        st, want = orc.sample_draft_batch(logits.numpy(), V, V, row0.numpy(), (dl + 1).numpy(), B, seed)
    else:
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_sample_draft(d[0], d[1], d[2] + 1, gamma + 1, seed)
        every = torch.arange(rows)
        one = torch.ones(rows, dtype=torch.int32)
        sampled = sv.spec_sample_draft(d[0], every.cuda(), one.cuda(), 1, seed)
        st, want = orc.sample_draft_batch(logits.numpy(), V, V, every.numpy(), one.numpy(), rows, seed)
    used = torch.cat([torch.arange(int(a), int(a) + k + 1) for a, k in zip(row0, n)])
    assert st == 0 and torch.equal(sampled.cpu()[used], torch.from_numpy(want)[used])
    out = sv.spec_tree_accept(sampled, d[3], d[4], d[1], d[5], d[2], gamma)
    assert int(out["status"]) == sv.SV_OK
    for r in range(B):
        path, emitted = pr.accept(sampled.tolist(), tokens.tolist(), parents.tolist(), row0.tolist(),
                                  draft_row0.tolist(), n, r)
        assert out["accepted_len"][r] == len(path)
        assert out["path"][r].tolist() == path + [-1] * (gamma - len(path))
        assert out["out_tokens"][r].tolist() == emitted + [-1] * (gamma - len(path))
