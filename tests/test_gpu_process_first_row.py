"""spec_process_logits with a first row behind all rows: nothing is processed, up to the largest value
the argument can have (the kernel adds a group of rows to it)."""
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


@pytest.mark.parametrize("B", [1, 3, 200])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("first_row", [4, 5, 2**31 - 4, 2**31 - 1])
def test_first_row_behind_all_rows(sv, first_row, in_place, B):
    g, V = 3, 1000
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.randn((B * (g + 1), V), device="cuda")
    before = x.clone()
    out = x if in_place else torch.full_like(x, 5.0)
    want = out.clone()
    t0 = torch.arange(B, device="cuda") * (g + 1)
    st = torch.full((1,), 9, **i32)
    counts, pb, ob = (torch.full((B, n), -1, **i32) for n in (V, 32, 32))
    counts.fill_(3)
    kw = dict(out=out, counts=counts, prompt_bits=pb, output_bits=ob, status=st,
              repetition=torch.full((B,), 2.0, device="cuda"), first_row=first_row,
              mask=torch.zeros((1, 32), **i32), mask_row=torch.zeros(B * (g + 1), **i32))
    args = (x, t0, torch.arange(B, device="cuda") * g, torch.full((B,), g, **i32), g)
    sv.spec_process_logits(*args, torch.zeros(B * g, **i32), **kw)
    assert int(st) == 0
    # what the request itself says is still checked
    sv.spec_process_logits(*args, torch.full((B * g,), V, **i32), **kw)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    assert torch.equal(out, want) and torch.equal(x, before if not in_place else want)
