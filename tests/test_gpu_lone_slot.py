"""The history of a single slot: its rows have no stride, so their buffers may be of any widths."""
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


@pytest.mark.parametrize("marshalled", [True, False])
@pytest.mark.parametrize("reset", [True, False])
def test_bit_rows_of_different_buffers(sv, reset, marshalled, monkeypatch):
    sv.lib()
    if not marshalled:
        monkeypatch.setattr(sv, "_fast", None)
        monkeypatch.setattr(sv, "_load_fast", lambda: None)
    i32 = dict(dtype=torch.int32, device="cuda")
    V = 300
    wide_c, wide_p, wide_o = (torch.full(s, 7, **i32) for s in ((2, 333), (3, 40), (2, 10)))
    counts, pb, ob = wide_c[1:, :V], wide_p[1:2, :10], wide_o[:1]
    for t in (counts, pb, ob):
        t.zero_()
    st = torch.zeros(1, **i32)
    hist = dict(counts=counts, prompt_bits=pb, output_bits=ob)
    tok = torch.tensor([[5, 299, 5]], **i32)
    sv.spec_history_append(tok, reset=reset, status=st, **hist)
    assert int(st) == 0
    sv.spec_history_append(torch.tensor([[64]], **i32), prompt=True, status=st, **hist)
    assert int(st) == 0 and counts.sum() == 3 and counts[0, 5] == 2 and counts[0, 299] == 1
    assert ob[0].tolist() == [32] + [0] * 8 + [1 << 11] and pb[0].tolist() == [0, 0, 1] + [0] * 7
    x = torch.ones((1, 304), device="cuda")
    zero = torch.zeros(1, **i32)
    sv.spec_process_logits(x[:, :V], zero.long(), None, zero, 0, None, status=st,
                           repetition=torch.full((1,), 2.0, device="cuda"), **hist)
    assert int(st) == 0 and (x == 0.5).nonzero()[:, 1].tolist() == [5, 64, 299]
    # nothing beside the rows was written
    assert (wide_c[0] == 7).all() and (wide_c[1, V:] == 7).all() and (wide_o[1] == 7).all()
    assert (wide_p[[0, 2]] == 7).all() and (wide_p[1, 10:] == 7).all()


@pytest.mark.parametrize("marshalled", [True, False])
def test_strides_of_several_slots_must_agree(sv, marshalled, monkeypatch):
    sv.lib()
    if not marshalled:
        monkeypatch.setattr(sv, "_fast", None)
        monkeypatch.setattr(sv, "_load_fast", lambda: None)
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sv.spec_history_append(torch.zeros((2, 3), **i32), torch.zeros((2, 64), **i32),
                               torch.zeros((2, 2), **i32), torch.zeros((2, 4), **i32)[:, :2],
                               status=torch.zeros(1, **i32))
