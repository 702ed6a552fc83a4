"""The status word of the calls around verification: reset by every call, also by one that has
nothing to do, and only there where the caller gives it (a call that returns no status makes none)."""
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


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


def _allocations(call):
    """How many tensors torch allocated on the device during the call."""
    call()  # whatever is made once
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    call()
    return torch.cuda.memory_stats()["allocation.all.allocated"] - before


@pytest.mark.parametrize("marshalled", [True, False])
def test_no_status_is_made_that_nobody_can_read(sv, marshalled, monkeypatch):
    """spec_process_logits and spec_project_fp4 return their output only: without a status they
    allocate nothing (a word of their own would be free again before the kernel writes it)."""
    if not marshalled:
        monkeypatch.setattr(sv, "_fast", None)
        monkeypatch.setattr(sv, "_load_fast", lambda: None)
    x = torch.randn((2, 64), device="cuda")
    row0 = torch.arange(2, device="cuda")
    mask, rows = _i32(1, 2), torch.tensor([0, -1], dtype=torch.int32, device="cuda")
    lens = _i32(2)
    q = sv.spec_quantize_fp4(torch.randn((8, 64), device="cuda"), sv.SV_FP4_E8M0_32)
    y = torch.zeros((8, 8), device="cuda")
    assert _allocations(lambda: sv.spec_process_logits(x, row0, None, lens, 0, None, mask=mask,
                                                       mask_row=rows)) == 0
    assert _allocations(lambda: sv.spec_project_fp4(q, q, out=y)) == 0
    assert torch.isneginf(x[0]).all() and torch.isfinite(x[1]).all()
    assert torch.equal(y, sv.spec_project_fp4(q, q, dtype=torch.float32))


@pytest.mark.parametrize("marshalled", [True, False])
def test_a_call_with_nothing_to_do_resets_the_status(sv, marshalled, monkeypatch):
    if not marshalled:
        monkeypatch.setattr(sv, "_fast", None)
        monkeypatch.setattr(sv, "_load_fast", lambda: None)
    st = _i32(1)
    hist = dict(counts=_i32(2, 40), prompt_bits=_i32(2, 2), output_bits=_i32(2, 2), status=st)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    x = torch.randn((3, 64), device="cuda")
    calls = [lambda: sv.spec_history_append(_i32(2, 0), **hist),  # no columns
             lambda: sv.spec_history_append(_i32(0, 5), **hist),  # no rows
             lambda: sv.spec_history_append(_i32(0, 5), reset=True, **hist),
             lambda: sv.spec_process_logits(x, none, none, _i32(0), 4, _i32(1), status=st)]
    for fmt in (sv.SV_FP4_E8M0_32, sv.SV_FP4_E4M3_16):
        w = sv.spec_quantize_fp4(x, fmt)
        e = sv.spec_quantize_fp4(x[:0], fmt)
        rs = e["row_scales"]
        calls += [lambda fmt=fmt, e=e, rs=rs: sv.spec_quantize_fp4(
                      x[:0], fmt, packed=e["packed"], scales=e["scales"], row_scales=rs, status=st),
                  lambda e=e, w=w: sv.spec_project_fp4(e, w, out=torch.zeros((0, 8), device="cuda")[:, :3],
                                                       status=st)]
    for k, call in enumerate(calls):
        st.fill_(sv.SV_ERR_BAD_INPUT)
        call()
        assert int(st) == sv.SV_OK, k
