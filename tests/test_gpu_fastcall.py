"""The marshalling module (_fastcall) makes the same calls as the Python checks, declines what is not
plain, and is the path that short calls take."""
import numpy as np
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
    sv.lib()
    assert sv._fast is not None
    return sv


def _calls(sv, stream=None):
    """Every call once, with all its outputs given; returns the outputs."""
    g = torch.Generator("cuda").manual_seed(3)
    i32 = dict(dtype=torch.int32, device="cuda")
    B, G, V, H = 3, 2, 1009, 100
    st = torch.full((1,), 5, **i32)
    counts, pb, ob = (torch.zeros(s, **i32) for s in ((4, V), (4, 32), (4, 32)))
    slots = torch.tensor([3, 0, 1], **i32)
    tok = torch.randint(-1, V, (B, 9), generator=g, **i32)
    kw = dict(status=st, stream=stream)
    sv.spec_history_append(tok, counts, pb, ob, slots=slots, **kw)
    sv.spec_history_append(tok[:, :4], counts, pb, ob, slots=slots, prompt=True,
                           lens=torch.tensor([4, 0, 2], **i32), **kw)
    x = torch.randn((B * (G + 1), 1016), generator=g, device="cuda")
    out = torch.zeros_like(x)
    f = lambda lo, hi: torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
    sv.spec_process_logits(
        x[:, :V], torch.arange(B, device="cuda") * (G + 1), torch.arange(B, device="cuda") * G,
        torch.tensor([2, 0, 1], **i32), G, torch.randint(0, V, (B * G,), generator=g, **i32),
        slots=slots, counts=counts, prompt_bits=pb, output_bits=ob, repetition=f(1, 2),
        presence=f(0, 1), frequency=f(0, 1), bias_start=torch.tensor([0, 2, 2, 3], **i32),
        bias_tokens=torch.tensor([4, 7, 1008], **i32), bias_values=f(-1, 1),
        mask=torch.randint(-2**31, 2**31, (2, 32), generator=g, device="cuda").int(),
        mask_row=torch.tensor([0, -1, 1, 0, 0, 0, -1, 1, 0], **i32), out=out[:, :V], **kw)
    ops = []
    for n, dt in ((40, torch.float32), (6, torch.bfloat16)):
        rs = torch.zeros(n, device="cuda")
        ops.append(sv.spec_quantize_fp4(
            torch.randn((n, H), generator=g, device="cuda").to(dt), 1, row_scales=rs,
            packed=torch.zeros((n, 64), dtype=torch.uint8, device="cuda"),
            scales=torch.zeros(2048, dtype=torch.uint8, device="cuda"),
            values=torch.zeros((n, H), dtype=torch.bfloat16, device="cuda"), **kw))
    y = torch.zeros((6, 40), device="cuda")
    sv.spec_project_fp4(ops[1], ops[0], out=y, **kw)
    torch.cuda.synchronize()
    assert int(st) == 0
    return [counts, pb, ob, out, y] + [o[k] for o in ops for k in ("packed", "scales", "row_scales")]


def test_same_as_python_checks(sv, monkeypatch):
    codes = []

    class Spy:
        def __getattr__(self, name):
            real = getattr(sv._fastcall, name)
            return lambda *a: codes.append(real(*a)) or codes[-1]

    with monkeypatch.context() as m:
        m.setattr(sv, "_fast", Spy())
        quick = _calls(sv)
    assert codes == [0] * 6  # every call went through the module
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = _calls(sv, side)
    monkeypatch.setattr(sv, "_fast", None)
    monkeypatch.setattr(sv, "_load_fast", lambda: None)
    slow = _calls(sv)
    for a, b, c in zip(quick, slow, on_side):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_declined_arguments_are_refused_by_name(sv):
    i32 = dict(dtype=torch.int32, device="cuda")
    st = torch.zeros(1, **i32)
    mk = lambda *s: torch.zeros(s, **i32)  # noqa: E731
    good = dict(tokens=mk(2, 3), counts=mk(2, 64), prompt_bits=mk(2, 2), output_bits=mk(2, 2),
                status=st)
    sv.spec_history_append(**good)
    for name, bad, error in [
            ("tokens", mk(2, 3).long(), TypeError), ("tokens", mk(6), ValueError),
            ("tokens", mk(3, 2).t(), ValueError), ("tokens", mk(2, 3).cpu(), ValueError),
            ("tokens", mk(3, 3), ValueError), ("counts", mk(2, 65), ValueError),
            ("prompt_bits", mk(1, 2), ValueError), ("output_bits", mk(2, 1), ValueError),
            ("output_bits", mk(2, 4)[:, :2], ValueError), ("lens", mk(3), ValueError),
            ("slots", mk(2).float(), TypeError), ("status", st.long(), TypeError),
            ("counts", None, TypeError), ("slots", [0, 1], TypeError),
            ("slots", np.zeros(2, np.int32), TypeError)]:
        with pytest.raises(error):
            sv.spec_history_append(**{**good, name: bad})
    # a synchronous refusal of the library keeps its code
    x = torch.zeros((2, 1001), device="cuda")
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_process_logits(x, torch.zeros(2, dtype=torch.int64, device="cuda"), None, mk(2), 0,
                               None, status=st)
    assert e.value.code == sv.SV_ERR_UNSUPPORTED
