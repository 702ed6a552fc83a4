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


def test_wrong_arguments_of_the_other_calls(sv):
    """Shapes, types and devices that do not fit, with and without the marshalling module."""
    i32 = dict(dtype=torch.int32, device="cuda")
    z = lambda *n: torch.zeros(n, **i32)  # noqa: E731
    f = lambda *n: torch.zeros(n, device="cuda")  # noqa: E731
    L = lambda *n: torch.zeros(n, dtype=torch.int64, device="cuda")  # noqa: E731
    B, V = 2, 64
    good = dict(logits=f(2, V), row0=torch.arange(2, device="cuda"), draft_row0=L(2), draft_len=z(2),
                max_draft_len=0, draft_tokens=z(1), counts=z(2, V), prompt_bits=z(2, 2),
                output_bits=z(2, 2), repetition=f(2) + 1, status=z(1))
    sv.spec_process_logits(**good)
    bad = [(dict(logits=f(2, V).half()), TypeError), (dict(logits=f(2, V).cpu()), ValueError),
           (dict(row0=z(2)), TypeError), (dict(row0=L(3)), ValueError),
           (dict(draft_row0=L(1)), ValueError), (dict(draft_tokens=L(1)), TypeError),
           (dict(draft_len=z(2).float()), TypeError), (dict(repetition=f(3)), ValueError),
           (dict(presence=f(2).double()), TypeError), (dict(counts=z(2, V + 1)), ValueError),
           (dict(counts=None), ValueError), (dict(counts=z(1, V), prompt_bits=z(1, 2),
                                                  output_bits=z(1, 2)), ValueError),
           (dict(slots=z(1)), ValueError), (dict(bias_start=z(2)), ValueError),
           (dict(bias_start=z(3), bias_tokens=z(1)), ValueError),
           (dict(bias_start=z(3), bias_tokens=z(2), bias_values=f(1)), ValueError),
           (dict(mask_row=z(3), mask=z(1, 2)), ValueError),
           (dict(mask_row=z(2), mask=z(1, 1)), ValueError), (dict(mask_row=z(2)), TypeError),
           (dict(out=f(2, V + 8)), ValueError), (dict(out=f(1, V)), ValueError),
           (dict(out=f(2, V).bfloat16()), TypeError)]
    for change, error in bad:
        for status in (good["status"], None):
            with pytest.raises(error):
                sv.spec_process_logits(**{**good, **change, "status": status})
    u8 = dict(dtype=torch.uint8, device="cuda")
    x = f(5, 100)
    for kw, error in [(dict(fmt=2), ValueError), (dict(packed=torch.zeros((5, 63), **u8)), ValueError),
                      (dict(scales=torch.zeros(7, **u8)), ValueError),
                      (dict(fmt=1, row_scales=f(4)), ValueError), (dict(values=f(5, 100)), TypeError),
                      (dict(values=f(5, 108).bfloat16()), ValueError), (dict(x=x.half()), TypeError),
                      (dict(x=x.t()), ValueError), (dict(x=x[0]), ValueError)]:
        with pytest.raises(error):
            sv.spec_quantize_fp4(**{**dict(x=x, fmt=0), **kw})
    q = {fmt: sv.spec_quantize_fp4(x, fmt) for fmt in (0, 1)}
    other = sv.spec_quantize_fp4(f(5, 99), 0)
    st = z(1)
    for a, b, kw, error in [
            (q[0], q[1], {}, ValueError), (q[0], other, {}, ValueError),
            (q[0], q[0], dict(out=f(5, 8)), ValueError), (q[0], q[0], dict(out=f(4, 5)), ValueError),
            (q[0], q[0], dict(out=torch.zeros((5, 8), **i32)[:, :5]), TypeError),
            (q[0], {**q[0], "scales": q[0]["scales"][:512]}, {}, ValueError),
            (q[0], {**q[0], "packed": q[0]["packed"][:4]}, {}, ValueError),
            (q[1], {**q[1], "row_scales": f(4)}, {}, ValueError),
            (q[1], {**q[1], "row_scales": None}, {}, (TypeError, ValueError, sv.SpecVerifyError))]:
        for status in (st, None):
            with pytest.raises(error):
                sv.spec_project_fp4(a, b, **{**dict(out=f(5, 8)[:, :5]), **kw}, status=status)


def test_two_host_threads_on_two_streams(sv):
    """Calls from two threads at once, each on its stream and tensors: the results of calls alone."""
    import threading
    want = _calls(sv)
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got[k] = [_calls(sv) for _ in range(10)]
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for runs in got.values():
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))
