"""The calls around verification on a stream that is not the current one, with tensors of their own
(status, outputs): these belong to that stream, whatever the current one does meanwhile."""
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


def _inputs():
    g = torch.Generator("cuda").manual_seed(11)
    i32 = dict(dtype=torch.int32, device="cuda")
    V, H, rows = 1009, 320, 6
    s = dict(V=V, H=H, rows=rows, x=torch.randn((rows, H), generator=g, device="cuda"),
             w=torch.randn((V, H), generator=g, device="cuda"),
             counts=torch.zeros((rows, V), **i32), pb=torch.zeros((rows, 32), **i32),
             ob=torch.zeros((rows, 32), **i32), rep=torch.full((rows,), 1.5, device="cuda"),
             tok=torch.randint(0, V, (rows, 9), generator=g, **i32),
             row0=torch.arange(rows, device="cuda"), zero=torch.zeros(rows, **i32))
    s["bad_tok"] = s["tok"].clone()
    s["bad_tok"][2, 3] = V
    s["bad_x"] = s["x"].clone()
    s["bad_x"][1, 7] = float("nan")
    return s


def _calls(sv, s, fmt, stream):
    """All four calls, every tensor that may be left out left out.  Returns results and statuses."""
    h = dict(counts=s["counts"], prompt_bits=s["pb"], output_bits=s["ob"])
    st = [sv.spec_history_append(s["tok"], stream=stream, **h)]
    wq = sv.spec_quantize_fp4(s["w"], fmt, stream=stream)
    xq = sv.spec_quantize_fp4(s["x"], fmt, stream=stream)
    y = sv.spec_project_fp4(xq, wq, dtype=torch.float32, stream=stream)
    sv.spec_process_logits(y, s["row0"], None, s["zero"], 0, None, repetition=s["rep"],
                           stream=stream, **h)
    st += [wq["status"], xq["status"],
           sv.spec_history_append(s["bad_tok"], stream=stream, **h),
           sv.spec_quantize_fp4(s["bad_x"], fmt, stream=stream)["status"]]
    return [y, xq["packed"], xq["scales"], wq["packed"], wq["scales"], s["counts"], s["ob"]], st


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("busy", ["side", "current"])
def test_tensors_of_the_call_belong_to_its_stream(sv, busy, fmt):
    """With long work ahead on the side stream, memory that the calls gave back must not be handed to
    the current stream's tensors before the calls have run; with long work ahead on the current
    stream, nothing of it may reach a word or output of the calls."""
    want, want_st = _calls(sv, _inputs(), fmt, None)
    s = _inputs()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    mine = []
    if busy == "side":
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)  # some 20 ms
    else:
        # freed blocks of every size the calls ask for, still to be written by the current stream
        torch.cuda._sleep(40_000_000)
        sizes = [1, s["rows"], s["V"], 1024, 2048, 8192, 65536, s["V"] * 160, s["rows"] * 1016]
        for n in sizes:
            for _ in range(8):
                torch.full((n,), 7, dtype=torch.int32, device="cuda")
    got, st = _calls(sv, s, fmt, side)
    for n in (1, 2, s["rows"], 256, 1024, 2048, 8192, s["rows"] * 1016, s["V"] * 160):
        mine += [torch.full((n,), 7, dtype=torch.int32, device="cuda") for _ in range(16)]
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in mine)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    codes = [sv.SV_OK] * 3 + [sv.SV_ERR_BAD_INPUT] * 2
    assert [int(t) for t in st] == codes and [int(t) for t in want_st] == codes


def test_results_may_be_used_and_dropped_on_the_current_stream(sv):
    """A result taken over by the current stream (after a wait) and dropped while that stream still
    reads it: the next call on the side stream must not write into its memory."""
    g = torch.Generator("cuda").manual_seed(5)
    x = sv.spec_quantize_fp4(torch.randn((64, 256), generator=g, device="cuda"), 0)
    w = [sv.spec_quantize_fp4(torch.randn((2000, 256), generator=g, device="cuda"), 0)
         for _ in range(2)]
    want = sv.spec_project_fp4(x, w[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = sv.spec_project_fp4(x, w[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(40_000_000)
    copy = y.clone()
    del y
    later = [sv.spec_project_fp4(x, w[1], stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(later) == 4


def test_a_stream_known_by_its_handle(sv):
    """Any object with a cuda_stream will do."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    s = _inputs()
    want, _ = _calls(sv, _inputs(), 1, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = _calls(sv, s, 1, Handle(side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_on_a_stream_beside_the_capturing_one(sv):
    """A captured step that forks to a second stream: the calls' tensors come from the graph's pool."""
    s = _inputs()
    want, _ = _calls(sv, _inputs(), 1, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in (s["counts"], s["ob"]):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got, st = _calls(sv, s, 1, side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in (s["counts"], s["ob"]):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert [int(t) for t in st] == [sv.SV_OK] * 3 + [sv.SV_ERR_BAD_INPUT] * 2


@pytest.mark.parametrize("marshalled", [True, False])
def test_every_tensor_given(sv, marshalled, monkeypatch):
    """All outputs and the status given, inputs made before: the calls on a side stream, behind long
    work there, equal those on the current one."""
    if not marshalled:
        monkeypatch.setattr(sv, "_fast", None)
        monkeypatch.setattr(sv, "_load_fast", lambda: None)

    def outputs(s):
        rows, V, H = s["rows"], s["V"], s["H"]
        u8 = dict(dtype=torch.uint8, device="cuda")
        n = [sv.spec_fp4_scale_bytes(k, H, 1) for k in (V, rows)]
        return dict(status=torch.full((1,), 9, dtype=torch.int32, device="cuda"),
                    w=dict(packed=torch.zeros((V, H // 2), **u8), scales=torch.zeros(n[0], **u8),
                           row_scales=torch.zeros(V, device="cuda")),
                    x=dict(packed=torch.zeros((rows, H // 2), **u8), scales=torch.zeros(n[1], **u8),
                           row_scales=torch.zeros(rows, device="cuda")),
                    y=torch.zeros((rows, 1016), device="cuda")[:, :V])

    def run(s, o, stream):
        kw = dict(status=o["status"], stream=stream)
        h = dict(counts=s["counts"], prompt_bits=s["pb"], output_bits=s["ob"])
        sv.spec_history_append(s["tok"], **h, **kw)
        wq = sv.spec_quantize_fp4(s["w"], 1, **o["w"], **kw)
        xq = sv.spec_quantize_fp4(s["x"], 1, **o["x"], **kw)
        sv.spec_project_fp4(xq, wq, out=o["y"], **kw)
        sv.spec_process_logits(o["y"], s["row0"], None, s["zero"], 0, None, repetition=s["rep"],
                               **h, **kw)
        return [o["status"], o["y"], s["counts"], s["ob"], *o["w"].values(), *o["x"].values()]

    ins = [_inputs(), _inputs()]
    outs = [outputs(s) for s in ins]
    want = run(ins[0], outs[0], None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(10_000_000)
    got = run(ins[1], outs[1], side)
    torch.cuda.synchronize()
    assert int(got[0]) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
