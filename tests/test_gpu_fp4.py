"""spec_quantize_fp4 and spec_project_fp4 against their definitions in binary64.

Quantisation rounds on exact quotients, so codes, scales and values must be equal.  A product's
terms are exact in binary32; the tensor cores add 64 of them into a step and H / 64 steps into the
accumulator.  An addition that truncates is off by at most 2^-23 of the largest partial sum, which is
at most sum |x w|: (64 + H / 64) 2^-23 sum |x w| bounds a row's error in any order of the additions.
A bf16 result is rounded once more, by at most 2^-8 of its value."""
import numpy as np
import pytest
import torch

import plain_serving as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return sv


def _check_quantized(q, values, x, fmt):
    rows, H = x.shape
    code, byte, g, val = plain.quantize(x.double().cpu().numpy(), fmt)
    got, zero_pad = plain.unpack_codes(q["packed"].cpu().numpy(), H)
    assert zero_pad
    assert ((got & 7) == code).all()
    neg = x.cpu().numpy() if x.dtype == torch.float32 else x.float().cpu().numpy()
    nz = code > 0
    assert ((got >> 3) == (neg < 0))[nz].all()
    sc, rest_zero = plain.scale_bytes(q["scales"].cpu().numpy(), rows, byte.shape[1])
    assert rest_zero and (sc == byte).all()
    if fmt == 1:
        assert (q["row_scales"].double().cpu().numpy() == g).all()
    if values is not None:
        # rounding to bf16 changes only what it has no number for: a row whose maximum is the
        # largest binary32 number has g = 2^117, s = 352 and the value 6 * 352 * 2^117 =
        # 1.03125 * 2^128, past the largest bf16 number
        want = torch.from_numpy(val).float().to(torch.bfloat16)
        small = np.abs(val) < 2.0 ** 127
        assert (want.double().numpy() == val)[small].all()
        assert torch.equal(values.cpu(), want)
    assert int(q["status"]) == 0


def _rows(rows, H, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, H), generator=g)
    if kind == "normal":
        x = x * torch.exp(torch.randn((rows, 1), generator=g))
    elif kind == "wide":  # forty binades within a row, some blocks far below the row's scale
        x = torch.ldexp(x, torch.randint(-30, 10, (rows, H), generator=g))
    elif kind == "ties":  # multiples of an eighth: many quotients on the middle of two codes
        x = torch.round(x * 32) / 8
    x[torch.rand((rows, H), generator=g) < 0.05] = 0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["normal", "wide", "ties"])
@pytest.mark.parametrize("rows,H", [(1, 1), (1, 16), (3, 33), (5, 255), (129, 256), (7, 1001),
                                    (130, 320), (2, 8192)])
def test_quantize(sv, rows, H, dtype, kind, fmt):
    x = _rows(rows, H, dtype, rows * 31 + H, kind)
    values = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device="cuda")
    q = sv.spec_quantize_fp4(x.cuda(), fmt, values=values)
    _check_quantized(q, values, x, fmt)
    assert torch.equal(sv.spec_quantize_fp4(x.cuda(), fmt)["packed"], q["packed"])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("H", [200, 500, 700, 1024, 1200, 2561, 3800, 5000, 5121, 7168, 8200, 10000,
                               10241, 16000, 20480, 20481])
def test_quantize_rows_of_every_length(sv, H, shift, dtype, fmt):
    """So many rows that each is held by as few warps as can; five of them against the plain form."""
    rows = 2100
    buf = torch.zeros((rows, H + 9), dtype=dtype, device="cuda")
    x = buf[:, shift:shift + H]
    x[:] = torch.randn((rows, H), device="cuda", generator=torch.Generator("cuda").manual_seed(H))
    few = _rows(5, H, dtype, H)
    x[:5] = few.cuda()
    x[-5:] = few.cuda()
    wide = torch.full((rows, H + 9), 5.0, dtype=torch.bfloat16, device="cuda")
    v = wide[:, shift:shift + H]
    q = sv.spec_quantize_fp4(x, fmt, values=v)
    small = torch.empty((5, H), dtype=torch.bfloat16, device="cuda")
    want = sv.spec_quantize_fp4(few.cuda(), fmt, values=small)
    _check_quantized(want, small, few, fmt)
    n = -(-H // plain.BLOCK[fmt])
    got_scales, clear = plain.scale_bytes(q["scales"].cpu().numpy(), rows, n)
    want_scales, _ = plain.scale_bytes(want["scales"].cpu().numpy(), 5, n)
    assert clear
    for part in (slice(0, 5), slice(rows - 5, rows)):
        assert torch.equal(q["packed"][part], want["packed"]) and torch.equal(v[part], small)
        assert (got_scales[part] == want_scales).all()
        if fmt == 1:
            assert torch.equal(q["row_scales"][part], want["row_scales"])
    assert (wide[:, :shift] == 5).all() and (wide[:, shift + H:] == 5).all()


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_strided_rows(sv, fmt):
    """Rows of a wider tensor (aligned and not), values into a wider tensor, guards kept."""
    for lead, width in ((8, 1024), (3, 1001)):
        base = _rows(9, width, torch.bfloat16, 3).cuda()
        x = base[:, lead:lead + 320]
        wide = torch.full((9, 400), 5.0, dtype=torch.bfloat16, device="cuda")
        v = wide[:, 40:360]
        q = sv.spec_quantize_fp4(x, fmt, values=v)
        _check_quantized(q, v, x.cpu(), fmt)
        assert (wide[:, :40] == 5).all() and (wide[:, 360:] == 5).all()


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantize_extremes(sv, fmt):
    """Zero rows, the largest and smallest numbers, halves of the smallest scale."""
    x = torch.zeros((6, 64))
    x[1] = torch.finfo(torch.float32).max
    x[2, 0] = torch.finfo(torch.float32).tiny
    x[3, ::2] = 2.0 ** -126
    x[3, 1::2] = -(2.0 ** -128)
    x[4, :16] = 448.0 * 6
    x[4, 16:] = 6 * 2.0 ** -10
    x[5, :40] = torch.arange(40) * 0.25
    values = torch.zeros((6, 64), dtype=torch.bfloat16, device="cuda")
    q = sv.spec_quantize_fp4(x.cuda(), fmt, values=values)
    _check_quantized(q, values, x, fmt)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_reports_non_finite(sv, fmt, bad):
    x = torch.randn((5, 96))
    x[2, 40] = bad
    q = sv.spec_quantize_fp4(x.cuda(), fmt)
    assert int(q["status"]) == sv.SV_ERR_BAD_INPUT
    n = plain.BLOCK[fmt]
    sc, _ = plain.scale_bytes(q["scales"].cpu().numpy(), 5, 96 // n)
    nan = sc == (0xFF if fmt == 0 else 0x7F)
    want = np.zeros_like(nan)
    if fmt == 0:
        want[2, 40 // n] = True
    else:
        want[2] = True
    assert (nan == want).all()
    # the product shows it in that row and nowhere else
    w = sv.spec_quantize_fp4(torch.randn((40, 96), device="cuda"), fmt)
    y = sv.spec_project_fp4(q, w, dtype=torch.float32)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4]]).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,H", [(1, 16), (3, 2560), (6, 2560), (17, 500), (32, 256), (64, 256),
                                    (65, 256), (300, 700), (20, 500), (30, 300), (1, 8192)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1])
def test_quantize_status_is_of_the_call(sv, fmt, rows, H, dtype, shift):
    """The status of a call with a NaN, then of one without, in one word and without a wait; and the
    codes are those of a larger batch (whose CTAs are others).  With a shift no row is aligned."""
    buf = torch.zeros((rows, H + shift), dtype=dtype, device="cuda")
    buf[:, shift:] = _rows(rows, H, dtype, rows + H).cuda()
    x = buf[:, shift:]
    st = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    q = sv.spec_quantize_fp4(x, fmt, status=st)
    bad = buf.clone()[:, shift:]
    bad[rows - 1, H - 1] = float("nan")
    seen = []
    for t in (bad, x, bad, bad, x):
        sv.spec_quantize_fp4(t, fmt, packed=torch.empty_like(q["packed"]),
                             scales=torch.empty_like(q["scales"]),
                             row_scales=None if fmt == 0 else torch.empty_like(q["row_scales"]),
                             status=st)
        seen.append(st.clone())
    assert [int(s) for s in seen] == [sv.SV_ERR_BAD_INPUT, 0, sv.SV_ERR_BAD_INPUT,
                                      sv.SV_ERR_BAD_INPUT, 0]
    many = sv.spec_quantize_fp4(torch.cat([x, torch.randn((1000, H), device="cuda").to(dtype)]), fmt)
    assert torch.equal(many["packed"][:rows], q["packed"])
    n = -(-H // plain.BLOCK[fmt])
    a, clear = plain.scale_bytes(q["scales"].cpu().numpy(), rows, n)
    b, _ = plain.scale_bytes(many["scales"].cpu().numpy(), rows + 1000, n)
    assert clear and (a == b[:rows]).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rows,H", [(2, 2560), (20, 500), (300, 700), (130, 2560), (5, 70001)])
@pytest.mark.parametrize("shift", [0, 1])
def test_quantize_values_over_x(sv, fmt, rows, H, shift):
    """values = x: the elements become the numbers their codes stand for."""
    buf = torch.zeros((rows, H + shift + 7), dtype=torch.bfloat16, device="cuda")
    buf[:, shift:shift + H] = _rows(rows, H, torch.bfloat16, rows + H).cuda()
    x, before = buf[:, shift:shift + H], buf.clone()
    y = torch.empty((rows, H), dtype=torch.bfloat16, device="cuda")
    want = sv.spec_quantize_fp4(x, fmt, values=y)
    got = sv.spec_quantize_fp4(x, fmt, values=x)
    assert torch.equal(x, y) and torch.equal(got["packed"], want["packed"])
    before[:, shift:shift + H] = y
    assert torch.equal(buf, before)  # nothing beside the rows changed


# ---- the product ---------------------------------------------------------------------------------

def _project(sv, M, V, H, fmt, dtype, spread, seed, ld=None):
    rng = np.random.default_rng(seed)
    a, b = plain.operand(M, H, fmt, rng, spread), plain.operand(V, H, fmt, rng, spread)
    ld = ld or (V + 7) // 8 * 8 + 8
    buf = torch.full((M + 1, ld), 7.0, dtype=dtype, device="cuda")
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    y = sv.spec_project_fp4(plain.device_operand(a, M, H, fmt), plain.device_operand(b, V, H, fmt),
                            out=buf[:M, :V], status=st)
    assert int(st) == 0
    assert (buf[M] == 7).all() and (buf[:, V:] == 7).all()  # nothing behind the rows and columns
    got = y.double().cpu().numpy()
    want = a[3] @ b[3].T
    return got, want, np.abs(a[3]) @ np.abs(b[3]).T


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,V,H", [(1, 128, 256), (16, 128, 64), (1, 1, 1), (3, 200, 31),
                                   (17, 129, 257), (64, 1000, 512), (100, 513, 2560),
                                   (128, 300, 1024), (192, 777, 320)])
def test_project_exact_sums(sv, fmt, M, V, H):
    """All scales one: products are multiples of a quarter and sums below 2^24 quarters, so the
    fp32 result is exact whatever the order."""
    got, want, _ = _project(sv, M, V, H, fmt, torch.float32, 0, M + V + H)
    assert (got == want).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,V,H", [(1, 257, 96), (6, 1000, 2560), (15, 130, 1000), (33, 128, 800),
                                   (129, 400, 256), (193, 391, 544), (320, 640, 288),
                                   (385, 200, 2048), (1000, 150, 512)])
def test_project(sv, M, V, H, fmt, dtype):
    got, want, mag = _project(sv, M, V, H, fmt, dtype, 3, 7 * M + V + H)
    tol = (64 + H / 64) * 2.0 ** -23 * mag
    if dtype == torch.bfloat16:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


def test_project_many_tiles(sv):
    """More tiles than CTAs, so that accumulators and ring stages are reused in every order."""
    for M, V, H in ((20, 40000, 192), (200, 30000, 128)):
        got, want, mag = _project(sv, M, V, H, 0, torch.float32, 2, M)
        assert (np.abs(got - want) <= (64 + H / 64) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M,H", [(512, 1000), (600, 2560), (700, 4096), (300, 1600)])
def test_project_rows_do_not_depend_on_the_batch(sv, M, H, fmt, dtype):
    """Several tiles per vocabulary tile and more of those than CTAs: the rows of smaller batches (of
    one tile, whose figures are tested above), bit for bit: each sum is formed in the order of K."""
    g = torch.Generator("cuda").manual_seed(M + H)
    V = 50001
    x = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    w = sv.spec_quantize_fp4(torch.randn((V, H), generator=g, device="cuda").to(torch.bfloat16), fmt)
    out = torch.full((M, V + 7), 3.0, dtype=dtype, device="cuda")
    y = sv.spec_project_fp4(sv.spec_quantize_fp4(x, fmt), w, out=out[:, :V])
    for a in range(0, M, 128):
        part = sv.spec_quantize_fp4(x[a:a + 128], fmt)
        assert torch.equal(y[a:a + 128], sv.spec_project_fp4(part, w, out=torch.empty(
            (part["rows"], V + 7), dtype=dtype, device="cuda")[:, :V]))
    assert (out[:, V:] == 3).all()


def test_project_same_tensor_and_reruns(sv):
    """Both operands the same tensor; the same bits from every run."""
    x = torch.randn((150, 640), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    q = sv.spec_quantize_fp4(x, 1)
    y = sv.spec_project_fp4(q, q, dtype=torch.float32)
    assert torch.equal(y, y.t())
    for _ in range(3):
        assert torch.equal(sv.spec_project_fp4(q, q, dtype=torch.float32), y)


def test_project_right_behind_a_new_w(sv):
    """W quantised and multiplied back to back, ever another one, without a wait in between: the
    product must not see the W before."""
    g = torch.Generator("cuda").manual_seed(2)
    V, H = 20000, 1024
    xs = torch.randn((40, H), generator=g, device="cuda").to(torch.bfloat16)
    w = [torch.randn((V, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    x = sv.spec_quantize_fp4(xs, 0)
    alone = []
    for t in w:
        q = sv.spec_quantize_fp4(t, 0)
        torch.cuda.synchronize()
        alone.append(sv.spec_project_fp4(x, q, dtype=torch.float32))
        torch.cuda.synchronize()
    packed, scales = torch.empty_like(q["packed"]), torch.empty_like(q["scales"])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(alone[0]) for _ in range(40)]
    for k, o in enumerate(outs):
        q = sv.spec_quantize_fp4(w[k % 4], 0, packed=packed, scales=scales, status=st)
        sv.spec_project_fp4(x, q, out=o, status=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[k % 4]) for k, o in enumerate(outs))


def test_offsets_past_32_bits(sv):
    """Hidden rows, packed rows and logits that lie more than 4 GiB into their tensors."""
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.zeros((140000, 16384), dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    x[-3:] = torch.randn((3, 16384), generator=g, device="cuda")
    for fmt in (0, 1):
        q = sv.spec_quantize_fp4(x, fmt)
        part = sv.spec_quantize_fp4(x[-96:].contiguous(), fmt)  # rows 139904 .. 139999, a whole tile
        assert torch.equal(q["packed"][-96:], part["packed"])
        assert 139904 % 128 == 0 and torch.equal(q["scales"][-part["scales"].numel():], part["scales"])
        assert q["packed"][:-3].count_nonzero() == 0
        del q
    del x
    M, V, H = 17000, 131072, 32
    h = sv.spec_quantize_fp4(torch.randn((M, H), generator=g, device="cuda"), 0)
    w = sv.spec_quantize_fp4(torch.randn((V, H), generator=g, device="cuda"), 0)
    y = sv.spec_project_fp4(h, w)  # 4.5 GB
    some = torch.tensor([0, 255, 256, 9000, 16383, 16384, 16999], device="cuda")
    few = sv.spec_quantize_fp4(torch.zeros((7, H), device="cuda"), 0)
    few["packed"].copy_(h["packed"][some])
    sc, _ = plain.scale_bytes(h["scales"].cpu().numpy(), M, 1)
    at = torch.arange(7) * 16
    few["scales"][at.cuda()] = torch.from_numpy(sc[some.cpu().numpy(), 0]).cuda()
    assert torch.equal(y[some], sv.spec_project_fp4(few, w))


def test_chain_to_verification(sv, orc):
    """The operators as they are used: hidden rows and W quantised, logits from the product, the
    history's penalties and masks in place on target and draft rows, verification, and the verified
    tokens into the history -- captured as one graph and replayed over three rounds, against the
    library's own calls one by one; the verified tokens against the oracle on the processed rows."""
    B, g, V, H = 6, 3, 2053, 320
    gen = torch.Generator().manual_seed(4)
    w = (torch.randn((V, H), generator=gen) * 3 / H ** 0.5).to(torch.bfloat16).cuda()
    th = torch.randn((B * (g + 1), H), generator=gen)
    dh = th.view(B, g + 1, H)[:, :g].reshape(B * g, H) + 0.3 * torch.randn((B * g, H), generator=gen)
    th, dh = th.to(torch.bfloat16).cuda(), dh.to(torch.bfloat16).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    t0 = torch.arange(B, device="cuda") * (g + 1)
    d0 = torch.arange(B, device="cuda") * g
    ln = torch.full((B,), g, **i32)
    rep = torch.full((B,), 1.2, device="cuda")
    freq = torch.full((B,), 0.1, device="cuda")
    mask = torch.full((1, (V + 31) // 32), 0x7FFFFFF7, **i32)
    mrow_t = torch.where(torch.arange(B * (g + 1), device="cuda") < 8, 0, -1).to(torch.int32)
    mrow_d = torch.where(torch.arange(B * g, device="cuda") < 6, 0, -1).to(torch.int32)
    wq = sv.spec_quantize_fp4(w, sv.SV_FP4_E4M3_16)
    ws = torch.empty(sv.spec_verify_workspace_bytes(B, g, V, sv.SV_BF16), dtype=torch.uint8,
                     device="cuda")

    def state():
        return dict(counts=torch.zeros((B, V), **i32),
                    prompt_bits=torch.zeros((B, (V + 31) // 32), **i32),
                    output_bits=torch.zeros((B, (V + 31) // 32), **i32))

    def round_(h):
        dl = sv.spec_project_fp4(sv.spec_quantize_fp4(dh, 1), wq)
        tl = sv.spec_project_fp4(sv.spec_quantize_fp4(th, 1), wq)
        # drafts: sampled row by row from the processed draft rows
        tok = torch.zeros(B * g, **i32)
        for i in range(g):
            sv.spec_process_logits(dl, d0, d0, torch.full((B,), i, **i32), g, tok, first_row=i,
                                   repetition=rep, frequency=freq, mask=mask, mask_row=mrow_d, **h)
            sv.spec_sample_draft(dl, d0, torch.full((B,), i + 1, **i32), g, 5, draft_tokens=tok,
                                 workspace=ws)
        sv.spec_process_logits(tl, t0, d0, ln, g, tok, repetition=rep, frequency=freq, mask=mask,
                               mask_row=mrow_t, **h)
        out = sv.spec_verify_token(tl, dl, t0, d0, ln, g, tok, 5, workspace=ws)
        sv.spec_history_append(out["out_tokens"], **h)
        return tok, dl, tl, out

    h = state()
    eager = []
    for _ in range(3):
        tok, dl, tl, out = round_(h)
        torch.cuda.synchronize()
        assert int(out["status"]) == 0
        eager.append([t.clone() for t in (tok, out["out_tokens"], out["accepted_len"])])
        # masked tokens are never drafted nor emitted by the masked requests
        banned = [t for t in range(V) if t % 32 in (3, 31)]
        assert not set(tok[:6].tolist()) & set(banned)
        assert not set(out["out_tokens"][:2].flatten().tolist()) & set(banned)
        ref = orc.verify_batch(0, tl.float().cpu().numpy(), dl.float().cpu().numpy(), V, V,
                               t0.cpu().numpy(), d0.cpu().numpy(), ln.cpu().numpy(),
                               tok.cpu().numpy(), B, 5, out_ld=g + 1)
        ok = (ref["out_tokens"] == out["out_tokens"].cpu().numpy()).all(1)
        near = (ref["decision_margin"] < 1e-5) | (ref["race_margin"] < 1e-5)
        assert (ok | near).all()
    # every emitted token was counted
    emitted = torch.cat([e[1] for e in eager], 1)
    want = torch.zeros((B, V), dtype=torch.int32)
    for r in range(B):
        for t in emitted[r].tolist():
            if t >= 0:
                want[r, t] += 1
    assert torch.equal(h["counts"].cpu(), want)
    bits = plain.bits_to_bool(h["output_bits"].cpu().numpy(), V)
    assert (bits == (want.numpy() > 0)).all()

    h2 = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        round_(h2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tok, dl, tl, out = round_(h2)
    for t in h2.values():
        t.zero_()
    for e in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, e[0]) and torch.equal(out["out_tokens"], e[1])
        assert torch.equal(out["accepted_len"], e[2])
    assert torch.equal(h2["counts"], h["counts"])
