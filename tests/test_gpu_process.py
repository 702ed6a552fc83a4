"""spec_history_append and spec_process_logits against their definitions in binary64.

History results are whole numbers and must be equal.  Processed logits: the plain form returns,
beside the value, the sum of |intermediate results| * 2^-24 -- every binary32 step rounds by at most
half a step of its result -- and a bf16 result is rounded once more, by at most 2^-8 of its value."""
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


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---- history -----------------------------------------------------------------------------------

def _history_state(rng, S, V):
    counts = rng.integers(0, 3, (S, V)).astype(np.int32)
    return counts, rng.random((S, V)) < 0.3, counts > 0


@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("B,n,V", [(1, 1, 1), (3, 6, 31), (5, 17, 1000), (7, 2000, 16385),
                                   (2, 33, 151936), (64, 6, 33), (3, 9000, 40001),
                                   (2, 500, 262145)])
def test_history_append(sv, B, n, V, prompt, reset):
    rng = np.random.default_rng(B * 1000 + n + V)
    S = B + 2
    counts, pb, ob = _history_state(rng, S, V)
    tokens = rng.integers(-1, V, (B, n)).astype(np.int32)
    lens = rng.integers(0, n + 1, B).astype(np.int32)
    slots = rng.permutation(S)[:B].astype(np.int32)
    # rows padded on the device: strides larger than the widths, guard columns kept
    W = (V + 31) // 32
    ldc, ldb = V + 3, W + 1
    d_counts = torch.full((S, ldc), 77, dtype=torch.int32, device="cuda")
    d_pb = torch.full((S, ldb), 77, dtype=torch.int32, device="cuda")
    d_ob = torch.full((S, ldb), 77, dtype=torch.int32, device="cuda")
    d_counts[:, :V] = _dev(counts)
    d_pb[:, :W] = _dev(plain.bool_to_bits(pb))
    d_ob[:, :W] = _dev(plain.bool_to_bits(ob))
    d_tok = torch.full((B, n + 2), 5, dtype=torch.int32, device="cuda")
    d_tok[:, :n] = _dev(tokens)
    st = sv.spec_history_append(d_tok[:, :n], d_counts[:, :V], d_pb[:, :W], d_ob[:, :W],
                                slots=_dev(slots), lens=_dev(lens), prompt=prompt, reset=reset)
    plain.history_append(tokens, counts, pb, ob, slots, lens, prompt, reset)
    assert int(st) == 0
    assert (d_counts[:, :V].cpu().numpy() == counts).all()
    assert (d_pb[:, :W].cpu().numpy() == plain.bool_to_bits(pb)).all()
    assert (d_ob[:, :W].cpu().numpy() == plain.bool_to_bits(ob)).all()
    assert (d_counts[:, V:] == 77).all() and (d_pb[:, W:] == 77).all() and (d_ob[:, W:] == 77).all()


def test_history_slots_listed_twice(sv):
    """Without reset both rows count; with reset the slot is refused and left alone."""
    V = 100
    mk = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    counts, pb, ob = mk(3, V), mk(3, 4), mk(3, 4)
    tok = torch.tensor([[5, 5], [5, 7], [9, -1]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([1, 1, 2], dtype=torch.int32, device="cuda")
    assert int(sv.spec_history_append(tok, counts, pb, ob, slots=slots)) == 0
    assert counts[1, 5] == 3 and counts[1, 7] == 1 and counts[2, 9] == 1 and counts.sum() == 5
    assert ob[1, 0] == (1 << 5) + (1 << 7)
    st = sv.spec_history_append(tok, counts, pb, ob, slots=slots, reset=True)
    assert int(st) == sv.SV_ERR_BAD_INPUT
    assert counts[1, 5] == 3 and counts[2, 9] == 1 and counts.sum() == 5


def test_history_bad_data_is_reported(sv):
    """Slots, lengths and tokens out of range leave their row (or token) out."""
    V = 50
    mk = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for reset in (False, True):
        for slots, lens, tok in [(t(0, 2), t(1, 1), t(1, 1)), (t(-1, 0), t(1, 1), t(1, 1)),
                                 (t(0, 1), t(2, 1), t(1, 1)), (t(0, 1), t(-1, 1), t(1, 1)),
                                 (t(0, 1), t(1, 1), t(50, 1))]:
            counts, pb, ob = mk(2, V), mk(2, 2), mk(2, 2)
            st = sv.spec_history_append(tok[:, None].contiguous(), counts, pb, ob, slots=slots,
                                        lens=lens, reset=reset)
            assert int(st) == sv.SV_ERR_BAD_INPUT
            assert counts.sum() == 1  # the good row's token


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("V,n", [(50, 1), (1000, 700), (40001, 9000), (300000, 20)])
def test_history_of_one_row_replaced(sv, V, n, prompt):
    """Status of calls with one row, good and bad, over what the word held before."""
    W = (V + 31) // 32
    mk = lambda *s: torch.full(s, 3, dtype=torch.int32, device="cuda")  # noqa: E731
    good = torch.randint(0, V, (1, n), dtype=torch.int32, device="cuda")
    for at, value, ln, slot, want in ((0, None, n, 1, 0), (n - 1, V, n, 1, 1), (0, None, n + 1, 1, 2),
                                      (0, None, -1, 1, 2), (0, None, n, 2, 2), (n - 1, V, n - 1, 0, 0)):
        counts, pb, ob = mk(2, V), mk(2, W), mk(2, W)
        tok = good.clone()
        if value is not None:
            tok[0, at] = value
        for stale in (0, sv.SV_ERR_BAD_INPUT):
            st = torch.full((1,), stale, dtype=torch.int32, device="cuda")
            sv.spec_history_append(tok, counts, pb, ob, prompt=prompt, reset=True, status=st,
                                   slots=torch.tensor([slot], dtype=torch.int32, device="cuda"),
                                   lens=torch.tensor([ln], dtype=torch.int32, device="cuda"))
            assert int(st) == (sv.SV_ERR_BAD_INPUT if want else 0)
        if want == 2:  # the row is left out
            assert (counts == 3).all() and (pb == 3).all() and (ob == 3).all()
            continue
        x = tok[0, :ln].cpu().numpy()
        c = np.bincount(x[x < V], minlength=V)
        bits = plain.bool_to_bits((c > 0)[None])
        zero = np.zeros_like(bits)
        assert (counts[slot].cpu().numpy() == (0 if prompt else c)).all()
        assert (pb[slot].cpu().numpy() == (bits if prompt else zero)[0]).all()
        assert (ob[slot].cpu().numpy() == (zero if prompt else bits)[0]).all()
        assert (counts[1 - slot] == 3).all() and (pb[1 - slot] == 3).all()


def test_history_reset_without_tokens(sv):
    V = 100
    counts = torch.ones((2, V), dtype=torch.int32, device="cuda")
    pb = torch.full((2, 4), 5, dtype=torch.int32, device="cuda")
    ob = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    tok = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    sl = torch.tensor([1], dtype=torch.int32, device="cuda")
    assert int(sv.spec_history_append(tok, counts, pb, ob, slots=sl, reset=True)) == 0
    assert counts[1].sum() == 0 and counts[0].sum() == V
    assert (pb[1] == 0).all() and (ob[1] == 0).all() and (pb[0] == 5).all() and (ob[0] == -1).all()


# ---- logits processing ---------------------------------------------------------------------------

def _case(seed, B, gamma, V, dtype, bias=0, masked=False, ragged=True, first_row=0, bonus=True,
          neutral=()):
    rng = np.random.default_rng(seed)
    S = B + 1
    R = gamma + 1
    rows = B * R + 2
    l = rng.normal(0, 3, (rows, V)).astype(np.float32)
    l[rng.random((rows, V)) < 0.05] = 0.0
    l[rng.random((rows, V)) < 0.02] = -np.inf
    l = torch.from_numpy(l).to(dtype)
    counts = np.where(rng.random((S, V)) < 0.2, rng.integers(1, 9, (S, V)), 0).astype(np.int32)
    c = {"B": B, "gamma": gamma, "V": V, "first_row": first_row, "bonus": bonus,
         "logits": l, "counts": counts, "prompt": rng.random((S, V)) < 0.2, "output": counts > 0,
         "slots": rng.permutation(S)[:B].astype(np.int32),
         "row0": (rng.permutation(B) * R + 1).astype(np.int64),
         "draft_row0": (rng.permutation(B) * max(gamma, 1)).astype(np.int64),
         "draft_len": (rng.integers(0, gamma + 1, B) if ragged
                       else np.full(B, gamma)).astype(np.int32),
         # few distinct tokens, so that rows draft the same token twice
         "draft_tokens": rng.choice(rng.integers(0, V, max(2, gamma // 2)),
                                    B * max(gamma, 1)).astype(np.int32),
         "rep": rng.uniform(0.7, 1.5, B).astype(np.float32),
         "pres": rng.uniform(-1, 1, B).astype(np.float32),
         "freq": rng.uniform(-0.5, 0.5, B).astype(np.float32),
         "bias": None, "mask": None, "mask_row": None}
    for r in neutral:
        c["rep"][r], c["pres"][r], c["freq"][r] = 1.0, 0.0, 0.0
    if bias:
        lens = rng.integers(0, min(bias, V) + 1, B)
        lens[-1] = min(bias, V)
        start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        toks = np.concatenate([np.sort(rng.permutation(V)[:n]) for n in lens]).astype(np.int32)
        vals = rng.normal(0, 4, len(toks)).astype(np.float32)
        vals[rng.random(len(vals)) < 0.1] = -np.inf
        c["bias"] = (start, toks, vals)
    if masked:
        n = max(1, rows // 2)
        m = rng.random((n, V)) < rng.choice([0.0, 0.01, 0.5, 0.97, 1.0], n)[:, None]
        c["mask"] = m
        c["mask_row"] = rng.integers(-1, n, rows).astype(np.int32)
        # whatever stands in a masked place must not matter
        for i in range(rows):
            if c["mask_row"][i] >= 0:
                junk = ~m[c["mask_row"][i]] & (rng.random(V) < 0.3)
                l[i, torch.from_numpy(junk)] = torch.from_numpy(rng.choice(
                    [np.nan, np.inf, torch.finfo(dtype).min], junk.sum()).astype(np.float32)).to(dtype)
    return c


def _expected(c):
    """(binary64 rows with untouched rows as they were, bounds, which rows were processed)."""
    out = c["logits"].double().numpy().copy()
    tol = np.zeros_like(out)
    done = np.zeros(len(out), bool)
    for r in range(c["B"]):
        bias = np.zeros(c["V"])
        if c["bias"] is not None:
            a, b = c["bias"][0][r], c["bias"][0][r + 1]
            bias[c["bias"][1][a:b]] = c["bias"][2][a:b]
        s = c["slots"][r]
        for i in range(c["first_row"], c["draft_len"][r] + int(c["bonus"])):
            row = c["row0"][r] + i
            allowed = np.ones(c["V"], bool)
            if c["mask"] is not None and c["mask_row"][row] >= 0:
                allowed = c["mask"][c["mask_row"][row]]
            d0 = c["draft_row0"][r]
            out[row], tol[row] = plain.process_row(
                out[row], c["draft_tokens"][d0:d0 + i], c["counts"][s], c["prompt"][s],
                c["output"][s], c["rep"][r], c["freq"][r], c["pres"][r], bias, allowed)
            done[row] = True
    return out, tol, done


def _device_args(c, ld):
    rows, V = c["logits"].shape
    buf = torch.full((rows, ld), 3.5, dtype=c["logits"].dtype, device="cuda")
    buf[:, :V] = c["logits"].cuda()
    W = (V + 31) // 32
    kw = dict(slots=_dev(c["slots"]), counts=_dev(c["counts"]),
              prompt_bits=_dev(plain.bool_to_bits(c["prompt"])),
              output_bits=_dev(plain.bool_to_bits(c["output"])), repetition=_dev(c["rep"]),
              presence=_dev(c["pres"]), frequency=_dev(c["freq"]), first_row=c["first_row"],
              bonus_row=c["bonus"])
    if c["bias"] is not None:
        kw.update(zip(("bias_start", "bias_tokens", "bias_values"), map(_dev, c["bias"])))
    if c["mask"] is not None:
        m = torch.full((len(c["mask"]), W + 2), -1, dtype=torch.int32, device="cuda")
        m[:, :W] = _dev(plain.bool_to_bits(c["mask"]))
        kw.update(mask=m[:, :W], mask_row=_dev(c["mask_row"]))
    args = (_dev(c["row0"]), _dev(c["draft_row0"]), _dev(c["draft_len"]), c["gamma"],
            _dev(c["draft_tokens"]))
    return buf, args, kw


def _check_rows(got, want, tol, dtype):
    g = got.double().cpu().numpy()
    bad = ~np.isfinite(want)
    assert ((g == want) | (np.isnan(g) & np.isnan(want)))[bad].all()
    if dtype == torch.bfloat16:  # one more rounding, of a value that may be off by tol
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    with np.errstate(invalid="ignore"):
        off = np.abs(g - want) - tol
    assert (off[~bad] <= 0).all(), off[~bad].max()


def _run(sv, c, in_place, ld=None):
    V = c["V"]
    ld = ld or (V + 7) // 8 * 8 + 8
    buf, args, kw = _device_args(c, ld)
    before = buf.clone()
    want, tol, done = _expected(c)
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    if in_place:
        out = sv.spec_process_logits(buf[:, :V], *args, status=st, **kw)
        assert out.data_ptr() == buf.data_ptr()
        whole = buf
        want_else = before
    else:
        whole = torch.full((buf.shape[0], ld + 8), -2.5, dtype=buf.dtype, device="cuda")
        want_else = whole.clone()
        sv.spec_process_logits(buf[:, :V], *args, out=whole[:, :V], status=st, **kw)
        bits = torch.int32 if buf.dtype == torch.float32 else torch.int16
        assert torch.equal(buf.view(bits), before.view(bits))
    assert int(st) == 0
    d = torch.from_numpy(done).cuda()
    _check_rows(whole[:, :V][d], want[done], tol[done], buf.dtype)
    bits = torch.int32 if buf.dtype == torch.float32 else torch.int16
    # rows of no request, and columns behind the vocabulary, are left as they were
    assert torch.equal(whole[~d].view(bits), want_else[~d].view(bits))
    assert torch.equal(whole[:, V:].contiguous().view(bits), want_else[:, V:].contiguous().view(bits))
    # what nothing touches keeps its bits
    same = torch.from_numpy((tol == 0) & np.isfinite(want) & done[:, None]).cuda()
    src = before[:, :V]
    assert torch.equal(whole[:, :V][same], src[same])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,gamma,V,bias,masked", [
    (1, 0, 1, 1, True), (1, 0, 7, 0, False), (2, 3, 33, 5, True), (3, 1, 1000, 0, True),
    (5, 5, 4099, 300, False), (4, 7, 8193, 2000, True), (2, 64, 517, 40, True),
    (9, 16, 2048, 17, True)])
def test_process(sv, B, gamma, V, bias, masked, dtype, in_place):
    _run(sv, _case(B + 10 * gamma + V, B, gamma, V, dtype, bias, masked), in_place)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_process_serving_size(sv, dtype):
    """Rows of the token-level benchmark's vocabulary, in place and copied."""
    c = _case(77, 2, 5, 151936, dtype, 300, True, ragged=False)
    _run(sv, c, True, ld=151936)
    _run(sv, c, False, ld=151936)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,gamma,V,bias,masked", [
    (70, 5, 9000, 4000, True), (330, 4, 1003, 30, True), (140, 0, 20000, 17, False),
    (60, 20, 4097, 0, True)])
def test_process_many_requests(sv, B, gamma, V, bias, masked, dtype, in_place):
    """More parts of rows than SMs can hold at once."""
    _run(sv, _case(B + 10 * gamma + V, B, gamma, V, dtype, bias, masked), in_place)


@pytest.mark.parametrize("in_place", [True, False])
def test_process_draft_side_and_single_rows(sv, in_place):
    """Draft rows (no bonus row), one row of an autoregressive draft, and requests without any
    penalty among requests with some."""
    _run(sv, _case(5, 4, 6, 999, torch.bfloat16, bonus=False, neutral=(1,)), in_place)
    _run(sv, _case(6, 4, 3, 999, torch.float32, first_row=3, ragged=False, neutral=(0, 3)), in_place)
    _run(sv, _case(7, 3, 9, 640, torch.float32, 20, True, first_row=2), in_place)


def test_process_without_penalties(sv):
    """Biases or masks alone need no history; with nothing asked rows are copied."""
    V, rows = 1000, 3
    x = torch.randn((rows, V), device="cuda")
    row0 = torch.arange(rows, device="cuda")
    ln = torch.zeros(rows, dtype=torch.int32, device="cuda")
    y = sv.spec_process_logits(x, row0, None, ln, 0, None, out=torch.zeros_like(x))
    assert torch.equal(x, y)
    start = torch.tensor([0, 0, 2, 2], dtype=torch.int32, device="cuda")
    toks = torch.tensor([3, 999], dtype=torch.int32, device="cuda")
    vals = torch.tensor([1.5, -2.0], device="cuda")
    y = sv.spec_process_logits(x, row0, None, ln, 0, None, bias_start=start, bias_tokens=toks,
                               bias_values=vals, out=torch.zeros_like(x))
    want = x.clone()
    want[1, 3] += 1.5
    want[1, 999] -= 2.0
    assert torch.equal(y, want)


@pytest.mark.parametrize("in_place", [True, False])
def test_process_everything_seen(sv, in_place):
    """Every token of the vocabulary in the history and in the bias list: lists as long as a chunk."""
    c = _case(21, 2, 3, 9000, torch.bfloat16, 9000, True, ragged=False)
    c["counts"][:] = 1 + np.arange(9000) % 5
    c["output"][:] = True
    start = np.array([0, 9000, 18000], np.int32)
    c["bias"] = (start, np.tile(np.arange(9000, dtype=np.int32), 2),
                 np.linspace(-2, 2, 18000).astype(np.float32))
    _run(sv, c, in_place)


def test_same_history_for_several_requests(sv):
    """Requests may share a slot; its history is only read."""
    c = _case(22, 5, 2, 1500, torch.float32)
    c["slots"][:] = 3
    _run(sv, c, True)


def test_offsets_past_32_bits(sv):
    """Rows, counts and tokens that lie more than 4 GiB into their tensors."""
    V, rows, S = 131072, 17000, 8400
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")  # 4.5 GB
    counts = torch.zeros((S, V), **i32)                              # 4.4 GB
    pb, ob = torch.zeros((S, V // 32), **i32), torch.zeros((S, V // 32), **i32)
    slots = torch.tensor([S - 1], **i32)
    tok = torch.tensor([[V - 1, 7, V - 1]], **i32)
    st = sv.spec_history_append(tok, counts, pb, ob, slots=slots)
    assert int(st) == 0 and counts[S - 1, V - 1] == 2 and counts[S - 1, 7] == 1
    assert counts[:S - 1].count_nonzero() == 0
    x[rows - 1] = 4.0
    kw = dict(slots=slots, counts=counts, prompt_bits=pb, output_bits=ob,
              frequency=torch.ones(1, device="cuda"))
    row0 = torch.tensor([rows - 1], device="cuda")
    zero = torch.zeros(1, **i32)
    out = torch.zeros_like(x)
    sv.spec_process_logits(x, row0, None, zero, 0, None, out=out, **kw)
    sv.spec_process_logits(x, row0, None, zero, 0, None, **kw)
    want = torch.full((V,), 4.0, dtype=torch.bfloat16, device="cuda")
    want[V - 1], want[7] = 2.0, 3.0
    assert torch.equal(x[rows - 1], want) and torch.equal(out[rows - 1], want)
    assert x[:rows - 1].count_nonzero() == 0 and out[:rows - 1].count_nonzero() == 0
    st = sv.spec_history_append(tok, counts, pb, ob, slots=slots, prompt=True, reset=True)
    assert int(st) == 0 and counts[S - 1].count_nonzero() == 0 and ob.count_nonzero() == 0
    assert pb[S - 1, 0] == 1 << 7 and pb[S - 1, V // 32 - 1] == -2**31


def test_single_row_of_odd_width(sv):
    """A lone row's stride says nothing: [1, 1001] is as good as a padded row."""
    x = torch.randn((1, 1001), device="cuda")
    row0 = torch.zeros(1, dtype=torch.int64, device="cuda")
    ln = torch.zeros(1, dtype=torch.int32, device="cuda")
    mask = torch.full((1, 32), -1, dtype=torch.int32, device="cuda")
    mask[0, 31] = 0  # tokens 992 .. 1000 banned
    y = sv.spec_process_logits(x, row0, None, ln, 0, None, mask=mask, mask_row=ln,
                               out=torch.zeros_like(x))
    assert torch.equal(y[:, :992], x[:, :992]) and torch.isneginf(y[:, 992:]).all()
    w = sv.spec_quantize_fp4(torch.randn((1001, 96), device="cuda"), 0)
    h = sv.spec_quantize_fp4(torch.randn((2, 96), device="cuda"), 0)
    one = sv.spec_quantize_fp4(torch.zeros((1, 96), device="cuda"), 0)
    one["packed"].copy_(h["packed"][:1])
    one["scales"].copy_(h["scales"])
    out = torch.full((1, 1001), 7.0, device="cuda")
    sv.spec_project_fp4(one, w, out=out)
    assert torch.equal(out, sv.spec_project_fp4(h, w, dtype=torch.float32)[:1])


def test_process_parts_of_the_penalties(sv):
    """Each of the three penalties may be left out."""
    c = _case(8, 3, 4, 777, torch.float32)
    for keep in ("rep", "pres", "freq"):
        d = dict(c)
        if keep != "rep":
            d["rep"] = np.ones(3, np.float32)
        if keep != "pres":
            d["pres"] = np.zeros(3, np.float32)
        if keep != "freq":
            d["freq"] = np.zeros(3, np.float32)
        want, tol, done = _expected(d)
        buf, args, kw = _device_args(c, 784)
        names = {"rep": "repetition", "pres": "presence", "freq": "frequency"}
        for k, name in names.items():
            if k != keep:
                kw[name] = None
        sv.spec_process_logits(buf[:, :777], *args, **kw)
        dn = torch.from_numpy(done).cuda()
        _check_rows(buf[:, :777][dn], want[done], tol[done], torch.float32)


def test_process_bad_data_is_reported(sv):
    def status(**change):
        c = _case(9, 2, 3, 100, torch.float32, 4, True, ragged=False)
        buf, args, kw = _device_args(c, 104)
        args = list(args)
        for k, v in change.items():
            if k == "draft_len":
                args[2] = v
            elif k == "draft_tokens":
                args[4] = v
            else:
                kw[k] = v
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.spec_process_logits(buf[:, :100], *args, status=st, **kw)
        return int(st)

    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    assert status() == 0
    bad = sv.SV_ERR_BAD_INPUT
    assert status(slots=i(0, 3)) == bad and status(slots=i(-1, 0)) == bad
    assert status(draft_len=i(3, 4)) == bad and status(draft_len=i(-1, 3)) == bad
    assert status(draft_tokens=i(0, 1, 2, 3, 4, 100)) == bad
    assert status(draft_tokens=i(0, 1, 2, 3, 4, -1)) == bad
    for v in (0.0, -1.0, float("nan"), float("inf")):
        assert status(repetition=f(1.1, v)) == bad
    for v in (float("nan"), float("inf"), -float("inf")):
        assert status(presence=f(0.1, v)) == bad and status(frequency=f(v, 0.1)) == bad
    lists = lambda a, t: dict(bias_start=i(*a), bias_tokens=i(*t),  # noqa: E731
                              bias_values=torch.zeros(len(t), device="cuda"))
    assert status(**lists((0, 2, 4), (1, 5, 0, 99))) == 0
    assert status(**lists((0, 2, 4), (5, 1, 0, 99))) == bad     # not ascending
    assert status(**lists((0, 2, 4), (5, 5, 0, 99))) == bad     # a token twice
    assert status(**lists((0, 2, 4), (1, 5, 0, 100))) == bad    # outside the vocabulary
    assert status(**lists((0, 2, 5), (1, 5, 0, 99))) == bad     # past the list
    assert status(**lists((0, 3, 2), (1, 5, 7, 99))) == bad     # runs backwards
    assert status(mask_row=i(*([99] * 10))) == bad and status(mask_row=i(*([-2] * 10))) == bad


@pytest.mark.parametrize("first_row,bonus", [(0, True), (0, False), (2, True)])
@pytest.mark.parametrize("B", [3, 40, 64, 100, 130])
def test_process_bad_data_of_one_request(sv, B, first_row, bonus):
    """Each value of one request that can be wrong, in batches of several sizes; a word that held
    something else before; lists that descend from one request to the next are none."""
    c = _case(B, B, 3, 100, torch.float32, 4, True, ragged=False, first_row=first_row, bonus=bonus)
    start, toks, _ = c["bias"]
    n = len(toks)
    r = int(np.argmax(start[1:] - start[:-1] >= 2))  # a request with two biases at least
    assert start[r + 1] - start[r] >= 2
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def status(stale, name=None, at=0, value=0):
        buf, args, kw = _device_args(c, 104)
        d = dict(draft_len=args[2], draft_tokens=args[4], **{k: v for k, v in kw.items()
                                                               if torch.is_tensor(v)})
        if name:
            d[name][at] = value
        st.fill_(stale)
        sv.spec_process_logits(buf[:, :100], *args, status=st, **kw)
        return int(st)

    bad = sv.SV_ERR_BAD_INPUT
    k = int(start[r])
    row = int(c["row0"][r]) + first_row
    for name, at, value in (
            ("slots", r, -1), ("slots", r, B + 1), ("draft_len", r, -1), ("draft_len", r, 4),
            ("draft_tokens", int(c["draft_row0"][r]) + 2, 100),
            ("draft_tokens", int(c["draft_row0"][r]), -1), ("repetition", r, 0.0),
            ("repetition", r, float("nan")), ("presence", r, float("inf")),
            ("frequency", r, float("nan")), ("bias_start", 0, -1), ("bias_start", B, n + 1),
            ("bias_start", r, k + 9), ("bias_tokens", k, -1), ("bias_tokens", k + 1, 100),
            ("bias_tokens", k + 1, int(toks[k])), ("mask_row", row, -2),
            ("mask_row", row, len(c["mask"])), ("mask_row", row + 2 - first_row, -2)):
        assert status(0, name, at, value) == bad, (name, at, value)
    assert status(bad) == 0 and status(0) == 0
    # a row that the request does not have is not looked at
    if not bonus:
        assert status(7, "mask_row", int(c["row0"][r]) + 3, -2) == 0


def test_empty_mask_is_reported_by_verification(sv):
    """A mask that allows nothing leaves a row of -inf; spec_verify_token reports it."""
    V, g = 256, 2
    t = torch.randn((g + 1, V), device="cuda")
    d = torch.randn((g, V), device="cuda")
    row0 = torch.zeros(1, dtype=torch.int64, device="cuda")
    ln = torch.full((1,), g, dtype=torch.int32, device="cuda")
    tok = torch.zeros(g, dtype=torch.int32, device="cuda")
    mask = torch.zeros((1, 8), dtype=torch.int32, device="cuda")
    sv.spec_process_logits(t, row0, row0, ln, g, tok, mask=mask,
                           mask_row=torch.tensor([-1, 0, -1], dtype=torch.int32, device="cuda"))
    assert torch.isneginf(t[1]).all() and torch.isfinite(t[0]).all() and torch.isfinite(t[2]).all()
    out = sv.spec_verify_token(t, d, row0, row0, ln, g, tok, 0)
    assert int(out["status"]) == sv.SV_ERR_BAD_INPUT


def test_calls_captured_behind_memsets_and_copies(sv):
    """Programmatic dependents whose predecessor in the captured stream is no kernel."""
    V = 517
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, pb, ob = torch.zeros((1, V), **i32), torch.zeros((1, 17), **i32), torch.zeros((1, 17), **i32)
    tok, st = torch.tensor([[3, 3, 9]], **i32), torch.zeros(1, **i32)
    src = torch.randn((1, 520), device="cuda")
    x = torch.zeros_like(src)
    row0, ln = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, **i32)
    rep = torch.full((1,), 2.0, device="cuda")
    h = torch.randn((5, 64), device="cuda")
    out = torch.zeros((5, 8), device="cuda")
    wq = sv.spec_quantize_fp4(torch.randn((8, 64), device="cuda"), 0)
    hq = sv.spec_quantize_fp4(h, 0)
    kw = dict(counts=counts, prompt_bits=pb, output_bits=ob, status=st)

    def step():
        counts.zero_(), ob.zero_()
        sv.spec_history_append(tok, **kw)
        x.copy_(src)
        sv.spec_process_logits(x[:, :V], row0, row0, ln, 0, tok[0], repetition=rep, **kw)
        hq["packed"].copy_(hq["packed"].clone())
        out.zero_()
        sv.spec_project_fp4(hq, wq, out=out, status=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [t.clone() for t in (counts, ob, x, out)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (counts, ob, x, out):
            t.fill_(1)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip((counts, ob, x, out), want))
    assert counts[0, 3] == 2 and x[0, 3] == (src[0, 3] / 2 if src[0, 3] > 0 else src[0, 3] * 2)


def test_process_and_history_in_a_graph(sv):
    """Captured on a side stream and replayed on new inputs: equal to eager calls."""
    c = _case(12, 6, 4, 3001, torch.bfloat16, 12, True, ragged=False)
    V = c["V"]
    buf, args, kw = _device_args(c, 3008)
    src = buf.clone()
    eager_counts = kw["counts"].clone()
    new = torch.randint(0, V, (6, 5), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(counts, x, s):
        sv.spec_process_logits(x[:, :V], *args, status=s, **{**kw, "counts": counts})
        sv.spec_history_append(new, counts, kw["prompt_bits"], kw["output_bits"],
                               slots=kw["slots"], status=s)

    ob = kw["output_bits"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kw["counts"].clone(), buf.clone(), st)
    torch.cuda.current_stream().wait_stream(side)
    kw["output_bits"].copy_(ob)
    g = torch.cuda.CUDAGraph()
    g_counts, x = eager_counts.clone(), src.clone()
    with torch.cuda.graph(g):
        step(g_counts, x, st)
    kw["output_bits"].copy_(ob)
    g_counts.copy_(eager_counts)
    for k in range(3):  # the graph: three rounds on new tokens each
        new.copy_(torch.full_like(new, 17 * k + 1))
        x.copy_(src)
        g.replay()
    got, got_counts, got_bits = x.clone(), g_counts.clone(), kw["output_bits"].clone()
    kw["output_bits"].copy_(ob)
    for k in range(3):
        new.copy_(torch.full_like(new, 17 * k + 1))
        x = src.clone()
        step(eager_counts, x, st)
    assert torch.equal(got.view(torch.int16), x.view(torch.int16))
    assert torch.equal(got_counts, eager_counts) and torch.equal(got_bits, kw["output_bits"])
    assert int(st) == 0
