"""Timed cases of the serving operators around verification: the token history, the logits
processor, 4-bit quantisation and the 4-bit output projection.

Each case is one call as an engine makes it.  With `own` false, `run` computes the call in its
plain form (elementary torch operations in binary32, rounded once at the end); with `own` true it
makes the library's call on the same state.  `exact` evaluates the definitions in binary64.

  history   spec_history_append: tokens added to per-slot output counts and seen bits
  process   spec_process_logits: repetition / presence / frequency penalties, logit biases and
            grammar masks on the rows of a speculative round (row i of a request is conditioned on
            its history and on its first i drafted tokens)
  quantize  spec_quantize_fp4: rows of hidden states or weights to blocks of 4-bit values
  project   spec_project_fp4: logits = hidden rows times the output projection, both in 4 bits
"""
import math

import torch

own = False

E8M0_32, E4M3_16 = 0, 1
_BLOCK = {E8M0_32: 32, E4M3_16: 16}


# ---- cases -------------------------------------------------------------------------------------

def _history(name, B, n, V, prompt):
    return {"name": name, "op": "history", "B": B, "n": n, "V": V, "prompt": prompt}


def _process(name, B, gamma, V, dtype, in_place, ragged, history, bias, masked, allow):
    return {"name": name, "op": "process", "B": B, "gamma": gamma, "V": V, "dtype": dtype,
            "in_place": in_place, "ragged": ragged, "history": history, "bias": bias,
            "masked": masked, "allow": allow}


def _quantize(name, rows, H, dtype, fmt):
    return {"name": name, "op": "quantize", "rows": rows, "H": H, "dtype": dtype, "fmt": fmt}


def _project(name, M, V, H, fmt, dtype):
    return {"name": name, "op": "project", "M": M, "V": V, "H": H, "fmt": fmt, "dtype": dtype}


def listed():
    return [
        # the tokens of one verified round of 64 requests (5 drafts and a correction each)
        _history("append a round, 64x5", 64, 6, 151936, False),
        # 32 requests admitted: their slots cleared, ragged prompts of up to 8192 tokens
        _history("admit prompts, 32x8192", 32, 8192, 129280, True),
        # one request decoding without drafts: a single row, penalised where it lies
        _process("one row in place", 1, 0, 151936, "f32", True, False, 700, 0, False, 1.0),
        # the token-level benchmark's round: every row copied with penalties and biases
        _process("round 64x5", 64, 5, 151936, "bf16", False, False, 2000, 300, False, 1.0),
        # the block benchmark's round, half the requests under a grammar that allows few tokens
        _process("grammar 128x7 in place", 128, 7, 129280, "bf16", True, False, 1500, 0, True, 0.02),
        # a large ragged round with everything on: most tokens allowed (inside a string)
        _process("ragged 256x8", 256, 8, 129280, "bf16", False, True, 4000, 50, True, 0.9),
        # hidden rows of a small odd batch, odd width
        _quantize("hidden 7x1001", 7, 1001, "f32", E4M3_16),
        # target hidden rows of the 64 x 5 round
        _quantize("hidden 384x2560", 384, 2560, "bf16", E8M0_32),
        # an output projection quantised when a model is loaded
        _quantize("weights 151936x2560", 151936, 2560, "bf16", E4M3_16),
        # one request's target rows
        _project("logits 6x2560", 6, 151936, 2560, E8M0_32, "bf16"),
        # the 64 x 5 round's target rows, logits kept in 32 bits
        _project("logits 384x2560", 384, 151936, 2560, E8M0_32, "f32"),
        # 128 requests of 7 drafts and a bonus row, wider model
        _project("logits 1024x4096", 1024, 129280, 4096, E4M3_16, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("history", "process", "quantize", "project"))
    if op == "history":
        prompt = rng.random() < 0.5
        n = _log(rng, 16, 8192) if prompt else rng.randint(1, 17)
        c = _history("", _log(rng, 1, 256 if not prompt else 32), n, _log(rng, 1000, 160000), prompt)
    elif op == "process":
        gamma = rng.randint(0, 16)
        V = _log(rng, 1000, 152000)
        most = max(1, min(256, int(2.9e8 // (V * (gamma + 1)))))
        masked = rng.random() < 0.5
        c = _process("", _log(rng, 1, most), gamma, V, rng.choice(("bf16", "f32")),
                     rng.random() < 0.5, rng.random() < 0.5, _log(rng, 1, 8000),
                     rng.choice((0, 0, 1, 17, 300)), masked,
                     rng.choice((0.001, 0.05, 0.5, 0.95)) if masked else 1.0)
    elif op == "quantize":
        H = rng.choice((rng.randint(1, 300), 128 * rng.randint(1, 56), _log(rng, 300, 8192)))
        most = max(1, min(152000, int(3.8e8 // H)))
        c = _quantize("", _log(rng, 1, most), H, rng.choice(("bf16", "f32")),
                      rng.choice((E8M0_32, E4M3_16)))
    else:
        H = rng.choice((128 * rng.randint(1, 56), _log(rng, 33, 7168)))
        V = _log(rng, 500, 152000)
        M = _log(rng, 1, 1100)
        M = max(1, min(M, int(5.0e11 // (H * V))))
        c = _project("", M, V, H, rng.choice((E8M0_32, E4M3_16)), rng.choice(("bf16", "f32")))
    del c["name"]
    return c


# ---- inputs ------------------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _zipf_tokens(shape, V, g):
    """Token ids whose frequency falls like 1 / rank, spread over the vocabulary."""
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return ((rank * 7919 + 13) % V).to(torch.int32)


def _pack_bits(b):
    """[n, V] truth values -> [n, ceil(V / 32)] words, token v in bit v % 32 of word v // 32."""
    n, V = b.shape
    W = (V + 31) // 32
    out = torch.empty((n, W), dtype=torch.int32, device=b.device)
    weight = (1 << torch.arange(32, device=b.device, dtype=torch.int64))
    step = max(1, (1 << 27) // (W * 32))
    for a in range(0, n, step):
        p = torch.zeros((min(step, n - a), W * 32), dtype=torch.int64, device=b.device)
        p[:, :V] = b[a:a + step]
        s = (p.view(-1, W, 32) * weight).sum(-1)
        out[a:a + step] = (s - ((s >> 31) << 32)).to(torch.int32)
    return out


def _prepare_history(c, g):
    B, n, V = c["B"], c["n"], c["V"]
    W = (V + 31) // 32
    slots = torch.randperm(B + 3, generator=g, device="cuda")[:B].to(torch.int32)
    lens = torch.randint(0 if B > 1 else 1, n + 1, (B,), generator=g, device="cuda",
                         dtype=torch.int32)
    tokens = _zipf_tokens((B, n), V, g)
    tokens[torch.arange(n, device="cuda")[None] >= lens[:, None]] = -1
    # what the slots hold from earlier rounds (or from the requests that had them before)
    counts = torch.zeros((B + 3, V), dtype=torch.int32, device="cuda")
    old = _zipf_tokens((B + 3, 500), V, g).long()
    counts.scatter_add_(1, old, torch.ones_like(old, dtype=torch.int32))
    seen = torch.zeros((B + 3, V), dtype=torch.bool, device="cuda")
    seen.scatter_(1, _zipf_tokens((B + 3, 500), V, g).long(), True)
    return {"tokens": tokens, "lens": lens, "slots": slots, "counts": counts,
            "prompt_bits": _pack_bits(seen), "output_bits": _pack_bits(counts > 0),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "V": V, "W": W,
            "prompt": c["prompt"]}


def _prepare_process(c, g):
    B, G, V = c["B"], c["gamma"], c["V"]
    rows = B * (G + 1)
    ld = (V + 7) // 8 * 8
    prior = -1.1 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
    prior = prior[(torch.arange(V, device="cuda") * 7919 + 13) % V]
    buf = torch.zeros((rows, ld), dtype=_DT[c["dtype"]], device="cuda")
    step = max(1, (1 << 28) // V)
    for a in range(0, rows, step):
        k = min(step, rows - a)
        buf[a:a + k, :V] = torch.randn((k, V), generator=g, device="cuda") * 3 + prior
    if c["ragged"]:
        draft_len = torch.randint(0, G + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    else:
        draft_len = torch.full((B,), G, dtype=torch.int32, device="cuda")
    # histories: prompt and output tokens of each request, of its own lengths
    H = c["history"]
    at = torch.arange(H, device="cuda")[None]
    plen = torch.randint(0, H + 1, (B, 1), generator=g, device="cuda")
    olen = torch.randint(0, H + 1, (B, 1), generator=g, device="cuda")
    # (a masked token scatters into a spare last column)
    pt = torch.where(at < plen, _zipf_tokens((B, H), V, g).long(), V)
    ot = torch.where(at < olen, _zipf_tokens((B, H), V, g).long(), V)
    seen = torch.zeros((B, V + 1), dtype=torch.bool, device="cuda").scatter_(1, pt, True)[:, :V]
    counts = torch.zeros((B, V + 1), dtype=torch.int32, device="cuda")
    counts = counts.scatter_add_(1, ot, torch.ones_like(ot, dtype=torch.int32))[:, :V].contiguous()
    slots = torch.randperm(B, generator=g, device="cuda").to(torch.int32)

    def uniform(lo, hi):
        v = torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo
        return v

    # one request in four uses no repetition penalty, one in four none of the additive ones
    rep = torch.where(torch.rand(B, generator=g, device="cuda") < 0.25, 1.0, uniform(1.0, 1.3))
    add = (torch.rand(B, generator=g, device="cuda") >= 0.25).float()
    s = {"logits": buf[:, :V], "out": None, "row0": torch.arange(B, device="cuda") * (G + 1),
         "draft_row0": torch.arange(B, device="cuda") * max(G, 1), "draft_len": draft_len,
         "gamma": G, "draft_tokens": _zipf_tokens((B * max(G, 1),), V, g), "slots": slots,
         "counts": counts, "prompt_bits": _pack_bits(seen), "output_bits": _pack_bits(counts > 0),
         "repetition": rep, "presence": uniform(0.0, 1.0) * add,
         "frequency": uniform(0.0, 0.5) * add, "bias_start": None, "bias_tokens": None,
         "bias_values": None, "mask": None, "mask_row": None,
         "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "B": B, "V": V}
    s["out"] = s["logits"] if c["in_place"] else torch.zeros_like(buf)[:, :V]
    if c["bias"]:
        n = min(c["bias"], V)
        w = V // n
        t = torch.randint(0, w, (B, n), generator=g, device="cuda")
        t = t + torch.arange(n, device="cuda") * w  # ascending, no token twice
        s["bias_start"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
        s["bias_tokens"] = t.reshape(-1).to(torch.int32)
        s["bias_values"] = torch.randn(B * n, generator=g, device="cuda") * 4
    if c["masked"]:  # every other request is under a grammar: a mask row for each of its rows
        req = torch.arange(rows, device="cuda") // (G + 1)
        on = req % 2 == 0
        n_mask = int(on.sum())
        s["mask_row"] = torch.where(on, torch.cumsum(on, 0) - 1, -1).to(torch.int32)
        s["mask"] = torch.cat([_pack_bits(torch.rand((min(step, n_mask - a), V), generator=g,
                                                     device="cuda") < c["allow"])
                               for a in range(0, n_mask, step)])
    return s


def _prepare_quantize(c, g):
    rows, H = c["rows"], c["H"]
    # rows of unequal size and a few large channels, as hidden states and weights have
    x = torch.randn((rows, H), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    x *= torch.where(torch.rand((1, H), generator=g, device="cuda") < 0.02, 8.0, 1.0)
    return {"x": x.to(_DT[c["dtype"]]), "fmt": c["fmt"],
            "values": torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda"),
            "packed": torch.zeros((rows, (H + 31) // 32 * 16), dtype=torch.uint8, device="cuda"),
            "scales": torch.zeros(_scale_shape(rows, H, c["fmt"]), dtype=torch.uint8,
                                  device="cuda"),
            "row_scales": (torch.zeros(rows, device="cuda") if c["fmt"] == E4M3_16 else None),
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prepare_project(c, g):
    M, V, H, fmt = c["M"], c["V"], c["H"], c["fmt"]
    x = torch.randn((M, H), generator=g, device="cuda")
    w = torch.randn((V, H), generator=g, device="cuda") * (3.0 / math.sqrt(H))
    ld = (V + 7) // 8 * 8
    return {"x": _quantized(x.to(torch.bfloat16), fmt), "w": _quantized(w.to(torch.bfloat16), fmt),
            "out": torch.zeros((M, ld), dtype=_DT[c["dtype"]], device="cuda")[:, :V],
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    return {"op": case["op"], **globals()["_prepare_" + case["op"]](case, _gen(seed))}


# ---- plain forms -------------------------------------------------------------------------------

def _unpack_bits(w, V):
    return ((w[:, :, None] >> torch.arange(32, device=w.device, dtype=torch.int32)) & 1).view(
        w.shape[0], -1)[:, :V].bool()


def _plain_history(s):
    V, W = s["V"], s["W"]
    slots = s["slots"].long()
    bits = s["prompt_bits"] if s["prompt"] else s["output_bits"]
    if s["prompt"]:
        s["counts"][slots] = 0
        s["prompt_bits"][slots] = 0
        s["output_bits"][slots] = 0
    tok = s["tokens"].long()
    tok = torch.where(tok >= 0, tok, W * 32)
    add = torch.zeros((tok.shape[0], W * 32 + 1), dtype=torch.int32, device=tok.device)
    add = add.scatter_add_(1, tok, torch.ones_like(tok, dtype=torch.int32))[:, :W * 32]
    if not s["prompt"]:
        s["counts"][slots] += add[:, :V]
    set_ = (add.view(-1, W, 32) > 0).to(torch.int32)
    words = (set_ << torch.arange(32, device=tok.device, dtype=torch.int32)).sum(
        -1, dtype=torch.int32)
    bits[slots] |= words
    return {"counts": s["counts"], "prompt_bits": s["prompt_bits"], "output_bits": s["output_bits"]}


def _plain_process(s):
    B, G, V = s["B"], s["gamma"], s["V"]
    R = G + 1
    slots = s["slots"].long()
    lane = torch.arange(R, device=slots.device)
    used = lane[None] <= s["draft_len"][:, None]  # [B, R]
    # tokens drafted before each row, counted
    out_count = s["counts"][slots][:, None, :].repeat(1, R, 1)
    if G:
        tok = s["draft_tokens"].view(B, 1, G).expand(B, R, G).long()
        before = (torch.arange(G, device=slots.device)[None] < lane[:, None]).to(torch.int32)
        out_count.scatter_add_(2, tok, before[None].expand(B, R, G).contiguous())
    seen = _unpack_bits(s["prompt_bits"][slots], V)[:, None, :] | (out_count > 0)
    x = s["logits"].float().view(B, R, V)
    rep = s["repetition"][:, None, None]
    y = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    y = y - s["frequency"][:, None, None] * out_count
    y = y - torch.where(out_count > 0, s["presence"][:, None, None], 0.0)
    if s["bias_tokens"] is not None:
        dense = torch.zeros((B, V), device=x.device)
        dense.scatter_(1, s["bias_tokens"].view(B, -1).long(), s["bias_values"].view(B, -1))
        y = y + dense[:, None, :]
    y = y.view(B * R, V)
    if s["mask"] is not None:
        row = s["mask_row"].long()
        ok = _unpack_bits(s["mask"], V)[row.clamp_min(0)] | (row < 0)[:, None]
        y = torch.where(ok, y, -math.inf)
    s["out"].copy_(torch.where(used.view(-1, 1), y.to(s["out"].dtype), s["out"]))
    return s["out"]


def _scale_shape(rows, H, fmt):
    """Scales lie in tiles of 128 rows by 4 blocks (512 bytes): byte (r % 32) * 16 + (r // 32) * 4 +
    k of a tile is row r's scale of block k; the blocks of a row are padded to 256 elements."""
    return ((rows + 127) // 128, (H + 255) // 256 * (64 // _BLOCK[fmt]), 512)


def _tile_scales(s, rows, H, fmt):
    t, k, _ = _scale_shape(rows, H, fmt)
    full = torch.zeros((t * 128, k * 4), dtype=torch.uint8, device=s.device)
    full[:rows, :s.shape[1]] = s
    return full.view(t, 4, 32, k, 4).permute(0, 3, 2, 1, 4).reshape(t, k, 512).contiguous()


def _untile_scales(tiles, rows, n):
    t, k, _ = tiles.shape
    return tiles.view(t, k, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(t * 128, k * 4)[:rows, :n]


def _pow2(e):
    """2^e exactly, in binary64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _codes(a):
    """Nearest 4-bit magnitude (0, .5, 1, 1.5, 2, 3, 4, 6) of a >= 0, ties to the even code."""
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c


def _quantize_plain(x, fmt):
    """(codes [rows, Hp], scale bytes [rows, blocks], power-of-two row scales or None, values)."""
    rows, H = x.shape
    n = _BLOCK[fmt]
    Hp = (H + n - 1) // n * n
    xf = torch.zeros((rows, Hp), device=x.device)
    xf[:, :H] = x
    xb = xf.view(rows, -1, n)
    amax = xb.abs().amax(-1)
    if fmt == E8M0_32:
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)  # floor(log2 amax) - 2
        e = torch.where(amax > 0, e, -127)
        byte = (e + 127).to(torch.uint8)
        scale = _pow2(e).float()
        row = None
    else:
        m, k = torch.frexp(amax.amax(-1))  # m in [0.5, 1): row maximum m * 2^k
        k = torch.where(m <= 0.65625, k - 12, k - 11)  # smallest 2^k with maximum / 2^k <= 6 * 448
        k = torch.where(m > 0, k, 0).clamp(-120, 120)
        row = _pow2(k).float()
        # in 64 bits: a quotient by 6 must not be rounded onto the middle of two scales
        t = (amax.double() / 6 / row[:, None].double())
        ex = (torch.frexp(t)[1] - 1).clamp_min(-6)
        q = _pow2(ex - 3)
        t = (torch.round(t / q) * q).float()
        byte = t.to(torch.float8_e4m3fn).view(torch.uint8)
        scale = t * row[:, None]
    inv = torch.where(scale > 0, scale, 1.0)[:, :, None].double()
    a = torch.where(scale[:, :, None] > 0, xb.abs().double() / inv, 0.0)
    c = _codes(a)
    level = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    v = level[c.int()] * scale[:, :, None]
    v = torch.where(xb < 0, -v, v).view(rows, Hp)[:, :H]
    c = torch.where(xb < 0, c + 8, c).view(rows, Hp)
    return c, byte, row, v


def _quantized(x, fmt):
    rows, H = x.shape
    pad = (H + 31) // 32 * 32
    packed = torch.zeros((rows, pad // 2), dtype=torch.uint8, device=x.device)
    scales = torch.zeros(((rows + 127) // 128 * 128, (H + _BLOCK[fmt] - 1) // _BLOCK[fmt]),
                         dtype=torch.uint8, device=x.device)
    row_scales = torch.zeros(rows, device=x.device) if fmt == E4M3_16 else None
    step = max(1, (1 << 27) // H)
    for a in range(0, rows, step):
        c, byte, row, _ = _quantize_plain(x[a:a + step], fmt)
        full = torch.zeros((c.shape[0], pad), dtype=torch.uint8, device=x.device)
        full[:, :c.shape[1]] = c
        packed[a:a + step] = full[:, 0::2] | (full[:, 1::2] << 4)
        scales[a:a + c.shape[0]] = byte
        if row is not None:
            row_scales[a:a + step] = row
    return {"packed": packed, "scales": _tile_scales(scales[:rows], rows, H, fmt),
            "row_scales": row_scales, "rows": rows, "H": H, "format": fmt}


def _dequantize(t):
    rows, H, fmt = t["rows"], t["H"], t["format"]
    n = _BLOCK[fmt]
    p = t["packed"]
    code = torch.stack((p & 15, p >> 4), -1).view(rows, -1)
    level = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6],
                         device=p.device)
    byte = _untile_scales(t["scales"], rows, code.shape[1] // n)
    if fmt == E8M0_32:
        scale = _pow2(byte.int() - 127).float()
    else:
        scale = byte.contiguous().view(torch.float8_e4m3fn).float() * t["row_scales"][:, None]
    return (level[code.int()].view(rows, -1, n) * scale[:, :, None]).view(rows, -1)[:, :H]


def _plain_quantize(s):
    c, byte, row, v = _quantize_plain(s["x"], s["fmt"])
    s["values"].copy_(v)
    return s["values"]


def _plain_project(s):
    s["out"].copy_(_dequantize(s["x"]) @ _dequantize(s["w"]).t())
    return s["out"]


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    if not own:
        return _PLAIN[state["op"]](state)
    return _OWN[state["op"]](state)


def _own_history(s):
    import speculative_decoding_verification_token_gb300 as sv
    sv.spec_history_append(s["tokens"], s["counts"], s["prompt_bits"], s["output_bits"],
                           slots=s["slots"], prompt=s["prompt"], reset=s["prompt"],
                           status=s["status"])
    return {"counts": s["counts"], "prompt_bits": s["prompt_bits"], "output_bits": s["output_bits"]}


def _own_process(s):
    import speculative_decoding_verification_token_gb300 as sv
    sv.spec_process_logits(s["logits"], s["row0"], s["draft_row0"], s["draft_len"], s["gamma"],
                           s["draft_tokens"], out=s["out"], slots=s["slots"], counts=s["counts"],
                           prompt_bits=s["prompt_bits"], output_bits=s["output_bits"],
                           repetition=s["repetition"], presence=s["presence"],
                           frequency=s["frequency"], bias_start=s["bias_start"],
                           bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
                           mask=s["mask"], mask_row=s["mask_row"], status=s["status"])
    return s["out"]


def _own_quantize(s):
    import speculative_decoding_verification_token_gb300 as sv
    sv.spec_quantize_fp4(s["x"], s["fmt"], packed=s["packed"], scales=s["scales"],
                         row_scales=s["row_scales"], values=s["values"], status=s["status"])
    return s["values"]


def _own_project(s):
    import speculative_decoding_verification_token_gb300 as sv
    sv.spec_project_fp4(s["x"], s["w"], out=s["out"], status=s["status"])
    return s["out"]


_PLAIN = {"history": _plain_history, "process": _plain_process, "quantize": _plain_quantize,
          "project": _plain_project}
_OWN = {"history": _own_history, "process": _own_process, "quantize": _own_quantize,
        "project": _own_project}


# ---- what a pass cannot do without ---------------------------------------------------------------

def _distinct(n, V):
    """Expected distinct tokens among n draws of probability 1 / (rank ln V), by rank octaves."""
    octaves = ((2 ** i, min(2 ** (i + 1), V + 1)) for i in range(V.bit_length()))
    return sum((1 - (1 - min(1.0, 1 / (1.4 * a * math.log(V)))) ** n) * (b - a)
               for a, b in octaves if a <= V)


def work(case):
    c = case
    if c["op"] == "history":
        n = c["B"] * c["n"] / 2  # lengths are uniform over 0 .. n
        if c["prompt"]:
            clear = c["B"] * (4 * c["V"] + 2 * c["V"] / 8)
            return {"bytes": n * 4 + c["B"] * _distinct(c["n"] / 2, c["V"]) * 4 + clear, "flops": n}
        return {"bytes": n * (4 + 8 + 8), "flops": n}
    if c["op"] == "process":
        e = 2 if c["dtype"] == "bf16" else 4
        V, B = c["V"], c["B"]
        rows = B * (c["gamma"] / 2 + 1 if c["ragged"] else c["gamma"] + 1)
        # bits of every slot, counts and logits of the tokens that a history or a bias touches
        out_tokens = _distinct(c["history"] / 2, V)
        touched = _distinct(c["history"], V) + c["bias"]
        b = B * (2 * V / 8 + 4 * out_tokens + 8 * c["bias"])
        masked = (rows + (c["gamma"] + 1 if B % 2 else 0)) / 2 if c["masked"] else 0.0
        b += masked * V / 8
        if c["in_place"]:
            b += masked * V * (1 - c["allow"]) * e
            b += 2 * e * touched * (rows - masked + masked * c["allow"])
        else:
            b += e * V * (2 * rows - masked * (1 - c["allow"]))
        return {"bytes": b, "flops": 4 * rows * touched}
    if c["op"] == "quantize":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["rows"] * c["H"]
        b = n * (e + 0.5 + 2) + n / _BLOCK[c["fmt"]]
        return {"bytes": b + (4 * c["rows"] if c["fmt"] == E4M3_16 else 0), "flops": 3 * n}
    e = 2 if c["dtype"] == "bf16" else 4
    M, V, H = c["M"], c["V"], c["H"]
    b = (M + V) * H * (0.5 + 1 / _BLOCK[c["fmt"]]) + M * V * e
    return {"bytes": b + (4 * (M + V) if c["fmt"] == E4M3_16 else 0), "flops": 2 * M * V * H}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _exact_process(s):
    """One request at a time, its rows in binary64."""
    V, R = s["V"], s["gamma"] + 1
    out = s["out"].double()
    shift = torch.arange(32, device=out.device)
    for r in range(s["B"]):
        slot = int(s["slots"][r])
        n = int(s["draft_len"][r]) + 1
        prompt = ((s["prompt_bits"][slot][:, None] >> shift) & 1).reshape(-1)[:V] != 0
        base = s["counts"][slot].double()
        theta, f, p = (float(s[k][r]) for k in ("repetition", "frequency", "presence"))
        add = torch.zeros(V, dtype=torch.float64, device=out.device)
        if s["bias_tokens"] is not None:
            a, b = int(s["bias_start"][r]), int(s["bias_start"][r + 1])
            add[s["bias_tokens"][a:b].long()] = s["bias_values"][a:b].double()
        drafted = torch.zeros(V, dtype=torch.float64, device=out.device)
        for i in range(n):
            if i:
                drafted[int(s["draft_tokens"][int(s["draft_row0"][r]) + i - 1])] += 1
            count = base + drafted
            x = s["logits"][r * R + i].double()
            y = torch.where(prompt | (count > 0), torch.where(x > 0, x / theta, x * theta), x)
            y = y - f * count - p * (count > 0).double() + add
            if s["mask"] is not None and int(s["mask_row"][r * R + i]) >= 0:
                m = s["mask"][int(s["mask_row"][r * R + i])]
                y[((m[:, None] >> shift) & 1).reshape(-1)[:V] == 0] = -math.inf
            out[r * R + i] = y
    return out


def _two_to(e):
    return torch.ones((), dtype=torch.float64, device=e.device).view(torch.int64).add(
        e.long() * 2 ** 52).view(torch.float64)


def _exact_quantize(s):
    """Nearest representable value, found among all of them."""
    x, fmt = s["x"].double(), s["fmt"]
    rows, H = x.shape
    n = _BLOCK[fmt]
    out = torch.empty((rows, H), dtype=torch.float64, device=x.device)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64,
                        device=x.device)
    if fmt == E4M3_16:  # the 127 finite scales in order; their index is their byte
        i = torch.arange(127, device=x.device)
        man, ex = (i & 7).double() / 8, (i >> 3)
        scales = torch.where(ex > 0, (1 + man) * _two_to(ex - 7), man / 64)

    def nearest(v, grid):  # ties to the even index
        hi = torch.searchsorted(grid, v.contiguous()).clamp(1, len(grid) - 1)
        lo = hi - 1
        d = (v - grid[lo]) - (grid[hi] - v)
        return torch.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)

    step = max(1, (1 << 26) // H)
    for a in range(0, rows, step):
        xs = torch.nn.functional.pad(x[a:a + step], (0, -H % n)).view(-1, (H + n - 1) // n, n)
        top = xs.abs().amax(-1)
        if fmt == E8M0_32:
            e = torch.floor(torch.log2(top))
            e = torch.where(top > 0, e, 0.0)
            e = torch.where(_two_to(e) > top, e - 1, torch.where(_two_to(e + 1) <= top, e + 1, e))
            sc = torch.where(top > 0, _two_to((e - 2).clamp(-127, 127)), 0.0)
        else:
            most = top.amax(-1, keepdim=True)
            g = torch.where(most > 0, torch.ceil(torch.log2(most / 2688)), 0.0)
            g = torch.where(most > 2688 * _two_to(g), g + 1, g)
            g = torch.where(most > 2688 * _two_to(g - 1), g, g - 1)
            g = torch.where(most > 0, _two_to(g.clamp(-120, 120)), 1.0)
            sc = scales[nearest(top / 6 / g, scales)] * g
        q = torch.where(sc[..., None] > 0, xs.abs() / sc[..., None], 0.0)
        v = grid[nearest(q, grid)] * sc[..., None] * torch.sign(xs)
        out[a:a + step] = v.view(xs.shape[0], -1)[:, :H]
    return out


def _exact_project(s):
    def values(t):
        rows, H, fmt = t["rows"], t["H"], t["format"]
        p = t["packed"].int()
        code = torch.stack((p & 15, p >> 4), -1).reshape(rows, -1)[:, :H]
        m = code & 7
        mag = torch.where(m < 2, m * 0.5, (1 + 0.5 * (m & 1)) * _two_to((m >> 1) - 1))
        k = torch.arange(H, device=p.device) // _BLOCK[fmt]
        r = torch.arange(rows, device=p.device)
        flat = t["scales"].view(t["scales"].shape[0], -1)
        b = flat[r[:, None] // 128, (k // 4 * 512 + k % 4)[None] +
                 ((r % 32) * 16 + (r % 128) // 32 * 4)[:, None]].int()
        if fmt == E8M0_32:
            sc = _two_to(b - 127)
        else:
            e, f = b >> 3, (b & 7).double() / 8
            sc = torch.where(e > 0, (1 + f) * _two_to(e - 7), f / 64)
            sc = sc * t["row_scales"].double()[:, None]
        return torch.where(code > 7, -mag, mag) * sc

    x = values(s["x"])
    w = s["w"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=x.device)
    step = 128 * max(1, (1 << 26) // (128 * w["H"]))
    for a in range(0, w["rows"], step):  # whole scale tiles at a time
        b = min(a + step, w["rows"])
        part = {"packed": w["packed"][a:b], "scales": w["scales"][a // 128:(b + 127) // 128],
                "row_scales": None if w["row_scales"] is None else w["row_scales"][a:b],
                "rows": b - a, "H": w["H"], "format": w["format"]}
        out[:, a:b] = x @ values(part).t()
    return out


def exact(case, seed):
    if case["op"] == "history":
        return None  # whole numbers
    return {"process": _exact_process, "quantize": _exact_quantize,
            "project": _exact_project}[case["op"]](prepare(case, seed))
