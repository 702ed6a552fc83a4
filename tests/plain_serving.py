"""Plain binary64 forms of the operators around verification, written from their definitions in
include/specverify.h for the tests: history, logits processing, 4-bit blocks.  CPU only."""
import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bits_to_bool(words, V):
    """int32 words [n, W] -> bool [n, V]."""
    w = np.ascontiguousarray(words).view(np.uint32)
    return ((w[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(len(w), -1)[:, :V] != 0


def bool_to_bits(b):
    """bool [n, V] -> int32 words [n, ceil(V / 32)]."""
    n, V = b.shape
    W = (V + 31) // 32
    p = np.zeros((n, W * 32), dtype=np.uint64)
    p[:, :V] = b
    w = (p.reshape(n, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def history_append(tokens, counts, prompt, output, slots, lens, is_prompt, reset):
    """In place on counts [S, V] and bool prompt / output [S, V]."""
    if reset:
        for s in slots:
            counts[s] = 0
            prompt[s] = False
            output[s] = False
    for r, s in enumerate(slots):
        for x in tokens[r, :lens[r]]:
            if x < 0:
                continue
            if is_prompt:
                prompt[s, x] = True
            else:
                counts[s, x] += 1
                output[s, x] = True


def process_row(l, drafted, counts, prompt, output, theta, freq, pres, bias, allowed):
    """One row: (binary64 result, bound on binary32 rounding).  drafted: the tokens before it."""
    n = np.where(output, counts, 0).astype(np.float64)
    for x in drafted:
        n[x] += 1
    seen = prompt | (n > 0)
    l = l.astype(np.float64)
    theta, freq, pres = float(theta), float(freq), float(pres)
    with np.errstate(invalid="ignore", over="ignore"):
        a = np.where(seen, np.where(l > 0, l / theta, l * theta), l)
        b = a - freq * n
        c = b - np.where(n > 0, pres, 0.0)
        d = c + bias
        # one rounding of each step that changes something, relative to its result, and one of f n
        steps = (np.where(seen, np.abs(a), 0) + np.where(n > 0, np.abs(freq * n) + np.abs(b)
                                                         + np.abs(c), 0)
                 + np.where(bias != 0, np.abs(d), 0))
    return np.where(allowed, d, -np.inf), np.where(allowed, steps, 0.0) * 2.0 ** -24 * 1.0001


# ---- 4-bit blocks ------------------------------------------------------------------------------

BLOCK = {0: 32, 1: 16}


def e4m3_values():
    i = np.arange(127)
    e, m = i >> 3, i & 7
    return np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)


def nearest(v, grid):
    """Index of the nearest grid value (ascending grid, v >= 0), ties to the even index."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    d = (v - grid[hi - 1]) - (grid[hi] - v)
    return np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, hi - 1)


def quantize(x, fmt):
    """x float64 [rows, H] -> magnitude codes [rows, H], scale bytes [rows, blocks], row scales,
    values [rows, H]."""
    rows, H = x.shape
    n = BLOCK[fmt]
    nb = (H + n - 1) // n
    xp = np.zeros((rows, nb * n))
    xp[:, :H] = x
    xb = xp.reshape(rows, nb, n)
    amax = np.abs(xb).max(-1)
    if fmt == 0:
        _, e = np.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
        e = np.where(amax > 0, np.clip(e - 3, -127, 127), -127)
        byte, S, g = e + 127, np.ldexp(1.0, e), None
    else:
        top = amax.max(-1)
        m, k = np.frexp(top)
        k = np.where(m > 0.65625, k - 11, k - 12)  # 2688 = 0.65625 * 2^12
        k = np.where(top > 0, np.clip(k, -120, 120), 0)
        g = np.ldexp(1.0, k)
        grid = e4m3_values()
        byte = nearest(amax / 6 / g[:, None], grid)
        S = grid[byte] * g[:, None]
    q = np.divide(np.abs(xb), S[..., None], out=np.zeros_like(xb), where=S[..., None] > 0)
    code = nearest(q, LEVELS)
    val = LEVELS[code] * S[..., None] * np.where(xb < 0, -1.0, 1.0)
    flat = lambda a: a.reshape(rows, -1)[:, :H]  # noqa: E731
    return flat(code), byte.astype(np.uint8), g, flat(val)


def scale_bytes(tiles, rows, nb):
    """The [rows, nb] scale bytes of a tiled scale buffer, each looked up by its address; the rest
    of the buffer must be zero."""
    flat = np.asarray(tiles).reshape(-1)
    row_tiles = (rows + 127) // 128
    groups = len(flat) // 512 // row_tiles
    r, k = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    at = (r // 128 * groups + k // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + k % 4
    rest = flat.copy()
    rest[at] = 0
    return flat[at], not rest.any()


def unpack_codes(packed, H):
    p = np.asarray(packed)
    c = np.stack((p & 15, p >> 4), -1).reshape(len(p), -1)
    return c[:, :H], not c[:, H:].any()


def operand(rows, H, fmt, rng, spread=3):
    """Random codes, scales and row scales: (packed, tiled scales, row scales, float64 values)."""
    n = BLOCK[fmt]
    nb = (H + n - 1) // n
    pad = (H + 31) // 32 * 32
    code = rng.integers(0, 16, (rows, H))
    full = np.zeros((rows, pad), np.uint8)
    full[:, :H] = code
    packed = full[:, 0::2] | (full[:, 1::2] << 4)
    if fmt == 0:
        byte = rng.integers(127 - spread, 128 + spread, (rows, nb)).astype(np.uint8)
        S = np.ldexp(1.0, byte.astype(int) - 127)
        g = None
    else:
        byte = rng.integers(0, 127 if spread else 57, (rows, nb)).astype(np.uint8)
        if not spread:
            byte[:] = 56  # 1.0
        g = np.ldexp(1.0, rng.integers(-spread - 1, spread + 1, rows)) if spread else np.ones(rows)
        S = e4m3_values()[byte] * g[:, None]
    if fmt == 0 and not spread:
        byte[:] = 127
        S[:] = 1.0
    groups = (H + 255) // 256 * (2 if fmt == 0 else 4)
    tiles = np.zeros((rows + 127) // 128 * groups * 512, np.uint8)
    r, k = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    tiles[(r // 128 * groups + k // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + k % 4] = byte
    val = LEVELS[code & 7] * np.where(code > 7, -1.0, 1.0) * np.repeat(S, n, 1)[:, :H]
    return packed, tiles, g, val


def device_operand(parts, rows, H, fmt):
    packed, tiles, g, _ = parts
    return {"packed": torch.from_numpy(packed).cuda(), "scales": torch.from_numpy(tiles).cuda(),
            "row_scales": None if g is None else torch.from_numpy(g).float().cuda(),
            "rows": rows, "H": H, "format": fmt}
