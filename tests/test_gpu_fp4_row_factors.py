"""Row factors of SV_FP4_E4M3_16 at the ends of their range, 2^-120 .. 2^117.  They are powers of two,
so a logit is the one of the same codes and block scales under row factors of one, scaled exactly --
whatever f * w_factor alone would be, f the sum before the factors (2^-20 <= |f| < 2^47 where it is
not 0).  Where the scaled number leaves binary32's range it is rounded there, once."""
import numpy as np
import pytest
import torch

import plain_serving as plain

pytestmark = pytest.mark.gpu

# both sides of 2^-100 and 2^64, between which the kernel multiplies in binary32, among them
FACTORS = [-120, -119, -106, -101, -100, -99, -60, -23, 0, 1, 30, 63, 64, 65, 81, 100, 116, 117]


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return sv


def _with_factors(op, k):
    return {**op, "row_scales": torch.from_numpy(np.ldexp(1.0, k)).float().cuda()}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,H", [(1, 33, 16), (18, 260, 320), (40, 300, 2560), (200, 70, 100)])
@pytest.mark.parametrize("scales", ["all", "largest", "smallest"])
def test_project_with_factors_of_every_size(sv, M, V, H, dtype, scales):
    rng = np.random.default_rng(M + V + H)
    fmt = sv.SV_FP4_E4M3_16
    ops = []
    for n in (M, V):
        packed, tiles, _, _ = plain.operand(n, H, fmt, rng)
        if scales != "all":  # 448, or 2^-9 with codes of -1.5 .. 1.5
            tiles[tiles > 0] = 126 if scales == "largest" else 1
        if scales == "smallest":
            packed &= 0xBB
        ops.append(plain.device_operand((packed, tiles, np.ones(n), None), n, H, fmt))
    # every pair of factors: rows of X one after the other through them, rows of W a step behind
    kx = [FACTORS[i % len(FACTORS)] for i in range(M)]
    kw = [FACTORS[(i + i // len(FACTORS)) % len(FACTORS)] for i in range(V)]
    ld = (V + 7) // 8 * 8
    for shift in range(0, len(FACTORS), 1 if M < len(FACTORS) else len(FACTORS)):
        k = kx[shift:] + kx[:shift] if M > 1 else [FACTORS[shift]]
        one = sv.spec_project_fp4(ops[0], ops[1], out=torch.zeros((M, ld), device="cuda")[:, :V])
        got = sv.spec_project_fp4(_with_factors(ops[0], k), _with_factors(ops[1], kw),
                                  out=torch.zeros((M, ld), dtype=dtype, device="cuda")[:, :V])
        e = np.array(k)[:, None] + np.array(kw)[None]
        want = torch.from_numpy(np.ldexp(one.double().cpu().numpy(), e)).float().to(dtype)
        assert torch.equal(got.cpu(), want)
