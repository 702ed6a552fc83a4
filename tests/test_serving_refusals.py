"""The operators around verification refuse invalid arguments synchronously: nothing is launched, so
no GPU is needed."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    build.build()
    return sv


FAKE = C.c_void_p(4096)  # never dereferenced: validation fails first
ODD = C.c_void_p(4100)


def test_history_refusals(sv):
    def call(ld=8, n=8, B=4, kind=0, reset=0, V=1000, n_slots=4, ldc=1000, ldb=32, ptr=FAKE):
        return sv.lib().spec_history_append(ptr, ld, None, n, None, B, kind, reset, V, n_slots,
                                            ptr, ldc, ptr, ptr, ldb, None, None)
    assert call(ld=7) == sv.SV_ERR_INVALID
    assert call(n=-1) == sv.SV_ERR_INVALID
    assert call(B=-1) == sv.SV_ERR_INVALID
    assert call(kind=2) == sv.SV_ERR_INVALID
    assert call(reset=2) == sv.SV_ERR_INVALID
    assert call(V=0) == sv.SV_ERR_INVALID
    assert call(ldc=999) == sv.SV_ERR_INVALID
    assert call(ldb=31) == sv.SV_ERR_INVALID
    assert call(n_slots=-1) == sv.SV_ERR_INVALID
    assert call(ptr=None) == sv.SV_ERR_INVALID
    assert call(V=2**31, ldc=2**31, ldb=2**26) == sv.SV_ERR_UNSUPPORTED
    assert call(B=2**30, n=2**12, ld=2**12) == sv.SV_ERR_UNSUPPORTED  # more blocks than a grid holds
    assert call(n=2**31 - 8192, ld=2**31) == sv.SV_ERR_UNSUPPORTED
    assert call(n=2**31 - 1, ld=2**31, reset=1) == sv.SV_ERR_UNSUPPORTED
    assert call(B=0) == sv.SV_OK and call(n=0, ld=0) == sv.SV_OK      # nothing to do


def test_process_refusals(sv):
    def call(logits=FAKE, out=FAKE, ld=1000, ldo=1000, dtype=0, V=1000, gmax=4, first=0, bonus=1,
             B=4, row0=FAKE, slots=4, counts=FAKE, ldc=1000, ldb=32, rep=FAKE, tokens=FAKE,
             bias=None, n_bias=0, bias_tok=None, mask=None, ldm=0, n_mask=0, mask_row=None):
        return sv.lib().spec_process_logits(
            logits, ld, out, ldo, dtype, V, row0, FAKE, FAKE, gmax, first, bonus, tokens, B, None,
            slots, counts, ldc, FAKE, FAKE, ldb, rep, None, None, bias, bias_tok, bias_tok, n_bias,
            mask, ldm, n_mask, mask_row, None, None)
    assert call(V=0) == sv.SV_ERR_INVALID
    assert call(ld=996) == sv.SV_ERR_INVALID
    assert call(ldo=1004) == sv.SV_ERR_INVALID                   # in place under another stride
    assert call(out=C.c_void_p(8192), ldo=996) == sv.SV_ERR_INVALID
    assert call(dtype=2) == sv.SV_ERR_INVALID
    assert call(gmax=65) == sv.SV_ERR_INVALID
    assert call(gmax=-1) == sv.SV_ERR_INVALID
    assert call(first=-1) == sv.SV_ERR_INVALID
    assert call(bonus=2) == sv.SV_ERR_INVALID
    assert call(B=-1) == sv.SV_ERR_INVALID
    assert call(logits=None) == sv.SV_ERR_INVALID
    assert call(row0=None) == sv.SV_ERR_INVALID
    assert call(counts=None) == sv.SV_ERR_INVALID                # penalties without a history
    assert call(slots=0) == sv.SV_ERR_INVALID
    assert call(ldc=999) == sv.SV_ERR_INVALID
    assert call(ldb=31) == sv.SV_ERR_INVALID
    assert call(tokens=None) == sv.SV_ERR_INVALID
    assert call(bias=FAKE, n_bias=-1) == sv.SV_ERR_INVALID
    assert call(bias=FAKE, n_bias=3) == sv.SV_ERR_INVALID        # no entries given
    assert call(mask_row=FAKE, n_mask=2, mask=None, ldm=32) == sv.SV_ERR_INVALID
    assert call(mask_row=FAKE, n_mask=2, mask=FAKE, ldm=31) == sv.SV_ERR_INVALID
    assert call(logits=ODD, out=ODD) == sv.SV_ERR_UNSUPPORTED
    assert call(V=1001, ld=1001, ldo=1001, ldc=1001) == sv.SV_ERR_UNSUPPORTED  # rows not 16 B apart
    assert call(V=2**31 - 4096, ld=2**31, ldo=2**31) == sv.SV_ERR_UNSUPPORTED
    assert call(B=0) == sv.SV_OK


def test_quantize_refusals(sv):
    def call(x=FAKE, dtype=1, rows=8, H=64, ldx=64, fmt=0, packed=FAKE, scales=FAKE, row=None,
             values=None, ldv=0):
        return sv.lib().spec_quantize_fp4(x, dtype, rows, H, ldx, fmt, packed, scales, row, values,
                                          ldv, None, None)
    assert call(dtype=2) == sv.SV_ERR_INVALID
    assert call(fmt=2) == sv.SV_ERR_INVALID
    assert call(rows=-1) == sv.SV_ERR_INVALID
    assert call(H=0) == sv.SV_ERR_INVALID
    assert call(ldx=63) == sv.SV_ERR_INVALID
    assert call(values=FAKE, ldv=63) == sv.SV_ERR_INVALID
    assert call(x=None) == sv.SV_ERR_INVALID
    assert call(packed=None) == sv.SV_ERR_INVALID
    assert call(fmt=1) == sv.SV_ERR_INVALID                      # no row scales
    assert call(packed=ODD) == sv.SV_ERR_UNSUPPORTED
    assert call(scales=ODD) == sv.SV_ERR_UNSUPPORTED
    assert call(x=C.c_void_p(4097)) == sv.SV_ERR_UNSUPPORTED     # not on an element boundary
    assert call(rows=0) == sv.SV_OK
    assert sv.spec_fp4_row_bytes(1) == 16 and sv.spec_fp4_row_bytes(33) == 32
    assert sv.spec_fp4_row_bytes(0) == 0
    # one tile of 128 rows by 4 blocks is 512 bytes; blocks padded to 256 elements
    assert sv.spec_fp4_scale_bytes(1, 1, 0) == 1024 and sv.spec_fp4_scale_bytes(129, 257, 0) == 4096
    assert sv.spec_fp4_scale_bytes(128, 256, 1) == 2048
    assert sv.spec_fp4_scale_bytes(0, 8, 0) == 0 and sv.spec_fp4_scale_bytes(8, 8, 2) == 0


def test_project_refusals(sv):
    def call(x=FAKE, xr=FAKE, M=8, w=FAKE, wr=FAKE, V=1000, H=64, fmt=1, out=FAKE, dtype=1,
             ld=1000):
        return sv.lib().spec_project_fp4(x, x, xr, M, w, w, wr, V, H, fmt, out, dtype, ld, None,
                                         None)
    assert call(dtype=2) == sv.SV_ERR_INVALID
    assert call(fmt=-1) == sv.SV_ERR_INVALID
    assert call(M=-1) == sv.SV_ERR_INVALID
    assert call(V=0) == sv.SV_ERR_INVALID
    assert call(H=0) == sv.SV_ERR_INVALID
    assert call(ld=999) == sv.SV_ERR_INVALID
    assert call(x=None) == sv.SV_ERR_INVALID
    assert call(out=None) == sv.SV_ERR_INVALID
    assert call(xr=None) == sv.SV_ERR_INVALID
    assert call(wr=None) == sv.SV_ERR_INVALID
    assert call(V=2**31 - 1, ld=2**31) == sv.SV_ERR_UNSUPPORTED
    assert call(M=2**24 + 1) == sv.SV_ERR_UNSUPPORTED
    assert call(H=2**24 + 1) == sv.SV_ERR_UNSUPPORTED
    assert call(out=ODD) == sv.SV_ERR_UNSUPPORTED
    assert call(w=ODD) == sv.SV_ERR_UNSUPPORTED
    assert call(V=999, ld=1001) == sv.SV_ERR_UNSUPPORTED          # rows not 16 bytes apart
    assert call(M=0) == sv.SV_OK


def test_host_tensors_are_refused(sv):
    """The binding has no CPU path for these calls either."""
    z = torch.zeros
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.spec_history_append(z((2, 3), **i32), z((2, 64), **i32), z((2, 2), **i32),
                               z((2, 2), **i32))
    with pytest.raises(ValueError):
        sv.spec_process_logits(z((2, 64)), z(2, dtype=torch.int64), None, z(2, **i32), 0, None)
    with pytest.raises(ValueError):
        sv.spec_quantize_fp4(z((2, 64)), sv.SV_FP4_E8M0_32)
    op = {"packed": z((2, 32), dtype=torch.uint8), "scales": z(1024, dtype=torch.uint8),
          "row_scales": None, "rows": 2, "H": 64, "format": 0}
    with pytest.raises(ValueError):
        sv.spec_project_fp4(op, op)
