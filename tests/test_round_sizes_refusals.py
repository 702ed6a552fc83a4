"""Numbers of rows next to 2^31 are refused by spec_tree_attention before anything is launched: no GPU is needed."""
import ctypes as C

import pytest

FAKE = C.c_void_p(4096)  # never dereferenced: validation fails first


@pytest.mark.parametrize("rows", [2**31 - 256, 2**31 - 1, 2**40])
def test_rows(rows):
    import speculative_decoding_verification_token_gb300 as sv
    from speculative_decoding_verification_token_gb300 import build
    build.build()
    assert sv.lib().spec_tree_attention(
        FAKE, 512, 64, rows, 4, 2, 64, 0.1, FAKE, FAKE, 5, 1, None, 2, FAKE, FAKE, 4, 4, FAKE, FAKE, 9, 16, 2048,
        128, 64, FAKE, 256, 64, None, 0, None, FAKE, 1 << 40, None) == sv.SV_ERR_UNSUPPORTED
