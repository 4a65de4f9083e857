"""Activation rows so far apart that a tile's rows past the last one would pass 32-bit offsets (no GPU needed)."""
import pytest

import block_scaled_fp8_linear_amd as B

FAKE = 1 << 40


# 20 tokens at 40 MB take 0.8 GB; a tile's row 108 lies past 2^32 bytes, at a wrapped offset inside the 0.8 GB
@pytest.mark.parametrize("M,ldx", [(20, 20_000_000), (2, 16_909_320), (63, 16_909_320), (100, 8_421_504)])
def test_dense_refuses_what_would_wrap(M, ldx):
    N = 33000 if M == 100 else 300      # 258 tiles of 128: the plan takes 129 tiles of 256
    assert M * ldx * 2 < 2 ** 31 and (255 if M == 100 else 127) * ldx * 2 + 512 > 2 ** 32
    st = B.lib().bsf8_linear_dense(FAKE, N, 256, FAKE, M, ldx, FAKE, B.DT_F32, N, None, 0, None)
    assert B.status_name(st) == "UNSUPPORTED"
