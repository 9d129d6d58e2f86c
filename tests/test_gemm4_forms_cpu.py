"""Which form a product in 4 bits takes (the library's own rule, read through the test controls; no GPU)."""
import ctypes

import pytest

import invariant_bi_gemm_gb300 as bg
from invariant_bi_gemm_gb300 import build as bgbuild

I64, I32 = ctypes.c_int64, ctypes.c_int32


def form(K, N, kind, f32, M, sms=152):
    """(rows of w a CTA, CTAs an SM, stages, slots a stage) of the smaller tiles, zeros for CTA pairs."""
    f = ctypes.CDLL(bgbuild.lib_path("libbi_gemm_controls.so")).bi_ctl_gemm4_form
    f.argtypes = [I64, I64, I32, I32, I32, I64] + [ctypes.POINTER(I32)] * 3
    per_sm, stages, slots = I32(), I32(), I32()
    rows = f(K, N, kind, f32, sms, M, *map(ctypes.byref, (per_sm, stages, slots)))
    return rows, per_sm.value, stages.value, slots.value


@pytest.mark.parametrize("kind", [bg.BI_MXFP4, bg.BI_NVFP4])
@pytest.mark.parametrize("f32", [0, 1])
def test_few_rows_take_the_smaller_tiles(kind, f32):
    """Up to 128 rows (bi_gemm4_config.few_rows), however wide w is: every edge of the rule's sizes."""
    for sms in (132, 148, 152, 160):
        for M in (1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128):
            for N in (8, 128, 4096, 128 * sms - 8, 128 * sms, 128 * sms + 8, 19464, 20480, 32000, 128256, 1 << 24):
                for K in (128, 1024, 1152, 4096, 14336):
                    rows, per_sm, stages, slots = form(K, N, kind, f32, M, sms)
                    fine = rows in (32, 64, 128) and per_sm in (1, 2) and stages >= 2 and slots in (2, 4)
                    assert fine, (sms, M, N, K)


@pytest.mark.parametrize("kind", [bg.BI_MXFP4, bg.BI_NVFP4])
@pytest.mark.parametrize("f32", [0, 1])
def test_more_rows_take_them_where_their_tiles_run_at_once(kind, f32):
    for M in (129, 257, 700, 4096):
        for N in (8, 1000, 4096, 10000, 128256):
            rows, per_sm, _, _ = form(1024, N, kind, f32, M)
            once = -(-M // 128) * -(-N // 128) <= 152
            assert (rows > 0) == once and per_sm == int(once), (M, N)
