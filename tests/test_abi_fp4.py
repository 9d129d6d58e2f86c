"""Host-side checks of the entry points in 4 bits that need no GPU: every declared symbol is exported, the binding's
structures match the headers, and bad arguments are refused with the documented codes before any CUDA call."""
import ctypes

import numpy as np
import pytest

import fp4_ref as ref
import invariant_bi_gemm_gb300 as bg
from invariant_bi_gemm_gb300 import build as bgbuild
from test_abi import _declared, _structs

INVALID, UNSUPPORTED = bg.BI_GEMM_ERR_INVALID_ARG, bg.BI_GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("header,names", [("bi_fp4.h", bg.FP4_EXPORTED_SYMBOLS),
                                          ("bi_attention4.h", bg.ATTENTION4_EXPORTED_SYMBOLS)])
def test_header_symbols_exported(header, names):
    declared = _declared(header)
    assert set(declared) == set(names)
    L = ctypes.CDLL(bgbuild.lib_path("libbi_gemm.so"))
    for name in declared:
        assert hasattr(L, name), name


@pytest.mark.parametrize("header,name", [("bi_fp4.h", "bi_quant4_config"), ("bi_fp4.h", "bi_gemm4_config"),
                                         ("bi_attention4.h", "bi_attention4_config")])
def test_binding_structs_match_the_header(header, name):
    assert [n for _, n in _structs(header)[name]] == [n for n, _ in getattr(bg, name)._fields_]
    assert all(t == "int32_t" for t, _ in _structs(header)[name])


@pytest.mark.parametrize("Hq,Hkv,D,page,scale,ks,vs,split,want", [
    (0, 8, 128, 16, 0.1, 1, 1, 0, INVALID), (32, 8, 128, 0, 0.1, 1, 1, 0, INVALID), (32, 8, 128, 16, 0.0, 1, 1, 0, INVALID),
    (32, 8, 128, 16, float("nan"), 1, 1, 0, INVALID), (32, 8, 128, 16, 0.1, 0, 1, 0, INVALID),
    (32, 8, 128, 16, 0.1, 1, float("inf"), 0, INVALID), (32, 8, 128, 16, 0.1, 1, 2.0 ** 65, 0, INVALID),
    (32, 8, 128, 16, 0.1, 1, 1, -128, INVALID), (32, 8, 96, 16, 0.1, 1, 1, 0, UNSUPPORTED),
    (32, 2, 128, 16, 0.1, 1, 1, 0, UNSUPPORTED), (12, 4, 128, 16, 0.1, 1, 1, 0, UNSUPPORTED),
    (32, 8, 128, 16, 0.1, 1, 1, 64, UNSUPPORTED), (32, 8, 128, 16, 0.1, 1, 1, 8192, UNSUPPORTED),
    (32, 8, 128, (1 << 20) + 1, 0.1, 1, 1, 0, UNSUPPORTED),
])
def test_attention4_create_refuses_before_touching_cuda(Hq, Hkv, D, page, scale, ks, vs, split, want):
    h = ctypes.c_void_p()
    assert bg.library().bi_attention4_create(ctypes.byref(h), Hq, Hkv, D, page, scale, ks, vs, split) == want
    assert h.value is None


@pytest.mark.parametrize("K,fmt,g,want", [
    (0, 1, 1.0, INVALID), (256, 2, 1.0, INVALID), (256, 1, 0.0, INVALID), (256, 1, -1.0, INVALID),
    (256, 1, float("nan"), INVALID), (256, 1, float("inf"), INVALID), (256, 1, 2.0 ** -65, INVALID),
    (256, 0, 0.5, INVALID), (192, 1, 1.0, UNSUPPORTED), ((1 << 24) + 128, 1, 1.0, UNSUPPORTED),
])
def test_quant4_create_refuses_before_touching_cuda(K, fmt, g, want):
    h = ctypes.c_void_p()
    assert bg.library().bi_quant4_create(ctypes.byref(h), K, fmt, g) == want
    assert h.value is None


@pytest.mark.parametrize("K,N,fmt,f32,want", [
    (0, 64, 1, 0, INVALID), (256, 0, 1, 0, INVALID), (256, 64, 2, 0, INVALID), (256, 64, 1, 2, INVALID),
    (192, 64, 1, 0, UNSUPPORTED), (256, 60, 1, 0, UNSUPPORTED), (256, (1 << 24) + 8, 1, 0, UNSUPPORTED),
])
def test_gemm4_create_refuses_before_touching_cuda(K, N, fmt, f32, want):
    h = ctypes.c_void_p()
    assert bg.library().bi_gemm4_create(ctypes.byref(h), K, N, fmt, f32) == want
    assert h.value is None


def test_null_arguments():
    L = bg.library()
    assert L.bi_quant4_create(None, 256, 1, 1.0) == INVALID
    assert L.bi_quant4_run(None, None, 1, 256, None, None, None) == INVALID
    assert L.bi_quant4_expand(None, None, None, 1, None, None) == INVALID
    assert L.bi_quant4_scale_bytes(None, 1, None) == INVALID
    assert L.bi_quant4_get_config(None, None) == INVALID
    assert L.bi_quant4_destroy(None) == bg.BI_GEMM_OK
    assert L.bi_attention4_create(None, 32, 8, 128, 16, 0.1, 1.0, 1.0, 0) == INVALID
    assert L.bi_attention4_run(None, None, 1, *[None] * 6, 1, None, 1, 1, 1, None, None) == INVALID
    assert L.bi_attention4_expand(None, *[None] * 4, 1, None, 1, None, None, None) == INVALID
    assert L.bi_attention4_workspace_size(None, 1, 1, None) == INVALID
    assert L.bi_attention4_get_device_error(None, None) == INVALID
    assert L.bi_attention4_get_config(None, None) == INVALID
    assert L.bi_attention4_destroy(None) == bg.BI_GEMM_OK
    assert L.bi_qkrope_run4(None, None, 1, 6144, None, None, None, 1, *[None] * 6, 1.0, 1.0, 1, None, 1, 1, None,
                            None) == INVALID
    assert L.bi_gemm4_create(None, 256, 64, 1, 0) == INVALID
    assert L.bi_gemm4_run(None, None, None, 1, None, None, 1.0, None, None) == INVALID
    assert L.bi_gemm4_get_device_error(None, None) == INVALID
    assert L.bi_gemm4_get_config(None, None) == INVALID
    assert L.bi_gemm4_destroy(None) == bg.BI_GEMM_OK


def test_the_tests_own_format():
    """The reference's pieces against facts of the format: landmarks, ties, round trips and the tiles' permutation."""
    assert list(ref.E4M3[[1, 8, 0x38, 126]]) == [2.0 ** -9, 2.0 ** -6, 1.0, 448.0]
    assert (np.diff(ref.E4M3) > 0).all()
    assert np.array_equal(ref.e4m3_nearest(ref.E4M3), np.arange(127))
    assert list(ref.e4m3_nearest(np.array([1.0625, 1.1875, 500.0, 0.0, 2.0 ** -10]))) == [0x38, 0x3A, 126, 0, 0]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.0])
    assert list(ref.e2m1_nearest(ties)) == [0, 2, 2, 4, 4, 6, 6, 7, 8]
    codes, byte = ref.quantise(np.array([[6.0] + [0.0] * 14 + [1.0]], np.float32).repeat(8, 1)[:, :16], "nvfp4")
    assert byte[0, 0] == 0x38 and codes[0, 0] == 7
    s = np.arange(200 * 8, dtype=np.uint32).astype(np.uint8).reshape(200, 8)
    assert np.array_equal(ref.from_tiles(ref.to_tiles(s), 200), s)
    t = ref.to_tiles(s)
    for r, c in ((0, 0), (31, 3), (32, 4), (127, 7), (128, 0), (199, 5)):
        assert t[r // 128, c // 4, r % 32, r // 32 % 4, c % 4] == s[r, c]


@pytest.mark.parametrize("scale,ks,fine", [(2.0 ** 100, 2.0 ** 64, False), (3e38, 1.0, False), (2.0 ** 64, 2.0 ** 64, False),
                                           (2.0 ** 63, 2.0 ** 64, True), (2e38, 1.0, True), (1e-38, 2.0 ** -64, True)])
def test_attention4_create_refuses_factors_beyond_fp32(scale, ks, fine):
    """scale k_scale log2(e), the factor of every score, has to be a finite fp32 number; scales that it is for get as far
    as the device (none here, or a handle)."""
    h = ctypes.c_void_p()
    rc = bg.library().bi_attention4_create(ctypes.byref(h), 32, 8, 128, 16, scale, ks, 1.0, 0)
    assert (rc != INVALID) == fine
    bg.library().bi_attention4_destroy(h)
