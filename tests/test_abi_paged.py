"""Host-side checks of the entry points around the paged cache that need no GPU: every declared
symbol is exported, the binding's structures match the headers, and bad arguments are refused with
the documented codes before any CUDA call."""
import ctypes

import pytest

import invariant_bi_gemm_gb300 as bg
from invariant_bi_gemm_gb300 import build as bgbuild
from test_abi import _declared, _structs

INVALID, UNSUPPORTED = bg.BI_GEMM_ERR_INVALID_ARG, bg.BI_GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("header,names", [("bi_qkrope.h", bg.QKROPE_EXPORTED_SYMBOLS),
                                          ("bi_prompt.h", bg.PROMPT_EXPORTED_SYMBOLS)])
def test_header_symbols_exported(header, names):
    declared = _declared(header)
    assert set(declared) == set(names)
    L = ctypes.CDLL(bgbuild.lib_path("libbi_gemm.so"))
    for name in declared:
        assert hasattr(L, name), name


@pytest.mark.parametrize("header,name", [("bi_qkrope.h", "bi_qkrope_config"), ("bi_prompt.h", "bi_prompt_config")])
def test_binding_structs_match_the_headers(header, name):
    assert [n for _, n in _structs(header)[name]] == [n for n, _ in getattr(bg, name)._fields_]
    assert all(t == "int32_t" for t, _ in _structs(header)[name])


@pytest.mark.parametrize("Hq,Hkv,D,page,rot,inter,eps,want", [
    (32, 8, 128, 16, 128, 0, -1.0, INVALID),
    (32, 8, 128, 16, 128, 0, float("nan"), INVALID),
    (32, 8, 128, 16, 128, 2, 1e-6, INVALID),
    (32, 8, 128, 0, 128, 0, 1e-6, INVALID),
    (0, 8, 128, 16, 128, 0, 1e-6, INVALID),
    (32, 8, 128, 16, 0, 0, 1e-6, INVALID),
    (32, 8, 96, 16, 96, 0, 1e-6, UNSUPPORTED),         # head dim
    (32, 8, 64, 16, 128, 0, 1e-6, UNSUPPORTED),        # rot_dim > head_dim
    (32, 8, 128, 16, 24, 0, 1e-6, UNSUPPORTED),        # rot_dim % 16
    (4000, 80, 128, 16, 128, 0, 1e-6, UNSUPPORTED),    # heads
    (32, 8, 128, (1 << 20) + 1, 128, 0, 1e-6, UNSUPPORTED),
])
def test_qkrope_create_refuses_before_touching_cuda(Hq, Hkv, D, page, rot, inter, eps, want):
    h = ctypes.c_void_p()
    assert bg.library().bi_qkrope_create(ctypes.byref(h), Hq, Hkv, D, page, rot, inter, eps) == want
    assert h.value is None


def test_qkrope_null_arguments():
    L = bg.library()
    assert L.bi_qkrope_create(None, 32, 8, 128, 16, 128, 0, 1e-6) == INVALID
    assert L.bi_qkrope_run(None, None, 1, 6144, None, None, None, 1, None, None, None, None, 1, None, 1, 1, None,
                           None) == INVALID
    assert L.bi_qkrope_get_device_error(None, None) == INVALID
    assert L.bi_qkrope_get_config(None, None) == INVALID
    assert L.bi_qkrope_destroy(None) == bg.BI_GEMM_OK


@pytest.mark.parametrize("Hq,Hkv,D,page,scale,want", [
    (32, 8, 128, 16, 0.0, INVALID),
    (32, 8, 128, 16, float("nan"), INVALID),
    (32, 8, 128, 0, 0.1, INVALID),
    (32, -8, 128, 16, 0.1, INVALID),
    (30, 8, 128, 16, 0.1, UNSUPPORTED),        # heads not a multiple
    (24, 8, 128, 16, 0.1, UNSUPPORTED),        # group of 3
    (32, 2, 128, 16, 0.1, UNSUPPORTED),        # group of 16
    (32, 8, 96, 16, 0.1, UNSUPPORTED),
    (32, 8, 128, (1 << 20) + 1, 0.1, UNSUPPORTED),
])
def test_prompt_create_refuses_before_touching_cuda(Hq, Hkv, D, page, scale, want):
    h = ctypes.c_void_p()
    assert bg.library().bi_prompt_create(ctypes.byref(h), Hq, Hkv, D, page, scale) == want
    assert h.value is None


def test_prompt_null_arguments():
    L = bg.library()
    b = ctypes.c_uint64()
    assert L.bi_prompt_create(None, 32, 8, 128, 16, 0.1) == INVALID
    assert L.bi_prompt_run(None, None, 1, None, None, 1, None, None, 1, None, 1, 0, None, None) == INVALID
    assert L.bi_prompt_workspace_size(None, 1, 1, ctypes.byref(b)) == INVALID
    assert L.bi_prompt_get_device_error(None, None) == INVALID
    assert L.bi_prompt_get_config(None, None) == INVALID
    assert L.bi_prompt_destroy(None) == bg.BI_GEMM_OK


def test_shared_attention_null_arguments():
    L = bg.library()
    b = ctypes.c_uint64()
    assert L.bi_attention_run_shared(None, None, 1, None, None, None, None, 1, None, 1, 1, 0, None, None, 1, None,
                                     None) == INVALID
    assert L.bi_attention_shared_workspace_size(None, 1, 1, 1, ctypes.byref(b)) == INVALID


def test_the_scratch_limit_names_captured_calls():
    """The prompt and shared-prefix calls return it too, and have no fixed array."""
    assert "captured" in bg.bi_gemm_strerror(bg.BI_GEMM_ERR_SCRATCH_LIMIT)


def test_controls_symbols_exported():
    declared = [n for n in _declared("bi_paged_controls.h") if n.startswith("bi_ctl_")]
    assert len(declared) == 10
    L = ctypes.CDLL(bgbuild.lib_path("libbi_gemm_controls.so"))
    for name in declared:
        assert hasattr(L, name), name
    for name in bg.PROMPT_EXPORTED_SYMBOLS + bg.QKROPE_EXPORTED_SYMBOLS:
        assert not hasattr(L, name), name
