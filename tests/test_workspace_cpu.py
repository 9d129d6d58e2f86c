"""How handles give their device memory back, without a GPU: csrc/workspace.cuh compiled against a CUDA runtime that
only keeps a record of its calls."""
import ctypes
import os
import subprocess

import pytest

from invariant_bi_gemm_gb300 import build as bgbuild

FAKE = r"""
#include <cstdio>
#include <string>
#include "workspace.cuh"

static std::string record;
static int device = 0, synced = -1, next_block = 0, failing = 0;
static void note(const char* what, long n) { record += what + std::to_string(n) + " "; }

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaSetDevice(int d) {
  if (failing == 2 && d) return cudaErrorInvalidDevice;
  device = d;
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() {
  if (failing == 1) return cudaErrorLaunchFailure;
  note("wait", device);
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) { note("free", long(size_t(p))); return cudaSuccess; }
cudaError_t cudaFreeAsync(void* p, cudaStream_t) { note("later", long(size_t(p))); return cudaSuccess; }
cudaError_t cudaMallocAsync(void** p, size_t, cudaStream_t) { *p = (void*)size_t(++next_block); return cudaSuccess; }
static cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { *s = capturing; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }

// A handle of device `owner` makes `calls` calls, each larger than the last and with a captured one behind it, and is
// released while `current` is current.  Returns the record of the release and, behind a bar, the device left current.
const char* released(int owner, int current, int calls, int fail) {
  record.clear();
  device = owner, next_block = 0, failing = 0;
  biattn_tc::Workspace ws;
  for (int i = 0; i < calls; ++i) {
    ws.need(size_t(1000) << (2 * i), nullptr);
    capturing = cudaStreamCaptureStatusActive;
    ws.need(1000, nullptr);
    capturing = cudaStreamCaptureStatusNone;
  }
  record.clear();
  device = current, failing = fail;
  ws.release(owner);
  record += "| " + std::to_string(device);
  return record.c_str();
}
}
"""


@pytest.fixture(scope="module")
def released(tmp_path_factory):
    out = tmp_path_factory.mktemp("workspace")
    (out / "fake.cpp").write_text(FAKE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(bgbuild.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", bgbuild.CSRC, "-I", cuda,
                    str(out / "fake.cpp"), "-o", str(out / "fake.so")], check=True)
    f = ctypes.CDLL(str(out / "fake.so")).released
    f.restype = ctypes.c_char_p
    return lambda *a: f(*a).decode()


@pytest.mark.parametrize("owner,current", [(0, 0), (1, 1), (1, 0), (0, 1)])
def test_memory_goes_back_behind_its_own_device(released, owner, current):
    """The handle's device is waited for, whichever is current, before anything is freed, and the current one stays."""
    assert released(owner, current, 1, 0) == f"wait{owner} free1 | {current}"
    assert released(owner, current, 3, 0) == f"wait{owner} free3 free1 free2 | {current}"


def test_a_handle_without_memory_waits_for_nothing(released):
    assert released(1, 0, 0, 0) == "| 0"


@pytest.mark.parametrize("fail", [1, 2])
def test_memory_stays_where_its_device_cannot_be_waited_for(released, fail):
    assert released(1, 0, 2, fail) == "| 0"
