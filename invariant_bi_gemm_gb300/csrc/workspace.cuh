// workspace.cuh — device scratch of the handles, on the host: how it grows in stream order, and how it is given back
// behind the calls that use it.
#pragma once
#include <cstddef>
#include <cuda_runtime_api.h>
#include <vector>

#include "../../include/bi_gemm.h"

namespace bigemm {

// Gives a handle's memory back (`free_all`) behind everything that its device has queued: cudaFree does not wait for
// the users of memory that came from cudaMallocAsync, and a handle may be dropped right behind its last call, with
// any device current.  Where the device cannot be waited for the memory stays: better lost than freed under a kernel.
template <class F>
void behind(int device, F&& free_all) {
  int current = device;
  if (cudaGetDevice(&current) == cudaSuccess && (current == device || cudaSetDevice(device) == cudaSuccess) &&
      cudaDeviceSynchronize() == cudaSuccess)
    free_all();
  if (current != device) cudaSetDevice(current);
  cudaGetLastError();
}

}  // namespace bigemm

namespace biattn_tc {

// A handle's device scratch, grown in stream order.  A block that a captured call uses lives until the
// handle does, since the graph may still be replayed; any other is freed behind the calls that used it.
struct Workspace {
  // growth doubles up to this step, so that a bound that climbs with every call does not move the
  // scratch at each, and no handle holds more than this beyond what a call has asked for
  static constexpr size_t kStep = size_t(64) << 20;
  void* at = nullptr;
  size_t bytes = 0;
  bool captured = false;        // a captured call uses `at`
  std::vector<void*> earlier;

  // A call being captured cannot allocate for good: it uses what earlier calls left.
  int need(size_t n, cudaStream_t st) {
    if (n == 0) return BI_GEMM_OK;
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &capturing) != cudaSuccess) {
      cudaGetLastError();
      return BI_GEMM_ERR_CUDA;
    }
    if (n <= bytes) {
      captured |= capturing != cudaStreamCaptureStatusNone;
      return BI_GEMM_OK;
    }
    if (capturing != cudaStreamCaptureStatusNone) return BI_GEMM_ERR_SCRATCH_LIMIT;
    try {
      if (captured) earlier.reserve(earlier.size() + 1);
    } catch (...) {
      return BI_GEMM_ERR_OOM;
    }
    const size_t step = bytes + (bytes < kStep ? bytes : kStep);
    size_t size = n > step ? n : step;
    void* p = allocate(size, st);
    if (!p && size > n) p = allocate(size = n, st);
    if (!p && at && !captured) {          // the block that it replaces may be the room it needs
      cudaFreeAsync(at, st);
      at = nullptr;
      bytes = 0;
      p = allocate(size, st);
    }
    if (!p) return BI_GEMM_ERR_OOM;
    if (captured) earlier.push_back(at);
    else if (at) cudaFreeAsync(at, st);
    at = p;
    bytes = size;
    captured = false;
    return BI_GEMM_OK;
  }
  void release(int device) {
    if (at || !earlier.empty())
      bigemm::behind(device, [this] {
        if (at) cudaFree(at);
        for (void* p : earlier) cudaFree(p);
      });
    at = nullptr;
    bytes = 0;
    captured = false;
    earlier.clear();
  }
  static void* allocate(size_t n, cudaStream_t st) {
    void* p = nullptr;
    if (cudaMallocAsync(&p, n, st) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    return p;
  }
};

}  // namespace biattn_tc
