// abi_host.cuh -- host helpers shared by the C ABI's source files: the error
// message, argument checks, launches.
#pragma once

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <string>

#include <cuda_runtime.h>

#include "ssmscan.h"

namespace ssm_host {

extern thread_local std::string g_last_error;  // defined in ssmscan.cu

#ifdef SSM_DEBUG_BOUNDS
// Reads and clears the bounds word of block_ops.cu's kernels.
cudaError_t take_block_bounds_word(unsigned int *word);
#endif

inline ssm_status fail(ssm_status s, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline ssm_status ok() { return SSM_OK; }

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

inline bool supported_state(int64_t n) {
  return n == 1 || n == 2 || n == 4 || n == 8 || n == 16 || n == 32 || n == 64;
}

inline size_t esize(ssm_dtype t) { return t == SSM_BF16 ? 2 : 4; }

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A named byte range of one argument; NULL or empty ranges overlap nothing.
struct Span {
  const char *name;
  const void *p;
  int64_t bytes;
};

inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// Outputs (and in-place buffers) must not overlap an input or each other.
// same_out / same_in name one output allowed to be exactly the given input
// (the same address: h_last == h0); any other overlap is an error.
inline ssm_status check_disjoint(const char *what, std::initializer_list<Span> outs,
                                 std::initializer_list<Span> ins, const void *same_out = nullptr,
                                 const void *same_in = nullptr) {
  for (const Span &o : outs) {
    for (const Span &i : ins) {
      if (same_out && o.p == same_out && i.p == same_in && o.p == i.p && o.bytes == i.bytes) continue;
      if (overlap(o, i))
        return fail(SSM_ERR_INVALID_ARG, "%s: %s overlaps the input %s", what, o.name, i.name);
    }
    for (const Span &o2 : outs)
      if (&o2 != &o && overlap(o, o2))
        return fail(SSM_ERR_INVALID_ARG, "%s: outputs %s and %s overlap", what, o.name, o2.name);
  }
  return SSM_OK;
}

inline ssm_status check_launch(const char *what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SSM_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
  return ok();
}

// Launch with programmatic stream serialization: the kernel may start once
// every block of the previous kernel in the stream has called
// grid_dependents_launch (or exited), and calls grid_dependency_wait before
// it reads that kernel's results.
template <typename... KArgs, typename... Args>
ssm_status launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 threads, int smem,
                            cudaStream_t st, const char *what, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(SSM_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
  }
  return ok();
}

// A number above 0 for each device, found on its first use.  Any thread may ask at
// any time; two that find it at once find the same.
class PerDevice {
 public:
  // find(device) for the current device; `none` where there is none
  template <typename F> int get(F &&find, int none) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) {
      cudaGetLastError();
      return none;
    }
    int v = v_[dev].load(std::memory_order_relaxed);
    if (!v) v_[dev].store(v = find(dev), std::memory_order_relaxed);
    return v;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> v_[kDevices] = {};
};

// Opt a kernel into > 48 KB of dynamic shared memory once per device.
template <auto Kernel>
ssm_status ensure_smem(int bytes, const char *what) {
  static std::atomic<bool> done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return fail(SSM_ERR_CUDA, "%s: cudaGetDevice failed", what);
  if (!done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess)
      return fail(SSM_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", what, cudaGetErrorString(e));
    done[dev].store(true, std::memory_order_release);
  }
  return ok();
}

// SMs of the current device (148 on B200; also the answer when no device is
// visible, so the workspace query works on a host without a GPU).
inline int device_sms() {
  static PerDevice sms;
  return sms.get(
      [](int dev) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
          cudaGetLastError();
          n = 148;
        }
        return n;
      },
      148);
}

inline unsigned grid_for(int64_t n) {
  const int64_t blocks = (n + 255) / 256;
  return (unsigned)(blocks < 148 * 32 ? (blocks > 0 ? blocks : 1) : 148 * 32);
}

}  // namespace ssm_host
