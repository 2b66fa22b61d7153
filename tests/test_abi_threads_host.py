"""The C ABI may be called from several threads: what the host side remembers of
a device (its SMs, the CTAs of a kernel, that a kernel's shared memory was
raised) is shared between them.  The helpers of csrc/abi_host.cuh in a host
program with the thread sanitizer and stand-ins for the runtime's calls."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

PROGRAM = r"""
#include <thread>
#include <vector>
#include <cuda_runtime.h>
template <typename T> cudaError_t cudaFuncSetAttribute(T *, cudaFuncAttribute, int) { return cudaSuccess; }
#include "abi_host.cuh"
thread_local std::string ssm_host::g_last_error;
static thread_local int current = 0;
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = current; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int dev) { *v = 100 + dev; return cudaSuccess; }
const char *cudaGetErrorString(cudaError_t) { return ""; }
}
static void kernel(int) {}
int main() {
  std::vector<std::thread> t;
  bool ok[8];
  for (int k = 0; k < 8; ++k)
    t.emplace_back([k, &ok] {
      ok[k] = true;
      for (int n = 0; n < 1000; ++n) {
        current = (k + n) % 4;
        ok[k] = ok[k] && ssm_host::device_sms() == 100 + current &&
                ssm_host::ensure_smem<kernel>(1 << 16, "kernel") == SSM_OK;
      }
    });
  for (auto &x : t) x.join();
  for (bool o : ok)
    if (!o) return 3;
  return 0;
}
"""


def test_device_facts_are_shared_without_a_race(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(CUDA, "include", "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    flags = ["-std=c++17", "-O1", "-g", "-fsanitize=thread", "-pthread"]
    probe, src, exe = tmp_path / "probe.cc", tmp_path / "threads.cc", tmp_path / "threads"
    probe.write_text("int main() { return 0; }\n")
    if subprocess.run([cxx, *flags, str(probe), "-o", str(exe)], capture_output=True).returncode or \
            subprocess.run([str(exe)], capture_output=True).returncode:
        pytest.skip("no thread sanitizer here")
    src.write_text(PROGRAM)
    inc = [f"-I{os.path.join(ROOT, 'include')}", f"-I{CUDA}/include",
           f"-I{os.path.join(ROOT, 'selective_state_space_25_b200', 'csrc')}"]
    r = subprocess.run([cxx, *flags, *inc, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[:3000]
