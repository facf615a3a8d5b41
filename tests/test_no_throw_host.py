"""No C++ exception leaves the host helpers that the C entry points use: with every allocation failing they return an
error (or no answer).  Host code against a stand-in for the CUDA runtime.  No GPU."""

import os
import subprocess

from rotated_bit_kv_kvq_gb300 import build

SOURCE = r"""
#include <new>
#include <cstdio>
#include <cstdlib>
#include "kvq_internal.h"

static bool g_fail = false;
void* operator new(size_t n) { if (g_fail) throw std::bad_alloc(); return std::malloc(n); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

// the runtime's functions that the helpers call
extern "C" cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }
extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) { *n = 7; return cudaSuccess; }
extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) { return cudaSuccess; }

int main() {
  int a, b;  // two addresses
  g_fail = true;
  std::printf("%d %d %d\n", int(kvq::ensure_dynamic_smem(&a, 1000)), int(kvq::allow_large_clusters(&a)),
              kvq::cluster_limits(&a, 256, 1000) == nullptr);
  g_fail = false;
  const kvq::ClusterLimits* l = kvq::cluster_limits(&b, 256, 1000);
  std::printf("%d %d %d\n", int(kvq::ensure_dynamic_smem(&b, 1000)), int(kvq::allow_large_clusters(&b)), l ? l->clusters[2] : -1);
}
"""


def test_failing_allocations_become_errors(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(SOURCE)
    cuda = os.path.dirname(os.path.dirname(build.nvcc()))
    r = subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC, "-I",
                        os.path.join(cuda, "include"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["2", "2", "1", "0", "0", "7"]  # 2: cudaErrorMemoryAllocation
