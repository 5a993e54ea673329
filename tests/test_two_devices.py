"""Launches on a second device, on the CPU: the kernels' host code linked against a CUDA runtime of the test's own, which
keeps a kernel's shared memory limit for each device, as the real one does."""
import os
import shutil
import subprocess

import pytest

SOURCE = r"""
#include <cstdio>
#include <map>
#include <set>
#include <utility>

#include "internal.h"

static int current = 0;
static std::map<std::pair<int, const void*>, int> allowed;  // device, kernel
static int launches = 0, refused = 0;

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = current; return cudaSuccess; }
cudaError_t cudaSetDevice(int d) { current = d; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) allowed[{current, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  *n = 128 / (int)c->gridDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  ++launches;
  if (c->dynamicSmemBytes > 49152 && allowed[{current, f}] < (int)c->dynamicSmemBytes) {
    ++refused;
    return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}
cudaError_t cudaEventCreate(cudaEvent_t*) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
// what the compiler's registration code calls; nothing of it is needed
void** __cudaRegisterFatBinary(void*) { static void* p; return &p; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPopCallConfiguration(void*, void*, size_t*, void*) { return 0; }
cudaError_t __cudaGetKernel(void**, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaSuccess; }
}

static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}

using namespace dec;

int main() {
  uint8_t* at = reinterpret_cast<uint8_t*>(1 << 20);  // never read
  float* scales = reinterpret_cast<float*>(at);
  uint16_t* bf = reinterpret_cast<uint16_t*>(at);
  int bad = 0;
  for (int device : {0, 1, 5, 1, 0}) {
    current = device;
    dec_handle h;
    h.device = device;
    h.sms = 152;
    h.encode = encode;
    auto ok = [&](cudaError_t e, const char* what) {
      if (e != cudaSuccess) std::printf("device %d: %s refused\n", device, what), ++bad;
    };
    for (int m : {1, 16}) {
      const Linear8 L = {at, 7168, scales, 56, at, scales, nullptr, 0, bf, 4096, m, 4096, 7168};
      ok(launch_stream8_linear(&h, L, nullptr), "streaming product");
    }
    for (int n : {300, 4096, 7168, 12288})
      for (int m : {17, 64, 300, 4096}) {
        const Linear8 L = {at, 7168, scales, 56, at, scales, nullptr, 0, bf, n, m, n, 7168};
        ok(launch_gemm8(&h, L, at, nullptr), "tcgen05 product on 8 bits");
      }
    for (int m : {1, 8, 64}) {
      Experts8 X = {};
      X.x = at, X.ldx = 2048, X.xs = scales, X.ldxs = 16;
      X.M = m, X.k = 4, X.E = 16, X.H = 2048, X.I = 512;
      X.gate = X.down = {{at, at}, {scales, scales}};
      ok(launch_experts8(&h, X, experts8_plan(m, 4, 16, 2048, 512, false), reinterpret_cast<int*>(at), scales, scales,
                         nullptr), "experts");
    }
    for (int epi : {EPI_LINEAR, EPI_SWIGLU, EPI_F32})
      for (int rows : {16, 32, 64}) {
        EngineLaunch E;
        E.epi = epi, E.A = E.A2 = bf, E.a_rows = 512, E.B = bf, E.b_rows = rows, E.ldb = E.K = 1024, E.N = 512;
        E.count = rows, E.out = at, E.ldo = 512, E.partials = scales, E.counters = reinterpret_cast<int*>(at);
        ok(launch_engine(&h, E, nullptr), "tcgen05 product on 16 bits");
      }
    if (current != device) std::printf("device %d became %d\n", device, current), ++bad;
  }
  std::printf("%d launches, %d refused\n", launches, refused);
  return bad != 0 || launches < 100;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_every_device_allows_the_kernels_shared_memory(tmp_path):
    import moe_layers_gb300 as ML
    from moe_layers_gb300 import _build
    ML.build()
    (tmp_path / "main.cpp").write_text(SOURCE)
    objects = [os.path.join(_build.BUILD, f) for f in ("gemm8.o", "stream8.o", "umma.o")]
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    made = subprocess.run(["g++", "-std=c++17", "-I", cuda, "-I", _build.CSRC, str(tmp_path / "main.cpp"), *objects, "-o",
                           str(tmp_path / "prog")], capture_output=True, text=True)
    assert made.returncode == 0, made.stderr
    ran = subprocess.run([str(tmp_path / "prog")], capture_output=True, text=True, timeout=60)
    assert ran.returncode == 0, ran.stdout
