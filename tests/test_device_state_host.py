"""What a kernel's attributes are kept by: the device.  The header's helpers are compiled against a stand-in for the
CUDA calls they make, which plays several devices (no GPU needed)."""

import os
import shutil
import subprocess

import pytest

from gemma_dual_geometry_gb300 import build as g4build

MAIN = r"""
#include <cuda_runtime.h>
#include <stdio.h>

// The runtime header's form for functions, which it has for CUDA compilers only.
template <typename F>
cudaError_t cudaFuncSetAttribute(F* f, cudaFuncAttribute a, int v) {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(f), a, v);
}

#include "g4_internal.h"

// Device d: `raised` and `wide` are the attributes set while it was current.
static int current = 0;
static int raised[4], wide[4], sets[4], asks[4];
static size_t asked_smem;
static void kern() {}
static void other() {}

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = current; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, enum cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) raised[current] = v;
  if (a == cudaFuncAttributeNonPortableClusterSizeAllowed) {
    ++sets[current];
    if (current == 2) return cudaErrorNotSupported;
    wide[current] = v;
  }
  return cudaSuccess;
}
// device 1 has room for clusters of 16 with little shared memory only; device 3 for none
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  ++asks[current];
  asked_smem = c->dynamicSmemBytes;
  if (!wide[current] || raised[current] < static_cast<int>(asked_smem)) return cudaErrorInvalidClusterSize;
  *n = current == 0 || (current == 1 && asked_smem < 60000) ? 4 : 0;
  return c->numAttrs == 1 && c->attrs[0].val.clusterDim.x == 16 ? cudaSuccess : cudaErrorInvalidValue;
}
}

int main() {
  for (int turn = 0; turn < 2; ++turn)
    for (int d = 0; d < 4; ++d) {
      current = d;
      if (g4::set_smem_limit_once<kern>(100000) != cudaSuccess) return 1;
      printf("%u ", g4::cluster_limit_once<kern>(1024, 70000));
    }
  current = 1;
  (void)g4::set_smem_limit_once<other>(100000);
  printf("%u ", g4::cluster_limit_once<other>(1024, 50000));
  printf("sets %d %d %d %d asks %d %d %d %d smem %d", sets[0], sets[1], sets[2], sets[3], asks[0], asks[1], asks[2],
         asks[3], static_cast<int>(asked_smem));
  return 0;
}
"""


def test_cluster_limits_belong_to_devices(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs a C++ compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(g4build.nvcc_path()))), "include")
    src, exe = tmp_path / "devices.cpp", tmp_path / "devices"
    src.write_text(MAIN)
    subprocess.run([cxx, "-std=c++17", "-I", g4build.CSRC, "-I", include, str(src), "-o", str(exe), "-pthread"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out[:8] == ["16", "8", "8", "8"] * 2     # each device's own answer, whatever came first
    assert out[8] == "16"                           # and each kernel's
    # opted in and asked once per device and kernel (not asked where the opt-in fails), with the launch's shared memory
    assert " ".join(out[9:]) == "sets 1 2 1 1 asks 1 2 0 1 smem 50000"


def test_the_assignments_clusters_go_by_the_device():
    """No launch opts in by itself, past the helper that does so per device."""
    for name in g4build.SOURCES:
        text = open(os.path.join(g4build.CSRC, name)).read()
        assert "cudaFuncAttributeNonPortableClusterSizeAllowed" not in text, name
