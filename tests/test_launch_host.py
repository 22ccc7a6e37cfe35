"""The launchers' host code against fakes of the CUDA calls it makes."""

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "indexer_projection_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "pa_launch.h"
static int device = 0, calls = 0;
static cudaError_t result = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { ++calls; return result; }
extern "C" cudaError_t cudaDeviceGetAttribute(int *, cudaDeviceAttr, int) { return cudaErrorUnknown; }
static char kernels[100];
int main() {
  for (int turn = 0; turn < 2; ++turn)  // 100 kernels on each of 8 devices: set once
    for (device = 0; device < 8; ++device)
      for (char &k : kernels)
        if (pa::ensure_smem_attr(&k, 65536) != cudaSuccess) return 1;
  printf("%d\n", calls);
  calls = 0, device = 3;
  pa::ensure_smem_attr(kernels, 1024);    // held already
  pa::ensure_smem_attr(kernels, 100000);  // more than is held
  pa::ensure_smem_attr(kernels, 100000);
  pa::ensure_smem_attr(kernels, 65536);
  printf("%d\n", calls);
  calls = 0, result = cudaErrorInvalidValue;  // a refusal is not remembered
  if (pa::ensure_smem_attr(kernels, 200000) != result || pa::ensure_smem_attr(kernels, 200000) != result) return 1;
  printf("%d\n", calls);
}
"""


def test_the_shared_memory_attribute_is_set_once_a_kernel_and_device(tmp_path):
    from indexer_projection_gb300 import build

    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split()
    assert out == ["800", "1", "2"]
