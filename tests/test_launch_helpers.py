"""Kernel attributes are set once per device, for every device ordinal: the launch helper, compiled with g++ against a
runtime that only counts, must set them again on a device whose ordinal shares its low bits with another's."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_decoding_saga_b200", "csrc")

RUNTIME = r"""
#pragma once
#include <cstddef>
#include <cstdint>
typedef int cudaError_t;
typedef void* cudaStream_t;
constexpr cudaError_t cudaSuccess = 0;
struct dim3 { unsigned x, y, z; };
enum { cudaFuncAttributeMaxDynamicSharedMemorySize, cudaFuncAttributePreferredSharedMemoryCarveout };
enum { cudaSharedmemCarveoutMaxShared = 100 };
enum { cudaLaunchAttributeProgrammaticStreamSerialization };
struct cudaLaunchAttribute { int id; struct { int programmaticStreamSerializationAllowed; } val; };
struct cudaLaunchConfig_t { dim3 gridDim, blockDim; size_t dynamicSmemBytes; cudaStream_t stream; cudaLaunchAttribute* attrs; unsigned numAttrs; };
extern int device, sets;
inline cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
inline cudaError_t cudaFuncSetAttribute(const void*, int, int) { ++sets; return cudaSuccess; }
template <typename... A> cudaError_t cudaLaunchKernelEx(A&&...) { return cudaSuccess; }
"""

PROGRAM = r"""
#include <cstdio>
#include "cuda_runtime.h"
int device, sets;
#include "saga_launch.cuh"
int main() {
  std::atomic<uint64_t> done{0};
  const int ordinals[] = {0, 0, 1, 1, 63, 64, 65, 127, 1};
  const int want[] = {2, 0, 2, 0, 2, 2, 2, 2, 0};  // two attributes where the device has not had them
  int fails = 0;
  for (int i = 0; i < 9; ++i) {
    device = ordinals[i];
    sets = 0;
    if (saga::prepare_kernel(nullptr, 1024, done) != cudaSuccess || sets != want[i]) {
      std::printf("device %d: %d attributes set, expected %d\n", device, sets, want[i]);
      ++fails;
    }
  }
  return fails;
}
"""


def test_attributes_are_set_on_every_device(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "main")
    subprocess.run(["g++", "-std=c++17", "-I" + str(tmp_path), "-I" + CSRC, str(tmp_path / "main.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_no_other_code_masks_a_device_ordinal():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            src = open(os.path.join(CSRC, name)).read()
            assert "dev & 63" not in src and "device & 63" not in src, name
            if name not in ("saga_launch.cuh", "saga_merge.cu"):
                assert "cudaFuncSetAttribute(" not in src, name
