"""The launchers' once-per-device attributes (csrc/kda_launch.h) on the host: a
program with a CUDA runtime of its own, which counts the attribute calls of each
device."""

import os
import subprocess

import pytest

from linear_attention_ssm_step_gb300 import _build

PROGRAM = r"""
#include "kda_launch.h"

static int device = 0, calls[200], fails = 0;
static int bytes_seen = 0;

extern "C" cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute a, int value) {
  if (fails > 0) {
    --fails;
    return cudaErrorInvalidValue;
  }
  ++calls[device];
  bytes_seen = a == cudaFuncAttributeMaxDynamicSharedMemorySize ? value : -1;
  return cudaSuccess;
}

static void kernel(int) {}

#define CHECK(x) if (!(x)) return __LINE__

int main() {
  static kda::DeviceFlags smem, carveout;
  for (int d : {0, 1, 63, 1, 0, 63}) {
    device = d;
    CHECK(kda::set_smem_limit_once(kernel, 200000, smem) == cudaSuccess);
  }
  CHECK(calls[0] == 1 && calls[1] == 1 && calls[63] == 1 && bytes_seen == 200000);
  device = 2;  // a failed attempt is retried, and says so
  fails = 1;
  CHECK(kda::set_smem_limit_once(kernel, 200000, smem) == cudaErrorInvalidValue && calls[2] == 0);
  CHECK(kda::set_smem_limit_once(kernel, 200000, smem) == cudaSuccess && calls[2] == 1);
  CHECK(kda::set_smem_limit_once(kernel, 200000, smem) == cudaSuccess && calls[2] == 1);
  device = 150;  // past the flags: set every time, and no other device's bit
  for (int i = 0; i < 2; ++i) CHECK(kda::set_smem_limit_once(kernel, 200000, smem) == cudaSuccess);
  CHECK(calls[150] == 2);
  device = 150 - 128;
  CHECK(kda::set_smem_limit_once(kernel, 200000, smem) == cudaSuccess && calls[device] == 1);
  for (int d : {0, 1, 0, 1}) {
    device = d;
    CHECK(kda::set_carveout_once(kernel, carveout) == cudaSuccess && calls[d] == 2);
  }
  CHECK(bytes_seen == -1);
  return 0;
}
"""


def test_attributes_are_set_once_on_each_device(tmp_path):
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build._nvcc())), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("needs the CUDA headers")
    src, exe = tmp_path / "flags.cpp", tmp_path / "flags"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE, "-I", cuda, str(src), "-o", str(exe)],
                   check=True)
    assert subprocess.run([str(exe)]).returncode == 0
