"""A launch that fails leaves no error behind in the CUDA runtime, where a later call that asks
for the last error would take it for its own.  Checked on the CPU, against stand-ins for the
runtime's calls that fail when told to."""
import subprocess

from hyper_connection_mix_gb300 import build as hbuild

PROGRAM = r"""
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdio>
#include <string>

// the runtime's calls that a launch makes, each of which can be told to fail
static cudaError_t last = cudaSuccess;
static const char* failing = "";
static cudaError_t fake(const char* name) {
  if (std::string(name) != failing) return cudaSuccess;
  return last = cudaErrorInvalidValue;
}
#define cudaFuncSetAttribute(f, attr, value) fake(#attr)
#define cudaLaunchKernelEx(cfg, f, args) fake("launch")
#define cudaGetLastError() (last = cudaSuccess)
#include "hcmix_experts.cuh"
using namespace hcmix::sublayer;

struct Args {};
__global__ void kernel(const Args) {}

static int fails(const char* call, hcmix_status (*run)()) {
  failing = call, last = cudaSuccess;
  const hcmix_status st = run();
  std::printf("%s fails: status %d, left %d\n", call, (int)st, (int)last);
  return st != HCMIX_ERR_CUDA || last != cudaSuccess;
}

static hcmix_status launch_much() {
  return launch(kernel, dim3(1), dim3(32), 64 * 1024, 64 * 1024, nullptr, Args{});
}
static hcmix_status sort_many() {
  return launch_sort<int32_t>(SortArgs{nullptr, 100000, 128, nullptr, nullptr, nullptr}, nullptr);
}

int main() {
  int bad = launch_much() + sort_many();  // nothing fails yet
  bad += fails("launch", launch_much);
  bad += fails("cudaFuncAttributeMaxDynamicSharedMemorySize", launch_much);
  bad += fails("cudaFuncAttributeNonPortableClusterSizeAllowed", sort_many);
  return bad;
}
"""


def test_failed_launches_leave_no_error(tmp_path):
    source, program = tmp_path / "launch.cu", tmp_path / "launch"
    source.write_text(PROGRAM)
    subprocess.run([hbuild.nvcc(), *hbuild.ARCH, "-std=c++17", "-I", hbuild.INCLUDE, "-I", hbuild.CSRC,
                    "-o", str(program), str(source)], check=True)
    run = subprocess.run([str(program)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
