"""Rules on the kernels' sources that no run shows."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_03_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_tma_load_is_a_multicast(name):
    # the kernels run as replicas on several GPUs too, where a load into several CTAs may not be used
    # (a commit that signals both CTAs of a pair is no load)
    with open(os.path.join(CSRC, name)) as f:
        for line in f:
            assert not ("cp.async.bulk" in line and "multicast::cluster" in line), line


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_attribute_of_a_device_is_remembered_for_the_process(name):
    with open(os.path.join(CSRC, name)) as f:
        assert "static bool" not in f.read()


HARNESS = r"""
#include <cstdio>
#include "per_device.h"
static int device, sets;
static cudaError_t get_result, set_result;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return get_result; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute a, int bytes) {
    if (a != cudaFuncAttributeMaxDynamicSharedMemorySize || bytes != 200000) return cudaErrorInvalidValue;
    sets++;
    return set_result;
}
int main() {
    bsq::SharedMemory m, other;
    const auto go = [](bsq::SharedMemory& s, int d) { device = d; sets = 0; const int e = s.allow(&device, 200000); printf("%d:%d ", sets, e); };
    go(m, 0); go(m, 0); go(m, 1); go(m, 1); go(m, 0); go(m, 63); go(m, 63); go(m, 64); go(m, 64); go(other, 0);
    set_result = cudaErrorInvalidValue; go(m, 2);
    set_result = cudaSuccess; go(m, 2); go(m, 2);
    get_result = cudaErrorNoDevice; go(m, 3);
}
"""


def test_shared_memory_is_allowed_once_on_every_device(tmp_path):
    # cudaGetDevice and cudaFuncSetAttribute are stand-ins here: no GPU, 65 devices
    from block_scaled_precision_03_gb300._build import nvcc
    src, exe = tmp_path / "harness.cpp", tmp_path / "harness"
    src.write_text(HARNESS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-I", cuda, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    # attributes set : result, of every call
    assert out == ["1:0", "0:0", "1:0", "0:0", "0:0", "1:0", "0:0", "1:0", "1:0", "1:0", "1:1", "1:0", "0:0", "0:100"]
