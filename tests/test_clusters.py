"""The lookup of how many clusters a device runs at once, against a fake of the runtime: every kernel, launch shape and
device is asked for itself, and a failed question is neither kept nor left behind as an error."""
import os
import shutil
import subprocess

import pytest

PROGRAM = r"""
#include <cstdio>
#include "moe_clusters.cuh"

static int device = 0, asked = 0;
static bool fail_device = false, fail_query = false;
static cudaError_t last = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) {
    *d = device;
    return fail_device ? last = cudaErrorNoDevice : cudaSuccess;
}
extern "C" cudaError_t cudaGetLastError(void) {
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
extern "C" cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* kernel, const cudaLaunchConfig_t* c) {
    ++asked;
    if (fail_query) return last = cudaErrorInvalidConfiguration;
    *n = (int)(long long)kernel * 1000 + device * 100 + (int)c->attrs[0].val.clusterDim.x + (c->blockDim.x > 500 ? 10 : 0) +
         (c->dynamicSmemBytes > 1000 ? 20 : 0);
    return cudaSuccess;
}
#define CHECK(x) if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main() {
    const void *a = (const void*)1, *b = (const void*)2;
    using moe::active_clusters;
    CHECK(active_clusters(a, 100, 100, 4) == 1004 && asked == 1);
    CHECK(active_clusters(a, 100, 100, 4) == 1004 && asked == 1);
    CHECK(active_clusters(b, 100, 100, 4) == 2004 && asked == 2);  // another kernel
    CHECK(active_clusters(a, 600, 100, 4) == 1014 && asked == 3);  // other launch shapes
    CHECK(active_clusters(a, 100, 2000, 4) == 1024 && asked == 4);
    CHECK(active_clusters(a, 100, 100, 8) == 1008 && asked == 5);
    device = 3;
    CHECK(active_clusters(a, 100, 100, 4) == 1304 && asked == 6);
    fail_query = true;
    CHECK(active_clusters(b, 100, 100, 8) == 0 && last == cudaSuccess);
    CHECK(active_clusters(a, 100, 100, 4) == 1304);                // what is known stays known
    fail_query = false;
    CHECK(active_clusters(b, 100, 100, 8) == 2308);                // asked again
    fail_device = true;
    CHECK(active_clusters(a, 100, 100, 4) == 0 && last == cudaSuccess);
    return 0;
}
"""


def test_lookup(tmp_path):
    from combine_moe_layout_04_gb300 import _build
    include = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    if shutil.which("g++") is None or not os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "clusters.cpp", tmp_path / "clusters"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", include, "-I", _build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
