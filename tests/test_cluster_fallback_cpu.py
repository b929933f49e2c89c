"""Router losses where the device cannot place the cluster that they ask for: the launcher's host code with a runtime that
knows clusters up to a given size, on the CPU."""
import os
import subprocess

import pytest

from routed_grouped_gemm_dispatch_gb300 import _build

# The runtime: refuses what the device cannot place, and prints the grid, the cluster and the shared memory of a launch.
RUNTIME = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cuda_runtime.h>

#include "train_internal.h"

static unsigned largest;
static unsigned cluster_of(const cudaLaunchConfig_t* c) {
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
    return 1;
}
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
    *n = 0;
    if (cluster_of(c) > largest) return cudaErrorInvalidClusterSize;
    *n = 1;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
    if (cluster_of(c) > largest) return cudaErrorInvalidClusterSize;
    std::printf("%u %u %zu\n", c->gridDim.x, cluster_of(c), c->dynamicSmemBytes);
    return cudaSuccess;
}
cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaErrorUnknown; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorUnknown; }
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, CUstream_st*) { return 1; }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
char __cudaInitModule(void**) { return 0; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
}

int main(int, char** argv) {
    largest = static_cast<unsigned>(std::atoi(argv[1]));
    moe::RouterBalance a{};
    a.r.n_tokens = std::atoll(argv[2]);
    a.r.n_experts = std::atoi(argv[3]);
    a.r.top_k = 1;
    a.r.n_seqs = std::atoi(argv[4]);
    return launch_router_balance(a, nullptr);
}
"""


@pytest.fixture(scope="module")
def launcher(tmp_path_factory):
    d = tmp_path_factory.mktemp("cluster")
    (d / "runtime.cpp").write_text(RUNTIME)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    for cmd in ([_build.nvcc(), *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-Xcicc", "-O0", "-Xptxas", "-O0", "-I",
                 _build.INCLUDE, "-c", os.path.join(_build.CSRC, "router_loss.cu"), "-o", d / "loss.o"],
                ["g++", "-std=c++17", "-I", cuda, "-I", _build.CSRC, d / "runtime.cpp", d / "loss.o", "-o", d / "launch"]):
        r = subprocess.run([str(c) for c in cmd], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]

    def run(*args):
        r = subprocess.run([str(d / "launch"), *map(str, args)], capture_output=True, text=True)
        return r.returncode, [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    return run


# tokens, experts, sequences
CASES = [(4097, 64, 5), (64, 128, 16), (1500, 1000, 1), (700, 129, 9), (8000, 60, 1), (0, 64, 32)]


@pytest.mark.parametrize("tokens,experts,seqs", CASES)
def test_clusters_as_large_as_can_be_placed(launcher, tokens, experts, seqs):
    """One launch of the cluster that is wanted or of the largest that there is room for, or two launches without any."""
    err, wanted = launcher(16, tokens, experts, seqs)
    assert err == 0 and (len(wanted) == 1 or [w[1] for w in wanted] == [1, 1])
    grid, cluster, shared = wanted[0]
    if len(wanted) == 1:
        assert grid == cluster and cluster >= 8
    for largest in (8, 4, 2, 1):
        err, got = launcher(largest, tokens, experts, seqs)
        assert err == 0
        assert got == (wanted if len(wanted) == 2 else [(min(largest, cluster), min(largest, cluster), shared)])


def test_small_clusters_are_what_they_are(launcher):
    err, want = launcher(16, 300, 64, 1)
    assert err == 0 and want[0][0] < 8 and launcher(8, 300, 64, 1) == (0, want)
