"""The waits of the attention kernels' warps, alone: a barrier in shared memory
that nobody arrives at is given up after the polls asked for, the block's other
warps give up after one, and the warps that share a barrier learn of it
together.  Nothing is under way in these blocks."""
import ctypes
import importlib.util
import os
import subprocess
import time

import pytest
import torch

import paged_kv_cache_group_b200 as fp8q

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "fp4_async.cuh"
using namespace fp8q;

// Warp 0 of four waits for a phase.  out[w]: what warp w was told after they had
// agreed; out[4 + w]: what they agreed on; out[8]: the error word; out[9]: the
// block's flag.
__global__ void probe(uint32_t *out, uint32_t *error, int arrivals, int tries) {
    __shared__ alignas(8) uint64_t bar;
    __shared__ uint32_t gave_up;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        barrier_init(smem_addr(&bar), 1);
        gave_up = 0;
    }
    __syncthreads();
    if (threadIdx.x == 32 && arrivals) barrier_arrive(smem_addr(&bar));
    if (warp == 0) barrier_wait(smem_addr(&bar), 0, &gave_up, error, tries);
    const bool all = agree(1, 128, warp == 0 ? told(&gave_up) : true);
    if (warp != 0) barrier_wait(smem_addr(&bar), 0, &gave_up, error);   // one poll if warp 0 has given up
    const bool mine = told(&gave_up);
    if (lane == 0) out[warp] = mine, out[4 + warp] = all;
    __syncthreads();
    if (threadIdx.x == 0) out[8] = *error, out[9] = gave_up;
    let_land(&gave_up);
}

extern "C" __attribute__((visibility("default"))) int run(uint32_t *out, uint32_t *error, int arrivals, int tries, void *stream) {
    probe<<<1, 128, 0, static_cast<cudaStream_t>(stream)>>>(out, error, arrivals, tries);
    return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    path = os.path.join(root, "paged_kv_cache_group_b200", "build.py")
    spec = importlib.util.spec_from_file_location("_fp8q_build", path)
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    folder = tmp_path_factory.mktemp("waits")
    source, lib = folder / "waits.cu", folder / "libwaits.so"
    source.write_text(SOURCE)
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-shared",
                    "-o", str(lib), str(source)], check=True)
    fn = ctypes.CDLL(str(lib)).run
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def call(arrivals, tries):
        out = torch.full((16,), 9, dtype=torch.int32, device="cuda")
        error = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        since = time.monotonic()
        assert fn(out.data_ptr(), error.data_ptr(), arrivals, tries, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return out.tolist(), time.monotonic() - since

    return call


def test_a_wait_that_ends(probe):
    out, _ = probe(1, 1000)
    assert out[:10] == [1, 1, 1, 1, 1, 1, 1, 1, 0, 0]


@pytest.mark.parametrize("tries", [0, 1, 4, 50])
def test_a_wait_that_runs_out(probe, tries):
    out, seconds = probe(0, tries)
    assert out[:10] == [0] * 8 + [fp8q.DEVERR_WAIT, 1]
    assert seconds < 1.0                           # 50 polls of up to 2 us, at the end 1 ms
