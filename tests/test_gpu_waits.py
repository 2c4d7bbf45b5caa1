"""The operators' bounded waits: what a wait that runs out leaves, and that ordinary calls leave nothing."""
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

# One warp waits on a barrier that nothing arrives on: the wait gives up after kWaitClocks (a second or two),
# marks the block and latches the word; a second wait returns at once, and the kernel ends in the ordinary way.
# Then the same kernel with the arrival.
PROGRAM = r"""
#include <cstdio>
#include "hs_tc.h"

__global__ void wait_for(int arrive, int* error, int* marked, long long* clocks)
{
    __shared__ uint64_t bar;
    __shared__ int dead;
    const uint32_t at = tc::smem_addr(&bar);
    if (threadIdx.x == 0) {
        dead = 0;
        tc::mbar_init(at, 1);
        tc::mbar_init_fence();
    }
    __syncthreads();
    if (arrive && threadIdx.x == 0) tc::mbar_arrive(at);
    const long long t0 = clock64();
    tc::wait(at, 0, &dead, error);
    const long long t1 = clock64();
    tc::wait(at, 0, &dead, error);
    const long long t2 = clock64();
    __syncthreads();
    if (threadIdx.x == 0) *marked = dead, clocks[0] = t1 - t0, clocks[1] = t2 - t1;
}

int main()
{
    struct Out { int error, marked; long long clocks[2]; } *o;
    if (cudaMallocManaged(&o, sizeof *o) != cudaSuccess) return 2;
    for (int arrive = 0; arrive < 2; ++arrive) {
        *o = Out{};
        wait_for<<<1, 32>>>(arrive, &o->error, &o->marked, o->clocks);
        const cudaError_t e = cudaDeviceSynchronize();
        printf("%d %d %d %lld %lld %lld\n", (int)e, o->error, o->marked, o->clocks[0], o->clocks[1], (long long)tc::kWaitClocks);
    }
    return 0;
}
"""


def test_wait_that_runs_out_is_latched(tmp_path):
    from hierarchical_kv_cache_hs_gb300 import build
    src, exe = tmp_path / "wait.cu", tmp_path / "wait"
    src.write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    ran_out, came = ([int(x) for x in line.split()] for line in r.stdout.splitlines())
    assert ran_out[:3] == [0, 1, 1] and ran_out[3] >= ran_out[5] > 100 * ran_out[4]
    assert came[:3] == [0, 0, 0] and came[3] < came[5] // 100


@pytest.mark.parametrize("word", [0, 7])
def test_calls_leave_the_error_word(word):
    from hierarchical_kv_cache_hs_gb300 import hs
    bf = torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(bf)

    def workspace(n):
        space = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        hs.hs_workspace_clear(space)
        space[:4].view(torch.int32).fill_(word)
        return space

    length = torch.tensor([3000, 5], dtype=torch.int32, device="cuda")
    rows8 = torch.zeros((2, 3000, 592), dtype=torch.uint8, device="cuda")
    for heads, rows, form in ((64, randn(2, 3000, 576), hs.HS_ROWS_16BIT), (16, rows8, hs.HS_ROWS_E4M3),
                              (64, rows8, hs.HS_ROWS_E4M3)):
        out = torch.empty((2, 1, heads, 512), dtype=bf, device="cuda")
        space = workspace(hs.hs_latent_attend_workspace(2, 1, heads, 3000))
        hs.hs_latent_attend(randn(2, 1, heads, 576), rows, out, 0.1, lengths=length, row_format=form, workspace=space)
        assert hs.hs_workspace_error(space) == word
    start = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")
    out = torch.empty((2000, 4, 128), dtype=bf, device="cuda")
    space = workspace(hs.hs_latent_prefill_workspace(2000, 4))
    hs.hs_latent_prefill(randn(2000, 4, 192), randn(2000, 576), randn(4, 128, 512), randn(4, 128, 512), start, start, out,
                         0.1, workspace=space)
    assert hs.hs_workspace_error(space) == word
