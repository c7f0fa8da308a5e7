"""The bounded wait of two CTAs that work as one: a wait that nothing satisfies
runs out, says so once, and ends the other CTA's waits too."""
import ctypes
import subprocess

import pytest
import torch

from long_context_sparse_gb300 import build as dsa_build

# Both CTAs wait, a warp and a thread each, on barriers of their own that nothing
# arrives at.  The CTA `first` gives up after short_ns, the other one after long_ns
# unless it learns of that.  out[rank]: microseconds the CTA waited, with the top
# bit set for each wait that said that its barrier was ready (none may).
SOURCE = r"""
#include "pair_common.cuh"
using namespace dsa;
__global__ void __cluster_dims__(2, 1, 1) pair_wait(uint32_t* status, uint32_t* out,
                                                    uint32_t first, uint64_t short_ns,
                                                    uint64_t long_ns) {
  __shared__ uint64_t bars[2];
  __shared__ uint32_t flag, ready;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    flag = ready = 0u;
    fence_mbar_init();
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  const PairWaiter W{&flag, at_rank(smem_u32(&flag), rank ^ 1u), status,
                     rank == first ? short_ns : long_ns};
  const uint64_t t0 = globaltimer_ns();
  if (threadIdx.x < 32) {
    if (W.wait(smem_u32(&bars[0]), 0)) atomicOr(&ready, 1u);
  } else if (threadIdx.x == 32) {
    if (W.wait1(smem_u32(&bars[1]), 0)) atomicOr(&ready, 1u);
  }
  __syncthreads();
  if (threadIdx.x == 0) out[rank] = (uint32_t)((globaltimer_ns() - t0) / 1000u) | ready << 31;
  cluster_arrive();  // neither leaves while the other may still write its flag
  cluster_wait();
}
extern "C" __attribute__((visibility("default"))) int run(void* status, void* out, uint32_t first,
                                                          uint64_t short_ns, uint64_t long_ns,
                                                          void* stream) {
  pair_wait<<<2, 64, 0, (cudaStream_t)stream>>>((uint32_t*)status, (uint32_t*)out, first,
                                                short_ns, long_ns);
  return (int)cudaGetLastError();
}
"""


def library(at):
    (at / "wait.cu").write_text(SOURCE)
    subprocess.run([dsa_build._nvcc()] + dsa_build.FLAGS +
                   ["-I", dsa_build.CSRC, "-shared", "-o", str(at / "wait.so"),
                    str(at / "wait.cu")], check=True)
    return ctypes.CDLL(str(at / "wait.so"))


def test_the_check_builds(tmp_path):
    assert library(tmp_path).run


@pytest.mark.gpu
@pytest.mark.parametrize("first", [0, 1])
def test_a_wait_of_a_pair_runs_out_in_both(tmp_path, first):
    fn = library(tmp_path).run
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64,
                   ctypes.c_uint64, ctypes.c_void_p]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert fn(status.data_ptr(), out.data_ptr(), first, 20_000_000, 2_000_000_000,
              torch.cuda.current_stream().cuda_stream) == 0
    us = out.tolist()
    assert status.item() == 6                      # DSA_ERR_DEVICE_TIMEOUT
    # neither was ready; both left after the short limit, far from the long one
    assert 20_000 <= us[first] < 500_000 and 0 < us[1 - first] < 500_000
    assert (out + 1).tolist() == [x + 1 for x in us]    # the context serves on
