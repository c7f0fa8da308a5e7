"""The serving calls behind a kernel that lets its dependents start before it has
written anything: the calls are launched then, and may read what it writes only
once it has ended."""
import ctypes
import subprocess

import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build
from tests.test_serving import BF, DEV, Case, check

gpu = pytest.mark.gpu

# Lets its dependents start, idles 30 us, then copies `words` words.
SOURCE = r"""
#include <cuda_runtime.h>
#include <stdint.h>
__global__ void late_copy(uint32_t* dst, const uint32_t* src, int64_t words) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do {
    __nanosleep(1000);
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  } while (t - t0 < 30000u);
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words;
       i += (int64_t)gridDim.x * blockDim.x)
    dst[i] = src[i];
}
extern "C" __attribute__((visibility("default"))) int late(void* dst, const void* src,
                                                           int64_t words, void* stream) {
  late_copy<<<16, 256, 0, (cudaStream_t)stream>>>((uint32_t*)dst, (const uint32_t*)src, words);
  return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """late(dst, src): dst = src by that kernel, on the current stream."""
    at = tmp_path_factory.mktemp("late")
    (at / "late.cu").write_text(SOURCE)
    subprocess.run([dsa_build._nvcc()] + dsa_build.FLAGS +
                   ["-shared", "-o", str(at / "late.so"), str(at / "late.cu")], check=True)
    fn = ctypes.CDLL(str(at / "late.so")).late
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]

    def call(dst, src):
        n = dst.numel() * dst.element_size()
        assert dst.shape == src.shape and dst.dtype == src.dtype and n % 4 == 0
        assert dst.is_contiguous() and src.is_contiguous()
        assert fn(dst.data_ptr(), src.data_ptr(), n // 4,
                  torch.cuda.current_stream().cuda_stream) == 0

    return call


def replayed(step, captured, times=8):
    step()
    if not captured:
        for _ in range(times):
            step()
        return
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(times):
        g.replay()


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("last", ["slots", "k_new", "v_new"])
def test_append_behind_a_kernel_that_writes_late(late, last, captured):
    T, d, n_pages = 1024, 256, 80
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=1, max_blocks=1, page_size=16,
                          d_qk=d, d_v=d)
    g = torch.Generator(device=DEV).manual_seed(1)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_APPEND)
    want = dict(slots=torch.randperm(n_pages * 16, generator=g, device=DEV)[:T].to(torch.int32),
                k_new=torch.randn((T, d), generator=g, device=DEV).to(BF),
                v_new=torch.randn((T, d), generator=g, device=DEV).to(BF))
    have = {n: torch.zeros_like(x) for n, x in want.items()}
    pages = [torch.zeros((n_pages, 16, d), dtype=BF, device=DEV) for _ in range(2)]

    def step():
        for n, x in want.items():
            if n != last:
                have[n].copy_(x)
        have[last].fill_(-1 if last == "slots" else 7)
        for p in pages:
            p.zero_()
        late(have[last], want[last])
        dsa.append_cache(cfg, have["slots"], have["k_new"], pages[0], v_new=have["v_new"],
                         v_pages=pages[1], ws=ws)

    replayed(step, captured)
    assert dsa.get_device_status(ws) == 0
    for p, x in zip(pages, (want["k_new"], want["v_new"])):
        ref = torch.zeros_like(p).view(-1, d)
        ref[want["slots"].long()] = x
        assert torch.equal(p.view(-1, d), ref)


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("last", ["seq", "cu", "table", "ptable", "q", "k"])
def test_attention_behind_a_kernel_that_writes_late(late, last, captured):
    """What is written late holds another call's valid values before."""
    cases = [Case([1, 3], [40, 300], 500, 16, 512, 64, 1, seed=8),
             Case([2, 2], [7, 300], 500, 16, 512, 64, 1, seed=9)]
    c, other = cases
    assert other.k.shape[0] <= c.k.shape[0] and c.table.shape == other.table.shape
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    now, before = (dict(seq=i32(x.seq + [0, 0]), cu=i32(x.cu + [0]), table=x.table.to(DEV),
                        ptable=x.prefix_table.to(DEV), q=x.q.to(DEV)) for x in cases)
    now["k"] = torch.nan_to_num(c.k).to(DEV)
    before["k"] = torch.ones_like(now["k"])
    before["table"] = before["table"].clamp(min=0)
    have = {n: x.clone() for n, x in now.items()}
    o = torch.zeros((4, 16, 512), dtype=BF, device=DEV)
    lse = torch.zeros((4, 16), device=DEV)
    ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX)

    def step():
        have[last].copy_(before[last])
        o.zero_()
        late(have[last], now[last])
        dsa.prefix_attn(c.cfg, have["q"], have["k"], have["ptable"], 500, have["table"],
                        have["seq"][:2], have["cu"][:3], o=o, lse=lse, ws=ws)

    replayed(step, captured)
    assert dsa.get_device_status(ws) == 0
    check((o.cpu(), lse.cpu()), c.plain())
