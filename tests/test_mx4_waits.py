"""Bounded waits of the MX4 products: what they leave behind when one expires,
and what they must not count."""
import ctypes
import subprocess

import pytest
import torch

import invariant_gemm_gb300 as ig
from helpers import need_gpu
from test_mx4 import gemm, held, values

gpu = pytest.mark.gpu
IG_ERR_TIMEOUT = -8


@gpu
@pytest.mark.parametrize("M", [1, 16, 48])
def test_blocks_that_failed_do_not_keep_the_others_waiting(M):
    """K in four parts (a cluster of four blocks to a tile), no more stages than
    the copy ring holds: after an expired wait each block tells the owners of
    the tokens that its sums will not come, so all end as soon as their copies
    have landed. A block that waited for sums that never come would take 2^31
    clocks, over a second, and could leave before those of a slower block."""
    need_gpu()
    N, K = 264, 8192
    x, w = held(values(M, K, 3)), held(values(N, K, 4))
    ref = gemm(x, w, N, "f32")
    ws = ig.mx4_workspace()
    y = torch.full((M, N), 5.0, device="cuda")
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    ig.mx4_gemm(x[0], x[1], w[0], w[1], y, ws, flags=ig.FLAG_TEST_COPY_TIMEOUT)
    stop.record()
    assert ig.check_status(ws) == IG_ERR_TIMEOUT
    assert start.elapsed_time(stop) < 500
    assert ((y == 5) | (y == ref)).all() and (y == 5).any()
    assert torch.equal(gemm(x, w, N, "f32", ws=ws), ref)


@gpu
@pytest.mark.parametrize("y_t", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(4, 264, 256), (16, 264, 8192), (48, 520, 4096),
                                   (100, 512, 2048), (300, 136, 2048), (600, 4096, 1024),
                                   (257, 12288, 512)])
def test_expired_blocks_store_their_result_or_nothing(M, N, K, y_t):
    """Each element is as it was or, bit for bit, that of an undisturbed call."""
    need_gpu()
    x, w = held(values(M, K, 3)), held(values(N, K, 4))
    ref = gemm(x, w, N, y_t)
    ws = ig.mx4_workspace()
    y = torch.full_like(ref, 5.0)
    ig.mx4_gemm(x[0], x[1], w[0], w[1], y, ws, flags=ig.FLAG_TEST_COPY_TIMEOUT)
    assert ig.check_status(ws) == IG_ERR_TIMEOUT
    assert ((y == 5) | (y == ref)).all() and (y == 5).any()
    assert torch.equal(gemm(x, w, N, y_t, ws=ws), ref)


# A kernel that lets the next one on the stream start and then runs on for
# `clocks` (at most 2^32) of its SM's clock: two seconds or so.
DELAY = r"""
__global__ void delay_kernel(long long clocks) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long t0 = clock64();
  for (int i = 0; i < 20000000 && clock64() - t0 < clocks; ++i) __nanosleep(1000);
}
extern "C" int delay(long long clocks, void* stream) {
  if (clocks < 0 || clocks > (1ll << 32)) return -1;
  delay_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(clocks);
  return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def delay(tmp_path_factory):
    need_gpu()
    from invariant_gemm_gb300 import build
    d = tmp_path_factory.mktemp("delay")
    (d / "delay.cu").write_text(DELAY)
    subprocess.run([build._nvcc(), "-shared", "-Xcompiler", "-fPIC", *build.ARCH, "-o",
                    str(d / "delay.so"), str(d / "delay.cu")], check=True)
    fn = ctypes.CDLL(str(d / "delay.so")).delay
    fn.argtypes = [ctypes.c_longlong, ctypes.c_void_p]
    return lambda clocks: fn(clocks, torch.cuda.current_stream().cuda_stream)


@gpu
@pytest.mark.parametrize("flags", [0, ig.FLAG_STATIC_WEIGHTS])
@pytest.mark.parametrize("M,N,K", [(4, 264, 256), (16, 1024, 2048), (3, 264, 8192),
                                   (40, 1024, 28672), (300, 12288, 512)])
def test_the_kernel_before_may_run_long(delay, M, N, K, flags):
    """A product behind a kernel that releases it early and then runs on for
    1.5 * 2^31 clocks is right: its waits do not count what that kernel takes."""
    x, w = held(values(M, K, 3)), held(values(N, K, 4))
    ref = gemm(x, w, N, "f32")
    ws = ig.mx4_workspace()
    y = torch.full((M, N), 5.0, device="cuda")
    torch.cuda.synchronize()
    assert delay(3 << 30) == 0
    ig.mx4_gemm(x[0], x[1], w[0], w[1], y, ws, flags=flags)
    assert ig.check_status(ws) == 0
    assert torch.equal(y, ref)
