"""Bounded waits of the MX4 products: what they leave behind when one expires,
and what they must not count."""
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
