"""Gates of one value per row that are columns of a wider tensor."""
import pytest
import torch

from helpers import need_gpu
from test_block_norm import FAKE, c_norm, make, run


@pytest.mark.gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
@pytest.mark.parametrize("M,H,width", [(1, 64, 16), (5, 264, 16), (37, 4096, 7)])
def test_columns_of_a_wider_tensor(M, H, width, h_t):
    """Any column and any row stride: one value is read per row, so no 16-byte
    alignment is asked for."""
    need_gpu()
    d = make(M, H, h_t, "none", M + H)
    wide = torch.randn(M, width, device="cuda").to(torch.bfloat16)
    for col in range(width):
        ref = run(dict(d, gate=wide[:, col:col + 1].contiguous()), h_t)
        got = run(dict(d, gate=wide[:, col:col + 1]), h_t)
        assert torch.equal(got["h"], ref["h"]) and torch.equal(got["n"], ref["n"]), col


def test_alignment_that_is_still_asked_for():
    assert c_norm(gate=FAKE + 1, gcs=0) == -3
    assert c_norm(gate=FAKE + 2, gcs=1) == -3
    assert c_norm(gate=FAKE + 8, gcs=1) == -3
