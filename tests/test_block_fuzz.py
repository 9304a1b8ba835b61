"""Random sizes, types and operands of the quantised-block calls against the
FP64 oracle, with the tolerances of test_mx4.py and test_block_norm.py."""
import numpy as np
import pytest
import torch

import test_block_norm as norm
import test_mx4 as mx4
from helpers import need_gpu

pytestmark = pytest.mark.gpu


def log_uniform(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


@pytest.mark.parametrize("seed", range(24))
def test_product(seed):
    need_gpu()
    rng = np.random.default_rng(900 + seed)
    M, N, K = log_uniform(rng, 1, 900), 8 * log_uniform(rng, 1, 600), 32 * log_uniform(rng, 1, 130)
    x = mx4.held(mx4.values(M, K, seed, spread=3))
    w = mx4.held(mx4.values(N, K, seed + 1, spread=3))
    y_t = ("bf16", "f32")[seed % 2]
    pad = 8 * int(rng.integers(0, 4))
    wide = torch.full((M, N + pad), -3.0, dtype=mx4.DT[y_t], device="cuda")
    mx4.check_product(mx4.gemm(x, w, N, y_t, y=wide[:, :N]), x[2], w[2], y_t)
    assert (wide[:, N:] == -3).all()


@pytest.mark.parametrize("seed", range(16))
def test_quantize(seed):
    need_gpu()
    rng = np.random.default_rng(300 + seed)
    R, K = log_uniform(rng, 1, 1500), 32 * log_uniform(rng, 1, 60)
    mx4.check_quantized(mx4.values(R, K, seed, ("bf16", "f32")[seed % 2],
                                   spread=float(rng.integers(0, 40))).cuda())


@pytest.mark.parametrize("seed", range(24))
def test_norm(seed):
    need_gpu()
    rng = np.random.default_rng(500 + seed)
    H = 8 * log_uniform(rng, 1, 4096)
    M = min(log_uniform(rng, 1, 1500), max(1, (1 << 21) // H))
    h_t = ("bf16", "f32")[seed % 2]
    gate = ("none", "channel", "row", "token", "full")[int(rng.integers(5))]
    d = norm.make(M, H, h_t, gate, seed)
    norm.check(d, h_t, scale=float(rng.normal()), codes=H % 32 == 0)
