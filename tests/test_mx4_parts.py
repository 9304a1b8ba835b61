"""MX4 products with K in parts: eight of them (clusters of eight blocks, and
block pairs that take eight parts one after the other), and static weights,
whose copies start before the kernel ahead of the product has ended."""
import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from helpers import need_gpu
from test_mx4 import DT, check_product, gemm, held, values

pytestmark = pytest.mark.gpu


def quantized(x):
    codes = torch.empty(x.shape[0], x.shape[1] // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(ig.mx4_scale_bytes(*x.shape), dtype=torch.uint8, device="cuda")
    ig.mx4_quantize(x, codes, scales)
    return codes, scales


# 112 and 64 + 1 stages of 256 k; 3 and 1 tiles of 128 columns
@pytest.mark.parametrize("N,K", [(264, 28672), (72, 16416)])
@pytest.mark.parametrize("M", [1, 2, 17, 33, 64, 130])
def test_eight_parts_equal_oracle(M, N, K):
    """One to 33 groups of four tokens, dealt to eight owners: fewer groups than
    owners, one more, and a last group that is not full."""
    need_gpu()
    x, w = held(values(M, K, M + 7, spread=3)), held(values(N, K, N, spread=3))
    for y_t in ("bf16", "f32"):
        check_product(gemm(x, w, N, y_t), x[2], w[2], y_t)


@pytest.mark.parametrize("y_t", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(264, 28672), (2056, 16416)])
def test_eight_parts_do_not_depend_on_the_batch(N, K, y_t):
    """Rows of a product of many tokens (block pairs) and the same rows alone, in
    every kind of tile."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(N)
    full = torch.randn(9000, K, device="cuda", generator=g).to(torch.bfloat16)
    w = quantized(torch.randn(N, K, device="cuda", generator=g))
    ref = gemm(quantized(full), w, N, y_t)
    rng = np.random.default_rng(K)
    for M in (1, 3, 17, 33, 64, 65, 130, 200, 700, 3000):
        pos = torch.from_numpy(rng.permutation(9000)[:M]).cuda()
        assert torch.equal(gemm(quantized(full[pos]), w, N, y_t), ref[pos]), M


@pytest.mark.parametrize("N,K", [(4096, 4096), (264, 28672), (8192, 28672)])
@pytest.mark.parametrize("M", [1, 16, 64])
def test_static_weights_in_parts(M, N, K):
    """With IG_FLAG_STATIC_WEIGHTS, queued right behind a norm that writes x and
    behind another product, the bits are those without it."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(M + N)
    h = torch.randn(M, K, device="cuda", generator=g)
    one = torch.ones(K, device="cuda").to(torch.bfloat16)
    w = [quantized(torch.randn(N, K, device="cuda", generator=g)) for _ in range(2)]
    n = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    ig.block_norm(h, None, None, one, n_out=n)
    x = quantized(n)
    refs = [gemm(x, v, N, "bf16") for v in w]
    ws = ig.mx4_workspace()
    outs = [torch.zeros(M, N, dtype=DT["bf16"], device="cuda") for _ in range(12)]
    torch.cuda.synchronize()
    for i in range(0, 12, 3):
        for t in x:
            t.fill_(255)                     # not to be read
        ig.block_norm(h, None, None, one, codes=x[0], scales=x[1])
        for j in range(3):
            ig.mx4_gemm(*x, *w[j % 2], outs[i + j], ws, flags=ig.FLAG_STATIC_WEIGHTS)
    assert ig.check_status(ws) == 0
    for i, o in enumerate(outs):
        assert torch.equal(o, refs[i % 3 % 2]), i
