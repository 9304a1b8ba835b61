"""MX4 and norm calls whose offsets pass 32 bits: rows far apart, and long
tensors. Each row's bits are those of the same row in a small call (which the
other files hold against the oracle), so comparisons are exact, but for products
whose number of columns differs.
"""
import pytest
import torch

import invariant_gemm_gb300 as ig
from helpers import need_gpu

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FAR = (1 << 31) + 24          # values between two rows


@pytest.fixture
def room():
    """Asks for gigabytes of device memory; gives them back after the test."""
    need_gpu()

    def ask(gigabytes):
        torch.cuda.empty_cache()
        if torch.cuda.mem_get_info()[0] < gigabytes << 30:
            pytest.skip(f"needs {gigabytes} GB of device memory")
        torch.manual_seed(gigabytes)

    yield ask
    torch.cuda.empty_cache()


def quantize(x):
    R, K = x.shape
    codes = torch.full((R, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((ig.mx4_scale_bytes(R, K),), 0xEE, dtype=torch.uint8, device="cuda")
    ig.mx4_quantize(x, codes, scales)
    return codes, scales


def group(scales, first, rows, K):
    """Scale bytes of rows `first` (a multiple of 128) to first + rows."""
    tile = -(-K // 128) * 512
    return scales[first // 128 * tile:-(-(first + rows) // 128) * tile]


def spread(x, far=FAR):
    """x's rows, `far` values apart, in a buffer of their own."""
    R, K = x.shape
    out = torch.empty((R - 1) * far + K + 8, dtype=x.dtype, device="cuda")
    out = out.as_strided((R, K), (far, 1))
    out.copy_(x)
    return out


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise_rows_far_apart(room, dtype):
    room(60)
    x = torch.randn(3, 1056, device="cuda").to(DT[dtype])
    near, far = quantize(x), quantize(spread(x))
    assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1])
    out = spread(torch.zeros_like(x))
    flat = torch.empty_like(x)
    ig.mx4_dequantize(*far, out)
    ig.mx4_dequantize(*near, flat)
    assert torch.equal(out, flat)


@gpu
def test_quantise_long(room):
    """4.3e9 values: codes past 2^31 bytes, values past 2^32."""
    room(40)
    R, K = (1 << 20) + 130, 4128
    x = torch.randn(R, K, dtype=torch.bfloat16, device="cuda")
    codes, scales = quantize(x)
    out = torch.empty_like(x)
    ig.mx4_dequantize(codes, scales, out)
    for first in (0, 1 << 19, 1 << 20):
        rows = min(200, R - first)
        part = x[first:first + rows]
        c, s = quantize(part)
        assert torch.equal(codes[first:first + rows], c)
        kt = -(-K // 128)
        if rows % 128 == 0 or first + rows == R:      # all bytes of its groups are the rows'
            assert torch.equal(group(scales, first, rows, K), s)
        else:
            assert torch.equal(group(scales, first, 128, K), s[:kt * 512])
        o = torch.empty_like(part)
        ig.mx4_dequantize(c, s, o)
        assert torch.equal(out[first:first + rows], o)


@gpu
@pytest.mark.parametrize("y_t", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,far", [(9, 264, (1 << 29) + 8), (200, 136, (1 << 25) + 8),
                                     (12800, 256, (1 << 19) + 8)])
def test_product_rows_far_apart(room, M, N, far, y_t):
    room(40)
    K, ws = 544, ig.mx4_workspace()
    x = quantize(torch.randn(M, K, device="cuda"))
    w = quantize(torch.randn(N, K, device="cuda"))
    near = torch.empty(M, N, dtype=DT[y_t], device="cuda")
    out = spread(torch.zeros_like(near), far)
    ig.mx4_gemm(*x, *w, near, ws)
    ig.mx4_gemm(*x, *w, out, ws)
    assert torch.equal(near, out) and ig.check_status(ws) == 0


@gpu
@pytest.mark.parametrize("few", [False, True])
def test_product_long(room, few):
    """Codes past 2^32 bytes, as the tokens and as the weights."""
    room(20)
    R, K, ws = (1 << 20) + 333, 8224, ig.mx4_workspace()
    codes = torch.randint(0, 256, (R, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(120, 130, (ig.mx4_scale_bytes(R, K),), dtype=torch.uint8,
                           device="cuda")
    other = quantize(torch.randn(8, K, device="cuda"))
    if few:                                           # 8 tokens, R (a multiple of 8) columns
        R -= R % 8
        codes = codes[:R]
        y = torch.empty(8, R, device="cuda")
        ig.mx4_gemm(*other, codes, scales, y, ws)
    else:
        y = torch.empty(R, 8, device="cuda")
        ig.mx4_gemm(codes, scales, *other, y, ws)
    for first in (0, 1 << 19, 1 << 20):
        rows = min(328, R - first)
        part = (codes[first:first + rows], group(scales, first, rows, K))
        if few:
            # K is cut by the number of columns, so the order of a sum may differ:
            # the product's bound, not its bits
            z = torch.empty(8, rows, device="cuda")
            ig.mx4_gemm(*other, *part, z, ws)
            v = torch.empty(rows, K, device="cuda")
            o = torch.empty(8, K, device="cuda")
            ig.mx4_dequantize(*part, v)
            ig.mx4_dequantize(*other, o)
            bound = 1e-5 * (o.double().abs() @ v.double().abs().T)
            for got in (y[:, first:first + rows], z):
                assert ((got.double() - o.double() @ v.double().T).abs() <= bound).all()
        else:
            z = torch.empty(rows, 8, device="cuda")
            ig.mx4_gemm(*part, *other, z, ws)
            assert torch.equal(y[first:first + rows], z)
    assert ig.check_status(ws) == 0


def norm(h, y, gate, w, h_out, n_out, codes=None, scales=None):
    ig.block_norm(h, y, w[0], w[1], gate=gate, scale=0.5, eps=1e-6, h_out=h_out, n_out=n_out,
                  codes=codes, scales=scales)


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
def test_norm_rows_far_apart(room, h_t):
    room(100)
    M, H = 3, 1056
    h = torch.randn(M, H, device="cuda").to(DT[h_t])
    y, gate = (torch.randn(M, H, device="cuda").bfloat16() for _ in range(2))
    w = 1 + 0.2 * torch.randn(2, H, device="cuda").bfloat16()
    near = torch.zeros_like(h), torch.zeros_like(y)
    far = spread(near[0]), spread(near[1])
    norm(h, y, gate, w, *near)
    norm(spread(h), spread(y), spread(gate), w, *far)
    assert all(torch.equal(a, b) for a, b in zip(near, far))


@gpu
def test_norm_long(room):
    """4.8e9 values, MX4 output past 2^31 bytes."""
    room(80)
    M, H = 590000, 8224
    h, y = (torch.randn(M, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gate = torch.randn(M, 1, device="cuda").bfloat16()
    w = 1 + 0.2 * torch.randn(2, H, device="cuda").bfloat16()
    h_out, n_out = torch.empty_like(h), torch.empty_like(h)
    codes = torch.empty(M, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(ig.mx4_scale_bytes(M, H), dtype=torch.uint8, device="cuda")
    norm(h, y, gate, w, h_out, n_out, codes, scales)
    for first in (0, 294912, 589824):
        rows = min(128, M - first)
        at = slice(first, first + rows)
        a, b = torch.empty_like(h[at]), torch.empty_like(h[at])
        c = torch.empty(rows, H // 2, dtype=torch.uint8, device="cuda")
        s = torch.zeros(ig.mx4_scale_bytes(rows, H), dtype=torch.uint8, device="cuda")
        norm(h[at], y[at], gate[at], w, a, b, c, s)
        assert torch.equal(h_out[at], a) and torch.equal(n_out[at], b)
        assert torch.equal(codes[at], c)
        assert torch.equal(group(scales, first, rows, H), s)
