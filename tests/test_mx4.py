"""MX4 quantisation, its inverse and the MX4 product against the FP64 oracle.

Tolerances:
  quantise    codes and scale bytes equal; dequantised values equal (every
              one is exact in bf16)
  product     |y_gpu - y_ref| <= 1e-5 sum_k |x_k w_k| (FP32 result), and
              2^-8 |y_ref| more for a bf16 result, as for the LoRA products;
              equal to the rounded y_ref where every partial sum is a multiple
              of 1/4 below 2^22 (24 bits hold it, whatever the order)
"""
import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from helpers import need_gpu
from oracle import blocks

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def values(R, K, seed, dtype="bf16", spread=6.0):
    """Normal values whose rows and blocks differ by powers of two."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g)
    x *= torch.exp2(torch.randint(-int(spread), int(spread) + 1, (R, K // 32, 1),
                                  generator=g)).expand(-1, -1, 32).reshape(R, K)
    return x.to(DT[dtype])


def held(x):
    """MX4 tensors of x on the GPU, from the oracle, and their FP64 values."""
    codes, exps = blocks.mx4_encode(x.double().numpy())
    packed, scales = blocks.mx4_pack(codes, exps)
    return torch.from_numpy(packed).cuda(), torch.from_numpy(scales).cuda(), \
        blocks.mx4_values(codes, exps)


def quantize(x, pad=0):
    R, K = x.shape
    codes = torch.full((R, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((ig.mx4_scale_bytes(R, K),), 0xEE, dtype=torch.uint8, device="cuda")
    ig.mx4_quantize(x, codes, scales)
    return codes, scales


def check_quantized(x):
    """GPU codes and scales of x (a GPU tensor) equal the oracle's."""
    R, K = x.shape
    codes, scales = quantize(x)
    c, e = blocks.mx4_encode(x.cpu().double().numpy())
    cg, eg = blocks.mx4_unpack(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(eg, e)
    assert np.array_equal(cg, c)
    # scale bytes that only pad K are 1 for every row that exists
    if K % 128:
        kt = -(-K // 128)
        s = scales.cpu().numpy().reshape(-1, kt, 32, 4, 4).transpose(0, 3, 2, 1, 4)
        s = s.reshape(-1, kt * 4)[:R, K // 32:]
        assert (s == 127).all()
    for out_t in ("bf16", "f32"):
        out = torch.empty(R, K, dtype=DT[out_t], device="cuda")
        ig.mx4_dequantize(codes, scales, out)
        ref = blocks.mx4_values(c, e)
        assert np.array_equal(out.cpu().double().numpy(), ref, equal_nan=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 4096), (3, 64), (5, 96), (31, 160), (127, 256),
                                 (128, 1056), (129, 4128), (300, 2080), (1000, 32), (2, 11008),
                                 (4, 28672), (33, 352)])
def test_quantize_equals_oracle(R, K, dtype):
    need_gpu()
    check_quantized(values(R, K, R + K, dtype).cuda())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_ties_and_extremes(dtype):
    """Every midpoint between neighbouring values, both signs, beside a block
    maximum that fixes the scale at 1, 2^-127 and 2^k; zeros, subnormals,
    the largest finite value, infinities and NaN."""
    need_gpu()
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0, 6.0, 7.0, 7.9375, 0.0, -0.0,
                         0.2490234375, 0.251953125, 2.484375])
    row = torch.cat([mids, -mids])
    rows = [row, row * 2.0 ** -20, row * 2.0 ** 100, row * 2.0 ** -126, row * 2.0 ** -129,
            torch.zeros(32), -torch.zeros(32)]
    big = torch.finfo(DT[dtype]).max
    for v in (big, float("inf"), -float("inf"), float("nan"), 2.0 ** -133, 2.0 ** -126):
        r = torch.ones(32)
        r[7] = v
        rows.append(r)
        r = torch.zeros(32)
        r[31] = v
        rows.append(r)
    x = torch.stack(rows).to(DT[dtype])
    x = torch.cat([x, torch.ones_like(x)], 1)   # a plain block beside each
    check_quantized(x.cuda())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_row_strides(dtype):
    need_gpu()
    wide = values(70, 512, 9, dtype).cuda()
    x = wide[:, 64:64 + 160]
    a, b = quantize(x), quantize(x.contiguous())
    r = np.arange(70)
    assert torch.equal(a[0], b[0])
    _, ea = blocks.mx4_unpack(a[0].cpu().numpy(), a[1].cpu().numpy())
    _, eb = blocks.mx4_unpack(b[0].cpu().numpy(), b[1].cpu().numpy())
    assert np.array_equal(ea, eb) and len(ea) == len(r)
    out = torch.zeros(70, 512, dtype=DT[dtype], device="cuda")
    ig.mx4_dequantize(a[0], a[1], out[:, 64:64 + 160])
    flat = torch.empty(70, 160, dtype=DT[dtype], device="cuda")
    ig.mx4_dequantize(a[0], a[1], flat)
    assert torch.equal(out[:, 64:64 + 160], flat)
    assert not out[:, :64].any() and not out[:, 224:].any()


@gpu
def test_quantize_offsets_past_32_bits():
    """rows x K past 2^32 elements: the last rows equal those of a small call."""
    need_gpu()
    R, K = 135000, 32768
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    tail = values(130, K, 3).cuda()
    x[-130:] = tail
    codes, scales = quantize(x)
    out = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    ig.mx4_dequantize(codes, scales, out)
    c, s = quantize(tail)
    ref = torch.empty(130, K, dtype=torch.bfloat16, device="cuda")
    ig.mx4_dequantize(c, s, ref)
    assert torch.equal(out[-130:], ref)
    assert torch.equal(codes[-130:], c)
    assert not out[:8].any() and not out[R // 2:R // 2 + 8].any()


@gpu
def test_empty_tensors():
    need_gpu()
    codes, scales = quantize(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    ig.mx4_dequantize(codes, scales, torch.zeros(0, 64, device="cuda"))
    w = held(values(64, 64, 1))
    y = torch.zeros(0, 64, device="cuda")
    ig.mx4_gemm(codes, scales, w[0], w[1], y, ig.mx4_workspace())
    torch.cuda.synchronize()


# ---------------------------------------------------------------- product

def gemm(x, w, N, y_t, ws=None, y=None, flags=0):
    M = x[0].shape[0]
    ws = ig.mx4_workspace() if ws is None else ws
    if y is None:
        y = torch.full((M, N), float("nan"), dtype=DT[y_t], device="cuda")
    ig.mx4_gemm(x[0], x[1], w[0], w[1], y, ws, flags=flags)
    assert ig.check_status(ws) == 0
    return y


def check_product(y, xv, wv, y_t):
    ref, terms = blocks.product(xv, wv)
    got = y.cpu().double().numpy()
    tol = 1e-5 * terms + (2.0 ** -8 * np.abs(ref) if y_t == "bf16" else 0.0)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


SIZES = [(1, 8, 32), (1, 4096, 4096), (2, 136, 64), (7, 128, 96), (15, 264, 160), (16, 512, 256),
         (17, 1000, 288), (31, 72, 4128), (33, 4104, 1056), (64, 128, 11008), (65, 520, 2048),
         (128, 384, 512), (129, 256, 4096), (200, 2056, 1024), (255, 120, 544), (257, 4096, 768),
         (333, 4104, 1056), (640, 1304, 2080), (1025, 520, 8192), (3, 8192, 28672),
         (300, 12288, 512), (2049, 1024, 992)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_equals_oracle(M, N, K):
    need_gpu()
    x = held(values(M, K, M + K, spread=3))
    w = held(values(N, K, N + K + 1, spread=3))
    for y_t in ("bf16", "f32"):
        check_product(gemm(x, w, N, y_t), x[2], w[2], y_t)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (16, 8, 32), (48, 264, 1120), (130, 1032, 2048),
                                   (300, 136, 11008), (700, 512, 4096)])
def test_product_exact_on_small_numbers(M, N, K):
    """All scales 1: every sum is a multiple of 1/4 below 36 K < 2^22, which
    FP32 holds in any order."""
    need_gpu()
    rng = np.random.default_rng(M + N + K)
    xc, wc = (rng.integers(0, 16, (R, K), dtype=np.uint8) for R in (M, N))
    ops = []
    for c in (xc, wc):
        e = np.full((c.shape[0], K // 32), 127, dtype=np.uint8)
        p, s = blocks.mx4_pack(c, e)
        ops.append((torch.from_numpy(p).cuda(), torch.from_numpy(s).cuda(),
                    blocks.mx4_values(c, e)))
    ref, _ = blocks.product(ops[0][2], ops[1][2])
    y = gemm(ops[0], ops[1], N, "f32")
    assert np.array_equal(y.cpu().double().numpy(), ref)
    yb = gemm(ops[0], ops[1], N, "bf16")
    assert torch.equal(yb, y.to(torch.bfloat16))


@gpu
def test_product_one_scale_at_a_time():
    """One-hot rows of x pick single elements of w: each (row, block) scale of
    both operands lands where it belongs, exactly."""
    need_gpu()
    M, N, K = 160, 264, 1056
    rng = np.random.default_rng(5)
    xc = np.zeros((M, K), dtype=np.uint8)
    pick = rng.permutation(K)[:M]
    xc[np.arange(M), pick] = 2                                  # 1.0
    xe = rng.integers(117, 138, (M, K // 32), dtype=np.uint8)
    wc = rng.integers(0, 16, (N, K), dtype=np.uint8)
    we = rng.integers(117, 138, (N, K // 32), dtype=np.uint8)
    x = [torch.from_numpy(a).cuda() for a in blocks.mx4_pack(xc, xe, pad=130)]
    w = [torch.from_numpy(a).cuda() for a in blocks.mx4_pack(wc, we, pad=125)]
    ref, _ = blocks.product(blocks.mx4_values(xc, xe), blocks.mx4_values(wc, we))
    y = gemm(x, w, N, "f32")
    assert np.array_equal(y.cpu().double().numpy(), ref)


@gpu
def test_product_nan_scales_and_garbage_padding():
    """A NaN scale reaches its row of x or column of w only; scale bytes of
    rows that do not exist (here NaN) reach nothing."""
    need_gpu()
    M, N, K = 40, 136, 352
    xc, xe = blocks.mx4_encode(values(M, K, 1).double().numpy())
    wc, we = blocks.mx4_encode(values(N, K, 2).double().numpy())
    clean = gemm([torch.from_numpy(a).cuda() for a in blocks.mx4_pack(xc, xe)],
                 [torch.from_numpy(a).cuda() for a in blocks.mx4_pack(wc, we)], N, "f32").cpu()
    xe[11, 3] = 255
    we[70, 10] = 255

    def operand(c, e):
        p, s = blocks.mx4_pack(c, e, pad=255)
        R, kt = c.shape[0], -(-K // 128)
        s = s.reshape(-1, kt, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-1, kt * 4).copy()
        s[:R, K // 32:] = 127             # blocks that pad K are finite
        s = s.reshape(-1, 4, 32, kt, 4).transpose(0, 3, 2, 1, 4).reshape(-1)
        return [torch.from_numpy(a).cuda() for a in (p, np.ascontiguousarray(s))]

    y = gemm(operand(xc, xe), operand(wc, we), N, "f32").cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[11], bad[:, 70] = True, True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@gpu
@pytest.mark.parametrize("N,K", [(4096, 4096), (520, 1056), (8192, 2048), (1032, 11008)])
def test_product_rows_do_not_depend_on_the_batch(N, K):
    """The same rows alone, in batches of many sizes and at other places give
    the same bits, in both result types."""
    need_gpu()
    base = held(values(12, K, 7, spread=3))
    w = held(values(N, K, 8, spread=3))
    c12, e12 = blocks.mx4_unpack(base[0].cpu().numpy(), base[1].cpu().numpy())
    for y_t in ("bf16", "f32"):
        ref = gemm(base, w, N, y_t)
        for M in (1, 5, 13, 16, 17, 33, 64, 65, 128, 129, 200, 256, 257, 500, 1000, 1500, 2100):
            rng = np.random.default_rng(M)
            c, e = blocks.mx4_encode(values(M, K, M).double().numpy())
            k = min(M, 12)
            pos = rng.permutation(M)[:k]
            c[pos], e[pos] = c12[:k], e12[:k]
            x = [torch.from_numpy(a).cuda() for a in blocks.mx4_pack(c, e)]
            y = gemm(x, w, N, y_t)
            assert torch.equal(y[torch.from_numpy(pos).cuda()], ref[:k]), (M, y_t)


@gpu
@pytest.mark.parametrize("M,N", [(5, 264), (300, 1032)])
@pytest.mark.parametrize("y_t", ["bf16", "f32"])
def test_product_strided_result(M, N, y_t):
    need_gpu()
    K = 512
    x, w = held(values(M, K, 3)), held(values(N, K, 4))
    ref = gemm(x, w, N, y_t)
    wide = torch.full((M, N + 48), -7.0, dtype=DT[y_t], device="cuda")
    gemm(x, w, N, y_t, y=wide[:, 16:16 + N])
    assert torch.equal(wide[:, 16:16 + N], ref)
    assert (wide[:, :16] == -7).all() and (wide[:, 16 + N:] == -7).all()


@gpu
def test_product_shares_a_lora_workspace_and_other_streams():
    """A LoRA workspace serves; calls on two streams with one workspace do not
    disturb each other; static weights give the same bits."""
    need_gpu()
    M, N, K = 96, 1024, 2048
    x, w = held(values(M, K, 3)), held(values(N, K, 4))
    ref = gemm(x, w, N, "bf16")
    ws = ig.workspace(ig.make_shape(8, 512, 512, 8))
    assert torch.equal(gemm(x, w, N, "bf16", ws=ws), ref)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        ig.mx4_gemm(x[0], x[1], w[0], w[1], o, ws, flags=ig.FLAG_STATIC_WEIGHTS,
                    stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    assert ig.check_status(ws) == 0


@gpu
def test_quantize_then_product_in_a_graph():
    """Quantise and multiply captured in one CUDA graph and replayed on new
    inputs."""
    need_gpu()
    M, N, K = 24, 512, 1024
    w = held(values(N, K, 4))
    x = values(M, K, 5).cuda()
    codes, scales = quantize(x)
    ws = ig.mx4_workspace()
    y = torch.zeros(M, N, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ig.mx4_quantize(x, codes, scales)
        ig.mx4_gemm(codes, scales, w[0], w[1], y, ws, flags=ig.FLAG_STATIC_WEIGHTS)
    for seed in (5, 6, 7):
        new = values(M, K, seed)
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        check_product(y, held(new)[2], w[2], "f32")


@gpu
@pytest.mark.parametrize("M,N,K", [(4, 264, 256), (30, 1024, 8192), (100, 512, 4096),
                                   (600, 4096, 1024)])
def test_expired_wait_is_reported_and_the_workspace_is_usable(M, N, K):
    """The first copy's wait runs out: IG_ERR_TIMEOUT, and the next call is
    right."""
    need_gpu()
    x, w = held(values(M, K, 3)), held(values(N, K, 4))
    ws = ig.mx4_workspace()
    y = torch.full((M, N), 5.0, device="cuda")
    ig.mx4_gemm(x[0], x[1], w[0], w[1], y, ws, flags=ig.FLAG_TEST_COPY_TIMEOUT)
    assert ig.check_status(ws) == -8
    assert (y == 5).sum() > y.numel() // 2       # expired blocks store nothing
    check_product(gemm(x, w, N, "f32", ws=ws), x[2], w[2], "f32")


# --------------------------------------------------------------- refusals

FAKE = 1 << 20     # an aligned address that no call below reads


def c_gemm(M=16, N=64, K=128, ld=None, t=0, flags=0, ptr=FAKE, ws_bytes=None, **over):
    import ctypes
    p = dict(xc=ptr, xs=ptr, wc=ptr, ws_=ptr, y=ptr, work=ptr)
    p.update(over)
    sh = ig.Mx4Shape(M, N, K, N if ld is None else ld, t, flags)
    n = ig.lib().ig_mx4_workspace_bytes() if ws_bytes is None else ws_bytes
    return ig.lib().ig_mx4_gemm(ctypes.byref(sh), p["xc"], p["xs"], p["wc"], p["ws_"], p["y"],
                                p["work"], n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(K=48), -2), (dict(K=0), -2), (dict(N=4), -2), (dict(N=12), -2), (dict(M=-1), -2),
    (dict(ld=56), -2), (dict(ld=68), -2), (dict(t=2), -1), (dict(flags=2), -1),
    (dict(M=1 << 31), -9), (dict(xc=None), -1), (dict(xs=None), -1), (dict(wc=None), -1),
    (dict(ws_=None), -1), (dict(y=None), -1), (dict(work=None), -1), (dict(xc=FAKE + 8), -3),
    (dict(y=FAKE + 2), -3), (dict(ws_bytes=256), -4)])
def test_gemm_refusals(kw, code):
    assert c_gemm(**kw) == code


def test_empty_calls_do_nothing():
    assert c_gemm(M=0) == 0
    assert ig.lib().ig_mx4_quantize(0, 64, None, 64, 0, None, None, None) == 0
    assert ig.lib().ig_mx4_dequantize(0, 64, None, None, None, 64, 0, None) == 0


@pytest.mark.parametrize("rows,K,ld,t,p,code", [
    (4, 33, 64, 0, FAKE, -2), (4, 64, 56, 0, FAKE, -2), (4, 64, 68, 0, FAKE, -2),
    (-1, 64, 64, 0, FAKE, -2), (4, 64, 64, 5, FAKE, -1), (4, 64, 64, 0, None, -1),
    (4, 64, 64, 1, FAKE + 4, -3), (1 << 31, 64, 64, 0, FAKE, -9)])
def test_quantize_refusals(rows, K, ld, t, p, code):
    assert ig.lib().ig_mx4_quantize(rows, K, p, ld, t, p, p, None) == code
    assert ig.lib().ig_mx4_dequantize(rows, K, p, p, p, ld, t, None) == code


def test_scale_bytes():
    assert ig.mx4_scale_bytes(1, 32) == 512
    assert ig.mx4_scale_bytes(128, 128) == 512
    assert ig.mx4_scale_bytes(129, 160) == 4 * 512
    assert ig.mx4_scale_bytes(0, 64) == 0
    with pytest.raises(ig.IGError):
        ig.mx4_scale_bytes(4, 40)


def test_binding_refuses_wrong_tensors():
    """Types, sizes, strides and devices are checked before the library runs."""
    u8, b16 = torch.uint8, torch.bfloat16
    x = torch.zeros(4, 64, dtype=b16)
    c, s = torch.zeros(4, 32, dtype=u8), torch.zeros(512, dtype=u8)
    for bad in (lambda: ig.mx4_quantize(x.half(), c, s),
                lambda: ig.mx4_quantize(x.t().contiguous().t(), c, s),
                lambda: ig.mx4_quantize(x, c[:, :16], s),
                lambda: ig.mx4_quantize(x, c[:3], s),
                lambda: ig.mx4_quantize(x, c.char(), s),
                lambda: ig.mx4_quantize(x, c, s[:100]),
                lambda: ig.mx4_quantize(x, c, s),                      # not on a GPU
                lambda: ig.mx4_dequantize(c, s, x.half()),
                lambda: ig.mx4_dequantize(c, s[:8], x),
                lambda: ig.mx4_gemm(c, s, c, s, torch.zeros(4, 5, dtype=b16), s),
                lambda: ig.mx4_gemm(c, s, c, s, torch.zeros(5, 4, dtype=b16), s),
                lambda: ig.mx4_gemm(c, s, c[:, :16], s, torch.zeros(4, 4, dtype=b16), s)):
        with pytest.raises(ig.IGError):
            bad()


def test_packed_shapes_are_the_structs():
    """The bytes the binding hands over are those of the declared structs."""
    a = bytes(ig.Mx4Shape(3, 64, 128, 72, 1, 1))
    assert ig._MX4_SHAPE(3, 64, 128, 72, 1, 1) == a
    b = bytes(ig.NormShape(3, 64, 72, 80, 88, 96, 104, 1, 1, 1, 1e-5, 0.5))
    packed = ig._NORM_SHAPE(3, 64, 72, 80, 88, 96, 104, 1, 1, 1, 1e-5, 0.5)
    assert packed == b[:len(packed)]
