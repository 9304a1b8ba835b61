"""Cases of the quantised-block operators: MX4 quantisation, the MX4 product and the block norm.

MX4: blocks of 32 values along K share one power-of-two scale (E8M0: the value
2^(byte - 127), 255 stands for NaN); a value is a 4-bit float (E2M1: 0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives). For a block with largest magnitude a the
scale is 2^(floor(log2 a) - 2), at least 2^-127; values are divided by it,
rounded to the nearest E2M1 value (ties to the even code) and held at +-6. A
block with an infinity or a NaN is all NaN.
Codes: uint8 [rows][K/2], the even k in the low four bits. Scales: uint8, per
128 rows and 4 blocks one tile [row % 32][row / 32][block % 4] of 512 bytes,
tiles of one row group one after the other along K.

  quantize  values = dequantize(quantize(x))
  gemm      y[m][n] = sum_k x[m][k] w[n][k], both sides MX4
  norm      t = y * rsqrt(mean(y^2) + eps) * w_post
            h' = h + scale * gate * t
            n = h' * rsqrt(mean(h'^2) + eps) * w_pre
"""
import math

import torch

own = False

EPS = 1e-5
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's activations on the way into a decode layer
        dict(name="quantize_M1_K4096", op="quantize", M=1, K=4096, x="bf16"),
        # a ragged prefill batch on its way into the down-projection
        dict(name="quantize_M4095_K11008", op="quantize", M=4095, K=11008, x="bf16"),
        # laying out a large down-projection weight once, from FP32
        dict(name="quantize_M8192_K28672_f32", op="quantize", M=8192, K=28672, x="f32"),
        # decode, one token
        dict(name="gemm_M1_K4096_N4096", op="gemm", M=1, K=4096, N=4096, y="bf16"),
        # decode, a full batch
        dict(name="gemm_M256_K4096_N4096", op="gemm", M=256, K=4096, N=4096, y="bf16"),
        # a few tokens through a large down-projection: the weights' bytes
        dict(name="gemm_M16_K28672_N8192", op="gemm", M=16, K=28672, N=8192, y="bf16"),
        # odd token count and a K that ends inside a tile, FP32 result (logits)
        dict(name="gemm_M333_K1056_N4104_f32", op="gemm", M=333, K=1056, N=4104, y="f32"),
        # stacked q/k/v of a prefill batch
        dict(name="gemm_M4096_K4096_N12288", op="gemm", M=4096, K=4096, N=12288, y="bf16"),
        # the largest prefill product of the large-model workload
        dict(name="gemm_M8192_K28672_N8192", op="gemm", M=8192, K=28672, N=8192, y="bf16"),
        # decode, one token between two blocks
        dict(name="norm_M1_H4096", op="norm", M=1, H=4096, h="bf16", gate="channel"),
        # ragged batch, FP32 residual stream, a gate value for each token and channel
        dict(name="norm_M1001_H11008_f32", op="norm", M=1001, H=11008, h="f32", gate="full"),
        # a large prefill batch, one gate value for each token
        dict(name="norm_M8192_H8192", op="norm", M=8192, H=8192, h="bf16", gate="token"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "norm"])
    M = _log(rng, 1, 8192)
    if op == "quantize":
        return dict(op=op, M=M, K=32 * _log(rng, 2, 896), x=rng.choice(["bf16", "f32"]))
    if op == "gemm":
        return dict(op=op, M=M, K=32 * _log(rng, 2, 896), N=8 * _log(rng, 8, 1024),
                    y=rng.choice(["bf16", "bf16", "f32"]))
    H = 8 * _log(rng, 8, 1376)
    return dict(op=op, M=min(M, 8192 * 8192 // H), H=H, h=rng.choice(["bf16", "f32"]),
                gate=rng.choice(["none", "channel", "token", "full"]))


def work(case):
    M = case["M"]
    if case["op"] == "quantize":
        K = case["K"]
        held = M * K // 2 + M * K // 32
        return {"bytes": M * K * (2 if case["x"] == "bf16" else 4) + 2 * held + 2 * M * K, "flops": 0}
    if case["op"] == "gemm":
        K, N = case["K"], case["N"]
        return {"bytes": (M + N) * (K // 2 + K // 32) + M * N * (2 if case["y"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    H = case["H"]
    gate = {"none": 0, "channel": H, "token": M, "full": M * H}[case["gate"]]
    return {"bytes": M * H * (2 * (2 if case["h"] == "bf16" else 4) + 2 + 2) + 2 * gate + 4 * H,
            "flops": 0}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _tokens(M, K, g):
    """Activations: unit normal values, a few channels of much larger size."""
    x = torch.randn(M, K, device="cuda", generator=g)
    c = torch.randint(0, K, (max(1, K // 128),), device="cuda", generator=g)
    x[:, c] *= 20.0
    return x


def _pack(codes, exps):
    """Codes [R][K] and scale bytes [R][K/32] in the layout given above; scale
    entries that stand for no block are 1."""
    R, K = codes.shape
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    rp, kp = -(-R // 128) * 128, -(-K // 128) * 4
    s = torch.full((rp, kp), 127, dtype=torch.uint8, device=codes.device)
    s[:R, :K // 32] = exps
    s = s.view(rp // 128, 4, 32, kp // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return packed.contiguous(), s.view(-1)


def _held(x):
    codes, exps = _quantize(x.float())
    return _pack(codes, exps)


def prepare(case, seed):
    g = _gen(seed)
    M, op = case["M"], case["op"]
    if own:
        import invariant_gemm_gb300 as ig
    if op == "quantize":
        K = case["K"]
        s = {"op": op, "x": _tokens(M, K, g).to(DTYPE[case["x"]])}
        if own:
            s["codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(ig.mx4_scale_bytes(M, K), dtype=torch.uint8, device="cuda")
            s["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        return s
    if op == "gemm":
        K, N = case["K"], case["N"]
        xc, xs = _held(_tokens(M, K, g))
        wc, ws = _held(torch.randn(N, K, device="cuda", generator=g) / math.sqrt(K))
        s = {"op": op, "y": case["y"], "xc": xc, "xs": xs, "wc": wc, "ws": ws, "M": M, "N": N}
        if own:
            s["out"] = torch.empty(M, N, dtype=DTYPE[case["y"]], device="cuda")
            s["work"] = ig.mx4_workspace()
        return s
    H = case["H"]
    h = DTYPE[case["h"]]
    s = {"op": op, "H": H, "scale": 0.5,
         "h": (4.0 * _tokens(M, H, g)).to(h), "y": _tokens(M, H, g).to(torch.bfloat16),
         "w_post": (1.0 + 0.1 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16),
         "w_pre": (1.0 + 0.1 * torch.randn(H, device="cuda", generator=g)).to(torch.bfloat16)}
    shape = {"none": None, "channel": (1, H), "token": (M, 1), "full": (M, H)}[case["gate"]]
    s["gate"] = None if shape is None else torch.rand(
        shape, device="cuda", generator=g).to(torch.bfloat16)
    if own:
        s["h_out"] = torch.empty_like(s["h"])
        s["n"] = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------ plain forms

_MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(byte):
    """2^(byte - 127) as FP32, NaN for 255."""
    b = byte.to(torch.int32)
    bits = torch.where(b > 0, b << 23, 1 << 22)
    return torch.where(b < 255, bits, 0x7fc00000).to(torch.int32).view(torch.float32)


def _quantize(x):
    """E2M1 codes [R][K] and scale bytes [R][K/32] of x (FP32)."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    bad = ~torch.isfinite(top)
    v = b * _power(127 - torch.where(bad, 0, e))[..., None]
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) +
            (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    code = torch.where(bad[..., None], 0, code).to(torch.uint8)
    return code.view(R, K), torch.where(bad, 255, e + 127).to(torch.uint8)


def _values(codes, exps):
    """What codes [R][K] and scale bytes [R][K/32] stand for, in FP32."""
    R, K = codes.shape
    table = torch.tensor(_MAG + tuple(-m for m in _MAG), device=codes.device)
    v = table[codes.int()].view(R, K // 32, 32) * _power(exps)[..., None]
    return v.view(R, K)


def _unpack(packed, s):
    R, half = packed.shape
    K = 2 * half
    codes = torch.stack((packed & 15, packed >> 4), -1).view(R, K)
    rt, kt = -(-R // 128), -(-K // 128)
    s = s.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)
    return _values(codes, s[:R, :K // 32])


def _norm(v, w):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()


def _plain(s):
    if s["op"] == "quantize":
        return {"values": _values(*_quantize(s["x"].float())).to(torch.bfloat16)}
    if s["op"] == "gemm":
        x, w = _unpack(s["xc"], s["xs"]), _unpack(s["wc"], s["ws"])
        return {"y": (x @ w.t()).to(DTYPE[s["y"]])}
    t = _norm(s["y"].float(), s["w_post"]) * s["scale"]
    if s["gate"] is not None:
        t = t * s["gate"].float()
    h = s["h"].float() + t
    return {"h": h.to(s["h"].dtype), "n": _norm(h, s["w_pre"]).to(torch.bfloat16)}


def run(s):
    if not own:
        return _plain(s)
    import invariant_gemm_gb300 as ig
    if s["op"] == "quantize":
        ig.mx4_quantize(s["x"], s["codes"], s["scales"])
        ig.mx4_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"]}
    if s["op"] == "gemm":
        ig.mx4_gemm(s["xc"], s["xs"], s["wc"], s["ws"], s["out"], s["work"],
                    flags=ig.FLAG_STATIC_WEIGHTS)
        return {"y": s["out"]}
    ig.block_norm(s["h"], s["y"], s["w_post"], s["w_pre"], gate=s["gate"], scale=s["scale"],
                  eps=EPS, h_out=s["h_out"], n_out=s["n"])
    return {"h": s["h_out"], "n": s["n"]}


# --------------------------------------------------------- 64-bit results

def _exact_quantized(x):
    """dequantize(quantize(x)) from the definition, in FP64 [R][K]."""
    if x.shape[0] > 1024:                       # FP64 copies of a large weight
        return torch.cat([_exact_quantized(c) for c in x.split(1024)])
    R, K = x.shape
    b = x.double().view(R, K // 32, 32)
    top = b.abs().amax(-1, keepdim=True)
    p = torch.floor(torch.log2(top))            # off by one only beside a power of two
    p = p + (torch.exp2(p + 1) <= top).double() - (torch.exp2(p) > top).double()
    scale = torch.exp2(torch.clamp(p - 2, min=-127.0))
    v = b / scale
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.copysign(q, v) * scale).view(R, K)


def _exact_held(packed, s):
    R, half = packed.shape
    K = 2 * half
    k = torch.arange(K, device=packed.device)
    r = torch.arange(R, device=packed.device)
    nib = (packed.long()[:, k // 2] >> (4 * (k % 2))) & 15
    e, m = (nib >> 1) & 3, nib & 1
    mag = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    blk = torch.arange(K // 32, device=packed.device)
    kt = -(-K // 128)
    at = ((r[:, None] // 128) * kt + blk // 4) * 512 + (r[:, None] % 32) * 16 + \
        ((r[:, None] % 128) // 32) * 4 + blk % 4
    scale = torch.exp2(s.long()[at].double() - 127)
    mag = torch.where(nib >= 8, -mag, mag).view(R, K // 32, 32)
    return (mag * scale[..., None]).view(R, K)


def _exact_norm(v, w):
    return v / torch.sqrt((v ** 2).sum(-1, keepdim=True) / v.shape[-1] + EPS) * w.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return {"values": _exact_quantized(s["x"])}
    if case["op"] == "gemm":
        w = _exact_held(s["wc"], s["ws"])
        y = torch.empty(s["M"], s["N"], dtype=torch.float64, device="cuda")
        torch.matmul(_exact_held(s["xc"], s["xs"]), w.t(), out=y)
        return {"y": y}
    t = _exact_norm(s["y"].double(), s["w_post"]) * s["scale"]
    if s["gate"] is not None:
        t = t * s["gate"].double()
    h = s["h"].double() + t
    return {"h": h, "n": _exact_norm(h, s["w_pre"])}
