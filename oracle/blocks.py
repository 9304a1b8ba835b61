"""FP64 oracle of the quantised-block operators (numpy): MX4 quantisation, the
MX4 product and the block norm, from their definitions. No code of the CUDA
path; layouts are walked element by element."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_encode(x):
    """x [R][K] -> (codes uint8 [R][K], scale bytes uint8 [R][K/32]).

    Nearest value of the E2M1 list by distance, a tie to the even code."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], b, 0.0)
    top = np.abs(b).max(-1)
    _, e = np.frexp(top)                                 # top = m 2^e, m in [0.5, 1)
    e = np.maximum(np.where(top > 0, e - 1 - 2, -127), -127)
    v = np.ldexp(b, -e[..., None])
    dist = np.abs(np.abs(v)[..., None] - E2M1)
    best = dist.min(-1, keepdims=True)
    near = dist == best                                  # one code, or two neighbours
    first = near.argmax(-1)
    tie = near.sum(-1) == 2
    code = np.where(tie & (first % 2 == 1), first + 1, first)
    code = code + 8 * np.signbit(v)
    code = np.where(finite[..., None], code, 0).astype(np.uint8).reshape(R, K)
    return code, np.where(finite, e + 127, 255).astype(np.uint8)


def mx4_values(codes, exps):
    """The values of codes [R][K] with scale bytes [R][K/32]."""
    R, K = codes.shape
    mag = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    scale = np.where(exps == 255, np.nan, np.ldexp(1.0, exps.astype(np.int64) - 127))
    return (mag.reshape(R, K // 32, 32) * scale[..., None]).reshape(R, K)


def mx4_pack(codes, exps, pad=127):
    """Codes and scale bytes in the library's layout; `pad` where there is no
    block."""
    R, K = codes.shape
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    kt = -(-K // 128)
    out = np.full(-(-R // 128) * kt * 512, pad, dtype=np.uint8)
    for kb in range(K // 32):
        r = np.arange(R)
        out[((r // 128) * kt + kb // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + kb % 4] = \
            exps[:, kb]
    return packed, out


def mx4_unpack(packed, scales):
    """Codes [R][K] and scale bytes [R][K/32] from the library's layout."""
    R, half = packed.shape
    K = 2 * half
    codes = np.empty((R, K), dtype=np.uint8)
    codes[:, 0::2] = packed & 15
    codes[:, 1::2] = packed >> 4
    kt = -(-K // 128)
    r, kb = np.arange(R)[:, None], np.arange(K // 32)[None, :]
    return codes, scales[((r // 128) * kt + kb // 4) * 512 + (r % 32) * 16 +
                         (r // 32 % 4) * 4 + kb % 4]


def product(x, w):
    """(x w^T, sum of |terms|)."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def rms_norm(v, w, eps):
    return v / np.sqrt((v ** 2).mean(-1, keepdims=True) + eps) * w


def block_norm(h, y, w_post, w_pre, gate, scale, eps):
    """(h', n or None, t scaled and gated); None operands as in the library."""
    t = 0.0
    if y is not None:
        t = rms_norm(y, w_post, eps) if w_post is not None else y
        t = scale * t * (gate if gate is not None else 1.0)
    out = (h if h is not None else 0.0) + t
    return out, (rms_norm(out, w_pre, eps) if w_pre is not None else None), t
