"""The block norm against the FP64 oracle.

Tolerances (t' = scale gate t, rounding unit u = 2^-24; a sum of squares is
nested at most 48 deep, so its relative error is below 48 u, half of that
after the root; rsqrtf and the products add less than 10 u: 34 u < 2^-18):
  h'  |err| <= E = 2^-18 |t'| + 2^-23 |h'|, and the rounding of its type
      (2^-8 |h'| for bf16)
  n   |err| <= (E + 2^-18 |h'|) |f w| + 2 |n| rms(E) / rms(h') and 2^-8 |n|,
      with f = 1 / sqrt(mean(h'^2) + eps)
MX4 output: the bits that mx4_quantize gives for n_out.
"""
import ctypes

import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from helpers import need_gpu
from oracle import blocks

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def make(M, H, h_t, gate, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    shape = {"none": None, "channel": (H,), "row": (1, H), "token": (M, 1), "full": (M, H)}[gate]
    d = dict(h=(3 * rnd(M, H)).to(DT[h_t]), y=(2 * rnd(M, H)).to(torch.bfloat16),
             w_post=(1 + 0.2 * rnd(H)).to(torch.bfloat16),
             w_pre=(1 + 0.2 * rnd(H)).to(torch.bfloat16),
             gate=None if shape is None else rnd(*shape).to(torch.bfloat16))
    return {k: None if v is None else v.to(device) for k, v in d.items()}


def f64(t):
    return None if t is None else t.cpu().double().numpy()


def reference(d, scale=1.0, eps=EPS, plus_one=0.0):
    w_post, w_pre = f64(d["w_post"]), f64(d["w_pre"])
    w_post = None if w_post is None else w_post + plus_one
    w_pre = None if w_pre is None else w_pre + plus_one
    h, n, t = blocks.block_norm(f64(d["h"]), f64(d["y"]), w_post, w_pre, f64(d["gate"]), scale,
                                eps)
    E = 2.0 ** -18 * np.abs(t) + 2.0 ** -23 * np.abs(h)
    En = None
    if n is not None:
        ms = (h ** 2).mean(-1, keepdims=True)
        f = 1.0 / np.sqrt(ms + eps)
        with np.errstate(divide="ignore", invalid="ignore"):
            spread = np.where(ms > 0, np.sqrt((E ** 2).mean(-1, keepdims=True) / ms), 0.0)
        En = (E + 2.0 ** -18 * np.abs(h)) * np.abs(f * w_pre) + 2 * np.abs(n) * spread + \
            2.0 ** -8 * np.abs(n)
    return h, n, E, En


def close(got, ref, tol):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def run(d, h_t, *, want=("h", "n"), codes=False, **kw):
    lead = d["h"] if d["h"] is not None else d["y"]
    M, H = lead.shape
    dev = lead.device
    out = {"h": torch.full((M, H), 99.0, dtype=DT[h_t], device=dev) if "h" in want else None,
           "n": torch.full((M, H), 99.0, dtype=torch.bfloat16, device=dev) if "n" in want else None}
    c = s = None
    if codes:
        c = torch.full((M, H // 2), 0xEE, dtype=torch.uint8, device=dev)
        s = torch.full((ig.mx4_scale_bytes(M, H),), 0xEE, dtype=torch.uint8, device=dev)
    ig.block_norm(d["h"], d["y"], d["w_post"], d["w_pre"], gate=d["gate"], h_out=out["h"],
                  n_out=out["n"], codes=c, scales=s, eps=kw.pop("eps", EPS), **kw)
    out["codes"], out["scales"] = c, s
    return out


def check(d, h_t, scale=1.0, **kw):
    o = run(d, h_t, scale=scale, **kw)
    h, n, E, En = reference(d, scale, plus_one=float(kw.get("flags", 0) == 1),
                            eps=kw.get("eps", EPS))
    if o["h"] is not None:
        close(o["h"], h, E + (2.0 ** -8 * np.abs(h) if h_t == "bf16" else 0))
    if o["n"] is not None:
        close(o["n"], n, En)
    return o


SIZES = [(1, 8), (1, 4096), (2, 16), (3, 248), (5, 256), (7, 264), (4, 2048), (9, 2056),
         (33, 4096), (2, 8192), (3, 8200), (2, 11008), (2, 16384), (2, 16392), (1, 32768),
         (129, 512), (700, 96)]


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "token", "full"])
@pytest.mark.parametrize("M,H", SIZES)
def test_equals_oracle(M, H, gate, h_t):
    need_gpu()
    check(make(M, H, h_t, gate, M + H), h_t, scale=0.75)


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
@pytest.mark.parametrize("drop", [("y", "w_post", "gate"), ("h",), ("w_post",), ("w_pre",),
                                  ("h", "w_post"), ("h", "gate", "w_pre"), ("gate", "w_post")])
def test_parts(drop, h_t):
    """Each part alone: only the norm before a block, only the one after, no
    residual, a plain residual."""
    need_gpu()
    for M, H in ((3, 264), (17, 4096)):
        d = make(M, H, h_t, "full", 40 + H)
        for k in drop:
            d[k] = None
        check(d, h_t, scale=-1.5, want=("h",) if d["w_pre"] is None else ("h", "n"))


@gpu
def test_weight_plus_one_and_outputs_left_out():
    need_gpu()
    d = make(5, 1024, "bf16", "channel", 3)
    check(d, "bf16", flags=ig.NORM_WEIGHT_PLUS_ONE)
    a = run(d, "bf16")
    assert torch.equal(run(d, "bf16", want=("n",))["n"], a["n"])
    d2 = dict(d, w_pre=None)
    assert torch.equal(run(d2, "bf16", want=("h",))["h"], a["h"])


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
@pytest.mark.parametrize("M,H", [(1, 32), (3, 96), (130, 4096), (2, 4128), (260, 352), (2, 32768)])
def test_codes_are_those_of_the_bf16_rows(M, H, h_t):
    need_gpu()
    d = make(M, H, h_t, "full", 77 + H)
    a = run(d, h_t, codes=True)
    b = run(d, h_t, want=("h",), codes=True)
    c = torch.full_like(a["codes"], 0xEE)
    s = torch.full_like(a["scales"], 0xEE)
    ig.mx4_quantize(a["n"], c, s)
    for o in (a, b):
        assert torch.equal(o["codes"], c) and torch.equal(o["scales"], s)
    assert torch.equal(a["h"], b["h"])
    assert torch.equal(a["n"], run(d, h_t)["n"])


@gpu
def test_rows_of_zeros_and_of_no_finite_sum():
    """Zero rows stay zero (eps > 0); a NaN or an infinity stays in its row."""
    need_gpu()
    d = make(6, 512, "f32", "none", 8)
    clean = run(d, "f32")
    d["h"][1] = 0
    d["y"][1] = 0
    d["y"][3, 100] = float("nan")
    d["h"][4, 5] = float("inf")
    o = run(d, "f32")
    assert not o["h"][1].any() and not o["n"][1].any()
    assert torch.isnan(o["h"][3]).all() and torch.isnan(o["n"][3]).all()
    assert torch.isinf(o["h"][4, 5])
    for r in (0, 2, 5):
        assert torch.equal(o["h"][r], clean["h"][r]) and torch.equal(o["n"][r], clean["n"][r])


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
def test_large_and_small_magnitudes(h_t):
    """Rows near 2^+-40: the squares stay inside FP32."""
    need_gpu()
    d = make(4, 1024, h_t, "none", 21)
    for r, e in enumerate((40, -40, 20, -20)):
        d["h"][r] *= 2.0 ** e
        d["y"][r] *= 2.0 ** e
    d["w_post"] = None
    check(d, h_t, eps=0.0)


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
def test_strides_and_in_place(h_t):
    need_gpu()
    M, H = 37, 520
    d = make(M, H, h_t, "full", 5)
    ref = run(d, h_t)
    wide = {k: torch.full((M, H + 88), 5.0, dtype=d[k].dtype, device="cuda")
            for k in ("h", "y", "gate")}
    e = dict(d)
    for k in wide:
        wide[k][:, 40:40 + H] = d[k]
        e[k] = wide[k][:, 40:40 + H]
    ig.block_norm(e["h"], e["y"], d["w_post"], d["w_pre"], gate=e["gate"], h_out=e["h"],
                  n_out=e["y"], eps=EPS)
    assert torch.equal(e["h"], ref["h"]) and torch.equal(e["y"], ref["n"])
    for k in wide:
        assert (wide[k][:, :40] == 5).all() and (wide[k][:, 40 + H:] == 5).all()
    # a gate broadcast by a zero stride is the gate of one row
    g = d["gate"][:1]
    a = run(dict(d, gate=g.expand(M, H)), h_t)
    b = run(dict(d, gate=g), h_t)
    assert torch.equal(a["h"], b["h"])
    t = d["gate"][:, :1].contiguous()
    a = run(dict(d, gate=t.expand(M, H)), h_t)
    b = run(dict(d, gate=t), h_t)
    assert torch.equal(a["h"], b["h"])


@gpu
@pytest.mark.parametrize("h_t", ["bf16", "f32"])
@pytest.mark.parametrize("H", [264, 4096, 11008])
def test_rows_do_not_depend_on_the_batch(H, h_t):
    need_gpu()
    big = make(3000, H, h_t, "full", H)
    ref = run(big, h_t)
    for M in (1, 2, 7, 64, 151, 500):
        d = {k: v if k.startswith("w") else v[:M].contiguous() for k, v in big.items()}
        o = run(d, h_t)
        assert torch.equal(o["h"], ref["h"][:M]) and torch.equal(o["n"], ref["n"][:M])


# --------------------------------------------------------------- refusals

FAKE = 1 << 20


def c_norm(M=4, H=64, lds=None, grs=64, gcs=1, t=0, flags=0, eps=1e-6, **over):
    p = dict(h=FAKE, y=FAKE, gate=FAKE, w_post=FAKE, w_pre=FAKE, h_out=FAKE, n_out=FAKE,
             codes=None, scales=None)
    p.update(over)
    lds = lds or (H,) * 4
    s = ig.NormShape(M, H, *lds, grs, gcs, t, flags, eps, 1.0)
    return ig.lib().ig_block_norm(ctypes.byref(s), *p.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=12), -2), (dict(H=0), -2), (dict(M=-1), -2), (dict(H=32776), -9),
    (dict(M=1 << 31), -9), (dict(t=2), -1), (dict(flags=2), -1), (dict(gcs=2), -1),
    (dict(grs=60), -2), (dict(grs=-8), -2), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(h=None, y=None, gate=None, w_post=None), -1), (dict(y=None), -1),
    (dict(h_out=None, n_out=None), -1), (dict(w_pre=None), -1), (dict(n_out=None), -1),
    (dict(codes=FAKE), -1), (dict(H=72, codes=FAKE, scales=FAKE, grs=72), -2),
    (dict(lds=(56, 64, 64, 64)), -2), (dict(lds=(64, 68, 64, 64)), -2),
    (dict(lds=(64, 64, 32, 64)), -2), (dict(lds=(64, 64, 64, 60)), -2),
    (dict(h=FAKE + 8), -3), (dict(w_post=FAKE + 2), -3), (dict(n_out=FAKE + 4), -3)])
def test_refusals(kw, code):
    assert c_norm(**kw) == code


def test_no_rows_is_a_no_op():
    assert c_norm(M=0) == 0
    assert c_norm(M=0, h=None, y=None, gate=None, h_out=None, n_out=None) == 0


@gpu
def test_empty_tensors():
    need_gpu()
    d = make(0, 64, "bf16", "full", 1)
    o = run(d, "bf16", codes=True)
    assert o["h"].shape == (0, 64)
    assert run(make(0, 64, "f32", "token", 1), "f32")["n"].shape == (0, 64)


def test_binding_refuses_wrong_tensors():
    d = make(4, 64, "bf16", "none", 1, device="cpu")
    h, y, w = d["h"], d["y"], d["w_pre"]
    for bad in (lambda: ig.block_norm(None, None, None, w, n_out=h.clone()),
                lambda: ig.block_norm(h.half(), y, w, w, n_out=h.clone()),
                lambda: ig.block_norm(h, y[:3], w, w, n_out=h.clone()),
                lambda: ig.block_norm(h, y, w[:32], w, n_out=h.clone()),
                lambda: ig.block_norm(h, y, w.float(), w, n_out=h.clone()),
                lambda: ig.block_norm(h, y, w, w, n_out=h.float()),
                lambda: ig.block_norm(h, y, w, w, n_out=h.clone(), h_out=h.float()),
                lambda: ig.block_norm(h, y, w, w, n_out=h.clone(), gate=h[:, :32]),
                lambda: ig.block_norm(h, y, w, w, n_out=h.clone(), gate=h[:3]),
                lambda: ig.block_norm(h, y, w, w, n_out=h.clone(), gate=h.float()),
                lambda: ig.block_norm(h, y, w, w, codes=torch.zeros(4, 32, dtype=torch.uint8)),
                lambda: ig.block_norm(h, y, w, w, n_out=h.clone())):   # not on a GPU
        with pytest.raises(ig.IGError):
            bad()
