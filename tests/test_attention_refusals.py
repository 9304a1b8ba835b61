"""What the attention calls refuse before anything is enqueued: by the library's own
checks (no call here reaches a launch) and by the binding's, for operands that are on a
GPU as far as it can see."""
import ctypes

import pytest
import torch

import invariant_gemm_gb300 as ig
from test_block_binding import library, on  # noqa: F401  (fixture)

U8, B16, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
FAKE = 0x100000        # never dereferenced
ARG, SHAPE, ALIGN, SMALL, UNSUPPORTED = -1, -2, -3, -4, -9
BIG = 1 << 62


def rope(T=4, table=100, ld_q=512, ld_k=256, ld_qo=512, ld_ko=256, hq=4, hk=2, D=128, rot=128,
         flags=0, eps=1e-6):
    return ig._ROPE_SHAPE(T, table, ld_q, ld_k, ld_qo, ld_ko, hq, hk, D, rot, flags, eps)


def cache(codes=FAKE, scales=FAKE, pages=8, ps=None, ss=None, page=16, heads=2, D=128, reserved=0):
    ps = 2 * heads * page * D if ps is None else ps
    ss = 2 * heads * page // 16 if ss is None else ss
    return ig._KV_CACHE(codes, scales, pages, ps, ss, page, heads, D, reserved)


def batch(cu=FAKE, kv=FAKE, table=FAKE, cols=4, B=2, max_q=4):
    return ig._BATCH(cu, kv, table, cols, B, max_q)


def attn(T=4, ld_q=512, ld_o=512, hq=4, flags=0, scale=0.1, reserved=0):
    return ig._ATTN_SHAPE(T, ld_q, ld_o, hq, flags, scale, reserved)


def call_qk(shape=None, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, cs=FAKE, pos=FAKE, qo=FAKE, ko=FAKE,
            ws=FAKE, n=BIG):
    return ig.lib().ig_qk_norm_rope(rope() if shape is None else shape, q, k, wq, wk, cs, pos, qo,
                                    ko, ws, n, None)


def call_append(shape=None, c=None, b=None, k=FAKE, v=FAKE, ld_v=256, q=FAKE, wq=FAKE, wk=FAKE,
                cs=FAKE, pos=FAKE, qo=FAKE, ws=FAKE, n=BIG):
    return ig.lib().ig_kv_append(rope() if shape is None else shape, cache() if c is None else c,
                                 batch() if b is None else b, k, v, ld_v, q, wq, wk, cs, pos, qo,
                                 ws, n, None)


def call_gather(c=None, b=None, T=4, k=FAKE, ld_k=256, v=FAKE, ld_v=256, ws=FAKE, n=BIG):
    return ig.lib().ig_kv_gather(cache() if c is None else c, batch() if b is None else b, T, k,
                                 ld_k, v, ld_v, ws, n, None)


def call_attn(shape=None, c=None, b=None, q=FAKE, out=2 * FAKE, ws=FAKE, n=BIG):
    return ig.lib().ig_paged_attention(attn() if shape is None else shape,
                                       cache() if c is None else c, batch() if b is None else b, q,
                                       out, ws, n, None)


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(q=None, k=None, qo=None, ko=None, wq=None, wk=None)), (ARG, dict(qo=None)),
    (ARG, dict(ko=None)), (ARG, dict(q=None)), (ARG, dict(pos=None)), (ARG, dict(cs=None)),
    (ARG, dict(ws=None)), (ARG, dict(shape=rope(flags=4))), (ARG, dict(shape=rope(eps=-1.0))),
    (ARG, dict(shape=rope(eps=float("nan")))),
    (SHAPE, dict(shape=rope(T=-1))), (SHAPE, dict(shape=rope(hq=0))),
    (SHAPE, dict(shape=rope(rot=24))), (SHAPE, dict(shape=rope(rot=144))),
    (SHAPE, dict(shape=rope(rot=0))), (SHAPE, dict(shape=rope(table=0))),
    (SHAPE, dict(shape=rope(ld_q=504))), (SHAPE, dict(shape=rope(ld_k=260))),
    (SHAPE, dict(shape=rope(ld_qo=516))), (SHAPE, dict(shape=rope(ld_ko=128))),
    (SHAPE, dict(shape=rope(ld_qo=1024), qo=FAKE)),         # in place, another stride
    (UNSUPPORTED, dict(shape=rope(D=96))), (UNSUPPORTED, dict(shape=rope(D=256, ld_q=1024))),
    (UNSUPPORTED, dict(shape=rope(T=(1 << 30) + 1))),
    (ALIGN, dict(q=FAKE + 8)), (ALIGN, dict(cs=FAKE + 8)), (ALIGN, dict(pos=FAKE + 2)),
    (ALIGN, dict(ko=FAKE + 2)), (ALIGN, dict(wq=FAKE + 4)), (ALIGN, dict(ws=FAKE + 4)),
    (SMALL, dict(n=100)),
])
def test_qk_norm_rope(code, kw):
    assert call_qk(**kw) == code


CACHES = [
    (ARG, dict(codes=0)), (ARG, dict(scales=0)), (ARG, dict(reserved=1)),
    (SHAPE, dict(page=8)), (SHAPE, dict(page=48)), (SHAPE, dict(pages=0)), (SHAPE, dict(ps=100)),
    (SHAPE, dict(ps=2 * 2 * 16 * 128 + 8)), (SHAPE, dict(ss=3)), (SHAPE, dict(heads=0)),
    (UNSUPPORTED, dict(page=512)), (UNSUPPORTED, dict(D=192)), (ALIGN, dict(codes=FAKE + 8)),
    (UNSUPPORTED, dict(pages=1 << 33)), (UNSUPPORTED, dict(ps=1 << 41)),
]
BATCHES = [
    (ARG, dict(cu=0)), (ARG, dict(kv=0)), (ARG, dict(table=0)), (SHAPE, dict(B=-1)),
    (SHAPE, dict(max_q=-1)), (SHAPE, dict(cols=0)), (UNSUPPORTED, dict(B=8193)),
    (ALIGN, dict(cu=FAKE + 2)), (ALIGN, dict(table=FAKE + 1)),
]


@pytest.mark.parametrize("code,kw", CACHES)
@pytest.mark.parametrize("call", [call_append, call_gather, call_attn])
def test_caches(call, code, kw):
    assert call(c=cache(**kw)) == code


@pytest.mark.parametrize("code,kw", BATCHES)
@pytest.mark.parametrize("call", [call_append, call_gather, call_attn])
def test_batches(call, code, kw):
    assert call(b=batch(**kw)) == code


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(k=None)), (ARG, dict(v=None)), (ARG, dict(q=None)), (ARG, dict(qo=None)),
    (ARG, dict(cs=None)), (SHAPE, dict(ld_v=128)), (SHAPE, dict(ld_v=260)),
    (SHAPE, dict(shape=rope(hk=3, ld_k=384))), (SHAPE, dict(shape=rope(D=64))),
    (ALIGN, dict(v=FAKE + 8)), (SMALL, dict(n=0)), (ARG, dict(ws=None)),
    (UNSUPPORTED, dict(shape=rope(T=1 << 30), b=batch(B=8192, max_q=1 << 30))),
])
def test_kv_append(code, kw):
    assert call_append(**kw) == code


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(k=None)), (ARG, dict(v=None)), (SHAPE, dict(ld_k=128)), (SHAPE, dict(ld_v=257)),
    (SHAPE, dict(T=-1)), (ALIGN, dict(k=FAKE + 8)), (SMALL, dict(n=16)), (ARG, dict(ws=None)),
])
def test_kv_gather(code, kw):
    assert call_gather(**kw) == code


@pytest.mark.parametrize("code,kw", [
    (ARG, dict(q=None)), (ARG, dict(out=None)), (ARG, dict(out=FAKE)), (ARG, dict(ws=None)),
    (ARG, dict(shape=attn(flags=1))), (ARG, dict(shape=attn(reserved=1))),
    (ARG, dict(shape=attn(scale=float("inf")))), (ARG, dict(shape=attn(scale=float("nan")))),
    (SHAPE, dict(shape=attn(hq=5, ld_q=640, ld_o=640))), (SHAPE, dict(shape=attn(ld_q=256))),
    (SHAPE, dict(shape=attn(ld_o=516))), (SHAPE, dict(shape=attn(T=-2))),
    (ALIGN, dict(q=FAKE + 4)), (ALIGN, dict(out=FAKE + 8)), (SMALL, dict(n=1 << 18)),
    (UNSUPPORTED, dict(shape=attn(T=1 << 30, hq=1024, ld_q=1 << 17, ld_o=1 << 17),
                       c=cache(heads=1, ps=4096, ss=2))),
    (UNSUPPORTED, dict(b=batch(max_q=(1 << 28) + 1))),
    (UNSUPPORTED, dict(b=batch(cols=1 << 24), c=cache(page=256, ps=1 << 20, ss=1 << 10))),
])
def test_paged_attention(code, kw):
    assert call_attn(**kw) == code


def test_workspace_bytes():
    """Grows with the sequences, new tokens and pages; enough for a smaller call."""
    size = lambda **kw: ig.lib().ig_attention_workspace_bytes(  # noqa: E731
        attn(T=kw.pop("T", 4)), cache(codes=0, scales=0, pages=0, ps=0, ss=0), batch(0, 0, 0, **kw))
    assert 0 < size(B=1) < size(B=2) < size(B=2, cols=400) < size(B=2, cols=400, max_q=40, T=80)
    assert size(B=2, max_q=200, T=400) >= size(B=2, max_q=100, T=200)
    assert ig.lib().ig_attention_workspace_bytes(attn(hq=3), cache(), batch()) == 0
    assert ig.lib().ig_attention_workspace_bytes(None, cache(), batch()) == 0
    s = size(B=2)
    assert call_attn(b=batch(B=2), n=s - 1) == SMALL


def test_nothing_to_do():
    """No tokens, no sequences: no operands are looked at."""
    assert call_qk(shape=rope(T=0), q=None, k=None, wq=None, wk=None, cs=None, pos=None, qo=None,
                   ko=None, ws=None, n=0) == 0
    assert call_append(shape=rope(T=0), k=None, v=None, q=None, wq=None, wk=None, cs=None, pos=None,
                       qo=None, ws=None, n=0) == 0
    assert call_append(b=batch(0, 0, 0, B=0), k=None, v=None, wk=None, q=None, wq=None, qo=None,
                       ws=None, n=0) == 0
    assert call_gather(T=0, k=None, v=None, ws=None, n=0) == 0
    assert call_attn(shape=attn(T=0), q=None, out=None, ws=None, n=0) == 0
    assert call_attn(b=batch(0, 0, 0, B=0), q=None, out=None, ws=None, n=0) == 0


# --- the binding --------------------------------------------------------------------

def operands():
    z = lambda *s, t=B16: on(torch.zeros(*s, dtype=t))  # noqa: E731
    return dict(q=z(4, 4, 128), k=z(4, 2, 128), v=z(4, 2, 128), qo=z(4, 4, 128), ko=z(4, 2, 128),
                w=z(128), cs=z(10, 128, t=F32), pos=z(4, t=I32), cache=z(3, 2, 2, 16, 128, t=U8),
                scales=z(3, 2, 2, 1, t=U8), cu=z(3, t=I32), kv=z(2, t=I32), table=z(2, 4, t=I32),
                ws=z(1 << 20, t=U8))


CALLS = {
    "qk_norm_rope": lambda o, **k: ig.qk_norm_rope(
        o["q"], o["k"], o["qo"], o["ko"], o["ws"], w_q=o["w"], w_k=o["w"], cos_sin=o["cs"],
        positions=o["pos"], **k),
    "kv_append": lambda o, **k: ig.kv_append(
        o["k"], o["v"], o["cache"], o["scales"], o["cu"], o["kv"], o["table"], o["ws"], w_k=o["w"],
        cos_sin=o["cs"], positions=o["pos"], q=o["q"], q_out=o["qo"], w_q=o["w"], **k),
    "kv_gather": lambda o, **k: ig.kv_gather(
        o["cache"], o["scales"], o["cu"], o["kv"], o["table"], o["ko"], o["v"], o["ws"], **k),
    "paged_attention": lambda o, **k: ig.paged_attention(
        o["q"], o["cache"], o["scales"], o["cu"], o["kv"], o["table"], o["qo"], o["ws"], **k),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, 0])
def test_operands_on_a_gpu_that_is_not_current(library, name, stream):  # noqa: F811
    CALLS[name](operands(), stream=stream)
    assert library.calls == ["ig_" + name]
    library.current = 0
    with pytest.raises(ig.IGError) as e:
        CALLS[name](operands(), stream=stream)
    assert e.value.code == -1 and "GPU 1" in str(e.value) and "GPU 0" in str(e.value)
    assert library.calls == ["ig_" + name]


def _z(*s, t=B16):
    return on(torch.zeros(*s, dtype=t))


@pytest.mark.parametrize("name,change", [
    ("qk_norm_rope", dict(q=_z(4, 512))), ("qk_norm_rope", dict(q=_z(4, 4, 128, t=F32))),
    ("qk_norm_rope", dict(qo=_z(4, 4, 64))), ("qk_norm_rope", dict(qo=_z(5, 4, 128))),
    ("qk_norm_rope", dict(k=_z(3, 2, 128))), ("qk_norm_rope", dict(k=_z(4, 2, 64))),
    ("qk_norm_rope", dict(q=_z(4, 128, 4).transpose(1, 2))),
    ("qk_norm_rope", dict(q=_z(4, 8, 128)[:, ::2])), ("qk_norm_rope", dict(w=_z(64))),
    ("qk_norm_rope", dict(pos=_z(5, t=I32))), ("qk_norm_rope", dict(pos=_z(4, t=torch.int64))),
    ("qk_norm_rope", dict(cs=_z(10, 128))), ("qk_norm_rope", dict(cs=_z(10, 256, t=F32)[:, ::2])),
    ("qk_norm_rope", dict(ws=_z(1 << 20))), ("qk_norm_rope", dict(q=torch.zeros(4, 4, 128).to(B16))),
    ("kv_append", dict(v=_z(4, 3, 128))), ("kv_append", dict(k=_z(4, 3, 128), v=_z(4, 3, 128))),
    ("kv_append", dict(q=_z(5, 4, 128))), ("kv_append", dict(cache=_z(3, 2, 2, 16, 128))),
    ("kv_append", dict(cache=_z(3, 1, 2, 16, 128, t=U8))),
    ("kv_append", dict(cache=_z(3, 2, 2, 16, 256, t=U8)[..., ::2])),
    ("kv_append", dict(scales=_z(3, 2, 2, 2, t=U8))), ("kv_append", dict(scales=_z(2, 2, 2, 1, t=U8))),
    ("kv_append", dict(cu=_z(2, t=I32))), ("kv_append", dict(kv=_z(3, t=I32))),
    ("kv_append", dict(table=_z(2, 8, t=I32)[:, ::2])), ("kv_append", dict(table=_z(8, t=I32))),
    ("kv_gather", dict(ko=_z(4, 2, 64))), ("kv_gather", dict(v=_z(3, 2, 128))),
    ("paged_attention", dict(q=_z(4, 4, 64), qo=_z(4, 4, 64))),
    ("paged_attention", dict(qo=_z(4, 3, 128))), ("paged_attention", dict(cu=_z(3, t=torch.int64))),
])
def test_operands_of_another_kind(library, name, change):  # noqa: F811
    o = operands()
    o.update(change)
    with pytest.raises(ig.IGError) as e:
        CALLS[name](o)
    assert e.value.code in (-1, -2) and library.calls == []


def test_pairs_of_operands(library):  # noqa: F811
    o = operands()
    for args in ((o["q"], None, None, None), (None, o["k"], None, None), (None,) * 4):
        with pytest.raises(ig.IGError):
            ig.qk_norm_rope(*args, o["ws"])
    with pytest.raises(ig.IGError):
        ig.kv_append(o["k"], o["v"], o["cache"], o["scales"], o["cu"], o["kv"], o["table"],
                     o["ws"], q=o["q"])
    assert library.calls == []


def test_structs_match_the_header():
    """Sizes as a C compiler lays them out (8-byte alignment, no tail padding lost)."""
    assert len(rope()) == 72 and len(cache()) == 56 and len(batch()) == 40 and len(attn()) == 40
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_workspace_follows_the_rows():
    """Not every sequence can have the most new tokens: 256 sequences, 64 query and 8 kv heads
    of 128, tables of 65536 tokens."""
    def size(T, max_q, B=256):
        return ig.lib().ig_attention_workspace_bytes(
            attn(T=T, hq=64, ld_q=8192, ld_o=8192),
            cache(codes=0, scales=0, pages=0, ps=0, ss=0, page=64, heads=8), batch(
                0, 0, 0, cols=1024, B=B, max_q=max_q))

    row = 4 * (128 + 4)                         # of a part: sums, maximum, sum of weights

    def close(got, rows):
        assert rows * row <= got <= rows * row + (1 << 20)

    close(size(256, 1), 256 * 8 * 64 * 8)       # single tokens: 8 rows in 64 parts of 8 heads
    # no bound on new tokens given: tiles of 16 rows as 256 sequences of 2048 rows can fill them,
    # 152 items for the prompts' rows
    close(size(256, 256), (256 + 128) * 8 * 64 * 16 + 2048 * 152)
    close(size(2304, 2048), 256 * 4 * 8 * 64 * 16 + 2304 * 8 * 152)
    close(size(2304, 2048, 16), 16 * 4 * 8 * 64 * 16 + 16 * 256 * 152)
