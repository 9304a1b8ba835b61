"""Head norms with the rotation, and the 8-bit paged cache, against FP64."""
import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from attention_helpers import B16, I32, Batch, f64
from helpers import need_gpu
from oracle import attention as ref

pytestmark = pytest.mark.gpu
EPS = 1e-6


def table(rows, rot):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def near(got, want):
    """bf16 (half a step: 2^-8) of a value whose FP32 steps (squares, their sum, the
    root, two products, a rotation of two products) leave at most 2^-20 of the
    pair's size, bounded by the head's largest value."""
    got = f64(got)
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all()
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(want).max(-1, keepdims=True)
    assert (np.abs(got - want) <= tol)[~nan].all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 40, 8), (3, 5, 0), (70, 12, 2), (2000, 33, 3)])
@pytest.mark.parametrize("rot,inter,plus", [(16, False, False), (64, False, True), (64, True, False),
                                            (48, True, True), (32, False, False), (0, False, True)])
def test_norm_and_rotation(D, T, hq, hk, rot, inter, plus):
    need_gpu()
    rng = np.random.default_rng(T + hq)
    rot = D if rot == 64 and D == 128 else rot
    x = torch.from_numpy(rng.standard_normal((T, hq + hk, D)) * 3).to(torch.float32).to(B16).cuda()
    x[0, 0] = 0
    q, k = x[:, :hq], x[:, hq:] if hk else None
    w = torch.from_numpy(rng.standard_normal((2, D))).to(B16).cuda()
    cs = table(5000, rot) if rot else None
    pos = rng.integers(0, 5000, T).astype(np.int32)
    kw = dict(w_q=w[0], w_k=w[1] if hk else None, eps=EPS,
              flags=(ig.NORM_WEIGHT_PLUS_ONE if plus else 0) | (ig.ROPE_INTERLEAVED if inter else 0))
    if rot:
        kw.update(cos_sin=torch.from_numpy(cs).cuda(), positions=torch.from_numpy(pos).cuda())
    ws = ig.mx4_workspace()
    out = torch.full((T, hq + hk + 1, D), 7.0, dtype=B16, device="cuda")
    ko = out[:, hq:hq + hk] if hk else None
    ig.qk_norm_rope(q, k, out[:, :hq], ko, ws, **kw)
    assert ig.check_status(ws) == 0
    near(out[:, :hq], ref.norm_rope(f64(q), f64(w[0]), cs, pos, EPS, inter, plus))
    if hk:
        near(ko, ref.norm_rope(f64(k), f64(w[1]), cs, pos, EPS, inter, plus))
    assert (out[:, hq + hk:] == 7).all()
    # in place, one side normed only
    kw.update(w_q=None)
    y = x.clone()
    ig.qk_norm_rope(y[:, :hq], y[:, hq:] if hk else None, y[:, :hq], y[:, hq:] if hk else None, ws,
                    **kw)
    near(y[:, :hq], ref.norm_rope(f64(q), None, cs, pos, EPS, inter, plus))
    if hk:
        assert torch.equal(y[:, hq:], ko)


def test_positions_outside_the_table():
    need_gpu()
    x = torch.randn(6, 3, 64, device="cuda").to(B16)
    cs = torch.from_numpy(table(10, 64)).cuda()
    pos = torch.tensor([0, 9, 10, -1, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda")
    ws = ig.mx4_workspace()
    out = torch.zeros_like(x)
    ig.qk_norm_rope(x, None, out, None, ws, cos_sin=cs, positions=pos)
    assert ig.check_status(ws) == -10 and ig.check_status(ws) == 0
    nan = out.isnan().all(-1).all(-1).cpu().numpy()
    assert (nan == [False, False, True, True, True, False]).all()


class Append:
    """One kv_append on the device and in the oracle, from the same cache."""

    def __init__(self, b, k, v, w=None, cs=None, pos=None, q=None, w_q=None, inter=False, **kw):
        self.b = b
        self.codes, self.scales = b.codes.copy(), b.scales.copy()
        args = b.device_args()
        self.args = args
        ws = ig.mx4_workspace()
        dev = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.q_out = None if q is None else torch.full(q.shape, 7.0, dtype=B16, device="cuda")
        ig.kv_append(k.cuda(), v.cuda(), *args, ws, w_k=dev(w), q=dev(q), q_out=self.q_out,
                     w_q=dev(w_q), cos_sin=None if cs is None else torch.from_numpy(cs).cuda(),
                     positions=None if pos is None else torch.from_numpy(pos).cuda(), eps=EPS,
                     max_q=b.max_q, flags=ig.ROPE_INTERLEAVED if inter else 0, **kw)
        self.status = ig.check_status(ws)
        at = np.concatenate([np.arange(kv - n, kv) for n, kv in b.lengths]) if pos is None else pos
        kk = ref.norm_rope(f64(k), None if w is None else f64(w), cs, at, EPS, inter)
        self.k = kk
        for s, (n, kv) in enumerate(b.lengths):
            r = slice(b.cu[s], b.cu[s + 1])
            ref.append(self.codes, self.scales, kk[r], b.table[s], kv - n, 0)
            ref.append(self.codes, self.scales, f64(v)[r], b.table[s], kv - n, 1)

    def same(self, keys_exact):
        codes, scales = self.args[0].cpu().numpy(), self.args[1].cpu().numpy()
        assert (scales == self.scales).all()
        sides = slice(0, 2) if keys_exact else slice(1, 2)
        assert (codes[:, sides] == self.codes[:, sides]).all()
        if not keys_exact:
            # FP32 keys may fall on the other side of a border between two codes
            a, b = codes[:, 0].astype(int), self.codes[:, 0].astype(int)
            off = a != b
            assert (np.abs(a - b)[off] == 1).all() and off.sum() <= 2e-5 * off.size + 2


@pytest.mark.parametrize("D,page", [(128, 16), (64, 32), (128, 256), (64, 128)])
@pytest.mark.parametrize("lengths", [
    [(1, kv) for kv in (1, 2, 15, 16, 17, 31, 32, 33, 100)],
    [(5, 5), (0, 9), (16, 16), (17, 40), (33, 33), (2, 17), (31, 47), (300, 333)],
])
def test_append_without_rotation(D, page, lengths):
    """Codes and scales to the last bit: values from bf16, some of them zeros, far
    apart in size, infinite or NaN; bytes of no new token stay."""
    need_gpu()
    b = Batch(lengths, 4, 3, D, page, seed=page)
    rng = b.rng
    k, v = b.rows(3), b.rows(3)
    for t in (k, v):
        t *= torch.from_numpy(2.0 ** rng.integers(-30, 30, (b.T, 3, 1))).to(B16)
        t[rng.random(tuple(t.shape)) < 0.02] = 0
        t[b.T // 2, 1, 5] = float("inf")
        t[b.T // 2, 2, 6:9] = float("nan")
        t[0, 0] = 0
        t[-1, 2] = 3e38
        t[-1, 1] = 1e-39
    a = Append(b, k, v)
    assert a.status == 0
    a.same(True)


@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, True), (128, 64, False)])
def test_append_with_norm_and_rotation(D, rot, inter):
    need_gpu()
    b = Batch([(1, 50), (40, 40), (100, 777), (1, 1), (7, 20)], 6, 2, D, 32, seed=rot)
    k, v, q = b.rows(2, 2.0), b.rows(2), b.rows(6)
    w = torch.from_numpy(b.rng.standard_normal((2, D))).to(B16)
    pos = b.rng.integers(0, 1000, b.T).astype(np.int32)
    cs = table(1000, rot)
    for kw in (dict(w=w[0], cs=cs, pos=pos, q=q, w_q=w[1], inter=inter), dict(w=w[0]),
               dict(cs=cs, q=q, inter=inter)):
        a = Append(b, k, v, **kw)
        assert a.status == 0
        a.same(False)
        if a.q_out is not None:
            at = kw.get("pos")
            if at is None:
                at = np.concatenate([np.arange(m - n, m) for n, m in b.lengths])
            near(a.q_out, ref.norm_rope(f64(q), f64(w[1]) if "w_q" in kw else None, cs, at, EPS,
                                        inter))


def test_append_one_by_one_grows_the_scale():
    """Sixteen tokens of growing and falling size into one block, one call each:
    every byte as the oracle has it after each call."""
    need_gpu()
    sizes = [0.1, 0.01, 3.0, 2.0, 500.0, 0.5, 1e5, 1.0, 1e5, 3e6, 1e-9, 0.0, 7.0, 1e9, 1e3, 2e9]
    codes = scales = None
    for j, size in enumerate(sizes):
        b = Batch([(1, 32 + j + 1)], 1, 2, 64, 16, seed=3)
        if codes is not None:
            b.codes, b.scales = codes, scales
        rng = np.random.default_rng(j)
        x = [torch.from_numpy(rng.standard_normal((1, 2, 64)) * size).float().to(B16)
             for _ in range(2)]
        # scales of an unused block mean nothing
        a = Append(b, *x)
        a.same(True)
        codes, scales = a.codes, a.scales


def test_one_by_one_and_at_once():
    """The same scales, and the same codes but for values under 2^-6 of the scale."""
    need_gpu()
    n = 40
    b = Batch([(n, n)], 1, 2, 128, 16, seed=4)
    k, v = b.rows(2), b.rows(2, 5.0)
    at_once = Append(b, k, v)
    one = Batch([(n, n)], 1, 2, 128, 16, seed=4)
    args = one.device_args()
    ws = ig.mx4_workspace()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for j in range(n):
        kv = torch.tensor([j + 1], dtype=torch.int32, device="cuda")
        ig.kv_append(k[j:j + 1].cuda(), v[j:j + 1].cuda(), args[0], args[1], cu, kv, args[4], ws)
    assert ig.check_status(ws) == 0
    assert torch.equal(args[1], at_once.args[1])
    a, c = args[0].cpu().numpy(), at_once.args[0].cpu().numpy()
    off = a != c
    assert ((a[off] & 127) < 8 + 1).all()
    assert (np.abs(a[off].astype(int) - c[off].astype(int)) <= 1).all()


def test_append_leaves_other_bytes_and_reports():
    need_gpu()
    b = Batch([(3, 40), (2, 20), (5, 3), (4, 18)], 2, 2, 64, 16, seed=5)
    k, v = b.rows(2), b.rows(2)
    before = b.codes.copy()
    b.table[1, 1] = b.pages + 7                       # the second sequence's new tokens
    args = b.device_args()
    ws = ig.mx4_workspace()
    ig.kv_append(k.cuda(), v.cuda(), *args, ws, max_q=b.max_q)
    assert ig.check_status(ws) == -10
    codes = args[0].cpu().numpy()
    touched = np.zeros(codes.shape[:1] + codes.shape[3:4], dtype=bool)
    for s, (n, kv) in enumerate(b.lengths):
        if s != 1:
            for j in range(max(kv - n, 0) // 16 * 16, kv):    # older tokens may be scaled again
                touched[b.table[s, j // 16], j % 16] = True
    assert (codes == before).transpose(0, 3, 1, 2, 4)[~touched].all()
    # more new tokens than there are in all: the first of them are not in it
    kk = f64(k)[b.cu[2] + 2:b.cu[3]]
    codes2, scales2 = b.codes.copy(), b.scales.copy()
    ref.append(codes2, scales2, kk, b.table[2], 0, 0)
    pg = b.table[2, 0]
    assert (codes[pg, 0, :, :3] == codes2[pg, 0, :, :3]).all()


@pytest.mark.parametrize("D,page", [(128, 16), (64, 256)])
def test_gather(D, page):
    """Exact, any number of last tokens, rows of no sequence left as they were."""
    need_gpu()
    b = Batch([(5, 5), (0, 9), (33, 60), (1, 1), (9, 4)], 2, 3, D, page, seed=6).fill()
    args = b.device_args()
    ko = torch.full((b.T + 4, 5, D), 7.0, dtype=B16, device="cuda")
    vo = torch.full((b.T + 4, 3, D), 7.0, dtype=B16, device="cuda")
    ws = ig.mx4_workspace()
    ig.kv_gather(*args, ko[:, 1:4], vo, ws)
    assert ig.check_status(ws) == 0
    want = []
    for s, (n, kv) in enumerate(b.lengths):
        x = ref.held(b.codes, b.scales, b.table[s], kv)
        pad = np.zeros((2, max(0, n - kv), 3, D))
        want.append(np.concatenate([pad, x[:, max(0, kv - n):]], 1))
    want = np.concatenate(want, 1)
    assert (f64(ko[:b.T, 1:4]) == want[0]).all() and (f64(vo[:b.T]) == want[1]).all()
    assert (ko[b.T:] == 7).all() and (vo[b.T:] == 7).all() and (ko[:, 0] == 7).all()


def test_every_code_and_scale_reads_back():
    need_gpu()
    b = Batch([(256, 256)], 1, 1, 64, 256, seed=7)
    b.codes[:] = np.arange(256).reshape(256, 1).astype(np.uint8)
    b.scales[:] = np.array([0, 1, 2, 7, 60, 100, 126, 127, 128, 129, 150, 200, 240, 246, 247, 255])
    args = b.device_args()
    ko, vo = (torch.empty(256, 1, 64, dtype=B16, device="cuda") for _ in range(2))
    ig.kv_gather(*args, ko, vo, ig.mx4_workspace())
    x = ref.held(b.codes, b.scales, b.table[0], 256)
    want = torch.from_numpy(x[0]).to(B16).double().numpy()
    np.testing.assert_array_equal(f64(ko), want)


def test_pools_of_more_than_4_gb_and_strides():
    need_gpu()
    b = Batch([(20, 50), (1, 17)], 2, 2, 128, 16, seed=8)
    k, v = b.rows(2), b.rows(2)
    a = Append(b, k, v)
    codes, scales, cu, kv, tab = b.device_args()
    far = (5 << 30) // (3 * codes[0].numel())
    n = far + b.pages
    pool = torch.zeros(n, 3, *codes.shape[1:], dtype=torch.uint8, device="cuda")[:, 1]
    spool = torch.zeros(n, 2, *scales.shape[1:], dtype=torch.uint8, device="cuda")[:, 1]
    pool[far:], spool[far:] = codes, scales
    ws = ig.mx4_workspace()
    qkv = torch.zeros(b.T, 6, 128, dtype=B16, device="cuda")
    qkv[:, 2:4], qkv[:, 4:] = k.cuda(), v.cuda()
    ig.kv_append(qkv[:, 2:4], qkv[:, 4:], pool, spool, cu, kv, tab + far, ws, max_q=b.max_q)
    assert ig.check_status(ws) == 0
    assert (pool[far:].cpu().numpy() == a.codes).all()
    assert (spool[far:].cpu().numpy() == a.scales).all()
    assert not pool[:far].any() and not spool[:far].any()


@pytest.mark.parametrize("D,n", [(128, 1), (128, 2), (64, 20)])
def test_append_and_gather_at_the_last_positions(D, n):
    """A sequence of 2^31 - 1 tokens, the most that a length can say, with blocks of another
    sequence's count behind its last one: only its own block is written, and reads back."""
    need_gpu()
    kv, page, cols = 2 ** 31 - 1, 256, 1 << 23
    b = Batch([(n, n), (150, 150)], 2, 2, D, page, seed=50)
    k, v = b.rows(2), b.rows(2)
    tables = [{cols - 1: int(b.table[0, 0])}, {0: int(b.table[1, 0])}]
    table = torch.zeros(2, cols, dtype=I32, device="cuda")
    table[0, -1], table[1, 0] = tables[0][cols - 1], tables[1][0]
    codes, scales, cu, _, _ = b.device_args()
    lengths = torch.tensor([kv, 150], dtype=I32, device="cuda")
    ws = ig.mx4_workspace()
    for max_q in ((150, None) if n > 1 else (150,)):
        codes.copy_(torch.from_numpy(b.codes))
        scales.copy_(torch.from_numpy(b.scales))
        ig.kv_append(k.cuda(), v.cuda(), codes, scales, cu, lengths, table, ws, max_q=max_q)
        assert ig.check_status(ws) == 0
        want_c, want_s = b.codes.copy(), b.scales.copy()
        for s, first in ((0, kv - n), (1, 0)):
            for side, x in ((0, k), (1, v)):
                ref.append(want_c, want_s, f64(x)[b.cu[s]:b.cu[s + 1]], tables[s], first, side)
        assert (codes.cpu().numpy() == want_c).all() and (scales.cpu().numpy() == want_s).all()
    ko, vo = (torch.zeros(b.T, 2, D, dtype=B16, device="cuda") for _ in range(2))
    ig.kv_gather(codes, scales, cu, lengths, table, ko, vo, ws)
    assert ig.check_status(ws) == 0
    for side, got in ((0, ko), (1, vo)):
        page_of, at = tables[0][cols - 1], np.arange(page - 1 - n, page - 1)
        unit = 2.0 ** (want_s[page_of, side][:, at // 16].astype(int) - 127.0)
        want = ref.decode(want_c[page_of, side][:, at]) * unit[..., None]
        np.testing.assert_array_equal(f64(got)[:n], want.transpose(1, 0, 2))
