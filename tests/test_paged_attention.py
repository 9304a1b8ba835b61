"""Attention over the 8-bit paged cache against FP64 from the held values."""
import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from attention_helpers import B16, Batch, f64
from helpers import need_gpu
from oracle import attention as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (6, 2), (16, 1), (21, 3), (40, 2)])
def test_single_tokens(D, hq, hkv):
    """One new token a sequence; contexts of 1 to more than one part."""
    need_gpu()
    lengths = [(1, kv) for kv in (1, 2, 15, 16, 17, 63, 64, 65, 129, 511, 512, 513, 700, 1500)]
    b = Batch(lengths, hq, hkv, D, 32, seed=hq).fill(spread=2)
    q = b.rows(hq, 2.0)
    b.check(q, b.attend(q))


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (128, 256), (64, 16)])
@pytest.mark.parametrize("lengths", [
    [(5, 5), (1, 40), (3, 300), (16, 17), (2, 2)],
    [(31, 31), (40, 500), (1, 1), (17, 1100)],
    [(130, 130), (257, 700)],
])
def test_several_tokens(D, page, lengths):
    need_gpu()
    b = Batch(lengths, 6, 2, D, page, seed=page).fill()
    q = b.rows(6, 2.0)
    b.check(q, b.attend(q))


@pytest.mark.parametrize("group", [1, 3, 4, 7, 8])
def test_heads_and_prompts(group):
    need_gpu()
    b = Batch([(90, 90), (33, 200), (1, 64)], 2 * group, 2, 128, 64, seed=group).fill()
    q = b.rows(2 * group, 2.0)
    b.check(q, b.attend(q))


@pytest.mark.parametrize("kv", [16384, 16385, 40000])
def test_long_contexts(kv):
    """More than 32 parts of 512 tokens: longer parts."""
    need_gpu()
    b = Batch([(1, kv), (2, 600)], 4, 1, 64, 128, seed=kv).fill()
    q = b.rows(4, 2.0)
    b.check(q, b.attend(q))


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (64, 9, 3), (128, 16, 1)])
def test_few_blocks_over_long_contexts(D, hq, hkv):
    """More than 64 rows a kv head, few blocks of them: a sequence's tokens are cut
    into parts. Tiles that end before the last parts; parts of a step and a bit."""
    need_gpu()
    lengths = [(65, 3000), (1, 50), (300, 900), (20, 4097), (9, 5000), (100, 100), (130, 4000)]
    b = Batch(lengths, hq, hkv, D, 32, seed=hq).fill()
    q = b.rows(hq, 2.0).cuda()
    args = b.device_args()
    got = b.attend(q, args=args)
    b.check(q, got)
    assert torch.equal(got, rows_alone(b, q, args))


def test_a_prompt_among_many_sequences():
    """More sequences than can have over 64 rows."""
    need_gpu()
    lengths = [(1, 40)] * 60 + [(20, 2000)] + [(1, 300)] * 40 + [(17, 3000)]
    b = Batch(lengths, 8, 2, 64, 32, seed=22).fill()
    q = b.rows(8, 2.0)
    b.check(q, b.attend(q))


def test_nan_in_parts():
    need_gpu()
    b = Batch([(40, 3000), (30, 2500)], 4, 2, 128, 16, seed=23).fill()
    b.codes[b.table[0, 2980 // 16], 1, 1, 2980 % 16, 37] = 0x7f        # seen by some rows
    b.codes[b.table[1, 10], 1, 0, 3, 5] = 0xff                         # by all
    q = b.rows(4)
    out = b.check(q, b.attend(q))
    assert np.isnan(out[20:40, 2, 37]).all() and not np.isnan(out[:20]).any()
    assert np.isnan(out[40:, 0, 5]).all()


def test_empty_sequences_and_rows_that_see_nothing():
    """No new tokens, no tokens at all, more new tokens than there are in all;
    rows of no sequence stay as they were."""
    need_gpu()
    b = Batch([(0, 0), (1, 0), (0, 70), (5, 3), (60, 2), (1, 33), (0, 0)], 4, 2, 128, 16).fill()
    q = b.rows(4)
    out = torch.full((b.T + 9, 4, 128), 7.0, dtype=B16, device="cuda")
    qq = torch.cat([q, torch.full((9, 4, 128), float("nan"), dtype=B16)]).cuda()
    ws = ig.attention_workspace(qq, b.device_args()[0], b.device_args()[4], b.max_q)
    ig.paged_attention(qq, *b.device_args(), out, ws, max_q=b.max_q)
    assert ig.check_status(ws) == 0
    assert (out[b.T:] == 7).all()
    want = b.check(q, out[:b.T])
    assert (want[0] == 0).all() and (f64(out[0]) == 0).all()     # sequence 1: no token
    assert (f64(out[1:3]) == 0).all() and (f64(out[3]) != 0).any()


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 20.0])
def test_scales_of_the_products(scale):
    need_gpu()
    b = Batch([(1, 700), (3, 90), (70, 140)], 4, 2, 64, 32, seed=5).fill()
    q = b.rows(4)
    b.check(q, b.attend(q, scale=scale), scale=scale)


@pytest.mark.parametrize("size,spread", [(1e-20, 0), (1e15, 0), (1.0, 8)])
def test_sizes_of_the_values(size, spread):
    """Value scales far from 1, and some binades apart from block to block."""
    need_gpu()
    b = Batch([(1, 300), (2, 1200), (80, 100)], 4, 2, 128, 16, seed=6)
    b.fill(spread=spread)
    e = int(np.log2(size))
    b.scales[:, 1] = np.clip(b.scales[:, 1].astype(int) + e, 1, 254).astype(np.uint8)
    q = b.rows(4, 0.3)
    b.check(q, b.attend(q))


def test_sizes_of_the_queries():
    """Rows of any size: what a row's largest value leaves of the others is kept."""
    need_gpu()
    b = Batch([(1, 100)] * 6, 4, 1, 128, 16, seed=7).fill()
    q = b.rows(4).float()
    for i, s in enumerate((0.0, 1e-30, 1e-3, 1.0, 30.0, 1e4)):
        q[i] *= s
    q[3, 0, ::2] *= 2.0 ** -12
    b.scales[:, 0] -= 8
    q = q.to(B16)
    b.check(q, b.attend(q))


@pytest.mark.parametrize("D", [64, 128])
def test_sizes_of_the_queries_of_a_prompt(D):
    need_gpu()
    b = Batch([(120, 150)], 4, 1, D, 32, seed=21).fill()
    q = b.rows(4).float()
    q *= torch.from_numpy(2.0 ** b.rng.integers(-60, 3, (b.T, 4, 1))).float()
    q[50:] *= torch.from_numpy(2.0 ** b.rng.integers(-14, 1, (b.T - 50, 4, D))).float()
    q[7] = 0
    q = q.to(B16)
    b.check(q, b.attend(q))


def test_a_sharp_maximum_late_and_early():
    """One token outweighs the others by more than p's range, at the first, a middle
    and the last place."""
    need_gpu()
    for at in (0, 333, 699):
        b = Batch([(1, 700)], 4, 1, 128, 16, seed=8).fill()
        q = b.rows(4)
        pg, row = b.table[0, at // 16], at % 16
        b.codes[pg, 0, 0, row] = ref.encode(np.sign(f64(q)[0, 0]) * 400)
        b.check(q, b.attend(q))


def test_equal_tokens():
    """All weights equal: the mean of the values."""
    need_gpu()
    b = Batch([(1, 5000), (64, 64)], 4, 1, 64, 16, seed=9).fill()
    b.codes[:, 0] = b.codes[0, 0, 0, 0]
    b.scales[:, 0] = 120
    q = b.rows(4)
    b.check(q, b.attend(q))


def test_nan_where_it_is_seen_only():
    """A NaN value or key of a token is in the rows that see the token, and in its
    own column (value) or all columns (key); NaN bytes behind the last token are in
    none."""
    need_gpu()
    for n, kv in ((8, 40), (100, 300)):
        b = Batch([(n, kv), (1, 33)], 4, 2, 128, 16, seed=10).fill()
        at = kv - n // 2
        b.codes[b.table[0, at // 16], 1, 1, at % 16, 37] = 0xff
        b.codes[b.table[0, (kv - 2) // 16], 0, 0, (kv - 2) % 16, 5] = 0x7f
        for s, (_, m) in enumerate(b.lengths):                     # behind the last token
            for j in range(m, -(-m // 16) * 16):
                b.codes[b.table[s, j // 16], :, :, j % 16] = 0x7f
        q = b.rows(4)
        out = b.check(q, b.attend(q))
        assert np.isnan(out[n // 2, 2, 37]) and not np.isnan(out[n // 2 - 1]).any()
        assert np.isnan(out[n - 1, 0]).all() and not np.isnan(out[n - 3, 0]).any()


def test_nan_scales():
    need_gpu()
    b = Batch([(20, 64), (1, 64), (1, 64)], 2, 2, 64, 16, seed=11).fill()
    b.scales[b.table[0, 3], 1, 0, 0] = 255          # tokens 48 .. 63, values
    b.scales[b.table[1, 1], 0, 1, 0] = 255          # keys
    q = b.rows(2)
    out = b.check(q, b.attend(q))
    assert not np.isnan(out[3, 0]).any() and np.isnan(out[4, 0]).all()
    assert np.isnan(out[20, 1]).all() and not np.isnan(out[20, 0]).any()
    assert not np.isnan(out[21]).any()


def test_not_finite_queries():
    need_gpu()
    b = Batch([(4, 50)], 2, 1, 64, 16, seed=12).fill()
    q = b.rows(2)
    q[1, 0, 3] = float("nan")
    q[2, 1, 9] = float("inf")
    got = f64(b.attend(q))
    assert np.isnan(got[1, 0]).all() and np.isnan(got[2, 1]).all()
    assert np.isnan(got).any(-1).sum() == 2


def rows_alone(b, q, args):
    """Each sequence in a batch of its own."""
    got = []
    for s in range(len(b.lengths)):
        one = Batch([b.lengths[s]], b.hq, b.hkv, b.D, b.page)
        cu = torch.tensor([0, b.lengths[s][0]], dtype=torch.int32, device="cuda")
        a = (args[0], args[1], cu, args[3][s:s + 1].contiguous(), args[4][s:s + 1].contiguous())
        got.append(one.attend(q[b.cu[s]:b.cu[s + 1]], args=a, max_q=b.lengths[s][0]))
    return torch.cat(got)


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (64, 6, 1)])
def test_rows_do_not_depend_on_the_batch(D, hq, hkv):
    """Bit for bit: alone or with others, at another place, on other pages, with
    another bound on the new tokens."""
    need_gpu()
    lengths = [(1, 3000), (4, 70), (60, 900), (1, 1), (2, 17000), (150, 150), (1, 513)]
    b = Batch(lengths, hq, hkv, D, 16, seed=13).fill()
    q = b.rows(hq, 2.0).cuda()
    args = b.device_args()
    whole = b.attend(q, args=args)
    assert torch.equal(whole, b.attend(q, args=args, max_q=b.max_q + 50))
    assert torch.equal(whole, rows_alone(b, q, args))
    # the same tokens on other pages
    perm = np.random.default_rng(1).permutation(b.pages)
    codes, scales = np.empty_like(b.codes), np.empty_like(b.scales)
    codes[perm], scales[perm] = b.codes, b.scales
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    moved = (dev(codes), dev(scales), args[2], args[3], dev(perm[b.table].astype(np.int32)))
    assert torch.equal(whole, b.attend(q, args=moved))


def test_runs_are_the_same_and_workspaces_reused():
    need_gpu()
    b = Batch([(1, kv) for kv in range(100, 9000, 370)], 8, 2, 128, 16, seed=14).fill()
    q = b.rows(8, 2.0).cuda()
    args = b.device_args()
    ws = ig.attention_workspace(q, args[0], args[4], 1)
    first = b.attend(q, args=args, ws=ws)
    for _ in range(20):
        assert torch.equal(first, b.attend(q, args=args, ws=ws))
    # a smaller call in the same workspace, then this one again
    small = Batch([(3, 600)], 8, 2, 128, 16, seed=15).fill()
    sq = small.rows(8)
    small.check(sq, small.attend(sq, ws=ws))
    assert torch.equal(first, b.attend(q, args=args, ws=ws))


def test_strided_operands_and_distant_pages():
    """q and out as columns of wider buffers; pages and their scales as every third
    of a larger pool."""
    need_gpu()
    b = Batch([(3, 200), (1, 30), (40, 90)], 4, 2, 128, 32, seed=16).fill()
    q = b.rows(4)
    codes, scales, cu, kv, table = b.device_args()
    pool = torch.randint(0, 256, (3 * b.pages, *codes.shape[1:]), dtype=torch.uint8, device="cuda")
    spool = torch.randint(0, 256, (3 * b.pages, *scales.shape[1:]), dtype=torch.uint8,
                          device="cuda")
    pool[1::3], spool[1::3] = codes, scales
    wide = torch.zeros(b.T, 6, 128, dtype=B16, device="cuda")
    wide[:, 1:5] = q.cuda()
    out = torch.full((b.T, 9, 128), 7.0, dtype=B16, device="cuda")
    got = b.attend(wide[:, 1:5], args=(pool[1::3], spool[1::3], cu, kv, table), out=out[:, 2:6])
    b.check(q, got)
    assert (out[:, :2] == 7).all() and (out[:, 6:] == 7).all()


def test_bad_pages_and_lengths_are_reported():
    """Tokens on pages that do not exist are absent, sequences out of range are left
    out; the status says so once."""
    need_gpu()
    b = Batch([(1, 100), (1, 64), (30, 80)], 4, 2, 64, 16, seed=17).fill()
    q = b.rows(4)
    b.table[0, 2], b.table[1, 0], b.table[2, 4] = b.pages, -1, 2 ** 31 - 1
    got = b.attend(q, status=-10)
    b.check(q, got)
    for name, change in (("kv beyond the table", lambda a: a[3][0:1].fill_(10 ** 6)),
                         ("negative", lambda a: a[3][0:1].fill_(-5)),
                         ("rows", lambda a: a[2][-1:].fill_(b.T + 1))):
        good = Batch([(1, 100), (1, 64), (30, 80)], 4, 2, 64, 16, seed=17).fill()
        args = good.device_args()
        change(args)
        out = good.attend(q, args=args, status=-10)
        seq = 2 if name == "rows" else 0
        rows = slice(good.cu[seq], good.cu[seq + 1])
        assert (out[rows] == 7).all(), name
        want, tol = good.reference(q)
        rest = np.ones(b.T, dtype=bool)
        rest[rows] = False
        assert (np.abs(f64(out) - want)[rest] <= tol[rest]).all(), name
    # more new tokens than max_q allows
    good = Batch([(1, 100), (1, 64), (30, 80)], 4, 2, 64, 16, seed=17).fill()
    out = good.attend(q, max_q=7, status=-10)
    assert (out[2:] == 7).all() and (out[:2] != 7).any()


def test_graph_and_another_stream():
    """Captured calls follow the lengths on the device."""
    need_gpu()
    b = Batch([(1, 900), (1, 40)], 8, 2, 128, 16, seed=18, cols=80).fill()
    q = b.rows(8).cuda()
    args = b.device_args()
    ws = ig.attention_workspace(q, args[0], args[4], 1)
    out = torch.zeros_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ig.paged_attention(q, *args, out, ws, max_q=1)
    for kv in ((900, 40), (17, 33), (0, 1), (513, 2)):
        args[3].copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b.attend(q, args=args)), kv


def test_expired_wait_ends_and_is_reported():
    need_gpu()
    b = Batch([(1, 900), (1, 40), (40, 100)], 8, 2, 128, 16, seed=19).fill()
    q = b.rows(8).cuda()
    args = b.device_args()
    ws = ig.attention_workspace(q, args[0], args[4], b.max_q)
    good = b.attend(q, args=args, ws=ws)
    b.attend(q, args=args, ws=ws, flags=ig.FLAG_TEST_COPY_TIMEOUT, status=-8)
    assert torch.equal(good, b.attend(q, args=args, ws=ws))


def test_offsets_past_32_bits():
    """A pool of more than 4 GB of codes: pages far from its start."""
    need_gpu()
    b = Batch([(1, 300), (20, 64)], 4, 2, 128, 64, seed=20).fill()
    q = b.rows(4)
    codes, scales, cu, kv, table = b.device_args()
    per = codes[0].numel()
    far = (5 << 30) // per
    pool = torch.zeros(far + b.pages, *codes.shape[1:], dtype=torch.uint8, device="cuda")
    spool = torch.zeros(far + b.pages, *scales.shape[1:], dtype=torch.uint8, device="cuda")
    pool[far:], spool[far:] = codes, scales
    b.check(q, b.attend(q, args=(pool, spool, cu, kv, table + far)))
