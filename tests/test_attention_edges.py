"""Attention at the ends of its ranges: NaN scales of tokens that some rows do not see, sequences
with no tokens, logits far beyond what FP32 tells apart, values whose scales lie far apart or
are as small as they get, lengths that change between replays."""
import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from attention_helpers import B16, I32, Batch, f64
from helpers import need_gpu
from oracle import attention as ref

pytestmark = pytest.mark.gpu


def at(b, s, token):
    """(page, block of the page) of a token of sequence s."""
    return b.table[s, token // b.page], token % b.page // 16


# (new tokens, tokens), query heads to one kv head: the kernel of few rows; one tile of rows
# (whose steps two tiles share), two tiles, several blocks; each also with its tokens cut
ROWS = [((20, 90), 2), ((100, 180), 1), ((200, 330), 1), ((300, 300), 1), ((90, 90), 4),
        ((100, 3000), 1), ((200, 3100), 1)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length,hq", ROWS)
def test_nan_scale_of_keys_stays_with_the_rows_that_see_it(length, hq, D):
    need_gpu()
    n, kv = length
    b = Batch([length, (n, kv)], hq, 1, D, 32, seed=40).fill()
    first = (kv - 10) // 16 * 16                # only the last rows see this block
    page, block = at(b, 0, first)
    b.scales[page, 0, 0, block] = 255
    q = b.rows(hq)
    out = b.check(q, b.attend(q))
    sees = np.arange(kv - n, kv) >= first
    assert 0 < sees.sum() < n
    assert np.isnan(out[:n][sees]).all() and not np.isnan(out[:n][~sees]).any()
    assert not np.isnan(out[n:]).any()


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_and_no_tokens(D):
    """Sequences of more than 64 rows that have no tokens at all: rows of 0, whatever the
    blocks before left in shared memory."""
    need_gpu()
    b = Batch([(100, 0), (70, 0), (300, 0), (129, 0), (128, 0), (200, 100)], 2, 1, D, 16, seed=45).fill()
    q = b.rows(2, 3.0)
    big = Batch([(300, 700)] * 12, 2, 1, D, 16, seed=46).fill(size=1e6)
    bq = big.rows(2, 1e4)
    for _ in range(3):
        big.attend(bq)
        got = f64(b.attend(q))
        assert (got[:-100] == 0).all() and (got[-100:] != 0).any()
    b.check(q, b.attend(q))


@pytest.mark.parametrize("size", [2.0 ** e for e in (10, 16, 18, 20, 24, 25, 26, 27, 28, 40)])
@pytest.mark.parametrize("length,hq", ROWS)
def test_logits_that_fp32_holds_in_steps(length, hq, size):
    """Queries and keys of one value that is not 0: equal tokens have equal logits in
    FP32, the others' are `size` / 4 below at least and weigh exp(-256) at most. What is left
    is the mean of the values of the largest keys, with FP16 weights (2^-11, over a sum of the
    same ones) and a result in bf16 (2^-8). Value scales differ from block to block where a
    logit has bits left for it."""
    need_gpu()
    n, kv = length
    b = Batch([length], hq, 1, 128, 32, seed=41).fill()
    rng = np.random.default_rng(1)
    codes = rng.choice([0x38, 0x3a, 0x3c, 0xb8], (kv,))         # 1, 1.25, 1.5, -1
    value = {0x38: 1.0, 0x3a: 1.25, 0x3c: 1.5, 0xb8: -1.0}
    for j in range(kv):
        page, block = at(b, 0, j)
        b.codes[page, 0, 0, j % 32] = 0
        b.codes[page, 0, 0, j % 32, 17] = codes[j]
        b.scales[page, 0, 0, block] = 127
        b.scales[page, 1, 0, block] = 121 + (block * 5 + j // 64 % 3 if size <= 2.0 ** 18 else 0)
    q = torch.zeros(n, hq, 128)
    q[:, :, 17] = size * (1 + torch.arange(n) % 16 / 16)[:, None]
    got = f64(b.attend(q.bfloat16(), scale=1.0))
    v = ref.held(b.codes, b.scales, b.table[0], kv)[1][:, 0]
    x = np.array([value[c] for c in codes])
    for i in range(n):
        see = slice(0, kv - n + i + 1)
        top = x[see] == x[see].max()
        want, mag = v[see][top].mean(0), np.abs(v[see][top]).mean(0)
        assert (np.abs(got[i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag).all(), i


def exact(b, s, q, scale):
    """(out, tolerance) of sequence s from what its rows see: half a step of bf16; twice, as
    in the sum of the weights too, 2^-11 of FP16 weights and 2^-16 of a logit's magnitudes
    (and 2^-17 of the row's largest query value times the keys' magnitudes where a query is
    two e4m3 numbers); of weights under 2^-14 half a step of 2^-24, times 448 of their block's
    scale, where the largest of weight times scale is 2^7 at least: 2^-32 times 448."""
    n, kv = b.lengths[s]
    k, v = ref.held(b.codes, b.scales, b.table[s], kv)
    j = np.arange(kv)
    page, block = b.table[s, j // b.page], j % b.page // 16
    x = f64(q)[b.cu[s]:b.cu[s + 1]]
    out, tol = np.zeros(x.shape), np.zeros(x.shape)
    group = b.hq // b.hkv
    for h in range(b.hq):
        kk, vv = k[:, h // group], v[:, h // group]
        unit = 2.0 ** (b.scales[page, 1, h // group, block] - 127.0)
        for i in range(n):
            see = slice(0, kv - n + i + 1)
            t = kk[see] @ x[i, h] * scale
            p = np.exp(t - t.max())
            p /= p.sum()
            logit = 2.0 ** -16 * abs(scale) * (np.abs(kk[see]) @ np.abs(x[i, h])).max()
            if n * group > 64:
                logit += 2.0 ** -17 * abs(scale) * np.abs(kk[see]).sum(-1).max() * np.abs(x[i, h]).max()
            out[i, h] = p @ vv[see]
            tol[i, h] = (2.0 ** -8 * np.abs(out[i, h]) + 2 * (2.0 ** -11 + logit) * (p @ np.abs(vv[see])) +
                         kv * 2.0 ** -32 * 448 * (p * unit[see]).max())
    return out, tol


def close(b, q, got, scale=None):
    got = f64(got)
    for s in range(len(b.lengths)):
        out, tol = exact(b, s, q, b.D ** -0.5 if scale is None else scale)
        err = np.abs(got[b.cu[s]:b.cu[s + 1]] - out)
        bad = ~(err <= tol)
        assert not bad.any(), (s, bad.sum(), np.argwhere(bad)[0], got[b.cu[s]:b.cu[s + 1]][bad][0],
                               out[bad][0], tol[bad][0])


@pytest.mark.parametrize("apart", [12, 24, 34, 45, 80])
@pytest.mark.parametrize("length,hq", ROWS)
def test_values_of_tokens_that_a_row_does_not_see(length, hq, apart):
    """The last tokens' values are 2^`apart` times the others': rows before them keep all
    their bits."""
    need_gpu()
    n, kv = length
    b = Batch([length], hq, 1, 128, 32, seed=42).fill()
    for j in range((kv - 20) // 16 * 16, kv, 16):
        page, block = at(b, 0, j)
        b.scales[page, 1, 0, block] += apart
    q = b.rows(hq, 0.5)
    close(b, q, b.attend(q))


@pytest.mark.parametrize("apart", [12, 24, 34, 45, 80, -34, -80])
@pytest.mark.parametrize("length,hq", ROWS)
def test_values_of_the_tokens_that_carry_the_weight(length, hq, apart):
    """Two tokens in three have nearly no weight (exp(-280)) and values 2^`apart` times those
    of the third, which make up the result."""
    need_gpu()
    n, kv = length
    b = Batch([length], hq, 1, 128, 32, seed=43).fill()
    for j in range(kv):
        page, block = at(b, 0, j)
        b.scales[page, 0, 0, block] = 127 - 4
        if j // 16 % 3 != 0:
            b.codes[page, 0, 0, j % 32, 5] = 0xf0           # -128
            if j % 16 == 0:
                b.scales[page, 1, 0, block] = int(b.scales[page, 1, 0, block]) + apart
        else:
            b.codes[page, 0, 0, j % 32, 5] = 0x70           # 128
    q = b.rows(hq, 2.0 ** -6).float()
    q[:, :, 5] = 17.5
    q = q.bfloat16()
    close(b, q, b.attend(q, scale=1.0), scale=1.0)


@pytest.mark.parametrize("byte", [2, 7, 9, 30, 190, 191, 246])
def test_the_smallest_and_largest_scales_over_long_contexts(byte):
    """Positive values of around 2^-118 and less, or 2^119, a sum of weights of 2^22 and
    more."""
    need_gpu()
    for length, hq in (((1, 40000), 2), ((1, 5000), 2), ((20, 2000), 4), ((2, 300), 1), ((150, 150), 1)):
        b = Batch([length], hq, 1, 64, 64, seed=44).fill()
        b.scales[:, 1] = byte
        b.codes[:, 1] &= 0x7f
        q = b.rows(hq, 0.3)
        close(b, q, b.attend(q))


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (64, 4, 4)])
def test_lengths_that_change_between_replays(D, hq, hkv):
    """One captured call of an append and the attention behind it: single tokens, prompts cut
    into parts and not, sequences of both kernels and empty ones, as the lengths on the device
    say at the time. Bit for bit what an eager run in a workspace of its own gives."""
    need_gpu()
    T, most, longest = 310, 300, 3000
    b = Batch([(0, longest)] * 4, hq, hkv, D, 64, seed=47).fill(spread=1)
    codes, scales, _, _, table = b.device_args()
    start = codes.clone(), scales.clone()
    x = torch.randn(T, hq + 2 * hkv, D, device="cuda").bfloat16()
    q, k, v = x.split([hq, hkv, hkv], 1)
    cu, kv = (torch.zeros(n, dtype=I32, device="cuda") for n in (5, 4))
    q_out, out = (torch.zeros(T, hq, D, dtype=B16, device="cuda") for _ in range(2))
    w = torch.ones(D, device="cuda").bfloat16()

    def run(ws):
        ig.kv_append(k, v, codes, scales, cu, kv, table, ws, w_k=w, q=q, q_out=q_out, w_q=w, max_q=most)
        ig.paged_attention(q_out, codes, scales, cu, kv, table, out, ws, max_q=most)

    def put(lengths):
        cu.copy_(torch.tensor(np.concatenate([[0], np.cumsum([n for n, _ in lengths])]), dtype=I32))
        kv.copy_(torch.tensor([m for _, m in lengths], dtype=I32))
        for t, s in zip((codes, scales), start):
            t.copy_(s)
        out.fill_(7.0)
        q_out.fill_(7.0)

    ws, other = (ig.attention_workspace(q, codes, table, most) for _ in range(2))
    put([(1, 5)] * 4)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        run(ws)
    for lengths in ([(1, 900), (200, 2900), (40, 40), (1, 1)], [(1, 5)] * 4,
                    [(300, 300), (1, 3000), (0, 0), (2, 70)], [(0, 0), (0, 17), (129, 3000), (90, 90)],
                    [(70, 3000)] * 4, [(16, 1024), (17, 17), (20, 2000), (100, 100)],
                    [(0, 0)] * 4, [(100, 60), (80, 2999), (65, 65), (64, 64)]):
        put(lengths)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, q_out, codes, scales)]
        put(lengths)
        run(other)
        assert all(torch.equal(g, t) for g, t in zip(got, (out, q_out, codes, scales))), lengths
        used = sum(n for n, _ in lengths)
        assert (out[used:] == 7).all() and not (out[:used] == 7).all(-1).any()
        one = Batch(lengths, hq, hkv, D, 64)
        one.table, one.pages = b.table, b.pages
        one.codes, one.scales = codes.cpu().numpy(), scales.cpu().numpy()
        one.check(q_out[:used], out[:used])
    assert ig.check_status(ws) == 0 and ig.check_status(other) == 0


@pytest.mark.parametrize("kv", [32767, 32768, 32769, 65537])
def test_where_parts_grow(kv):
    """64 parts of 512 tokens are the most; behind them parts of 1024, then 1536."""
    need_gpu()
    b = Batch([(1, kv), (2, kv - 5)], 4, 1, 64, 128, seed=kv).fill()
    q = b.rows(4, 2.0)
    b.check(q, b.attend(q))


@pytest.mark.parametrize("lengths", [[(1, 3000)] * 20 + [(0, 40)] + [(5, 2000)] * 7,
                                     [(1, 900)] * 15 + [(100, 2500), (0, 0), (300, 900), (70, 3000)],
                                     [(66, 2000)] * 9 + [(1, 1500)] * 9])
def test_parts_placed_by_rows(lengths):
    """With no bound on new tokens a sequence's parts are where its rows begin, not where its
    number says: the same bits, and nothing written behind the workspace."""
    need_gpu()
    b = Batch(lengths, 8, 2, 64, 32, seed=48).fill()
    q = b.rows(8, 2.0).cuda()
    args = b.device_args()
    b.check(q, b.attend(q, args=args))
    size = ig.attention_workspace(q, args[0], args[4], b.T).numel()
    buf = torch.full((size + (1 << 20),), 0xab, dtype=torch.uint8, device="cuda")
    buf[:size] = 0
    got = b.attend(q, args=args, max_q=b.T, ws=buf[:size])
    assert torch.equal(got, b.attend(q, args=args)) and (buf[size:] == 0xab).all()
