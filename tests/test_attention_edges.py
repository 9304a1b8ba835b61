"""Attention at the ends of its ranges: NaN scales of tokens that some rows do not see, sequences
with no tokens, logits far beyond what FP32 tells apart."""
import numpy as np
import pytest
import torch

from attention_helpers import Batch, f64
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
