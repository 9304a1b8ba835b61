"""Attention at the ends of its ranges: NaN scales of tokens that some rows do not see, sequences
with no tokens."""
import numpy as np
import pytest

from attention_helpers import Batch, f64
from helpers import need_gpu

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
