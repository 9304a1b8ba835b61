"""Batches, caches and tolerances for the tests of the attention calls."""
import numpy as np
import torch

import invariant_gemm_gb300 as ig
import oracle
from oracle import attention as ref

B16, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def f64(t):
    return t.double().cpu().numpy()


def bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.float32).to(B16)


class Batch:
    """Sequences of (new tokens, tokens in all) on shuffled pages, with pages of no
    sequence between them; unused bytes are noise, NaN codes among them."""

    def __init__(self, lengths, hq, hkv, D, page, seed=0, spare=3, device="cuda", cols=None):
        self.lengths, self.hq, self.hkv, self.D, self.page = lengths, hq, hkv, D, page
        rng = np.random.default_rng(seed)
        self.rng = rng
        need = [-(-kv // page) for _, kv in lengths]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        cols = max([1] + need) if cols is None else cols
        self.table = np.zeros((len(lengths), cols), dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.concatenate([[0], np.cumsum([q for q, _ in lengths])]).astype(np.int32)
        self.kv = np.array([kv for _, kv in lengths], dtype=np.int32)
        self.T = int(self.cu[-1])
        self.max_q = max([q for q, _ in lengths] + [0])
        self.codes = rng.integers(0, 256, (self.pages, 2, hkv, page, D)).astype(np.uint8)
        self.scales = rng.integers(100, 140, (self.pages, 2, hkv, page // 16)).astype(np.uint8)
        self.device = device

    def rows(self, heads, size=1.0):
        """bf16 rows [T][heads][D], as a torch tensor on the host."""
        x = self.rng.standard_normal((self.T, heads, self.D)) * size
        return bf16(x)

    def fill(self, size=1.0, spread=0):
        """The tokens of all sequences, appended at once by the oracle; spread:
        binades by which sizes differ from token to token."""
        for b, (_, kv) in enumerate(self.lengths):
            for side in (0, 1):
                x = self.rng.standard_normal((kv, self.hkv, self.D)) * size
                x = x * 2.0 ** self.rng.integers(-spread, spread + 1, (kv, self.hkv, 1))
                ref.append(self.codes, self.scales, x.astype(np.float32), self.table[b], 0, side)
        return self

    def device_args(self):
        dev = lambda a: torch.from_numpy(a).to(self.device)  # noqa: E731
        return (dev(self.codes), dev(self.scales), dev(self.cu), dev(self.kv), dev(self.table))

    def attend(self, q, scale=None, max_q=None, args=None, ws=None, out=None, flags=0, status=0):
        """paged_attention of q (host or device); (T, hq, D) on the device."""
        args = self.device_args() if args is None else args
        q = q.to(self.device)
        out = torch.full(q.shape, 7.0, dtype=B16, device=self.device) if out is None else out
        max_q = self.max_q if max_q is None else max_q
        ws = ig.attention_workspace(q, args[0], args[4], max_q) if ws is None else ws
        ig.paged_attention(q, *args, out, ws, max_q=max_q, scale=scale, flags=flags)
        assert ig.check_status(ws) == status
        return out

    def reference(self, q, scale=None):
        """(out, tolerance) over all rows.

        The stored result is off by half a bf16 step, 2^-8 |o|. Each p is an FP16
        value times 2^(e - E), e the exponent of its block's value scale and E the
        largest one: 2^-11 relative while it is normal. Under 2^-14 it is off by half
        a step of 2^-24, with values of at most 448 * 2^E < 2 max|v|, and the row's
        largest p, which the sum of p is not below, is at least 2^7 (m is less than
        one above the row's largest logit and p is 2^8 at m): each token adds at
        most 2^-25 2^-7 2 max|v| = 2^-31 max|v| to the error of o. The sum of p is an
        FP32 one. A logit of products that sum to A in
        magnitude is off by 2^-16 A at most: D / 16 tensor-core sums of 16 exact
        products into FP32 (each within 2^-20 of the magnitudes added), two FP32
        products and the rounding of the exponential's argument. Where a sequence
        has more than 64 rows a kv head, a query is two e4m3 numbers: exact but for
        values under 2^-9 of the row's largest, off by at most 2^-17 of it (steps of
        2^-9 where the largest is 2^7 at least). These count twice, in p and in the
        sum of p, over sum p |v|."""
        scale = self.D ** -0.5 if scale is None else scale
        q = f64(q)
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        for b, (n, kv) in enumerate(self.lengths):
            r = slice(self.cu[b], self.cu[b + 1])
            k, v = ref.held(self.codes, self.scales, self.table[b], kv)
            bad = self.table[b, np.arange(kv) // self.page]
            absent = (bad < 0) | (bad >= self.pages)
            o, size, big = ref.attention(q[r], k, v, scale, absent)
            out[r] = o
            logit = 2.0 ** -16 * big
            if n * self.hq // self.hkv > 64 and kv:
                kk = np.nan_to_num(np.abs(k)).sum(-1).max()
                logit = logit + 2.0 ** -17 * abs(scale) * kk * np.nan_to_num(
                    np.abs(q[r])).max(-1, keepdims=True)
            tol[r] = 2.0 ** -8 * np.abs(o) + 2 * (2.0 ** -11 + logit) * size
            top = np.abs(np.where(np.isfinite(v), v, 0)).max(initial=0.0)
            tol[r] += kv * 2.0 ** -31 * top
        return out, tol

    def check(self, q, got, scale=None):
        out, tol = self.reference(q, scale)
        got = f64(got)
        nan = np.isnan(out)
        assert (np.isnan(got) == nan).all(), "NaN in other places"
        err = np.abs(got - out)
        bad = ~nan & ~(err <= tol)
        assert not bad.any(), (
            f"{bad.sum()} of {bad.size} outside; first {tuple(np.argwhere(bad)[0])}: "
            f"{got[bad][0]} for {out[bad][0]}, tolerance {tol[bad][0]}")
        return out
