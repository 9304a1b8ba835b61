"""The attention calls together and in the ways a server uses them: drawn sizes, captured
runs, two streams at a time, padded batches, one workspace for several kinds of call."""
import numpy as np
import pytest
import torch

import invariant_gemm_gb300 as ig
from attention_helpers import B16, I32, Batch, f64
from helpers import need_gpu
from oracle import attention as ref


def draw(rng):
    hkv = int(rng.choice([1, 2, 3]))
    group = int(rng.choice([1, 2, 3, 5, 8, 16]))
    D, page = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256]))
    kind, lengths = rng.choice(["one", "few", "prompt", "mixed"]), []
    for _ in range(int(rng.integers(1, 7))):
        n = {"one": 1, "few": int(rng.integers(1, 9)), "prompt": int(rng.integers(9, 200)),
             "mixed": int(rng.choice([0, 1, 3, 40, 150]))}[str(kind)]
        lengths.append((n, n + int(round(2.0 ** rng.uniform(0, 11))) - 1))
    keep, rows = [], 0
    for n, kv in lengths:                   # (the oracle goes row by row)
        if rows + n * hkv * group <= 4000:
            keep.append((n, kv))
            rows += n * hkv * group
    return keep or [(1, 5)], hkv * group, hkv, D, page


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(24))
def test_drawn_sizes(seed):
    need_gpu()
    rng = np.random.default_rng(1000 + seed)
    lengths, hq, hkv, D, page = draw(rng)
    b = Batch(lengths, hq, hkv, D, page, seed=seed).fill(spread=int(rng.integers(0, 4)))
    q = b.rows(hq, float(2.0 ** rng.uniform(-3, 3)))
    b.check(q, b.attend(q))


@pytest.mark.parametrize("seed", range(30))
def test_workspace_is_enough_for_smaller_calls(seed):
    rng = np.random.default_rng(seed)
    hkv, group = int(rng.integers(1, 9)), int(rng.integers(1, 17))
    page = int(rng.choice([16, 64, 256]))

    def size(T, B, max_q, cols):
        return ig.lib().ig_attention_workspace_bytes(
            ig._ATTN_SHAPE(T, 0, 0, hkv * group, 0, 1.0, 0),
            ig._KV_CACHE(0, 0, 0, 0, 0, page, hkv, 128, 0), ig._BATCH(0, 0, 0, cols, B, max_q))

    top = [int(2 ** rng.uniform(0, x)) for x in (16, 9, 13, 10)]
    for _ in range(40):
        less = [int(rng.integers(1, t + 1)) for t in top]
        assert 0 < size(*less) <= size(*top), (less, top)


class Chain:
    """Append, attention and read-back of one batch, outputs in buffers of its own."""

    def __init__(self, lengths, hq, hkv, D, page, seed, longest=0):
        self.b = b = Batch(lengths, hq, hkv, D, page, seed=seed,
                           cols=-(-max(longest, *[kv for _, kv in lengths]) // page)).fill()
        self.codes, self.scales, self.cu, self.kv, self.table = b.device_args()
        self.start = (self.codes.clone(), self.scales.clone())
        x = b.rows(hq + 2 * hkv).cuda()
        self.q, self.k, self.v = x.split([hq, hkv, hkv], 1)      # columns of one buffer
        self.w = (1 + 0.1 * torch.randn(D)).to(B16).cuda()
        turn = torch.arange(4096)[:, None] * 10000.0 ** (-torch.arange(D // 2) * 2.0 / D)
        self.cs = torch.cat([turn.cos(), turn.sin()], 1).float().cuda()
        z = lambda h: torch.zeros(b.T, h, D, dtype=B16, device="cuda")  # noqa: E731
        self.q_out, self.out, self.k_out, self.v_out = z(hq), z(hq), z(hkv), z(hkv)
        self.ws = ig.attention_workspace(self.q_out, self.codes, self.table, b.max_q)

    def run(self):
        at = (self.codes, self.scales, self.cu, self.kv, self.table)
        ig.kv_append(self.k, self.v, *at, self.ws, w_k=self.w, cos_sin=self.cs, q=self.q,
                     q_out=self.q_out, w_q=self.w, max_q=self.b.max_q)
        ig.paged_attention(self.q_out, *at, self.out, self.ws, max_q=self.b.max_q)
        ig.kv_gather(*at, self.k_out, self.v_out, self.ws)

    def state(self):
        return [t.clone() for t in (self.codes, self.scales, self.q_out, self.out, self.k_out,
                                    self.v_out)]

    def again(self):
        self.codes.copy_(self.start[0])
        self.scales.copy_(self.start[1])
        for t in (self.q_out, self.out, self.k_out, self.v_out):
            t.zero_()
        torch.cuda.synchronize()

    def check(self):
        """Attention and read-back against the oracle over what the cache holds."""
        b = self.b
        b.codes, b.scales = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        b.check(self.q_out, self.out)
        for s, (n, kv) in enumerate(b.lengths):
            k, v = ref.held(b.codes, b.scales, b.table[s], kv)
            r = slice(b.cu[s], b.cu[s + 1])
            for got, want in ((self.k_out[r], k[kv - n:]), (self.v_out[r], v[kv - n:])):
                np.testing.assert_array_equal(f64(got), want)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [
    [(1, 1), (1, 17), (1, 300)],
    [(3, 3), (90, 90), (1, 2000), (200, 1500)],         # both kernels, a sequence cut into parts
])
def test_captured_runs(lengths):
    """The three calls in a graph on a stream of its own, replayed over the cache as it was
    at the start: the bits of an eager run, each time."""
    need_gpu()
    c = Chain(lengths, 8, 2, 64, 32, 30)
    c.run()
    assert ig.check_status(c.ws) == 0
    c.check()
    eager = c.state()
    c.again()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run()
    for _ in range(3):
        c.again()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, c.state()))
    assert ig.check_status(c.ws) == 0


@pytest.mark.gpu
def test_two_streams_at_a_time():
    """Two batches on two streams, eager and replayed, a workspace each."""
    need_gpu()
    pair = [Chain([(1, 3000), (1, 1), (70, 2900)], 8, 2, 128, 64, 31),
            Chain([(1, 2500), (200, 2500)], 8, 2, 128, 64, 32)]
    want = []
    for c in pair:
        c.run()
        want.append(c.state())
        c.again()
    streams = [torch.cuda.Stream() for _ in pair]
    graphs = [torch.cuda.CUDAGraph() for _ in pair]
    for c, s, g in zip(pair, streams, graphs):
        with torch.cuda.graph(g, stream=s):
            c.run()
    for replay in (False, True):
        for c in pair:
            c.again()
        for _ in range(5):
            for c, s, g in zip(pair, streams, graphs):
                with torch.cuda.stream(s):
                    c.codes.copy_(c.start[0])
                    c.scales.copy_(c.start[1])
                    g.replay() if replay else c.run()
        torch.cuda.synchronize()
        for c, w in zip(pair, want):
            assert all(torch.equal(a, b) for a, b in zip(w, c.state())), replay
            assert ig.check_status(c.ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[(1, 100), (1, 30)], [(80, 300), (2, 9)]])
def test_padded_batches(lengths):
    """Rows behind the last sequence (a batch padded to the size of a capture) and unused
    sequences without tokens: neither read nor written."""
    need_gpu()
    pad = 37
    c = Chain(lengths + [(0, 0), (0, 12)], 6, 2, 64, 16, 33)
    c.run()
    want = c.state()
    c.again()
    T = c.b.T

    def padded(t, fill):
        out = torch.full((T + pad, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")
        out[:T] = t
        return out

    nan = float("nan")
    c.q, c.k, c.v = padded(c.q, nan), padded(c.k, nan), padded(c.v, nan)
    c.q_out, c.out, c.k_out, c.v_out = (padded(t, 7.0) for t in (c.q_out, c.out, c.k_out, c.v_out))
    c.ws = ig.attention_workspace(c.q_out, c.codes, c.table, c.b.max_q)
    c.run()
    got = c.state()
    assert ig.check_status(c.ws) == 0
    for a, w in zip(got[:2], want[:2]):
        assert torch.equal(a, w)
    for a, w in zip(got[2:], want[2:]):
        assert torch.equal(a[:T], w) and (a[T:] == 7).all()


@pytest.mark.gpu
def test_one_workspace_for_many_kinds_of_call():
    """Attention of different sizes and the library's other calls, in turn, in one
    workspace: each as in one of its own."""
    need_gpu()
    chains = [Chain(n, 8, 2, 64, 32, 40 + i) for i, n in enumerate(
        ([(1, 900)], [(70, 1500), (1, 40)], [(4, 77)] * 9))]
    M, K, N, r = 64, 512, 256, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(B16)  # noqa: E731
    x, A, B = rnd(M, K), rnd(4, 1, r, K), rnd(4, 1, N, r)
    idx = torch.randint(-1, 4, (M,), device="cuda", dtype=I32, generator=g)
    shape = ig.make_shape(M, K, N, r, num_adapters=4)
    want = []
    for c in chains:
        c.run()
        want.append(c.state())
    y0, z = rnd(M, N), torch.empty(1, M, r, device="cuda")
    y = y0.clone()
    ig.lora_apply(shape, x, y, idx, A, B, 1.0, z, ig.workspace(shape))
    ws = ig.workspace(shape, min_bytes=max(c.ws.numel() for c in chains))
    for _ in range(2):
        for c, w in zip(chains, want):
            c.ws = ws
            c.again()
            c.run()
            got = y0.clone()
            ig.lora_apply(shape, x, got, idx, A, B, 1.0, z, ws)
            assert ig.check_status(ws) == 0
            assert torch.equal(got, y)
            assert all(torch.equal(a, b) for a, b in zip(w, c.state()))


@pytest.mark.gpu
def test_shared_pages():
    """Two sequences with the same pages for a common beginning read what one reads."""
    need_gpu()
    b = Batch([(1, 200), (1, 200)], 4, 2, 64, 16, seed=50).fill()
    b.table[1, :12] = b.table[0, :12]
    q = b.rows(4)
    b.check(q, b.attend(q))


@pytest.mark.gpu
def test_many_sequences():
    """The most sequences that a call takes, most of them without a token."""
    need_gpu()
    lengths = [(0, 0)] * 8192
    for i, n in ((0, (1, 33)), (4000, (30, 64)), (8000, (1, 5)), (8191, (2, 300))):
        lengths[i] = n
    for hq in (2, 16):                      # tiles of 8 and of 16 rows, prompts
        b = Batch(lengths, hq, 1, 128, 16, seed=51).fill()
        q = b.rows(hq)
        b.check(q, b.attend(q))


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(65, 1), (128, 1), (200, 2), (300, 1), (1024, 1)])
@pytest.mark.parametrize("lengths", [[(1, 70), (1, 1), (2, 300)], [(1, 3000)], [(3, 2), (0, 5), (1, 129)]])
def test_many_query_heads_of_one_kv_head(hq, hkv, lengths):
    """A token's rows alone are more than a tile, or than a block."""
    need_gpu()
    b = Batch(lengths, hq, hkv, 64, 32, seed=hq).fill()
    q = b.rows(hq)
    b.check(q, b.attend(q))


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_append_beyond_the_table_of_angles(inter):
    """Tokens whose place the table does not have: NaN keys and queries, values as they
    are, and the status says so."""
    need_gpu()
    b = Batch([(20, 25), (1, 9), (1, 11)], 4, 2, 64, 16, seed=60)
    q, k, v = b.rows(4), b.rows(2), b.rows(2)
    args = b.device_args()
    ws, out = ig.mx4_workspace(), torch.zeros(b.T, 4, 64, dtype=B16, device="cuda")
    cs = torch.ones(10, 64, device="cuda")
    ig.kv_append(k.cuda(), v.cuda(), *args, ws, cos_sin=cs, q=q.cuda(), q_out=out, max_q=b.max_q,
                 flags=ig.ROPE_INTERLEAVED if inter else 0)
    assert ig.check_status(ws) == -10 and ig.check_status(ws) == 0
    codes, scales = args[0].cpu().numpy(), args[1].cpu().numpy()
    at = np.concatenate([np.arange(kv - n, kv) for n, kv in b.lengths])
    assert (out.isnan().all(-1).all(-1).cpu().numpy() == (at >= 10)).all()
    assert not out.isnan()[torch.from_numpy(at < 10)].any()
    for s, (n, kv) in enumerate(b.lengths):
        kk, vv = ref.held(codes, scales, b.table[s], kv)
        new = np.arange(kv - n, kv)
        assert np.isnan(kk[new[new >= 10]]).all() and np.isfinite(kk[new[new < 10]]).all()
        assert np.isfinite(vv[new]).all()


@pytest.mark.gpu
def test_nothing_in_a_batch():
    """No sequences, no tokens, sequences of no tokens."""
    need_gpu()
    z = lambda *s, t=B16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    cache, scales = z(2, 2, 2, 16, 64, t=torch.uint8), z(2, 2, 2, 1, t=torch.uint8)
    for B, T in ((0, 0), (0, 5), (3, 0), (3, 5)):
        cu, kv, table = z(B + 1, t=I32), z(B, t=I32), z(B, 4, t=I32)
        q, k, out = z(T, 4, 64), z(T, 2, 64), torch.full((T, 4, 64), 7.0, device="cuda").to(B16)
        ws = ig.attention_workspace(q, cache, table)
        kept = torch.full((T, 2, 64), 7.0, device="cuda").to(B16)
        ig.kv_append(k, k, cache, scales, cu, kv, table, ws, q=q, q_out=out)
        ig.paged_attention(q, cache, scales, cu, kv, table, out, ws)
        ig.kv_gather(cache, scales, cu, kv, table, kept, kept.clone(), ws)
        assert ig.check_status(ws) == 0
        assert (out == 7).all() and (kept == 7).all() and not cache.any()


@pytest.mark.gpu
@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (64, 12, 3)])
def test_rows_of_cut_sequences_do_not_depend_on_the_batch(D, hq, hkv):
    """Sequences cut into parts, blocks of one tile and of two, few rows among them: each
    bit for bit as alone, wherever it stands."""
    need_gpu()
    lengths = [(25, 4000), (1, 500), (100, 3000), (17, 2500), (200, 2000), (3, 9)]
    b = Batch(lengths, hq, hkv, D, 32, seed=70).fill()
    q = b.rows(hq, 2.0).cuda()
    args = b.device_args()
    whole = b.attend(q, args=args)
    b.check(q, whole)
    for i, (n, kv) in enumerate(lengths):
        r = slice(int(b.cu[i]), int(b.cu[i + 1]))
        one = (args[0], args[1], torch.tensor([0, n], dtype=I32, device="cuda"), args[3][i:i + 1],
               args[4][i:i + 1])
        assert torch.equal(whole[r], b.attend(q[r], max_q=n, args=one)), (i, n, kv)


@pytest.mark.gpu
@pytest.mark.parametrize("D,inter", [(128, False), (64, True)])
def test_norms_and_appends_do_not_depend_on_the_batch(D, inter):
    """The same bits in calls of a token and of thousands, in and out of place."""
    need_gpu()
    flags = ig.ROPE_INTERLEAVED if inter else 0
    g = torch.Generator(device="cuda").manual_seed(3)
    T, hq, hk = 3001, 24, 5
    x = torch.randn(T, hq + 2 * hk, D, device="cuda", generator=g).to(B16)
    w = torch.rand(D, device="cuda", generator=g).to(B16)
    turn = torch.arange(4000)[:, None] * 10000.0 ** (-torch.arange(D // 2) * 2.0 / D)
    cs = torch.cat([turn.cos(), turn.sin()], 1).float().cuda()
    pos = torch.randint(0, 4000, (T,), dtype=I32, device="cuda", generator=g)
    ws = ig.mx4_workspace()

    def normed(r, place):
        q, k = x[r, :hq].clone(), x[r, hq:hq + hk].clone()
        qo, ko = (q, k) if place else (torch.empty_like(q), torch.empty_like(k))
        ig.qk_norm_rope(q, k, qo, ko, ws, w_q=w, w_k=w, cos_sin=cs, positions=pos[r], flags=flags)
        return qo, ko

    whole = normed(slice(0, T), False)
    for r in (slice(0, T), slice(0, 1), slice(1500, 1504), slice(T - 1, T)):
        for place in (False, True):
            for a, b in zip(whole, normed(r, place)):
                assert torch.equal(a[r], b)

    # sequences of one to many new tokens, together and each alone
    lengths = [(1, 17), (2, 40), (1, 1), (1000, 1200), (4, 4), (700, 703), (1, 3000)]
    b = Batch(lengths, hq, hk, D, 32, seed=71).fill()
    n = b.T
    q, k, v = x[:n, :hq], x[:n, hq:hq + hk], x[:n, hq + hk:]

    def appended(seqs):
        codes, scales, cu, kv, table = b.device_args()
        out = torch.zeros(n, hq, D, dtype=B16, device="cuda")
        for first, last in seqs:
            r = slice(int(b.cu[first]), int(b.cu[last]))
            ig.kv_append(k[r], v[r], codes, scales, cu[first:last + 1] - int(b.cu[first]),
                         kv[first:last], table[first:last], ws, w_k=w, cos_sin=cs, q=q[r],
                         q_out=out[r], w_q=w, flags=flags,
                         max_q=max(m for m, _ in lengths[first:last]))
        assert ig.check_status(ws) == 0
        return codes, scales, out

    together = appended([(0, len(lengths))])
    alone = appended([(i, i + 1) for i in range(len(lengths))])
    assert all(torch.equal(a, c) for a, c in zip(together, alone))


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot,inter,placed", [(128, 128, False, False), (64, 32, True, True)])
def test_keys_are_rounded_to_the_nearest_code(D, rot, inter, placed):
    """Of 8 million normed and rotated keys, against FP64: FP32's last place (2^-24, a few
    of them) next to middles 2^-4 apart gets about one of a million wrong, 8 here, and those
    as near as 2^-20 are worked out in FP64. What is left are keys whose error is above
    2^-20 of the larger value of their pair, 16 units: none to speak of, and keys under 2^-6
    of the scale. At most one."""
    need_gpu()
    T, heads = 2 ** 23 // (8 * D), 8
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(T, 2 * heads, D, device="cuda", generator=g).to(B16)
    w = (1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(B16)
    turn = torch.arange(T)[:, None] * 10000.0 ** (-torch.arange(rot // 2) * 2.0 / rot)
    cs = torch.cat([turn.cos(), turn.sin()], 1).float().cuda()
    pos = torch.randperm(T, device="cuda", generator=g).to(I32) if placed else None
    pages = -(-T // 64)
    cache = torch.zeros(pages, 2, heads, 64, D, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, 2, heads, 4, dtype=torch.uint8, device="cuda")
    cu, kv = (torch.tensor(a, dtype=I32, device="cuda") for a in ([0, T], [T]))
    table = torch.randperm(pages, device="cuda", generator=g).to(I32)[None]
    ws = ig.mx4_workspace()
    k, v = x[:, :heads], x[:, heads:]
    ig.kv_append(k, v, cache, scales, cu, kv, table, ws, w_k=w, cos_sin=cs, positions=pos, eps=1e-6,
                 flags=ig.ROPE_INTERLEAVED if inter else 0)
    got, _ = torch.empty(2, T, heads, D, dtype=B16, device="cuda")
    ig.kv_gather(cache, scales, cu, kv, table, got, torch.empty_like(got), ws)
    assert ig.check_status(ws) == 0
    y = k.double()
    y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    c, s = cs.double()[torch.arange(T) if pos is None else pos.long()][:, None].chunk(2, -1)
    a, b = (y[..., :rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    one, two = a * c - b * s, b * c + a * s
    y[..., :rot] = torch.stack([one, two], -1).flatten(-2) if inter else torch.cat([one, two], -1)
    scale = scales[table[0].long(), 0].permute(0, 2, 1).reshape(-1, heads)[:T // 16].double()
    z = y.view(-1, 16, heads, D) / torch.exp2(scale - 127)[:, None, :, None]
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    want = (z / step).round() * step * torch.exp2(scale - 127)[:, None, :, None]
    assert z.abs().max() <= 448
    assert (want.view(T, heads, D) != got.double()).sum() <= 1
