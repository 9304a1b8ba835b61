"""Cases of the served layer's attention: head norms with rotation, the 8-bit paged cache and
attention over it.

Cache: codes uint8 [pages][2][kv heads][page][D] (side 0 keys, 1 values; e4m3: 4 exponent and 3
mantissa bits, largest 448, 0x7f and 0xff NaN), scales uint8 [pages][2][kv heads][page / 16]: 16
tokens of a head share the scale 2^(byte - 127). Token j of sequence b is in row j % page of page
page_table[b][j / page]. Tokens of all sequences are stacked: sequence b has the rows
cu[b]..cu[b + 1] - 1, and they are its last ones, positions kv_len[b] - rows..kv_len[b] - 1.

  qk      x = x * rsqrt(mean(x^2) + eps) * w for each head, then pairs (x1, x2) of its first `rot`
          values become (x1 cos - x2 sin, x2 cos + x1 sin)
  append  q and k like that, q returned; k and v into the cache. A block's scale is the smallest
          power of two, at least 2^-120, with max|value| <= 448 scale over its tokens' finite
          values; where the block already holds older tokens it is at least their scale, and they
          are divided by what it grew. Rounded to nearest, ties to even. Returned: what the
          blocks with new tokens hold, up to the last token.
  attn    o = sum_j softmax_j(q.k_j / sqrt(D)) v_j over the tokens j up to the row's own
"""
import math
import random

import torch

own = False

EPS = 1e-6
BLOCK = 16
B16 = torch.bfloat16


def _case(name, op, B, q, kv, hq, hkv, d, page=64, rot=None, inter=False, norm=True, ragged=True):
    c = dict(op=op, B=B, q=q, kv=kv, hq=hq, hkv=hkv, d=d, page=page, rot=d if rot is None else rot,
             inter=inter, norm=norm, ragged=ragged)
    return c if name is None else dict(name=name, **c)


def listed():
    return [
        # one token on its way into a decode layer's attention
        _case("qk_T1_h32_8_d128", "qk", 1, 1, 1, 32, 8, 128),
        # a ragged batch, half of each head rotated, neighbours as pairs
        _case("qk_T1001_h16_2_d64", "qk", 1, 1001, 1001, 16, 2, 64, rot=32, inter=True),
        # a large prefill batch
        _case("qk_T8192_h64_8_d128", "qk", 1, 8192, 8192, 64, 8, 128),
        # decode, one token
        _case("append_B1_h32_8_d128", "append", 1, 1, 1000, 32, 8, 128),
        # decode, a full batch at every place of a block, no head norms
        _case("append_B256_h32_8_d128", "append", 256, 1, 4096, 32, 8, 128, norm=False),
        # five prompts of odd lengths behind earlier turns
        _case("append_B5_q3001_h64_8_d128", "append", 5, 3001, 5000, 64, 8, 128),
        # decode, one sequence: latency
        _case("attn_B1_kv777_h32_8_d128", "attn", 1, 1, 777, 32, 8, 128),
        # decode, a full batch of ragged contexts
        _case("attn_B64_kv8192_h64_8_d128", "attn", 64, 1, 8192, 64, 8, 128),
        # decode, long contexts
        _case("attn_B8_kv65536_h32_8_d128", "attn", 8, 1, 65536, 32, 8, 128),
        # a few drafted tokens a sequence, small heads and pages
        _case("attn_B33_q4_kv2500_h12_4_d64", "attn", 33, 4, 2500, 12, 4, 64, page=16),
        # prompts of odd lengths, nothing before them
        _case("attn_B3_q4095_h32_8_d128", "attn", 3, 4095, 4095, 32, 8, 128),
        # a chunk of a long prompt over what is there already
        _case("attn_q2048_kv32768_h32_8_d128", "attn", 1, 2048, 32768, 32, 8, 128, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "append", "attn", "attn", "attn"])
    hkv = rng.choice([1, 2, 4, 5, 8])
    d = rng.choice([64, 128, 128])
    hq = hkv * rng.choice([1, 2, 3, 4, 7, 8, 16] if hkv < 8 else [1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    rot = rng.choice([d, d, d // 2])
    inter, norm = rng.random() < 0.3, rng.random() < 0.6
    if op == "qk":
        T = _log(rng, 1, 8192 * 72 // (hq + hkv) * 128 // d)
        return _case(None, op, 1, min(T, 60000), min(T, 60000), hq, hkv, d, page, rot, inter, norm)
    kind = rng.choice(["one", "one", "few", "prompt"])
    if kind == "prompt":
        B = rng.choice([1, 1, 2, 3, 5])
        q = _log(rng, 17, 4096 // B)
        kv = q if rng.random() < 0.4 else q + _log(rng, 1, 24000 // B)
        kv = max(q, min(kv, 2048 * 32768 * 4096 // (B * q * hq * d)))
    else:
        q = 1 if kind == "one" else rng.randint(2, 16)
        kv = _log(rng, q, 65536)
        B = _log(rng, 1, max(1, min(256, (1 << 29) // max(4096, kv * hkv * d))))
    if op == "append":
        kv = min(kv, q + 4096)
    return _case(None, op, B, q, kv, hq, hkv, d, page, rot, inter, norm, rng.random() < 0.7)


def _lengths(case):
    """(new tokens, tokens in all) of each sequence: the largest first, where ragged the others
    between a tenth of it and all, and of the new ones between one and all."""
    r = random.Random(case["B"] * 1000003 + case["q"] * 101 + case["kv"])
    got = [(case["q"], case["kv"])]
    for _ in range(case["B"] - 1):
        if not case["ragged"]:
            got.append(got[0])
            continue
        q = case["q"] if case["q"] <= 2 else r.randint(max(1, case["q"] // 10), case["q"])
        alone = case["kv"] == case["q"]
        got.append((q, q if alone else max(q, r.randint(max(1, case["kv"] // 10), case["kv"]))))
    return got


def _blocks(lengths):
    """Tokens from the start of the first block with new tokens, for each sequence."""
    return [kv - (kv - q) // BLOCK * BLOCK for q, kv in lengths]


def work(case):
    n = _lengths(case)
    T, hq, hkv, d = sum(q for q, _ in n), case["hq"], case["hkv"], case["d"]
    table = 4 * case["rot"] * min(T, max(kv for _, kv in n))
    if case["op"] == "qk":
        return {"bytes": 4 * T * (hq + hkv) * d + table, "flops": 0}
    if case["op"] == "append":
        # q in and out, k and v in, their codes and scales out; what the blocks hold in and out
        held = sum(_blocks(n)) * hkv * d
        return {"bytes": 4 * T * hq * d + table + 2 * T * hkv * d * 3 + 2 * held * 3, "flops": 0}
    pairs = sum(q * (kv - q) + q * (q + 1) // 2 for q, kv in n)
    held = sum(kv * d + -(-kv // BLOCK) for _, kv in n) * 2 * hkv
    return {"bytes": held + 4 * T * hq * d, "flops": 4 * pairs * hq * d}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) % (1 << 62))
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(rows, rot):
    """cos and sin of the angles of each position, FP32 from angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _cache(pages, case, g):
    """Keys with a few large channels and values, each token a size of its own."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    codes = torch.empty(pages, 2, hkv, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, 2, hkv, page // BLOCK, dtype=torch.uint8, device="cuda")
    grow = torch.ones(2, hkv, 1, d, device="cuda")
    grow[0, :, :, :: 16] = 4.0
    step = max(1, (1 << 27) // (2 * hkv * page * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn(n, 2, hkv, page, d, device="cuda", generator=g) * grow
        x *= torch.rand(n, 2, hkv, page, 1, device="cuda", generator=g) + 0.5
        x = x.view(-1, BLOCK, d)
        e = _exponent(x.abs().amax((1, 2)))
        codes[a:a + n] = _encode(x, e[:, None, None]).view(n, 2, hkv, page, d)
        scales[a:a + n] = (e + 127).to(torch.uint8).view(n, 2, hkv, page // BLOCK)
    return codes, scales


def prepare(case, seed):
    if own:
        import invariant_gemm_gb300 as ig
    g = _gen(seed)
    rnd = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    n = _lengths(case)
    B, hq, hkv, d, page = len(n), case["hq"], case["hkv"], case["d"], case["page"]
    T, op = sum(q for q, _ in n), case["op"]
    cu = [0]
    for q, _ in n:
        cu.append(cu[-1] + q)
    s = {"op": op, "T": T, "max_q": max(q for q, _ in n), "max_kv": max(kv for _, kv in n)}
    if op != "attn":
        # q, k and v of a token side by side, as the projection leaves them
        qkv = (rnd(T, (hq + 2 * hkv) * d) * 1.5).to(B16)
        s["q"] = qkv[:, :hq * d].view(T, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
        w = (1 + 0.1 * rnd(2, d)).to(B16) if case["norm"] else (None, None)
        s["w_q"], s["w_k"] = w[0], w[1]
        s["inter"], s["rot"] = case["inter"], case["rot"]
        s["cos_sin"] = _table(max(kv for _, kv in n), case["rot"])
        s["pos"] = _ints([p for q, kv in n for p in range(kv - q, kv)])
        if own:
            s["flags"] = ig.ROPE_INTERLEAVED if case["inter"] else 0
            s["q_out"] = torch.empty(T, hq, d, dtype=B16, device="cuda")
            s["ws"] = ig.mx4_workspace()
    if op == "qk":
        if own:
            s["k_out"] = torch.empty(T, hkv, d, dtype=B16, device="cuda")
        return s
    # pages of all sequences in any order, some others between them
    need = [-(-kv // page) for _, kv in n]
    pages = sum(need) + max(1, sum(need) // 16)
    s["cache"], s["scales"] = _cache(pages, case, g)
    order = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["table"], s["cu"], s["kv_len"] = table, _ints(cu), _ints([kv for _, kv in n])
    if op == "append":
        rows = [0]
        for r in _blocks(n):
            rows.append(rows[-1] + r)
        s["cu_read"], s["R"] = _ints(rows), rows[-1]
        if own:
            s["k_read"] = torch.empty(rows[-1], hkv, d, dtype=B16, device="cuda")
            s["v_read"] = torch.empty(rows[-1], hkv, d, dtype=B16, device="cuda")
        return s
    s["q"] = (rnd(T, hq, d) * 1.5).to(B16)
    if own:
        s["out"] = torch.empty(T, hq, d, dtype=B16, device="cuda")
        s["ws"] = ig.attention_workspace(s["q"], s["cache"], s["table"], max_q=s["max_q"])
    return s


# ------------------------------------------------------------ plain forms

def _power(e):
    """2^e as FP32 for whole e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(top):
    """The smallest e, at least -120, with top <= 448 * 2^e."""
    m, x = torch.frexp(top)
    return torch.where(top > 0, x - 9 + (m > 0.875).int(), -120).clamp(min=-120)


def _encode(x, e):
    """e4m3 codes of x / 2^e (FP32, finite ones within 448), NaN for what is not finite."""
    v = x * _power(-e)
    a = v.abs()
    fine = torch.isfinite(a)
    a = torch.where(fine, a, 0)
    step = (torch.frexp(a)[1] - 1).clamp(min=-6)              # the binade
    q = torch.round(a * _power(3 - step)).int()               # whole steps, 8 to 16 in a binade
    code = torch.where(a > 0, q + (step + 6) * 8, 0)
    code = torch.where(fine, code, 127) | (torch.signbit(v).int() << 7)
    return code.to(torch.uint8)


def _decode(codes):
    """What e4m3 codes stand for, FP32."""
    c = codes.int()
    e, m = (c >> 3) & 15, c & 7
    mag = torch.where(e > 0, (8 + m).float() * _power(e - 10), m.float() * 2.0 ** -9)
    mag = torch.where((c & 127) == 127, float("nan"), mag)
    return torch.where(c >= 128, -mag, mag)


def _rotated(x, w, s):
    """Head norm and rotation of x [T][heads][D], FP32."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    half = s["rot"] // 2
    t = s["cos_sin"][s["pos"].long()][:, None]
    cos, sin = t[..., :half], t[..., half:]
    if s["inter"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _held(s, pos):
    """Keys and values [2][B][n][kv heads][D] of positions pos [B][n], FP32."""
    page = s["cache"].shape[3]
    p = torch.gather(s["table"].long(), 1, pos // page)
    codes = s["cache"][p, :, :, pos % page]                   # [B][n][2][heads][D]
    scales = s["scales"][p, :, :, pos % page // BLOCK].int() - 127
    return (_decode(codes) * _power(scales)[..., None]).permute(2, 0, 1, 3, 4)


def _append(s):
    cache, scales, cu, kv = s["cache"], s["scales"], s["cu"].long(), s["kv_len"].long()
    page = cache.shape[3]
    hkv, d = s["k"].shape[1:]
    q = _rotated(s["q"], s["w_q"], s).to(B16)
    new = torch.stack((_rotated(s["k"], s["w_k"], s), s["v"].float()), 1)     # [T][2][heads][D]
    # blocks with new tokens, padded to the longest sequence's
    first = kv - (cu[1:] - cu[:-1])
    nb = (s["max_q"] + 2 * BLOCK - 2) // BLOCK
    blk = first[:, None] // BLOCK + torch.arange(nb, device="cuda")           # [B][nb]
    pos = blk[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")         # [B][nb][16]
    is_new = (pos >= first[:, None, None]) & (pos < kv[:, None, None])
    is_old = pos < first[:, None, None]
    live = is_new.any(-1)
    at = torch.where(is_new, pos - first[:, None, None] + cu[:-1, None, None], 0)
    x = new[at][live]                                                         # [n][16][2][heads][D]
    fresh, old = is_new[live], is_old[live]
    p = torch.gather(s["table"].long(), 1, torch.where(live, blk * BLOCK // page, 0))[live]
    row = (pos % page)[live]                                                  # [n][16]
    inside = row[:, 0] // BLOCK
    codes = cache[p[:, None], :, :, row]                                      # [n][16][2][heads][D]
    was = scales[p, :, :, inside].int() - 127                                 # [n][2][heads]
    mine = fresh[:, :, None, None, None]
    top = torch.where(mine & torch.isfinite(x), x.abs(), 0).amax((1, 4))
    e = _exponent(top)
    e = torch.where(old.any(1)[:, None, None], torch.maximum(e, was), e)
    at_e = e[:, None, :, :, None]
    again = _encode(_decode(codes) * _power((was - e).clamp(min=-126))[:, None, :, :, None],
                    torch.zeros_like(at_e))
    codes = torch.where(mine, _encode(x, at_e), torch.where(old[:, :, None, None, None], again, codes))
    cache[p[:, None], :, :, row] = codes
    scales[p, :, :, inside] = (e + 127).to(torch.uint8)
    # what these blocks hold
    rows = torch.arange(s["R"], device="cuda")
    b = torch.bucketize(rows, s["cu_read"].long()[1:], right=True)
    read = kv[b] - s["cu_read"].long()[1:][b] + rows
    got = _decode(cache[s["table"].long()[b, read // page], :, :, read % page])
    sc = scales[s["table"].long()[b, read // page], :, :, read % page // BLOCK].int() - 127
    got = (got * _power(sc)[..., None]).to(B16)
    return {"q": q, "k": got[:, 0], "v": got[:, 1]}


def _attend(s):
    q, cu, kv = s["q"], s["cu"].long(), s["kv_len"].long()
    T, hq, d = q.shape
    hkv, mq, mkv = s["cache"].shape[2], s["max_q"], s["max_kv"]
    B = kv.shape[0]
    j = torch.arange(mkv, device="cuda")
    k, v = _held(s, torch.minimum(j, kv[:, None] - 1))                        # [B][kv][heads][D]
    t = torch.arange(mq, device="cuda")
    n = cu[1:] - cu[:-1]
    rows = torch.minimum(cu[:-1, None] + t, cu[1:, None] - 1)                 # [B][q]
    x = q.float()[rows].view(B, mq, hkv, hq // hkv, d)
    last = (kv - n)[:, None] + torch.minimum(t, n[:, None] - 1)               # [B][q]
    a = torch.einsum("bthgd,bjhd->bhgtj", x, k) * (1.0 / math.sqrt(d))
    a.masked_fill_((j > last[..., None])[:, None, None], float("-inf"))
    a = torch.exp_(a.sub_(a.amax(-1, keepdim=True)))
    o = torch.einsum("bhgtj,bjhd->bthgd", a, v) / a.sum(-1).permute(0, 3, 1, 2)[..., None]
    return {"o": o.reshape(B, mq, hq, d)[t < n[:, None]].to(B16)}


def run(s):
    if not own:
        if s["op"] == "qk":
            return {"q": _rotated(s["q"], s["w_q"], s).to(B16), "k": _rotated(s["k"], s["w_k"], s).to(B16)}
        return _append(s) if s["op"] == "append" else _attend(s)
    import invariant_gemm_gb300 as ig
    if s["op"] == "qk":
        ig.qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["ws"], w_q=s["w_q"], w_k=s["w_k"],
                        cos_sin=s["cos_sin"], positions=s["pos"], eps=EPS, flags=s["flags"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "append":
        ig.kv_append(s["k"], s["v"], s["cache"], s["scales"], s["cu"], s["kv_len"], s["table"], s["ws"],
                     w_k=s["w_k"], cos_sin=s["cos_sin"], positions=s["pos"], q=s["q"],
                     q_out=s["q_out"], w_q=s["w_q"], eps=EPS, max_q=s["max_q"], flags=s["flags"])
        ig.kv_gather(s["cache"], s["scales"], s["cu_read"], s["kv_len"], s["table"], s["k_read"],
                     s["v_read"], s["ws"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    ig.paged_attention(s["q"], s["cache"], s["scales"], s["cu"], s["kv_len"], s["table"], s["out"],
                       s["ws"], max_q=s["max_q"])
    return {"o": s["out"]}


# --------------------------------------------------------- 64-bit results

def _e4m3_values():
    """The 127 magnitudes of e4m3, by its definition."""
    return [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16)
                                                for m in range(8) if (e, m) != (15, 7)]


def _exact_rotated(x, w, s, angles):
    T, heads, d = x.shape
    y = x.double().clone()
    if w is not None:
        y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / d + EPS) * w.double()
    half = s["rot"] // 2
    c, n = angles[:, None, :half], angles[:, None, half:]
    one = torch.arange(half, device="cuda") * (2 if s["inter"] else 1)
    two = one + (1 if s["inter"] else half)
    a, b = y[..., one], y[..., two]
    y[..., one], y[..., two] = a * c - b * n, a * n + b * c
    return y


def _exact_rounded(v):
    """Nearest e4m3 value to v (64 bits, within 448), ties to the even code."""
    vals = torch.tensor(_e4m3_values(), dtype=torch.float64, device=v.device)
    a = v.abs()
    up = torch.searchsorted(vals, a).clamp(max=126)
    down = (up - 1).clamp(min=0)
    hi, lo = vals[up] - a, a - vals[down]
    take = torch.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, down)
    take = torch.where(a == vals[up], up, take)
    return torch.copysign(vals[take], v)


def _exact_held(s, b, first, last):
    """Keys and values [2][n][heads][D] of sequence b, tokens first..last - 1."""
    page = s["cache"].shape[3]
    mags = torch.tensor(_e4m3_values() + [math.nan], dtype=torch.float64, device="cuda")
    j = torch.arange(first, last, device="cuda")
    p = s["table"][b].long()[j // page]
    c = s["cache"][p, :, :, j % page].long()
    v = mags[c & 127] * (1 - 2 * (c >> 7)).double()
    sc = torch.exp2(s["scales"][p, :, :, j % page // BLOCK].double() - 127)
    return (v * sc[..., None]).transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attn":
        angles = s["cos_sin"].double()[s["pos"].long()]
        q = _exact_rotated(s["q"], s["w_q"], s, angles)
        k = _exact_rotated(s["k"], s["w_k"], s, angles)
    if case["op"] == "qk":
        return {"q": q, "k": k}
    n = _lengths(case)
    if case["op"] == "append":
        got, t = [], 0
        for b, (m, kv) in enumerate(n):
            start = (kv - m) // BLOCK * BLOCK
            rows = -(-kv // BLOCK) * BLOCK - start
            x = torch.zeros(2, rows, *k.shape[1:], dtype=torch.float64, device="cuda")
            older = kv - m - start
            if older:
                x[:, :older] = _exact_held(s, b, start, kv - m)
            x[0, older:kv - start], x[1, older:kv - start] = k[t:t + m], s["v"][t:t + m].double()
            x = x.view(2, rows // BLOCK, BLOCK, *k.shape[1:])
            fresh = x.clone()
            fresh[:, 0, :older] = 0
            top = fresh.abs().amax((2, 4), keepdim=True)
            e = torch.ceil(torch.log2(top / 448)).clamp(min=-120)
            e = e + (top > 448 * torch.exp2(e)).double()
            e = e - ((top <= 448 * torch.exp2(e - 1)) & (e > -120)).double()
            if older:
                page = s["cache"].shape[3]
                was = s["scales"][s["table"][b, start // page].long(), :, :, start % page // BLOCK]
                e[:, 0] = torch.maximum(e[:, 0], was.double()[:, None, :, None] - 127)
            x = _exact_rounded(x * torch.exp2(-e)) * torch.exp2(e)
            got.append(x.reshape(2, rows, *k.shape[1:])[:, :kv - start])
            t += m
        got = torch.cat(got, 1)
        return {"q": q, "k": got[0], "v": got[1]}
    hq, d = case["hq"], case["d"]
    hkv = case["hkv"]
    out, t = torch.empty(s["T"], hq, d, dtype=torch.float64, device="cuda"), 0
    for b, (m, kv) in enumerate(n):
        k, v = _exact_held(s, b, 0, kv)
        for a in range(0, m, 512):
            z = min(m, a + 512)
            for h in range(hkv):
                x = s["q"][t + a:t + z, h * (hq // hkv):(h + 1) * (hq // hkv)].double()
                w = torch.matmul(x, k[:, h].t()) / math.sqrt(d)
                seen = torch.arange(kv, device="cuda") <= torch.arange(kv - m + a, kv - m + z,
                                                                       device="cuda")[:, None]
                w = torch.where(seen[:, None], w, -math.inf)
                w = torch.softmax(w, -1)
                out[t + a:t + z, h * (hq // hkv):(h + 1) * (hq // hkv)] = torch.matmul(w, v[:, h])
        t += m
    return {"o": out}
