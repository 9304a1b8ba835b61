"""A served layer with its attention, with the library's calls alone: a ragged batch
of prompts, then single tokens in a CUDA graph.

    n      = norm(h)                  bf16 and MX4          block_norm
    qkv    = n_mx4 W_qkv^T                                  mx4_gemm
    qkv   += s (n A_i^T) B_i^T        per-token adapter     lora_apply
    cache <- norm, rotation of k; v;  q in place            kv_append
    a      = attention over the cache                       paged_attention
    y      = mx4(a) W_out^T                                 mx4_quantize, mx4_gemm
    h     += norm(y)                                        block_norm

The tokens' positions, the lengths and the page table live on the GPU and the graph
advances them, so that a replay is the next token of every sequence. Each step is
checked: what the cache holds against keys and values of FP32 torch operations (e4m3
with a scale per 16 tokens), the layer's result against attention over what it holds.

    python examples/served_attention.py [--prompts 700,33,1200] [--steps 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import invariant_gemm_gb300 as ig  # noqa: E402

EPS, SCALE, PAGE = 1e-6, 2.0, 64
B16, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


class Mx4Weight:
    def __init__(self, w):
        n, k = w.shape
        self.codes = torch.empty(n, k // 2, dtype=U8, device="cuda")
        self.scales = torch.empty(ig.mx4_scale_bytes(n, k), dtype=U8, device="cuda")
        ig.mx4_quantize(w, self.codes, self.scales)
        self.values = torch.empty_like(w)       # for the check
        ig.mx4_dequantize(self.codes, self.scales, self.values)


class Layer:
    """Weights laid out once and the cache of `batch` sequences of up to `longest` tokens."""

    def __init__(self, batch, longest, hidden=1024, heads=16, kv_heads=4, head_dim=64, rank=16,
                 adapters=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.heads, self.kv_heads, self.dim, self.hidden, self.rank = heads, kv_heads, head_dim, hidden, rank
        self.wide = (heads + 2 * kv_heads) * head_dim
        self.adapters = adapters
        self.w_qkv = Mx4Weight(rnd(self.wide, hidden) / hidden ** 0.5)
        self.w_out = Mx4Weight(rnd(hidden, heads * head_dim) / (heads * head_dim) ** 0.5)
        self.A = (rnd(adapters, 1, rank, hidden) / hidden ** 0.5).to(B16)
        self.B = (rnd(adapters, 1, self.wide, rank) / rank ** 0.5).to(B16)
        self.pre, self.post = ((1 + 0.1 * rnd(hidden)).to(B16) for _ in range(2))
        self.norm_q, self.norm_k = ((1 + 0.1 * rnd(head_dim)).to(B16) for _ in range(2))
        inv = 10000.0 ** (-torch.arange(head_dim // 2, device="cuda").double() * 2 / head_dim)
        turn = torch.arange(longest, device="cuda").double()[:, None] * inv
        self.cos_sin = torch.cat([turn.cos(), turn.sin()], 1).float()
        # pages in no order, as a server's pool hands them out
        cols = -(-longest // PAGE)
        order = torch.randperm(batch * cols, device="cuda", generator=g)
        self.table = order.to(I32).view(batch, cols)
        self.cache = torch.zeros(batch * cols, 2, kv_heads, PAGE, head_dim, dtype=U8, device="cuda")
        self.scales = torch.zeros(batch * cols, 2, kv_heads, PAGE // 16, dtype=U8, device="cuda")
        self.kv_len = torch.zeros(batch, dtype=I32, device="cuda")
        self.k = self.v = None

    def buffers(self, tokens, max_q):
        """What a step of so many tokens needs beside the weights."""
        e = lambda *s, t=B16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        wide = self.heads * self.dim
        s = dict(n=e(tokens, self.hidden), codes=e(tokens, self.hidden // 2, t=U8),
                 scales=e(ig.mx4_scale_bytes(tokens, self.hidden), t=U8),
                 qkv=e(tokens, self.heads + 2 * self.kv_heads, self.dim),
                 a=e(tokens, self.heads, self.dim), a_codes=e(tokens, wide // 2, t=U8),
                 a_scales=e(ig.mx4_scale_bytes(tokens, wide), t=U8), y=e(tokens, self.hidden),
                 z=e(1, tokens, self.rank, t=torch.float32), max_q=max_q,
                 shape=ig.make_shape(tokens, self.hidden, self.wide, self.rank,
                                     num_adapters=self.adapters, flags=ig.FLAG_STATIC_WEIGHTS))
        s["lora_ws"] = ig.workspace(s["shape"])
        s["ws"] = ig.attention_workspace(s["a"], self.cache, self.table, max_q)
        return s

    def step(self, s, h, cu, idx):
        """h [tokens][hidden] is updated in place; kv_len counts the new tokens already."""
        q, k, v = s["qkv"].split([self.heads, self.kv_heads, self.kv_heads], 1)
        ig.block_norm(h, None, None, self.pre, eps=EPS, n_out=s["n"], codes=s["codes"],
                      scales=s["scales"])
        ig.mx4_gemm(s["codes"], s["scales"], self.w_qkv.codes, self.w_qkv.scales,
                    s["qkv"].view(len(h), -1), s["ws"], flags=ig.FLAG_STATIC_WEIGHTS)
        ig.lora_apply(s["shape"], s["n"], s["qkv"], idx, self.A, self.B, SCALE, s["z"],
                      s["lora_ws"])
        ig.kv_append(k, v, self.cache, self.scales, cu, self.kv_len, self.table, s["ws"],
                     w_k=self.norm_k, cos_sin=self.cos_sin, q=q, q_out=q, w_q=self.norm_q, eps=EPS,
                     max_q=s["max_q"])
        ig.paged_attention(q, self.cache, self.scales, cu, self.kv_len, self.table, s["a"],
                           s["ws"], max_q=s["max_q"])
        ig.mx4_quantize(s["a"].view(len(h), -1), s["a_codes"], s["a_scales"])
        ig.mx4_gemm(s["a_codes"], s["a_scales"], self.w_out.codes, self.w_out.scales, s["y"],
                    s["ws"], flags=ig.FLAG_STATIC_WEIGHTS)
        ig.block_norm(h, s["y"], self.post, eps=EPS, h_out=h)

    def status(self, s):
        return ig.check_status(s["ws"]) or ig.check_status(s["lora_ws"])

    # --- the same in FP32 torch operations, rounded where the layer stores -----------
    def plain(self, s, h, lengths, idx):
        """h after the step and the relative error of the cache's new keys and values;
        lengths: (new tokens, tokens in all) of each sequence. Codes of the products'
        inputs and the cache are taken from the step, which has run."""
        def norm(x, w):
            return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()

        T, D = len(h), self.dim
        x = torch.empty(T, self.hidden, device="cuda")
        ig.mx4_dequantize(s["codes"], s["scales"], x)
        qkv = (x @ self.w_qkv.values.t()).to(B16).float()
        n = norm(h, self.pre).to(B16).float()
        z = SCALE * torch.einsum("mk,mrk->mr", n, self.A[idx.long(), 0].float())
        z = z.to(B16).float()
        qkv = (qkv + torch.einsum("mr,mnr->mn", z, self.B[idx.long(), 0].float())).to(B16).float()
        q, k, v = qkv.view(T, -1, D).split([self.heads, self.kv_heads, self.kv_heads], 1)
        pos = torch.cat([torch.arange(kv - q_, kv, device="cuda") for q_, kv in lengths])
        cos, sin = self.cos_sin[pos][:, None].chunk(2, -1)

        def rotate(t, w):
            one, two = norm(t, w).chunk(2, -1)
            return torch.cat([one * cos - two * sin, two * cos + one * sin], -1)

        q, k = rotate(q, self.norm_q).to(B16).float(), rotate(k, self.norm_k)
        held_k, held_v, out, row, worst = [], [], [], 0, 0.0
        for b, (q_, kv) in enumerate(lengths):
            hk, hv = (torch.empty(kv, self.kv_heads, D, dtype=B16, device="cuda") for _ in "kv")
            ig.kv_gather(self.cache, self.scales,
                         torch.tensor([0, kv], dtype=I32, device="cuda"), self.kv_len[b:b + 1],
                         self.table[b:b + 1], hk, hv, s["ws"])
            hk, hv = hk.float(), hv.float()
            new = slice(row, row + q_)
            for got, ref in ((hk[kv - q_:], k[new]), (hv[kv - q_:], v[new])):
                worst = max(worst, ((got - ref).norm() / ref.norm()).item())
            group = self.heads // self.kv_heads
            t = torch.einsum("qhd,khd->hqk", q[new], hk.repeat_interleave(group, 1)) * D ** -0.5
            seen = torch.arange(kv, device="cuda")[None] <= torch.arange(
                kv - q_, kv, device="cuda")[:, None]
            p = t.masked_fill(~seen, float("-inf")).softmax(-1)
            out.append(torch.einsum("hqk,khd->qhd", p, hv.repeat_interleave(group, 1)))
            row += q_
        a = torch.cat(out)
        rel = ((s["a"].float() - a).norm() / a.norm()).item()
        x = torch.empty(T, self.heads * D, device="cuda")
        ig.mx4_dequantize(s["a_codes"], s["a_scales"], x)
        y = (x @ self.w_out.values.t()).to(B16).float()
        return h + norm(y, self.post), worst, rel


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", default="700,33,1200")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--head-dim", type=int, default=64)
    a = ap.parse_args(argv)
    prompts = [int(x) for x in a.prompts.split(",")]
    B, T = len(prompts), sum(prompts)
    layer = Layer(B, max(prompts) + a.steps + 4, head_dim=a.head_dim)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda n: torch.randn(n, layer.hidden, device="cuda", generator=g)  # noqa: E731
    errors = []

    def check(s, before, after, lengths, idx):
        status = layer.status(s)
        assert status == 0, ig.status_string(status)
        ref, cache, rel = layer.plain(s, before, lengths, idx)
        errors.append((cache, rel, ((after - ref).norm() / ref.norm()).item()))

    # the prompts, all at once
    idx = torch.repeat_interleave(torch.arange(B, device="cuda", dtype=I32) % layer.adapters,
                                  torch.tensor(prompts, device="cuda"))
    cu = torch.tensor([0] + prompts, device="cuda").cumsum(0).to(I32)
    s = layer.buffers(T, max(prompts))
    layer.kv_len.copy_(torch.tensor(prompts))
    h = rnd(T)
    before = h.clone()
    layer.step(s, h, cu, idx)
    check(s, before, h, [(n, n) for n in prompts], idx)

    # single tokens: one eager step, then a graph whose replays are the next ones
    s = layer.buffers(B, 1)
    idx = torch.arange(B, device="cuda", dtype=I32) % layer.adapters
    cu = torch.arange(B + 1, device="cuda", dtype=I32)
    h, new = rnd(B), rnd(B)

    def one():
        layer.kv_len.add_(1)
        h.copy_(new)
        layer.step(s, h, cu, idx)

    one()
    check(s, new, h, [(1, n + 1) for n in prompts], idx)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        one()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(a.steps):
        graph.replay()
    stop.record()
    torch.cuda.synchronize()
    check(s, new, h, [(1, n + 1 + a.steps) for n in prompts], idx)
    us = start.elapsed_time(stop) * 1000 / a.steps
    for what, (cache, rel, full) in zip(("prompts", "one token", "replayed"), errors):
        print(f"{what}: cache {cache:.2e}, attention {rel:.2e}, layer {full:.2e}")
    print(f"prompts {prompts}, {a.steps} replays: {us:.1f} us a layer")
    return errors


if __name__ == "__main__":
    main()
