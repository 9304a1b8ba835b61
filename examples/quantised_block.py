"""One served layer around the adapters, with the library's calls alone:

    h' = h + scale * gate * norm(y_prev)          block_norm
    n  = norm(h')            bf16 and MX4         (the same call)
    y  = n_mx4 W_mx4^T                            mx4_gemm
    y += s (n A_i^T) B_i^T   per-token adapter    lora_apply
    h" = h' + scale * gate * norm(y)              block_norm

It runs the layer in a CUDA graph, checks it against a plain FP32 computation on
the same quantised operands and prints the error and the time of a replay.

    python examples/quantised_block.py [--tokens 256] [--hidden 4096] [--rank 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import invariant_gemm_gb300 as ig  # noqa: E402

EPS, SCALE = 1e-6, 2.0


class Layer:
    """Weights laid out once, buffers for up to `tokens` tokens, and run()."""

    def __init__(self, tokens, hidden, rank, adapters, seed=0, residual_scale=0.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        b16 = torch.bfloat16
        self.scale = residual_scale
        self.w = rnd(hidden, hidden) / hidden ** 0.5
        self.w_codes = torch.empty(hidden, hidden // 2, dtype=torch.uint8, device="cuda")
        self.w_scales = torch.empty(ig.mx4_scale_bytes(hidden, hidden), dtype=torch.uint8,
                                    device="cuda")
        ig.mx4_quantize(self.w, self.w_codes, self.w_scales)
        self.A = (rnd(adapters, 1, rank, hidden) / hidden ** 0.5).to(b16)
        self.B = (rnd(adapters, 1, hidden, rank) / rank ** 0.5).to(b16)
        self.norms = [(1 + 0.1 * rnd(hidden)).to(b16) for _ in range(3)]
        self.gate = torch.rand(1, hidden, device="cuda", generator=g).to(b16)

        self.shape = ig.make_shape(tokens, hidden, hidden, rank, num_adapters=adapters,
                                   flags=ig.FLAG_STATIC_WEIGHTS)
        self.ws = ig.workspace(self.shape)      # serves mx4_gemm as well
        self.z = torch.empty(1, tokens, rank, device="cuda")
        self.n = torch.empty(tokens, hidden, dtype=b16, device="cuda")
        self.codes = torch.empty(tokens, hidden // 2, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(ig.mx4_scale_bytes(tokens, hidden), dtype=torch.uint8,
                                  device="cuda")
        self.y = torch.empty(tokens, hidden, dtype=b16, device="cuda")
        torch.cuda.synchronize()                # the weights are laid out

    def run(self, h, y_prev, idx):
        """h [tokens][hidden] is updated in place."""
        post, pre, last = self.norms
        ig.block_norm(h, y_prev, post, pre, gate=self.gate, scale=self.scale, eps=EPS, h_out=h,
                      n_out=self.n, codes=self.codes, scales=self.scales)
        ig.mx4_gemm(self.codes, self.scales, self.w_codes, self.w_scales, self.y, self.ws,
                    flags=ig.FLAG_STATIC_WEIGHTS)
        ig.lora_apply(self.shape, self.n, self.y, idx, self.A, self.B, SCALE, self.z, self.ws)
        ig.block_norm(h, self.y, last, gate=self.gate, scale=self.scale, eps=EPS, h_out=h)

    def plain(self, h, y_prev, idx):
        """The same in FP32 torch operations, rounded where the layer stores."""
        def norm(v, w):
            return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.float()

        post, pre, last = self.norms
        gate = self.gate.float() * self.scale
        h1 = h.float() + gate * norm(y_prev.float(), post)
        n = norm(h1, pre).to(torch.bfloat16)
        x, w = torch.empty_like(n), torch.empty_like(self.w)
        ig.mx4_dequantize(self.codes, self.scales, x)
        ig.mx4_dequantize(self.w_codes, self.w_scales, w)
        y = (x.float() @ w.t()).to(torch.bfloat16).float()
        a, b = self.A[idx.long(), 0].float(), self.B[idx.long(), 0].float()
        z = SCALE * torch.einsum("mk,mrk->mr", n.float(), a)
        z = z.to(torch.bfloat16).float()
        y = (y + torch.einsum("mr,mnr->mn", z, b)).to(torch.bfloat16).float()
        h1 = h1.to(h.dtype).float()
        return h1 + gate * norm(y, last)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--adapters", type=int, default=8)
    a = ap.parse_args(argv)
    layer = Layer(a.tokens, a.hidden, a.rank, a.adapters)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(a.tokens, a.hidden, device="cuda", generator=g)
    y_prev = torch.randn(a.tokens, a.hidden, device="cuda", generator=g).to(torch.bfloat16)
    idx = torch.randint(0, a.adapters, (a.tokens,), device="cuda", dtype=torch.int32, generator=g)

    got = h.clone()
    layer.run(got, y_prev, idx)
    status = ig.check_status(layer.ws)
    assert status == 0, ig.status_string(status)
    # small batches: the plain form gathers an A and a B for every token
    ref = layer.plain(h, y_prev, idx)
    err = ((got - ref).norm() / ref.norm()).item()

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    work = h.clone()
    with torch.cuda.graph(graph, stream=stream):
        work.copy_(h)
        layer.run(work, y_prev, idx)
    graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(work, got)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    with torch.cuda.stream(stream):
        start.record()
        for _ in range(100):
            graph.replay()
        stop.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(stop) * 10
    print(f"tokens {a.tokens}, hidden {a.hidden}, rank {a.rank}: relative error {err:.2e}, "
          f"replay bit-identical: {same}, {us:.1f} us a layer")
    assert err < 5e-3 and same
    return err


if __name__ == "__main__":
    main()
