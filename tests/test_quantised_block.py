"""The layer of examples/quantised_block.py: norm, MX4 product, adapters and
norm on one stream, against the plain computation, and its rows in batches of
different sizes."""
import importlib.util
import os

import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "quantised_block.py")


def example():
    spec = importlib.util.spec_from_file_location("quantised_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,hidden,rank", [(1, 1024, 8), (24, 1024, 16), (200, 2048, 64)])
def test_layer_matches_plain_and_replays(tokens, hidden, rank):
    """bf16 rounding of y (2^-9) and of n, at a norm of about that of h: the
    relative error stays under 5e-3."""
    need_gpu()
    assert example().main(["--tokens", str(tokens), "--hidden", str(hidden), "--rank",
                           str(rank)]) < 5e-3


def test_layer_rows_do_not_depend_on_the_batch():
    need_gpu()
    mod = example()
    g = torch.Generator(device="cuda").manual_seed(3)
    H = 1024
    h = torch.randn(300, H, device="cuda", generator=g)
    y = torch.randn(300, H, device="cuda", generator=g).to(torch.bfloat16)
    idx = torch.randint(-1, 4, (300,), device="cuda", dtype=torch.int32, generator=g)
    ref = None
    for tokens in (300, 1, 17, 130):
        layer = mod.Layer(tokens, H, 16, 4)
        out = h[:tokens].clone()
        layer.run(out, y[:tokens].contiguous(), idx[:tokens].contiguous())
        torch.cuda.synchronize()
        ref = out if ref is None else ref
        assert torch.equal(out, ref[:tokens]), tokens
