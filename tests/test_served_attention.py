"""The layer of examples/served_attention.py: its calls one after the other over prompts,
single tokens and replayed ones, against the plain computation."""
import importlib.util
import os

import pytest

from helpers import need_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "served_attention.py")


@pytest.mark.parametrize("prompts,dim", [("700,33,1200", 64), ("1", 128), ("15,16,17,300", 128)])
def test_layer_matches_plain_and_replays(prompts, dim):
    """Cache: a code is off by half a step, 2^-4 of the value at most, or, where it is
    under 2^-6 scale, by 2^-10 scale. A scale is less than 2/448 of the block's largest value,
    itself less than 8 sqrt(D) times the root mean square of normed keys, so that adds under
    2^-10 * 2 / 448 * 8 * sqrt(128) = 4e-4: below 0.07. Attention: the same q on both
    sides but where FP32 values that differ in their last bits are next to a tie (a step,
    2^-7, of few elements); p within 2^-11, the result within 2^-8: under 1e-2. The layer's y
    is rounded to bf16 (2^-8 at most) from products of the same codes and its norm is that
    of h: under 5e-3."""
    need_gpu()
    spec = importlib.util.spec_from_file_location("served_attention", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for cache, attention, layer in mod.main(["--prompts", prompts, "--steps", "5", "--head-dim",
                                             str(dim)]):
        assert cache < 0.07 and attention < 1e-2 and layer < 5e-3
