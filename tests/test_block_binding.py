"""What the binding of the quantised-block calls refuses before the library is
called, for operands that are on a GPU as far as it can see: the tensors here
are CPU tensors that name a GPU, and the library is a stand-in that records its
calls. Nothing reaches a GPU."""
import pytest
import torch

import invariant_gemm_gb300 as ig

U8, B16, F32 = torch.uint8, torch.bfloat16, torch.float32


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on GPU 1."""

    def get_device(self):
        return 1


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


def on(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def library(monkeypatch):
    """Current GPU and library as the binding sees them."""
    rec = Recorder()
    rec.ig_status_string = ig.lib().ig_status_string
    rec.current = 1
    monkeypatch.setattr(ig, "_LIB", rec)
    monkeypatch.setattr(ig, "_ONE_GPU", False)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: rec.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return rec


def operands():
    M, H = 4, 64
    return dict(x=on(torch.zeros(M, H, dtype=B16)), c=on(torch.zeros(M, H // 2, dtype=U8)),
                s=on(torch.zeros(512, dtype=U8)), y=on(torch.zeros(M, M, dtype=F32)),
                ws=on(torch.zeros(512, dtype=U8)), w=on(torch.ones(H, dtype=B16)))


CALLS = {
    "mx4_quantize": lambda o, **k: ig.mx4_quantize(o["x"], o["c"], o["s"], **k),
    "mx4_dequantize": lambda o, **k: ig.mx4_dequantize(o["c"], o["s"], o["x"], **k),
    "mx4_gemm": lambda o, **k: ig.mx4_gemm(o["c"], o["s"], o["c"], o["s"], o["y"], o["ws"], **k),
    "block_norm": lambda o, **k: ig.block_norm(o["x"], o["x"], o["w"], o["w"], n_out=o["x"], **k),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, 0])
def test_operands_on_a_gpu_that_is_not_current(library, name, stream):
    """The library launches on the current GPU: operands on another one would be
    read there, on a stream of the wrong GPU."""
    CALLS[name](operands(), stream=stream)
    assert library.calls == ["ig_" + name]
    library.current = 0
    with pytest.raises(ig.IGError) as e:
        CALLS[name](operands(), stream=stream)
    assert e.value.code == -1 and "GPU 1" in str(e.value) and "GPU 0" in str(e.value)
    assert library.calls == ["ig_" + name]


@pytest.mark.parametrize("post,pre", [(128, 64), (64, 128), (32, 64), (64, 72)])
def test_norm_weights_of_another_size(library, post, pre):
    """A weight of more than H values is not one of H: its first row may be
    another layer's."""
    o = operands()
    w = {n: on(torch.ones(n, dtype=B16)) for n in (post, pre)}
    with pytest.raises(ig.IGError) as e:
        ig.block_norm(o["x"], o["x"], w[post], w[pre], n_out=o["x"])
    assert e.value.code == -2 and library.calls == []
