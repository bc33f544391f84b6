"""The training step's entry points take tensors of the current device only, every argument of them (no GPU needed:
stubs stand for the tensors, and a call that is refused reaches no kernel)."""
import math

import pytest

from tests.test_abi import moe  # noqa: F401

T, K, F, H = 64, 128, 512, 128
CFG = dict(hidden=128, num_experts=8, top_k=2, intermediate=256, block_size=8)
ROWS = T * 2 + 8 * 7


class Stub:
    """What the binding looks at in a tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        import torch
        self.dtype, self.shape, self.on = getattr(torch, dtype), shape, 0

    device = property(lambda self: f"cuda:{self.on}")

    def get_device(self):
        return self.on

    def is_contiguous(self):
        return True

    def numel(self):
        return math.prod(self.shape)

    def data_ptr(self):
        return 0x100000000 * (id(self) % 1000 + 1)


def bf(*s):
    return Stub("bfloat16", *s)


def f32(*s):
    return Stub("float32", *s)


def i32(*s):
    return Stub("int32", *s)


def grouped():
    return dict(sorted_route_ids=i32(ROWS), expert_counts=i32(8), ws=Stub("uint8", 256))


def swiglu():
    return dict(gu=bf(ROWS, 512), topk_gate=f32(T, 2), sorted_route_ids=i32(ROWS), num_padded=i32(1), a=bf(ROWS, 256))


# the tensors of each entry point, and its other arguments
CALLS = {
    "moe_grouped_gemm": (lambda: dict(x=bf(T, K), w=bf(8, K, F), y_perm=bf(ROWS, F), **grouped()),
                         dict(cfg=CFG, T=T, gather=True)),
    "moe_grouped_wgrad": (lambda: dict(x=bf(T, K), dy=bf(ROWS, F), dw=f32(8, K, F), dw_add=f32(8, K, F), **grouped()),
                          dict(cfg=CFG, T=T, gather_x=True)),
    "moe_swiglu": (swiglu, dict(cfg=CFG, T=T)),
    "moe_swiglu_backward": (lambda: dict(swiglu(), da=bf(ROWS, 256), dgu=bf(ROWS, 512), dgate=f32(T, 2)),
                            dict(cfg=CFG, T=T)),
    "moe_add_layer_norm": (lambda: dict(x=bf(T, H), residual=bf(T, H), weight=bf(H), bias=bf(H),
                                        residual_out=bf(T, H), out=bf(T, H)), dict(eps=1e-5)),
    "moe_norm_backward": (lambda: dict(v=bf(T, H), dout=bf(T, H), dresidual=bf(T, H), weight=bf(H), dx=bf(T, H),
                                       dweight=f32(H), dbias=f32(H), ws=Stub("uint8", 1 << 20)), dict(eps=1e-5)),
}


@pytest.mark.parametrize("name,tensor", [(n, t) for n, (make, _) in CALLS.items() for t in make()])
@pytest.mark.parametrize("current", [0, 1])
def test_a_tensor_of_another_device_is_refused(moe, monkeypatch, name, tensor, current):  # noqa: F811
    make, rest = CALLS[name]
    called = []
    monkeypatch.setattr(moe, "_current_device", lambda: current)
    monkeypatch.setattr(moe, "_current_stream", lambda: 0)
    monkeypatch.setattr(moe, "_lib", type("Lib", (), {name: staticmethod(lambda *a: called.append(a) or 0)}))
    tensors = make()
    for t in tensors.values():
        t.on = current
    getattr(moe, name)(**tensors, **rest)
    assert len(called) == 1   # on one device all of them are taken
    tensors[tensor].on = 1 - current
    with pytest.raises(ValueError, match=f"^{tensor}: on cuda:{1 - current}, but the current device is cuda:{current}"):
        getattr(moe, name)(**tensors, **rest)
    assert len(called) == 1
