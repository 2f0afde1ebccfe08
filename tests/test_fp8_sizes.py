"""Workspace sizes of the dense layers in 8 bits, and the cut of their products that they follow from."""
import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B

BF16 = torch.bfloat16


# ------------------------------------------------------------------ a layer that is used on two devices
class On(torch.Tensor):
    """A tensor that says it is on a device."""

    @classmethod
    def make(cls, index, *shape, dtype=BF16):
        t = torch.zeros(*shape, dtype=dtype).as_subclass(cls)
        t.index = index
        return t

    def get_device(self):
        return self.index


def weight(index, n, k):
    return On.make(index, n, k, dtype=torch.uint8), On.make(index, *B.fp8_scales_shape(n, k, M.MOE_B_SQUARE), dtype=torch.float32)


def test_one_layer_on_two_devices_takes_each_ones_sizes(monkeypatch):
    """The size of a workspace goes by the current device's number of SMs: here 100 bytes on device 0 and 200 on device 1."""
    now, given = [0], []
    for name in ("moe_linear_size", "moe_ffn_size"):
        monkeypatch.setattr(B, name, lambda cfg, T, backward=False: 100 * (now[0] + 1))

    def call(at):
        return lambda *args: given.append(args[at]) or 0

    lin, ffn = M.MoEFp8Linear(32, 64), M.MoEFeedForward(32, 64)
    for layer in (lin, ffn):
        layer._current, layer._stream = (lambda: now[0]), (lambda index: None)
        layer._forward, layer._backward = call(9), call(13 if layer is lin else 12)
    for index in (0, 1, 0, 1):
        now[0] = index
        x, y = On.make(index, 4, 32), On.make(index, 4, 64)
        w = weight(index, 64, 32)
        f = M.FeedForwardWeights(w, w, weight(index, 32, 64))
        column, row = weight(index, 4, 32)[0], weight(index, 4, 64)[0]
        kept = (column, On.make(index, 1, 32, dtype=torch.float32))
        gate = (row, On.make(index, 1, 4, dtype=torch.float32))
        given.clear()
        lin.forward(x, w)
        lin.backward(y, w, kept)
        ffn.forward(x, f)
        ffn.backward(x, f, (kept, gate, gate), grads=[On.make(index, *n) for n in ((64, 32), (64, 32), (32, 64))])
        assert given == [100 * (index + 1)] * 4
