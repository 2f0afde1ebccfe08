"""Workspace sizes of the dense layers in 8 bits, and the cut of their products that they follow from."""
import math
import random

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


# ------------------------------------------------------------------ how a product is cut, as the library says it
SMS = 152                      # of a GB300; what the library takes where there is no GPU, too
NT, NN, TN, GATED = "nt", "nn", "tn", "gated"


def blocks(n):
    return -(-n // 128)


def up(n, to):
    return -(-n // to) * to


def ways(op, outs, k_blocks, sms=SMS):
    """[(us by the library's model, (columns of a tile, CTAs of a tile, parts of K))] of products with outputs of the given sizes."""
    gated, found = op == GATED, []
    elements = sum(m * n for m, n in outs)
    small = sum(blocks(m) * blocks(n) for m, n in outs)
    wide = sum(blocks(m) * (blocks(n) if gated else -(-n // 256)) for m, n in outs)
    pairs = sum(-(-m // 256) * (blocks(n) if gated else -(-n // 256)) for m, n in outs)

    def look(bn, cg, splits):
        units, items = sms // cg, (pairs if cg == 2 else wide if bn == 256 else small) * splits
        busy = min(items / units, 1.0)
        chain = (0.3 + 0.25 * busy if bn == 128 else 0.42 + 0.08 * busy if cg == 2 else 0.45 + 0.15 * busy) + (0.35 if op == TN else 0.0)
        ends = (4.0 if bn == 128 else 6.0 if cg == 2 else 5.5) + (3.0 if gated and splits == 1 else 0.0)
        us = -(-items // units) * (ends + chain * -(-k_blocks // splits))
        if splits > 1:
            us += 2.7 + (1.5 if gated else 0.0) + elements * (2 if gated else 1) * splits * 0.8e-6
        found.append((us, (bn, cg, splits)))

    look(256, 2, 1)
    for splits in (1, 2, 3, 4, 5, 6, 8, 10, 12, 16):
        if splits > k_blocks or splits > 1 and wide > sms:
            break
        if gated or op == TN or splits == 1:
            look(256, 1, splits)
        if not gated:
            look(128, 1, splits)
    return found


def cut(op, outs, k_blocks):
    return min(ways(op, outs, k_blocks), key=lambda w: w[0])[1]       # the first of equals, as the library


def variant(op, outs, k_blocks):
    """(the kernel taken: columns, CTAs, whether K is in parts; by how much the next other kernel is slower in the model)."""
    kind = lambda c: (c[0], c[1], c[2] > 1)  # noqa: E731
    every = ways(op, outs, k_blocks)
    us, best = min(every, key=lambda w: w[0])
    return kind(best), min(t for t, c in every if kind(c) != kind(best)) / us - 1


def linear_products(T, K, N):
    return {"y": (NT, [(T, N)], blocks(K)), "dx": (NN, [(T, K)], blocks(N)), "dw": (TN, [(N, K)], blocks(T))}


def ffn_products(T, H, I):
    return {"h": (GATED, [(T, I)], blocks(H)), "y": (NT, [(T, H)], blocks(I)), "dx": (NN, [(T, I)], blocks(H)),     # (dh, by dx's kernels)
            "dx of two": (NN, [(T, H)], 2 * blocks(I)), "three dw": (TN, [(I, H), (I, H), (H, I)], blocks(T))}


def few(T, N, K, gated):
    units = T * blocks(K)
    return T <= 16 and units * 132 <= 128 << 10 and -(-N // (8 if gated else 16)) * units <= 600 * SMS


def codes(rows, cols, by_row):
    return up(rows * up(cols, 16), 256) + up(4 * (blocks(cols) * rows if by_row else blocks(rows) * cols), 256)


def parts(op, outs, k_blocks):
    splits = cut(op, outs, k_blocks)[2]
    return sum(up(4 * splits * (2 if op == GATED else 1) * m * up(n, 256), 256) for m, n in outs) if splits > 1 else 0


def linear_sizes(T, K, N):
    p = linear_products(T, K, N)
    forward = 0 if few(T, N, K, False) else codes(T, K, True) + parts(*p["y"])
    return forward, codes(T, N, True) + codes(T, N, False) + parts(*p["dx"]) + parts(*p["dw"])


def ffn_sizes(T, H, I):
    p = ffn_products(T, H, I)
    forward = codes(T, H, True) + codes(T, I, True) + parts(*p["h"]) + parts(*p["y"])
    if few(T, I, H, True) and few(T, H, I, False):
        forward = max(forward, up(4 * T * up(I, 4), 256))
    back = codes(T, H, True) + codes(T, H, False) + up(4 * T * up(I, 4), 256) + 2 * codes(T, I, True) + 3 * codes(T, I, False)
    return forward, back + parts(*p["dx"]) + parts(*p["dx of two"]) + parts(*p["three dw"])


@pytest.mark.skipif(torch.cuda.is_available(), reason="the sizes go by the GPU's SMs")
def test_sizes_are_those_of_the_cut():
    """Which holds the cut above to the library's own (the parts' sums are most of a workspace), for the tests below that go by it."""
    rng = random.Random(0)
    size = lambda lo, hi: round(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    for _ in range(1500):
        T, a, b = size(1, 16384), size(1, 8192), size(1, 8192)
        lin, ffn = B.moe_linear_config(a, b, 0, 0), B.moe_ffn_config(a, b, 0.0)
        assert (M.moe_linear_size(lin, T), M.moe_linear_size(lin, T, True)) == linear_sizes(T, a, b), (T, a, b)
        assert (M.moe_ffn_size(ffn, T), M.moe_ffn_size(ffn, T, True)) == ffn_sizes(T, a, b), (T, a, b)


def test_every_kernel_that_a_cut_takes_is_compared_with_the_formulas():
    """The kernels that some size takes are all met by a case that is compared with its 64-bit formulas, most of them by one where the next
    kernel is 5 % slower in the model, so that a constant of it may be measured anew."""
    from tests import test_gpu_fp8, test_gpu_fp8_cuts
    met = {}
    for T, K, N, *_ in test_gpu_fp8.LINEAR + test_gpu_fp8_cuts.LINEAR:
        for name, p in linear_products(T, K, N).items():
            kind, margin = variant(*p)
            met[name, kind] = max(met.get((name, kind), 0.0), margin)
    for T, H, I, L, *_ in test_gpu_fp8.FFN + test_gpu_fp8_cuts.FFN:
        for name, p in ffn_products(T, H, I).items():
            kind, margin = variant(*p)
            for key in [(name, kind), (name, kind, L > 0)] if name == "h" else [(name, kind)]:
                met[key] = max(met.get(key, 0.0), margin)
    whole, wide, pair = (128, 1, False), (256, 1, False), (256, 2, False)
    part, wide_part = (128, 1, True), (256, 1, True)
    taken = {"y": (whole, part, wide, pair), "dx": (whole, part, wide, pair), "dw": (whole, part, wide, wide_part, pair),
             "dx of two": (whole, part, wide, pair), "three dw": (whole, part, wide, wide_part, pair), "h": (wide, wide_part, pair)}
    missing = [(n, k) for n, kinds in taken.items() for k in kinds if met.get((n, k), 0.0) < 0.05]
    missing += [("h", k, clamp) for k in taken["h"] for clamp in (False, True) if met.get(("h", k, clamp), -1.0) < 0.0]
    assert not missing
    rng = random.Random(1)
    size = lambda lo, hi: round(math.exp(rng.uniform(math.log(lo), math.log(hi))))  # noqa: E731
    for _ in range(3000):           # there are no others
        T, a, b = size(1, 16384), size(1, 8192), size(1, 8192)
        for name, p in [*linear_products(T, a, b).items(), *ffn_products(T, a, b).items()]:
            assert variant(*p)[0] in taken[name]
