"""What a block's forward keeps is its backward's, whatever stream that runs on.

The kept tensors are of the stream that forward ran on, and the block alone holds them. The allocator gives a tensor's memory to the next one of
its stream as soon as it is let go, so a backward on another stream has to tell it of its reads (``record_stream``) before it lets them go.
The first tests look at that on the CPU, with tensors that note what is said of them; the GPU ones look at the gradients.
"""
import gc
import weakref

import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ on the CPU: streams by name, operators that only pass tensors on
class Noted(torch.Tensor):
    """A tensor that notes the streams that it is recorded on."""

    @classmethod
    def new(cls, *shape, dtype=BF16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(cls)

    @property
    def told(self):
        return self.__dict__.setdefault("streams", [])

    def record_stream(self, stream):
        self.told.append(stream)

    def get_device(self):
        return 0


class Streams:
    """The current stream, as the blocks ask for it."""

    def __init__(self, monkeypatch):
        self.now, self.capturing = "A", False
        monkeypatch.setattr(B, "_current_stream_of", lambda: lambda index: self.now)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.now)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        B._fp8_of_torch.cache_clear()


@pytest.fixture
def streams(monkeypatch):
    yield Streams(monkeypatch)
    monkeypatch.undo()
    B._fp8_of_torch.cache_clear()


T, H, I, E, K = 4, 8, 16, 3, 2


class Norm:
    def forward(self, x, weight, bias, residual=None, out_dtype=None):
        self.made = [Noted.new(T, H), Noted.new(T, H), Noted.new(T, dtype=F32), Noted.new(T, dtype=F32)]
        return tuple(self.made)

    def backward(self, dy, s, weight, mean, rstd, dsum=None, bias=False):
        self.seen = [list(t.told) for t in (s, mean, rstd)]
        return Noted.new(T, H), Noted.new(H), None


class FeedForward:
    def forward(self, y, weights):
        pair = [(Noted.new(T, n), Noted.new(T, dtype=F32)) for n in (H, I, I)]
        self.made = [t for p in pair for t in p]
        return Noted.new(T, H), tuple(pair)

    def backward(self, dout, weights, kept, grads=None, accumulate=False):
        self.seen = [list(t.told) for p in kept for t in p]
        return Noted.new(T, H), (None, None, None)


def dense_block():
    block = M.DenseBlock(64, 64, device="cpu")
    block.norm, block.ffn = Norm(), FeedForward()
    return block, M.DenseParams(Noted.new(H), None)


class Router:
    def forward(self, logits, select_bias=None):
        self.made = [Noted.new(T, K, dtype=torch.int32), Noted.new(E, dtype=torch.int32)]
        return self.made[0], Noted.new(T, K, dtype=F32), self.made[1], None

    def backward(self, logits, ids, dprobs, counts=None, loss_grad=1.0):
        self.seen = [list(t.told) for t in (logits, ids, counts)]
        return torch.zeros(T, E, dtype=BF16)


class Layer:
    prepared = None

    def forward_topk(self, y, ids, probs, weights):
        return Noted.new(T, H)

    def backward(self, dout, main_grads):
        return torch.zeros(T, H, dtype=BF16), torch.zeros(T, K)


def expert_block():
    block = M.MoEBlock.__new__(M.MoEBlock)      # (its constructor allocates on a GPU)
    block.norm, block.router, block.layer, block.decoder, block.decode_tokens = Norm(), Router(), Layer(), None, 0
    block._mx, block._kept, block._captured, block._held = False, None, None, []
    return block, M.BlockParams(Noted.new(H), torch.zeros(E, H, dtype=BF16), B.moe_weights())


def backward(block, d):
    return block.backward(d, None) if isinstance(block, M.MoEBlock) else block.backward(d)


@pytest.mark.parametrize("make", [dense_block, expert_block])
def test_a_backward_on_another_stream_is_told_to_the_allocator(make, streams):
    block, params = make()
    block.forward(Noted.new(T, H), params)
    streams.now = "B"
    backward(block, torch.zeros(T, H, dtype=BF16))
    parts = [block.norm, block.ffn if make is dense_block else block.router]
    for part in parts:
        assert part.seen and all(told == ["B"] for told in part.seen), "before the first of its reads"
    made = [t for part in parts for t in part.made]
    if make is dense_block:
        made = made[1:]                # y itself is not kept
    assert all(t.told == ["B"] for t in made)


@pytest.mark.parametrize("make", [dense_block, expert_block])
def test_a_backward_on_the_same_stream_tells_nothing(make, streams):
    block, params = make()
    block.forward(Noted.new(T, H), params)
    backward(block, torch.zeros(T, H, dtype=BF16))
    for part in (block.norm, block.ffn if make is dense_block else block.router):
        assert all(t.told == [] for t in part.made)


def left_alive(block, made):
    """Which of the tensors that `block`'s operators made are still held, once those have let them go."""
    refs = [weakref.ref(t) for t in made]
    for part in (block.norm, getattr(block, "ffn", None), getattr(block, "router", None)):
        if part is not None:
            part.made = None
    made.clear()
    gc.collect()
    return [r() is not None for r in refs]


@pytest.mark.parametrize("make", [dense_block, expert_block])
@pytest.mark.parametrize("captured_forward", [False, True])
def test_what_a_captured_backward_reads_outlives_it(make, captured_forward, streams):
    """The replays of a backward that was captured by itself read what an eager forward kept. Where forward is of the capture too, the tensors are of the
    graph's own memory, which the rest of the capture may use again."""
    block, params = make()
    streams.capturing = captured_forward
    block.forward(Noted.new(T, H), params)
    streams.capturing = True
    backward(block, torch.zeros(T, H, dtype=BF16))
    made = block.norm.made[2:] + (block.ffn.made if make is dense_block else block.router.made)
    alive = left_alive(block, made)
    assert all(alive) if not captured_forward else not any(alive)


# ------------------------------------------------------------------ on the GPU
def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def dense(T, H, I, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [M.fp8_quantize((randn(g, *n) * 0.05).bfloat16(), M.MOE_B_SQUARE) for n in ((I, H), (I, H), (H, I))]
    p = M.DenseParams(1 + 0.1 * randn(g, H), M.FeedForwardWeights(*w), 0.1 * randn(g, H))
    steps = [(randn(g, T, H).bfloat16(), randn(g, T, H).bfloat16(), randn(g, T, H).bfloat16()) for _ in range(2)]
    return M.DenseBlock(H, I, norm=B.MOE_NORM_LAYER), p, steps


def dense_step(block, p, x, res, dout):
    out, s = block.forward(x, p, residual=res)
    dx, grads = block.backward(dout)
    return [out, s, dx, *grads.values()]


@gpu
def test_a_dense_backward_on_another_stream_beside_the_next_forward():
    block, p, steps = dense(600, 520, 1100)
    want = [dense_step(block, p, *step) for step in steps]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        (x, res, dout), (x2, res2, dout2) = steps
        with torch.cuda.stream(a):
            out, s = block.forward(x, p, residual=res)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            torch.cuda._sleep(200_000_000)          # some 0.1 s: the backward's kernels wait behind it
            dx, grads = block.backward(dout)
        with torch.cuda.stream(a):                  # at once, of the same sizes
            out2, s2 = block.forward(x2, p, residual=res2)
            dx2, grads2 = block.backward(dout2)
        torch.cuda.synchronize()
        for got, ref in zip(([out, s, dx, *grads.values()], [out2, s2, dx2, *grads2.values()]), want):
            assert all(torch.equal(g, r) for g, r in zip(got, ref))


@gpu
def test_an_expert_backward_on_another_stream_beside_new_tensors():
    """The layer's steps are ordered, so that the first stream's next work is tensors of the sizes that the block kept. The library products in the
    block (logits, dy, the router's gradient) may be split otherwise on another stream: results whose bf16 rounding may go the other way, 2^-8 of an
    element each, doubled by the norm's projection at most: 2^-6 for all of them."""
    T, H, I, E, k = 300, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    w = [(randn(g, *n) * 0.06).bfloat16() for n in ((2 * I, H), (H, I), (E, 2 * I, H), (E, H, I))]
    p = M.BlockParams(1 + 0.1 * randn(g, H), (randn(g, E, H) * 0.1).bfloat16(), M.weights_from_combined(*w))
    block = M.MoEBlock(T, H, E, k, I, aux_coeff=0.01)
    x, res, dout = (randn(g, T, H).bfloat16() for _ in range(3))

    def gradients(before=lambda: None):
        mg = [torch.zeros_like(t, dtype=F32) for t in w]
        before()
        dx, grads = block.backward(dout, M.main_grads_from_combined(*mg))
        return [dx, grads["norm_weight"], grads["router_weight"], *mg]

    block.forward(x, p, residual=res)
    want = gradients()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            block.forward(x, p, residual=res)
        b.wait_stream(a)
        with torch.cuda.stream(b):
            got = gradients(lambda: torch.cuda._sleep(200_000_000))
        with torch.cuda.stream(a):
            junk = [torch.full(n, float("nan"), dtype=t, device="cuda") for _ in range(6)
                    for n, t in (((T, H), BF16), ((T, E), BF16), ((T,), F32))]
            junk += [torch.full((T, k), E - 1, dtype=torch.int32, device="cuda") for _ in range(6)]
        torch.cuda.synchronize()
        for t, ref in zip(got, want):
            assert (t.double() - ref.double()).norm() <= 2.0 ** -6 * ref.double().norm()
        del junk
    block.close()


@gpu
def test_a_dense_backward_captured_by_itself():
    """Its replays take other dout at what the eager forward kept, whatever the program allocates meanwhile."""
    T, H, I = 300, 264, 520
    block, p, ((x, res, dout), (_, _, dout2)) = dense(T, H, I)
    want = [dense_step(block, p, x, res, d)[2:] for d in (dout, dout2)]
    given = dout.clone()
    block.forward(x, p, residual=res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, grads = block.backward(given)
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (T * H, T * I, 2 * T * H, 4 * T, 4 * T * 3, 4 * T * 5) for _ in range(8)]
    for d, ref in zip((dout, dout2), want):
        given.copy_(d)
        graph.replay()
        assert all(torch.equal(g, r) for g, r in zip([dx, *grads.values()], ref))
    del junk
