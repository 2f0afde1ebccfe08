"""The dense layers in 8 bits at sizes that take the other cuts of a product: pairs of CTAs, wide tiles and K in parts, of the gated product, of the
two products that dx sums and of the three gradients of a launch. Held to the formulas and bounds of test_gpu_fp8; test_fp8_sizes says
which kernels these sizes take."""
import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from tests import test_gpu_fp8 as F

LINEAR = [
    # T, in, out, x, y, pad, shift
    (1311, 125, 140, F.BF16, F.BF16, 3, 1),
    (1003, 3999, 97, F.BF16, F.F32, 0, 0),
]
FFN = [
    # T, H, I, limit, pad, shift
    (936, 105, 101, 0.0, 3, 1),
    (2322, 1863, 143, 1.5, 0, 0),
    (3524, 2472, 1035, 2.0, 0, 0),
    (6788, 324, 1450, 0.0, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,xt,yt,pad,shift", LINEAR)
def test_linear(T, K, N, xt, yt, pad, shift):
    F.test_linear(T, K, N, xt, yt, pad, shift)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,L,pad,shift", FFN)
def test_feed_forward(T, H, I, L, pad, shift):
    F.test_feed_forward(T, H, I, L, pad, shift)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,L,pad,shift", FFN + [(200, 260, 300, 0.0, 3, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradients_into_fp32_buffers(T, H, I, L, pad, shift, accumulate):
    """Written and added to: one rounding of the sum, 2^-24 of it, beside the products' own bound."""
    g = F.gen(T)
    x, dy = F.activation(g, T, H).bfloat16(), F.randn(g, T, H).bfloat16()
    w = [F.weight(g, I, H), F.weight(g, I, H), F.weight(g, H, I)]
    ffn, fw = M.MoEFeedForward(H, I, swiglu_limit=L), M.FeedForwardWeights(*w)
    kept = ffn.forward(x, fw)[1]
    want = F.ffn_backward_ref(dy, F.values(kept[0], F.COL), *(F.values(k, F.ROW).float().double() for k in kept[1:]),
                              *(F.values(v, F.SQUARE) for v in w), L)
    bufs = [F.rows(F.randn(g, *n), pad, shift) for n in ((I, H), (I, H), (H, I))]
    first = [b.double() if accumulate else torch.zeros_like(b).double() for b in bufs]
    ffn.backward(dy, fw, kept, grads=bufs, accumulate=accumulate, need_dx=False)
    for got, f, name in zip(bufs, first, ("dgate", "dup", "ddown")):
        ref, tol = want[name]
        F.close(got, f + ref, tol + 2.0 ** -24 * (f + ref).abs(), name)


@pytest.mark.gpu
def test_backward_offsets_past_32_bits():
    """More than 2^31 elements of dx, of dh and of the five codes of the gate's backward pass. All rows but the last 300 are zeros, which add nothing
    to the gradients, so that those are the ones of the last whole blocks of rows."""
    T, H, I = 1_060_000, 64, 2040
    lo = T // 128 * 128 - 384
    g = F.gen(0)

    def last(n):
        t = torch.zeros(T, n, dtype=F.BF16, device="cuda")
        t[-300:] = F.randn(g, 300, n).bfloat16()
        return t

    x, dy, w = last(I), last(H), F.weight(g, H, I)
    lin = M.MoEFp8Linear(I, H)
    kept = lin.forward(x, w)[1]
    dx, dw = lin.backward(dy, w, kept)
    D, W = F.values(F.ref_codes(dy[lo:], F.ROW), F.ROW), F.values(w, F.SQUARE)
    F.close(dx[lo:], D @ W, F.sum_tol(D.abs() @ W.abs(), H), "dx")
    assert not dx[:-300].any()
    Dc, Xc = F.values(F.ref_codes(dy[lo:], F.COL), F.COL), F.values(F.ref_codes(x[lo:], F.COL), F.COL)
    F.close(dw, Dc.t() @ Xc, F.sum_tol(Dc.t().abs() @ Xc.abs(), T - lo), "dw")
    del x, kept, dx

    x = last(H)
    w = [F.weight(g, I, H), F.weight(g, I, H), F.weight(g, H, I)]
    ffn, fw = M.MoEFeedForward(H, I), M.FeedForwardWeights(*w)
    kept = ffn.forward(x, fw)[1]
    (xq, xs), *gu = kept
    tail = [F.values((q[lo:], s[:, lo:]), F.ROW).float().double() for q, s in gu]
    want = F.ffn_backward_ref(dy[lo:], F.values((xq[lo:], xs[lo // 128:]), F.COL), *tail, *(F.values(v, F.SQUARE) for v in w), 0.0)
    dx, grads = ffn.backward(dy, fw, kept)
    assert not dx[:-300].any()
    for got, name in zip((dx[lo:], *grads), ("dx", "dgate", "dup", "ddown")):
        F.close(got, *want[name], name)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 700, 300), (12, 700, 300), (90, 1500, 140), (400, 520, 400)])
def test_scales_whose_product_is_below_the_normal_range(T, K, N):
    """Rows of some 1e-36 against weights of 0.05: the product of two blocks' scales is rounded below 2^-126, by 2^-150 at most, which counts as often as the
    largest sum of a block's codes, 448^2 128: 2^-125.3 for each block along K beside the sums' own bound, and 2^-149 for each rounding of a result there."""
    g = F.gen(T)
    x, dy, w = (F.randn(g, T, K) * 1e-36), (F.randn(g, T, N) * 1e-36), F.weight(g, N, K)
    lin = M.MoEFp8Linear(K, N)
    y, kept = lin.forward(x, w)
    dx, _ = lin.backward(dy, w, kept, need_dweight=False)
    W = F.values(w, F.SQUARE)
    for got, a, b, k in ((y, x, W.t(), K), (dx, dy, W, N)):
        a = F.values(F.ref_codes(a, F.ROW), F.ROW)
        ref, tol = a @ b, F.sum_tol(a.abs() @ b.abs(), k)
        n = -(-k // 128)
        err = (got.double() - ref).abs() - tol - n * (448 ** 2 * 128 * 2.0 ** -150 + 20 * 2.0 ** -149)
        assert float(err.max()) <= 0.0 and got.any()
