"""Dense layers in 8-bit floating point (a scale for each block of 128) against their formulas in fp64.

Codes and scales are defined by fp32 operations and compared bitwise. Everything else is held to bounds:

* A product's terms are exact in fp32 up to the scales. A block of 128 is summed by the tensor cores in four steps, whose alignment
  may drop bits below 2^-22 of a step's largest magnitude: 2^-20 of the sum of the terms' magnitudes S, safely. The scaled
  sums over the blocks are fp32 (two roundings a block and one for the scales' product), partial sums included: (2 blocks + 20)
  2^-24 S. Together `sum_tol`.
* A result in bf16 is rounded once, 2^-8 of itself (half a step), a gradient added to bf16 twice.
* A value that is off by e before it is stored in 8 bits is off afterwards by the distance between the numbers that its lower and upper
  ends are stored as (`stored`), which a product carries on with the other operand's magnitudes. A block's scale moves with its
  largest value.
* The logistic function is taken with the hardware's exponential, of error 2 + 1.16 |z| units in the last place (2^-23), and its
  fast division, 2: with the sums around them each of h, dg, du is off by (16 + 2 |g|) 2^-23 of the magnitudes that it is made of.
* A kept g or u is code * scale in fp32. The gradient jumps where it passes the clamp's bound, so the backward's reference takes that
  fp32 number: the product in 64 bits may lie on the bound's other side (by less than 2^-24 of it).
"""
import math

import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B

gpu = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ROW, COL, SQUARE = B.MOE_B_ROW, B.MOE_B_COL, B.MOE_B_SQUARE
BLOCK = {ROW: (1, 128), COL: (128, 1), SQUARE: (128, 128)}


# ------------------------------------------------------------------ the definitions
def block_max(a, block):
    (R, C), (br, bc) = a.shape, BLOCK[block]
    p = torch.nn.functional.pad(a, (0, -C % bc, 0, -R % br))
    return p.reshape(p.shape[0] // br, br, p.shape[1] // bc, bc).amax(3).amax(1)


def each(s, shape, block):
    br, bc = BLOCK[block]
    return s.repeat_interleave(br, 0)[:shape[0]].repeat_interleave(bc, 1)[:, :shape[1]]


def e4m3(z):
    return z.clamp(-448, 448).to(torch.float8_e4m3fn)


def ref_codes(x, block):
    """Codes and scales (in the library's layout) of x, by fp32 operations."""
    x = x.float()
    seen = torch.where(torch.isnan(x), torch.zeros_like(x), x).abs()
    amax = block_max(seen, block)
    s = torch.maximum(amax / torch.full_like(amax, 448.0), torch.full_like(amax, 2.0 ** -126))
    codes = e4m3(x * each(torch.ones_like(s) / s, x.shape, block)).view(torch.uint8)
    return codes, (s.t().contiguous() if block == ROW else s)


def values(pair, block):
    q, s = pair
    return q.contiguous().view(torch.float8_e4m3fn).double() * each((s.t() if block == ROW else s).double(), q.shape, block)


def stored(v, err, block):
    """(values of v stored in 8 bits, how far off they are where v is off by up to err)."""
    amax = block_max(v.abs(), block)
    slack = block_max(err, block)
    s = each(torch.clamp(amax / 448, min=2.0 ** -126), v.shape, block)
    rel = each(slack / torch.clamp(amax, min=1e-300), v.shape, block) + 2.0 ** -22   # of the scale
    z, dz = v / s, err / s + (v / s).abs() * rel
    at, lo, hi = (e4m3(t).double() for t in (z, z - dz, z + dz))
    # |code' s' - code s| <= |code' - code| s + |code'| |s' - s|
    return at * s, (torch.maximum(hi - at, at - lo) + torch.maximum(hi.abs(), lo.abs()) * rel) * s


def sum_tol(S, K):
    return (2.0 ** -20 + (2 * math.ceil(K / 128) + 20) * 2.0 ** -24) * S


def close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    bad = ~(err <= tol + 1e-37)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / (tol + 1e-37)).max()):.3g} x the bound"


def matmul(a, b):
    return a @ b


def gated(g, u, L):
    if L > 0:
        g, u = g.clamp(max=L), u.clamp(-L, L)
    return g * torch.sigmoid(g) * u


def gated_backward(dh, g, u, L):
    """(dg, du, h) and the magnitudes that they are made of."""
    gc, uc = (g.clamp(max=L), u.clamp(-L, L)) if L > 0 else (g, u)
    sig = torch.sigmoid(gc)
    dg, du = dh * uc * sig * (1 + gc * (1 - sig)), dh * gc * sig
    size = (dh * uc * sig).abs() * (1 + gc.abs() * (1 - sig))
    if L > 0:
        dg, du = torch.where(g > L, 0.0, dg), torch.where(u.abs() > L, 0.0, du)
    return dg, du, gc * sig * uc, size


# ------------------------------------------------------------------ the formulas themselves, on the CPU
def test_gated_backward_is_the_gradient():
    gen = torch.Generator().manual_seed(3)
    for L in (0.0, 1.0):
        g, u, dh = (torch.randn(4, 5, generator=gen, dtype=F64) for _ in range(3))
        dg, du, *_ = gated_backward(dh, g, u, L)
        for x, grad, f in ((g, dg, lambda t: gated(t, u, L)), (u, du, lambda t: gated(g, t, L))):
            d = (f(x + 1e-6) - f(x - 1e-6)) / 2e-6 * dh
            assert (d - grad).abs().max() < 1e-8


def test_stored_band_holds_for_moved_values():
    gen = torch.Generator().manual_seed(4)
    for block in BLOCK:
        v = torch.randn(150, 140, generator=gen, dtype=F64)
        err = 1e-3 * v.abs()
        at, band = stored(v, err, block)
        for _ in range(5):
            moved, _ = stored(v + err * (2 * torch.rand(v.shape, generator=gen, dtype=F64) - 1), 0 * err, block)
            assert ((moved - at).abs() <= band * (1 + 1e-9)).all()


def test_codes_of_the_definition():
    x = torch.zeros(130, 129)
    x[0, 0], x[0, 1], x[129, 128] = 448.0, 17.0, -3.0
    q, s = ref_codes(x, SQUARE)
    assert s.shape == B.fp8_scales_shape(130, 129, SQUARE) == (2, 2)
    assert s[0, 0] == 1.0 and s[1, 1] == torch.tensor(3.0) / 448 and s[0, 1] == 2.0 ** -126
    assert values((q, s), SQUARE)[0, 1] == 16.0 and (values((q, s), SQUARE)[129, 128] + 3.0).abs() < 1e-6   # 17 lies between 16 and 18, ties to even


@pytest.mark.parametrize("bad", [dict(in_features=0), dict(out_features=0), dict(in_features=(1 << 20) + 1), dict(x_type=2), dict(y_type=-1)])
def test_linear_configs_are_checked(bad):
    cfg = B.moe_linear_config(**{**dict(in_features=64, out_features=64, x_type=0, y_type=0), **bad})
    with pytest.raises(B.MoeError) as e:
        M.moe_linear_size(cfg, 4)
    assert e.value.status == 1


@pytest.mark.parametrize("bad", [dict(hidden=0), dict(inter=0), dict(inter=(1 << 20) + 1), dict(swiglu_limit=-1.0),
                                 dict(swiglu_limit=math.nan), dict(swiglu_limit=math.inf)])
def test_feed_forward_configs_are_checked(bad):
    cfg = B.moe_ffn_config(**{**dict(hidden=64, inter=64, swiglu_limit=0.0), **bad})
    with pytest.raises(B.MoeError) as e:
        M.moe_ffn_size(cfg, 4)
    assert e.value.status == 1


def test_sizes_and_null_arguments():
    L = M.load()
    cfg, ffn = B.moe_linear_config(64, 64, 0, 0), B.moe_ffn_config(64, 64, 0.0)
    assert M.moe_linear_size(cfg, 0) == 0 and M.moe_linear_size(cfg, 5) < M.moe_linear_size(cfg, 50) < M.moe_linear_size(cfg, 500)
    assert M.moe_ffn_size(ffn, 0) == 0 and 0 < M.moe_ffn_size(ffn, 5) < M.moe_ffn_size(ffn, 500, True)
    for T in (-1, (1 << 24) + 1):
        with pytest.raises(B.MoeError):
            M.moe_linear_size(cfg, T)
    assert L.moe_linear_size(None, 1, 0, None) == 1 and L.moe_ffn_size(None, 1, 0, None) == 1
    assert L.moe_fp8_quantize(None, 0, 4, 4, 4, B.moe_fp8(), None, None, None) == 1
    assert L.moe_fp8_quantize(None, 0, 0, 4, 4, B.moe_fp8(), None, None, None) == 0         # no rows: nothing to do
    assert L.moe_fp8_quantize(None, 0, 4, 4, 3, None, None, None, None) == 1                # stride
    assert L.moe_fp8_dequantize(None, 0, 4, 4, None, 0, 4, None) == 1
    assert L.moe_fp8_dequantize(B.moe_fp8(), 3, 4, 4, None, 0, 4, None) == 1                # no such block
    assert L.moe_linear_forward(cfg, 4, None, 64, None, None, 64, None, None, 0, None) == 1
    assert L.moe_linear_forward(cfg, 4, None, 63, None, None, 64, None, None, 0, None) == 1
    assert L.moe_linear_backward(cfg, 4, None, 64, None, None, None, 64, None, 64, 2, 0, None, 0, None) == 1
    assert L.moe_ffn_forward(ffn, 4, None, 64, None, None, 64, None, None, 0, None) == 1
    assert L.moe_ffn_backward(ffn, 4, None, 64, None, None, None, 64, None, 0, 2, None, 0, None) == 1
    # places that the library would read or write are looked at before anything is launched (none of these is read here)
    fake = 1 << 20
    good = B.moe_fp8(fake, 64, fake)
    for v in (B.moe_fp8(fake + 8, 64, fake), B.moe_fp8(fake, 72, fake), B.moe_fp8(fake, 48, fake), B.moe_fp8(fake, 64, fake + 2), B.moe_fp8(fake, 64, None)):
        assert L.moe_fp8_quantize(fake, 0, 4, 64, 64, v, None, None, None) == 1
        assert L.moe_linear_forward(cfg, 4, fake, 64, v, fake, 64, None, fake, 1 << 30, None) == 1
        assert L.moe_linear_forward(cfg, 4, fake, 64, good, fake, 64, v, fake, 1 << 30, None) == 1
    need = M.moe_linear_size(cfg, 40)
    assert L.moe_linear_forward(cfg, 40, fake, 64, good, fake, 64, None, fake, need - 1, None) == 1
    assert L.moe_linear_forward(cfg, 40, fake, 64, good, fake, 64, None, fake + 128, need, None) == 1
    assert L.moe_linear_forward(cfg, 40, fake + 1, 64, good, fake, 64, None, fake, need, None) == 1


# ------------------------------------------------------------------ on the GPU
def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def rows(t, pad, shift):
    """t in rows of a buffer `pad` elements wider, starting `shift` elements into it; NaN around them."""
    wide = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 8,), math.nan, dtype=t.dtype, device=t.device)
    v = wide[shift:shift + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v


def activation(g, T, C):
    """Channels of very different sizes, a block of zeros."""
    x = randn(g, T, C) * torch.exp(randn(g, C))
    if C > 256:
        x[:, 128:256] = 0
    return x


def weight(g, n, k):
    w = randn(g, n, k) * 0.05
    return M.fp8_quantize(w.bfloat16(), SQUARE)


SIZES = [(1, 1), (1, 128), (3, 15), (128, 128), (129, 127), (130, 257), (1, 2051), (300, 16), (257, 1000), (1000, 31)]


@gpu
@pytest.mark.parametrize("block", [ROW, COL, SQUARE])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_codes_and_values_are_the_definitions(block, dtype):
    for n, (R, C) in enumerate(SIZES):
        for pad, shift in ((0, 0), (8, 0), (3, 1)):
            x = rows(activation(gen(n), R, C).to(dtype), pad, shift)
            ld = (C + 15) // 16 * 16 + 16
            q = torch.full((R, ld), 0xA5, dtype=torch.uint8, device="cuda")
            s = torch.empty(B.fp8_scales_shape(R, C, block), device="cuda")
            M.fp8_quantize(x, block, out=(q[:, :C], s))
            rq, rs = ref_codes(x, block)
            assert torch.equal(q[:, :C], rq) and torch.equal(s, rs), (R, C, pad)
            assert (q[:, C:] == 0xA5).all(), "bytes of a row past its columns are not written"
            for out_type in (BF16, F32):
                ref = values((rq, rs), block)
                out = rows(torch.zeros(R, C, dtype=out_type, device="cuda"), pad, shift)
                M.fp8_dequantize(q[:, :C], s, block, out=out)
                assert torch.equal(out, (ref.float()).to(out_type)), (R, C, pad, out_type)


@gpu
def test_both_directions_at_once_and_extremes():
    x = activation(gen(1), 260, 300)
    x[5, 7], x[140, 290], x[200, 20] = math.nan, math.inf, -math.inf
    x[60, :128] = 1e-41                     # below the smallest normal number: a scale of 2^-126
    x[61, :128] = 3e38
    x[3, 3] = -0.0
    row, col = (B._new_codes(torch, 260, 300, b, "cuda") for b in (ROW, COL))
    v = [B._codes(torch, p, 260, 300, b, 0, "") for p, b in ((row, ROW), (col, COL))]
    assert M.load().moe_fp8_quantize(x.data_ptr(), 1, 260, 300, 300, v[0], v[1], None, torch.cuda.current_stream().cuda_stream) == 0
    for pair, block in ((row, ROW), (col, COL)):
        q, s = ref_codes(x, block)
        nan = (q & 0x7F) == 0x7F
        assert torch.equal(pair[1], s)
        assert torch.equal((pair[0] & 0x7F) == 0x7F, nan) and torch.equal(pair[0][~nan], q[~nan])
        got, ref = M.fp8_dequantize(*pair, block, dtype=F32), values((q, s), block).float()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        inf = each((torch.isinf(s.t() if block == ROW else s)).float(), x.shape, block) > 0
        assert torch.isnan(got[inf]).all(), "a block with an infinity is NaN"
        assert torch.isnan(got[5, 7]) and torch.isfinite(got[5, 8]), "a NaN keeps to its place"


@gpu
def test_refusals():
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    with pytest.raises(ValueError):
        M.fp8_quantize(x.half(), ROW)
    with pytest.raises(ValueError):
        M.fp8_quantize(x, 3)
    with pytest.raises(ValueError):
        M.fp8_quantize(x.t(), ROW)
    with pytest.raises(ValueError):
        M.fp8_quantize(x.cpu(), ROW)
    pair = M.fp8_quantize(x, ROW)
    with pytest.raises(ValueError):
        M.fp8_dequantize(pair[0], pair[1].t().contiguous(), ROW)
    with pytest.raises(ValueError):
        M.fp8_dequantize(pair[0][:, :24].contiguous(), pair[1], ROW)
    lin = M.MoEFp8Linear(64, 32)
    w = M.fp8_quantize(torch.zeros(32, 64, device="cuda"), SQUARE)
    with pytest.raises(ValueError):
        lin.forward(x[:, :32], w)
    with pytest.raises(ValueError):
        lin.forward(x, M.fp8_quantize(torch.zeros(64, 32, device="cuda"), SQUARE))
    with pytest.raises(ValueError):
        lin.forward(x, (w[0].cpu(), w[1].cpu()))
    y, kept = lin.forward(x, w)
    with pytest.raises(ValueError):
        lin.backward(y, w, kept, accumulate=True)
    with pytest.raises(ValueError):
        lin.backward(y, w, kept, dweight=torch.zeros(64, 32, device="cuda"))
    with pytest.raises(ValueError):
        lin.backward(y, w, kept, dweight=torch.zeros(32, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        lin.backward(y, w, (kept[0][:2], kept[1]))
    ffn = M.MoEFeedForward(64, 32)
    down = M.fp8_quantize(torch.zeros(64, 32, device="cuda"), SQUARE)
    with pytest.raises(ValueError):
        M.FeedForwardWeights(w, w, w)
    fw = M.FeedForwardWeights(w, w, down)
    with pytest.raises(ValueError):
        ffn.forward(x.float(), fw)
    with pytest.raises(ValueError):
        M.MoEFeedForward(64, 48).forward(x, fw)
    y, kept = ffn.forward(x, fw)
    with pytest.raises(ValueError):
        ffn.backward(y, fw, kept[:1] + (kept[0],) + kept[2:])
    with pytest.raises(ValueError):
        ffn.backward(y, fw, kept, grads=[torch.zeros(32, 64, device="cuda")] * 3)
    with pytest.raises(ValueError):
        ffn.backward(y, fw, kept, accumulate=True)


LINEAR = [
    # T, in, out, x, y, pad, shift
    (1, 1, 1, BF16, BF16, 0, 0),
    (1, 128, 128, BF16, BF16, 0, 0),
    (2, 129, 5, F32, F32, 3, 1),
    (7, 200, 130, BF16, F32, 0, 0),
    (8, 300, 40, F32, F32, 0, 0),
    (9, 7168, 33, BF16, BF16, 3, 1),
    (16, 2048, 256, BF16, BF16, 8, 0),
    (33, 1500, 100, BF16, BF16, 0, 0),
    (65, 1160, 424, BF16, BF16, 0, 0),
    (17, 999, 1001, BF16, BF16, 3, 1),
    (64, 4096, 512, F32, BF16, 0, 0),
    (127, 300, 257, BF16, BF16, 0, 0),
    (128, 256, 256, BF16, BF16, 0, 0),
    (129, 260, 640, BF16, F32, 5, 0),
    (300, 1160, 424, BF16, BF16, 0, 0),
    (1000, 96, 4000, BF16, BF16, 0, 0),
    (2500, 700, 2050, BF16, BF16, 0, 0),
    (2305, 2304, 2300, F32, F32, 0, 0),
    (5000, 130, 1300, BF16, BF16, 0, 0),
    (40, 4099, 2100, BF16, BF16, 3, 1),
    (2400, 200, 4099, BF16, BF16, 3, 1),
    (2400, 257, 4099, F32, F32, 1, 1),
]


@gpu
@pytest.mark.parametrize("T,K,N,xt,yt,pad,shift", LINEAR)
def test_linear(T, K, N, xt, yt, pad, shift):
    g = gen(T + K)
    x = rows(activation(g, T, K).to(xt), pad, shift)
    w = weight(g, N, K)
    lin = M.MoEFp8Linear(K, N)
    y, kept = lin.forward(x, w, out_dtype=yt)
    W, X = values(w, SQUARE), values(ref_codes(x, ROW), ROW)
    close(y, X @ W.t(), sum_tol(X.abs() @ W.abs().t(), K), "y")
    rq, rs = ref_codes(x, COL)
    assert torch.equal(kept[0], rq) and torch.equal(kept[1], rs)
    assert torch.equal(lin.forward(x, w, keep=False, out_dtype=yt)[0], y)

    dy = rows(randn(g, T, N).to(yt), pad, shift)
    D, Dc, Xc = values(ref_codes(dy, ROW), ROW), values(ref_codes(dy, COL), COL), values(kept, COL)
    dx, dw = lin.backward(dy, w, kept, dx_dtype=xt)
    dw_ref, dw_tol = Dc.t() @ Xc, sum_tol(Dc.t().abs() @ Xc.abs(), T)
    close(dx, D @ W, sum_tol(D.abs() @ W.abs(), N), "dx")
    close(dw, dw_ref, dw_tol, "dw")
    for gt in (F32, BF16):          # into a buffer, overwritten and added to
        first = rows(randn(g, N, K).to(gt), pad, shift)
        buf = rows(first, pad, shift)
        _, again = lin.backward(dy, w, kept, dx_dtype=xt, dweight=buf, need_dx=False)
        assert again is buf
        close(buf, dw_ref, dw_tol, f"dw into {gt}")
        buf.copy_(first)
        lin.backward(dy, w, kept, dx_dtype=xt, dweight=buf, accumulate=True, need_dx=False)
        sum_ref = first.double() + dw_ref
        extra = 2.0 ** -8 * dw_ref.abs() if gt == BF16 else 2.0 ** -24 * sum_ref.abs()
        close(buf, sum_ref, dw_tol * (1 + 2.0 ** -8) + extra, f"dw added to {gt}")
    only, none = lin.backward(dy, w, None, dx_dtype=xt, need_dweight=False)
    assert none is None and torch.equal(only, dx)


FFN = [
    # T, H, I, limit, pad, shift
    (1, 1, 1, 0.0, 0, 0),
    (1, 256, 128, 0.0, 0, 0),
    (2, 130, 70, 1.0, 3, 1),
    (8, 2048, 1024, 0.0, 0, 0),
    (9, 200, 1000, 2.0, 3, 1),
    (17, 1160, 424, 2.0, 0, 0),
    (40, 264, 520, 0.0, 0, 0),
    (65, 264, 520, 0.0, 0, 0),
    (64, 512, 2049, 0.0, 8, 0),
    (128, 128, 128, 0.0, 0, 0),
    (200, 260, 300, 0.0, 3, 1),
    (515, 1160, 1000, 2.0, 0, 0),
    (2600, 520, 1400, 0.0, 0, 0),
    (4100, 300, 2600, 1.5, 0, 0),
]


def ffn_forward_ref(x, wg, wu, wd, L):
    """y, g, u and their bounds: sums, then h with the logistic function's error, stored, then the sum of the down product."""
    H, I = wg.shape[1], wg.shape[0]
    X = values(ref_codes(x, ROW), ROW)
    g, u = X @ wg.t(), X @ wu.t()
    eg, eu = sum_tol(X.abs() @ wg.abs().t(), H), sum_tol(X.abs() @ wu.abs().t(), H)
    h = gated(g, u, L)
    gc, uc = (g.clamp(max=L), u.clamp(-L, L)) if L > 0 else (g, u)
    silu = gc * torch.sigmoid(gc)
    # |silu'| <= 1.1; the clamps move by no more than their arguments
    eh = 1.1 * eg * (uc.abs() + eu) + (silu.abs() + 1.1 * eg) * eu + (16 + 2 * gc.abs()) * 2.0 ** -23 * h.abs()
    hs, band = stored(h, eh, ROW)
    y = hs @ wd.t()
    return y, band @ wd.abs().t() + sum_tol((hs.abs() + band) @ wd.abs().t(), I), g, eg, u, eu


def ffn_backward_ref(dy, xc, g, u, wg, wu, wd, L):
    H, I = wg.shape[1], wg.shape[0]
    D = values(ref_codes(dy, ROW), ROW)
    dh = D @ wd
    e = sum_tol(D.abs() @ wd.abs(), H)
    dg, du, h, size = gated_backward(dh, g, u, L)
    gc, uc = (g.clamp(max=L), u.clamp(-L, L)) if L > 0 else (g, u)
    near = (16 + 2 * gc.abs()) * 2.0 ** -23
    scale = torch.where(dh != 0, size / dh.abs().clamp(min=1e-300), (uc * torch.sigmoid(gc)).abs() * (1 + gc.abs()))
    eg, eu, eh = scale * e + near * size, (gc * torch.sigmoid(gc)).abs() * (e + near * dh.abs()), near * h.abs()
    if L > 0:
        eg, eu = torch.where(g > L, 0.0, eg), torch.where(u.abs() > L, 0.0, eu)
    (rg, bg), (ru, bu) = stored(dg, eg, ROW), stored(du, eu, ROW)
    out = {"dx": (rg @ wg + ru @ wu, bg @ wg.abs() + bu @ wu.abs() +
                  sum_tol((rg.abs() + bg) @ wg.abs() + (ru.abs() + bu) @ wu.abs(), 2 * I + 256))}
    T = dy.shape[0]
    Dc = values(ref_codes(dy, COL), COL)
    for name, (v, b), other in (("dgate", stored(dg, eg, COL), xc), ("dup", stored(du, eu, COL), xc)):
        out[name] = (v.t() @ other, b.t() @ other.abs() + sum_tol((v.abs() + b).t() @ other.abs(), T))
    v, b = stored(h, eh, COL)
    out["ddown"] = (Dc.t() @ v, Dc.t().abs() @ b + sum_tol(Dc.t().abs() @ (v.abs() + b), T))
    return out


@gpu
@pytest.mark.parametrize("T,H,I,L,pad,shift", FFN)
def test_feed_forward(T, H, I, L, pad, shift):
    gn = gen(T + H + I)
    x = rows(activation(gn, T, H).bfloat16(), pad, shift)
    w = [weight(gn, I, H), weight(gn, I, H), weight(gn, H, I)]
    wg, wu, wd = (values(v, SQUARE) for v in w)
    fw = M.FeedForwardWeights(*w)
    ffn = M.MoEFeedForward(H, I, swiglu_limit=L)
    y, kept = ffn.forward(x, fw)
    ref, tol, g, eg, u, eu = ffn_forward_ref(x, wg, wu, wd, L)
    close(y, ref, tol, "y")
    alone, none = ffn.forward(x, fw, keep=False)    # few tokens by other kernels
    assert none is None
    close(alone, ref, tol, "y, nothing kept")
    rq, rs = ref_codes(x, COL)
    assert torch.equal(kept[0][0], rq) and torch.equal(kept[0][1], rs)
    for pair, v, e, what in ((kept[1], g, eg, "g"), (kept[2], u, eu, "u")):
        at, band = stored(v, e, ROW)
        close(values(pair, ROW).float(), at, band + 2.0 ** -23 * at.abs(), "kept " + what)

    dy = rows(randn(gn, T, H).bfloat16(), pad, shift)
    xc, gk, uk = values(kept[0], COL), values(kept[1], ROW).float().double(), values(kept[2], ROW).float().double()
    want = ffn_backward_ref(dy, xc, gk, uk, wg, wu, wd, L)
    dx, grads = ffn.backward(dy, fw, kept)
    for got, name in zip((dx, *grads), ("dx", "dgate", "dup", "ddown")):
        close(got, *want[name], name)
    bufs = [rows(randn(gn, *t.shape).bfloat16(), pad, shift) for t in grads]
    first = [b.clone() for b in bufs]
    _, back = ffn.backward(dy, fw, kept, grads=bufs, accumulate=True, need_dx=False)
    for got, f, name in zip(back, first, ("dgate", "dup", "ddown")):
        r, t = want[name]
        close(got, f.double() + r, t * (1 + 2.0 ** -8) + 2.0 ** -8 * r.abs(), name + " added to bf16")
    only, none = ffn.backward(dy, fw, kept, need_grads=False)
    assert none is None and torch.equal(only, dx)


# ------------------------------------------------------------------ few tokens and weights of more rows than a block of them an SM
@gpu
@pytest.mark.parametrize("T,K,N,xt,pad,shift", [
    (1, 300, 2432, BF16, 0, 0), (1, 4500, 2433, BF16, 0, 0), (3, 257, 8000, F32, 3, 1), (8, 5000, 2600, BF16, 3, 1),
    (9, 700, 2600, BF16, 0, 0), (16, 1000, 5003, BF16, 8, 0), (16, 1, 4100, F32, 0, 0), (13, 2400, 2500, F32, 0, 0)])
def test_linear_of_few_tokens(T, K, N, xt, pad, shift):
    g = gen(T + K + N)
    x = rows(activation(g, T, K).to(xt), pad, shift)
    w = weight(g, N, K)
    lin = M.MoEFp8Linear(K, N)
    W, X = values(w, SQUARE), values(ref_codes(x, ROW), ROW)
    ref, tol = X @ W.t(), sum_tol(X.abs() @ W.abs().t(), K)
    for yt in (F32, BF16):
        y, none = lin.forward(x, w, keep=False, out_dtype=yt)
        assert none is None
        close(y, ref, tol, f"y {yt}")
        assert torch.equal(lin.forward(x, w, out_dtype=yt)[0], y)
    if T > 1:                       # a token's result does not depend on the others'
        assert torch.equal(lin.forward(x[1:2], w, keep=False, out_dtype=F32)[0], lin.forward(x, w, keep=False, out_dtype=F32)[0][1:2])


@gpu
@pytest.mark.parametrize("T,H,I,L", [(1, 2500, 1300, 0.0), (1, 4500, 1217, 2.0), (4, 300, 2600, 1.0), (9, 260, 1300, 0.0), (16, 700, 1500, 2.0)])
def test_feed_forward_of_few_tokens(T, H, I, L):
    gn = gen(T + H + I)
    x = activation(gn, T, H).bfloat16()
    w = [weight(gn, I, H), weight(gn, I, H), weight(gn, H, I)]
    y, none = M.MoEFeedForward(H, I, swiglu_limit=L).forward(x, M.FeedForwardWeights(*w), keep=False)
    assert none is None
    ref, tol = ffn_forward_ref(x, *(values(v, SQUARE) for v in w), L)[:2]
    close(y, ref, tol, "y")


# ------------------------------------------------------------------ the calls that a program makes of them
def ffn_setup(T, H, I, seed=0, limit=0.0):
    gn = gen(seed)
    x = activation(gn, T, H).bfloat16()
    w = M.FeedForwardWeights(weight(gn, I, H), weight(gn, I, H), weight(gn, H, I))
    return M.MoEFeedForward(H, I, limit), w, x, randn(gn, T, H).bfloat16()


def ffn_step(ffn, w, x, dy, **kw):
    y, kept = ffn.forward(x, w, **kw)
    dx, grads = ffn.backward(dy, w, kept, **kw)
    return (y, dx, *grads)


@gpu
@pytest.mark.parametrize("T,H,I", [(5, 256, 384), (300, 520, 400), (3000, 512, 1100)])
def test_results_repeat_bitwise(T, H, I):
    ffn, w, x, dy = ffn_setup(T, H, I)
    first = ffn_step(ffn, w, x, dy)
    for _ in range(3):
        for a, b in zip(first, ffn_step(ffn, w, x, dy)):
            assert torch.equal(a, b)


@gpu
def test_streams():
    sets = [ffn_setup(200, 384, 512, seed) for seed in range(4)]
    want = [ffn_step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [ffn_step(*s, stream=st) for s, st in zip(sets, streams)]     # four at a time
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
        for g, r in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, r))
    q = M.fp8_quantize(sets[0][2], COL, stream=streams[0])
    x = M.fp8_dequantize(*q, COL, stream=streams[0])
    torch.cuda.current_stream().wait_stream(streams[0])
    assert torch.equal(x, M.fp8_dequantize(*M.fp8_quantize(sets[0][2], COL), COL))


@gpu
@pytest.mark.parametrize("T", [3, 40, 700])
def test_graphs(T):
    """Two captured steps of one network, replayed in turn on other inputs, beside eager calls."""
    sets = [ffn_setup(T, 300, 260, seed) for seed in range(2)]
    ffn = sets[0][0]
    graphs = []
    for _, w, x, dy in sets:
        ffn_step(ffn, w, x, dy)
        ffn.forward(x, w, keep=False)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ffn_step(ffn, w, x, dy)
            alone = ffn.forward(x, w, keep=False)[0]
        graphs.append((g, out, alone))
    for turn in range(3):
        for (_, w, x, dy), (g, out, alone) in zip(sets, graphs):
            x.copy_(activation(gen(10 + turn), T, 300).bfloat16())
            dy.copy_(randn(gen(20 + turn), T, 300).bfloat16())
            g.replay()
            eager = ffn_step(ffn, w, x, dy)
            assert all(torch.equal(a, b) for a, b in zip(out, eager))
            assert torch.equal(alone, ffn.forward(x, w, keep=False)[0])


@gpu
def test_no_rows():
    ffn, w, x, dy = ffn_setup(4, 200, 130)
    y, kept = ffn.forward(x[:0], w)
    assert y.shape == (0, 200) and kept[0][1].shape == (0, 200)
    dx, grads = ffn.backward(dy[:0], w, kept)
    assert dx.shape == (0, 200) and all((g == 0).all() for g in grads)
    bufs = [torch.full_like(g, 3.0) for g in grads]
    ffn.backward(dy[:0], w, kept, grads=bufs, accumulate=True)
    assert all((b == 3).all() for b in bufs)
    lin, wl = M.MoEFp8Linear(200, 130), weight(gen(1), 130, 200)
    y, kept = lin.forward(x[:0], wl)
    dw = torch.full((130, 200), 5.0, device="cuda", dtype=BF16)
    dx, _ = lin.backward(y, wl, kept, dweight=dw)
    assert dx.shape == (0, 200) and (dw == 0).all()
    q, s = M.fp8_quantize(x[:0], ROW)
    assert q.shape == (0, 200) and s.shape == (2, 0) and M.fp8_dequantize(q, s, ROW).shape == (0, 200)


@gpu
@pytest.mark.parametrize("T", [4, 100, 600])
def test_a_bad_token_stays_alone(T):
    """NaN and infinities of one token reach its own rows only, and the weights' gradients as NaN."""
    ffn, w, x, dy = ffn_setup(T, 384, 256)
    for bad in (math.nan, math.inf):
        xb = x.clone()
        xb[1, 7] = bad
        y, yb = ffn.forward(x, w, keep=False)[0], ffn.forward(xb, w, keep=False)[0]
        assert torch.isnan(yb[1]).all()
        others = torch.arange(T, device="cuda") != 1
        assert torch.equal(y[others], yb[others])
        _, kept = ffn.forward(x, w)
        db = dy.clone()
        db[1, 7] = bad
        dx, _ = ffn.backward(dy, w, kept)
        dxb, grads = ffn.backward(db, w, kept)
        assert torch.isnan(dxb[1]).all() and torch.equal(dx[others], dxb[others])
        assert all(torch.isnan(g).any() for g in grads)


@gpu
@pytest.mark.parametrize("T", [1, 9, 33, 200])
def test_weights_in_wider_buffers(T):
    """gate and up as halves of one matrix, rows with other bytes behind them (NaN codes): nothing of those is read as a value."""
    H, I = 250, 256
    gn = gen(T)
    x = activation(gn, T, H).bfloat16()
    q, s = M.fp8_quantize((randn(gn, 2 * I, H) * 0.05).bfloat16(), SQUARE)
    wide = torch.full((2 * I, 288), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, :H] = q
    halves = [(wide[:I, :H], s[:2]), (wide[I:, :H], s[2:])]
    down = weight(gn, H, I)
    ffn = M.MoEFeedForward(H, I)
    w = M.FeedForwardWeights(*halves, down)
    plain = M.FeedForwardWeights((q[:I], s[:2].clone()), (q[I:], s[2:].clone()), down)
    dy = randn(gn, T, H).bfloat16()
    for a, b in zip(ffn_step(ffn, w, x, dy), ffn_step(ffn, plain, x, dy)):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    assert torch.equal(ffn.forward(x, w, keep=False)[0], ffn.forward(x, plain, keep=False)[0])
    lin = M.MoEFp8Linear(H, 2 * I)
    assert torch.equal(lin.forward(x, (wide[:, :H], s))[0], lin.forward(x, (q, s))[0])


@gpu
@pytest.mark.parametrize("T", [3, 70, 500])
def test_results_in_wider_buffers(T):
    """Through the C entry points: y, dx and the kept codes in rows of wider buffers, whose other elements stay."""
    K, N, L = 200, 330, M.load()
    gn = gen(T)
    x, dy, w = activation(gn, T, K).bfloat16(), randn(gn, T, N).bfloat16(), weight(gn, N, K)
    lin = M.MoEFp8Linear(K, N)
    y, kept = lin.forward(x, w)
    dx, dw = lin.backward(dy, w, kept)
    cfg, stream = lin._cfg(BF16, BF16), torch.cuda.current_stream().cuda_stream
    for pad in (1, 8):
        yb, xb = (torch.full((T + 1, n + pad), 7.0, dtype=BF16, device="cuda") for n in (N, K))
        kq = torch.full((T + 1, 224), 0x55, dtype=torch.uint8, device="cuda")
        ks = torch.full((kept[1].numel() + 8,), 9.0, device="cuda")
        ws = torch.empty(M.moe_linear_size(cfg, T, True) + M.moe_linear_size(cfg, T), dtype=torch.uint8, device="cuda")
        v = B._codes(torch, w, N, K, SQUARE, 0, "")
        k = B.moe_fp8(kq.data_ptr(), 224, ks.data_ptr())
        assert L.moe_linear_forward(cfg, T, x.data_ptr(), K, v, yb.data_ptr(), N + pad, k, ws.data_ptr(), ws.numel(), stream) == 0
        assert L.moe_linear_backward(cfg, T, dy.data_ptr(), N, v, k, xb.data_ptr(), K + pad, None, 0, 0, 0, ws.data_ptr(), ws.numel(), stream) == 0
        assert torch.equal(yb[:T, :N], y) and (yb[T] == 7).all() and (yb[:, N:] == 7).all()
        assert torch.equal(xb[:T, :K], dx) and (xb[T] == 7).all() and (xb[:, K:] == 7).all()
        assert torch.equal(kq[:T, :K], kept[0]) and (kq[T] == 0x55).all() and (kq[:, K:] == 0x55).all()
        assert torch.equal(ks[:-8].view_as(kept[1]), kept[1]) and (ks[-8:] == 9).all()


@gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows of codes, values and a product's results."""
    R, C = 2_150_000, 1016
    x = torch.zeros(R, C, dtype=BF16, device="cuda")
    x[-300:] = randn(gen(1), 300, C).bfloat16()
    for block in (ROW, COL):
        q, s = M.fp8_quantize(x, block)
        back = M.fp8_dequantize(q, s, block)
        lo = R // 128 * 128 - 128   # whole blocks of rows
        rq, rs = ref_codes(x[lo:], block)
        assert torch.equal(q[lo:], rq) and torch.equal(s[:, lo:] if block == ROW else s[lo // 128:], rs)
        assert torch.equal(back[lo:], values((rq, rs), block).float().bfloat16()) and not back[:lo - 300].any()
        del q, s, back
    del x
    T, K, N = 1_060_000, 64, 2040
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[-300:] = randn(gen(2), 300, K).bfloat16()
    w = weight(gen(3), N, K)
    y, _ = M.MoEFp8Linear(K, N).forward(x, w, keep=False)
    X, W = values(ref_codes(x[-300:], ROW), ROW), values(w, SQUARE)
    close(y[-300:], X @ W.t(), sum_tol(X.abs() @ W.abs().t(), K), "y")
    assert not y[:-300].any()


@gpu
def test_more_refusals():
    ffn, w, x, dy = ffn_setup(4, 64, 64)
    _, kept = ffn.forward(x, w)
    one = torch.zeros(64, 64, device="cuda")
    with pytest.raises(B.MoeError):       # one buffer for two gradients
        ffn.backward(dy, w, kept, grads=[one, one, torch.zeros_like(one)])
    with pytest.raises(ValueError):
        ffn.backward(dy, w, kept, grads=[one, one.clone(), one.bfloat16()])
    with pytest.raises(ValueError):
        ffn.backward(dy.float(), w, kept)
    with pytest.raises(ValueError):
        M.DenseBlock(64, 64).backward(dy)
    block = M.DenseBlock(64, 64)
    params = M.DenseParams(torch.ones(64, device="cuda"), w)
    out, s = block.forward(x, params)
    with pytest.raises(ValueError):
        block.backward(dy[:2])
    with pytest.raises(ValueError):
        block.backward(dy, ds=dy.float())
    with pytest.raises(ValueError):
        block.backward(dy.float())
    block.backward(dy)
    with pytest.raises(ValueError):       # once for each forward
        block.backward(dy)


@gpu
@pytest.mark.parametrize("T,xt,norm,bias", [(1, BF16, "rms", False), (20, F32, "layer", True), (500, BF16, "rms", True)])
def test_dense_block(T, xt, norm, bias):
    """The block is its operators one after the other; its forward and backward against the whole formula in 64 bits, normwise."""
    H, I = 264, 520
    gn = gen(T)
    x, res = randn(gn, T, H).to(xt), randn(gn, T, H).to(xt)
    p = M.DenseParams(1 + 0.1 * randn(gn, H), M.FeedForwardWeights(weight(gn, I, H), weight(gn, I, H), weight(gn, H, I)),
                      0.1 * randn(gn, H) if bias else None)
    kind = B.MOE_NORM_RMS if norm == "rms" else B.MOE_NORM_LAYER
    block = M.DenseBlock(H, I, norm=kind, eps=1e-5)
    out, s = block.forward(x, p, residual=res)
    dout, ds = randn(gn, T, H).bfloat16(), randn(gn, T, H).to(xt)
    dx, grads = block.backward(dout, ds=ds)
    y, s2, mean, rstd = M.MoENorm(H, 1e-5, kind).forward(x, p.norm_weight, p.norm_bias, residual=res, out_dtype=BF16)
    ffn = M.MoEFeedForward(H, I)
    o2, kept = ffn.forward(y, p.weights)
    assert torch.equal(out, o2) and torch.equal(s, s2)
    dy, g2 = ffn.backward(dout, p.weights, kept)
    dx2, dw2, db2 = M.MoENorm(H, 1e-5, kind).backward(dy, s2, p.norm_weight, mean, rstd, dsum=ds, bias=bias)
    assert torch.equal(dx, dx2) and torch.equal(grads["norm_weight"], dw2) and (not bias or torch.equal(grads["norm_bias"], db2))
    assert all(torch.equal(grads[n], g) for n, g in zip(("gate", "up", "down"), g2))

    # without any quantisation of activations, the weights' values as they are: each storing in 8 bits moves a value by at most 2^-4 of itself (or
    # of the smallest normal number, 2^-6 / 448 of its block's largest), and with independent signs by its 2-norm 2^-4 / sqrt(3) at most; y has two
    # of them in a row (x, h), the gradients up to four. Bounds of 2^-4 and 2^-3 of the 2-norm, then.
    wg, wu, wd = (values(v, SQUARE) for v in p.weights.tensors)
    leaf = s.double().requires_grad_(True)
    mu = leaf.mean(-1, keepdim=True) if norm == "layer" else 0
    yy = (leaf - mu) / torch.sqrt((leaf - mu).pow(2).mean(-1, keepdim=True) + 1e-5) * p.norm_weight.double()
    if bias:
        yy = yy + p.norm_bias.double()
    exact = (torch.nn.functional.silu(yy @ wg.t()) * (yy @ wu.t())) @ wd.t()
    (dleaf,) = torch.autograd.grad(exact, leaf, dout.double())
    assert (out.double() - exact).norm() <= 2.0 ** -4 * exact.norm()
    assert (dx.double() - ds.double() - dleaf).norm() <= 2.0 ** -3 * dleaf.norm() + 2.0 ** -8 * dx.double().norm()

    alone, s3 = block.decode(x, p, residual=res)
    assert torch.equal(s3, s) and (alone.double() - exact).norm() <= 2.0 ** -4 * exact.norm()


@gpu
def test_expert_and_dense_blocks_in_turn():
    """A dense block, an expert block and another dense one: the residual stream through all of them, forward, backward and decode."""
    T, H, I, E, k = 96, 256, 128, 4, 2
    gn = gen(5)
    dense = [M.DenseBlock(H, I) for _ in range(2)]
    dp = [M.DenseParams(torch.ones(H, device="cuda"), M.FeedForwardWeights(weight(gn, I, H), weight(gn, I, H), weight(gn, H, I))) for _ in dense]
    fc1, fc2 = (randn(gn, E, 2 * I, H) * 0.05).bfloat16(), (randn(gn, E, H, I) * 0.05).bfloat16()
    sfc1, sfc2 = (randn(gn, 2 * I, H) * 0.05).bfloat16(), (randn(gn, H, I) * 0.05).bfloat16()
    moe = M.MoEBlock(T, H, E, k, I)
    mp = M.BlockParams(torch.ones(H, device="cuda"), randn(gn, E, H) * 0.05, M.weights_from_combined(sfc1, sfc2, fc1, fc2))
    mg = [torch.zeros_like(t, dtype=F32) for t in (sfc1, sfc2, fc1, fc2)]
    x = randn(gn, T, H).bfloat16()

    def forward():
        a, s = dense[0].forward(x, dp[0])
        b, s, _ = moe.forward(a, mp, residual=s)
        return dense[1].forward(b, dp[1], residual=s)

    out, s = forward()
    dout, ds = randn(gn, T, H).bfloat16(), randn(gn, T, H).bfloat16()
    db, last = dense[1].backward(dout, ds=ds)
    da, _ = moe.backward(db, M.main_grads_from_combined(*mg), ds=db)
    dx, first = dense[0].backward(da, ds=da)
    for t in (out, s, dx, *[v for g in (first, last) for v in g.values() if v is not None], *mg):
        assert torch.isfinite(t).all() and t.abs().max() > 0
    again, s2 = forward()
    assert torch.equal(out, again) and torch.equal(s, s2)
    a, r = dense[0].decode(x, dp[0])
    b, r = moe.decode(a, mp, residual=r)
    alone, r = dense[1].decode(b, dp[1], residual=r)
    assert (alone.double() - out.double()).norm() <= 2.0 ** -4 * out.double().norm()
