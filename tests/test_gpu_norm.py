"""Layer norm and RMS norm, forward and backward, against their formulas in fp64.

Tolerances. u = 2^-24. A sum of n fp32 terms accumulated in any order by at
least 32 partial sums has an error of at most (n/32 + 32) u times the sum of the
terms' magnitudes (gamma below); each further fp32 operation adds u of its
result. With S = mean |s| the statistics are off by gamma S (mean) and, relative,
gamma plus the mean's effect (rstd), so every y by at most
    8 gamma |w| rstd (|s| + S) (1 + |xhat|) + 8 u |b|,
and bf16 results by 2^-8 of themselves more (round to nearest: 2^-9; the other
half covers a rounding midpoint). Sums over T rows in any order are off by at
most (T + 64) u times the sum of magnitudes.
"""
import math

import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B

gpu = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
KINDS = {"layer": B.MOE_NORM_LAYER, "rms": B.MOE_NORM_RMS}


def gamma(H):
    return (H / 32 + 32) * U


def ref_forward(s, w, b, eps, kind):
    mean = s.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(s[:, :1])
    rstd = 1 / torch.sqrt((s - mean).pow(2).mean(-1, keepdim=True) + eps)
    y = (s - mean) * rstd * w
    return (y if b is None else y + b), mean, rstd


def ref_backward(s, w, dy, mean, rstd, kind):
    """ds, dw, db, and bounds on the magnitudes that their fp32 evaluation adds up."""
    xh = (s - mean) * rstd
    g = dy * w
    mg = g.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(mean)
    mgx = (g * xh).mean(-1, keepdim=True)
    ds = rstd * (g - mg - xh * mgx)
    mag = rstd * (g.abs() + g.abs().mean(-1, keepdim=True) + (1 + xh.abs()) * (g * (xh.abs() + 1)).abs().mean(-1, keepdim=True))
    return ds, (dy * xh).sum(0), dy.sum(0), mag, (dy * xh).abs().sum(0), dy.abs().sum(0)


def test_the_backward_formula_is_the_gradient():
    """The fp64 formula the kernels are compared with, against central differences."""
    g = torch.Generator().manual_seed(5)
    for kind in KINDS:
        T, H, eps, h = 3, 7, 1e-3, 1e-6
        s, dy = torch.randn(T, H, generator=g, dtype=torch.float64), torch.randn(T, H, generator=g, dtype=torch.float64)
        w, b = torch.randn(H, generator=g, dtype=torch.float64), torch.randn(H, generator=g, dtype=torch.float64)
        _, mean, rstd = ref_forward(s, w, b, eps, kind)
        ds, dw, db, *_ = ref_backward(s, w, dy, mean, rstd, kind)

        def loss(s, w, b):
            return (ref_forward(s, w, b, eps, kind)[0] * dy).sum()

        for x, grad, at in ((s, ds, 0), (w, dw, 1), (b, db, 2)):
            for i in range(x.numel()):
                e = torch.zeros_like(x).view(-1)
                e[i] = h
                args = [s, w, b]
                args[at] = x + e.view_as(x)
                up = loss(*args)
                args[at] = x - e.view_as(x)
                assert abs((up - loss(*args)) / (2 * h) - grad.view(-1)[i]) < 1e-7


def rows(t, pad, shift):
    """t in rows of a buffer `pad` elements wider, starting `shift` elements into it; NaN around them."""
    wide = torch.full((t.shape[0] * (t.shape[1] + pad) + shift + 8,), math.nan, dtype=t.dtype, device=t.device)
    v = wide[shift:shift + t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v


def make(T, H, xt, yt, wt, seed, offset=0.0, pad=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rows((r(T, H) + offset).to(xt), pad, shift)
    res, dsum = rows(r(T, H).to(xt), pad, shift), rows(r(T, H).to(xt), pad, shift)
    return dict(x=x, res=res, dsum=dsum, dy=rows(r(T, H).to(yt), pad, shift), w=(1 + 0.2 * r(H)).to(wt), b=(0.3 * r(H)).to(wt))


def close(got, ref, tol, what):
    err = (got.double() - ref).abs()
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * ref.abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol.clamp(min=1e-300)).max()):.3g} x the bound"


CASES = [
    # T, H, x, y, w, residual, bias, offset, pad, shift
    (1, 1, F32, F32, F32, False, True, 0.0, 0, 0),
    (3, 2, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (5, 31, BF16, F32, F32, True, False, 0.0, 0, 0),
    (4, 64, BF16, BF16, F32, False, True, 0.0, 0, 0),
    (7, 256, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (130, 1000, BF16, BF16, F32, True, True, 3.0, 8, 0),
    (33, 1023, F32, BF16, BF16, True, True, 0.0, 0, 0),
    (33, 1025, BF16, BF16, F32, True, True, 0.0, 3, 1),
    (300, 2048, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (300, 2048, F32, BF16, F32, False, False, 0.0, 4, 3),
    (17, 2051, F32, F32, F32, True, True, 100.0, 5, 0),
    (9, 4096, F32, F32, BF16, True, True, 0.0, 0, 0),
    (12, 7168, BF16, BF16, F32, True, True, 0.0, 8, 8),
    (3, 12289, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (2, 32768, BF16, BF16, F32, True, True, 0.0, 0, 0),
    (2, 32767, F32, F32, F32, True, True, 0.0, 1, 1),
    (700, 96, BF16, BF16, F32, True, True, 0.0, 0, 0),
    (2500, 40, F32, F32, F32, False, True, 0.0, 0, 0),
    # many rows: every width of a block, whole and odd columns, rows that end inside a warp's share
    (400, 513, BF16, BF16, F32, True, True, 0.0, 3, 1),
    (400, 512, F32, F32, BF16, True, True, 2.0, 0, 0),
    (350, 1544, BF16, F32, BF16, True, True, 0.0, 0, 0),
    (320, 3001, F32, BF16, F32, True, False, 0.0, 1, 3),
    (320, 5001, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (310, 8192, F32, F32, F32, True, True, 0.0, 0, 0),
    (310, 8200, F32, F32, F32, False, True, 0.0, 0, 0),
    (310, 9001, BF16, BF16, F32, True, True, 0.0, 2, 1),
    (310, 12288, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (310, 12288, F32, BF16, F32, True, True, 0.0, 4, 4),
    (8200, 4104, BF16, BF16, BF16, True, True, 0.0, 0, 0),
    (40, 16384, BF16, BF16, F32, True, True, 0.0, 0, 0),
    (40, 14008, BF16, F32, BF16, False, True, 1.0, 8, 8),
]


@gpu
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("T,H,xt,yt,wt,residual,bias,offset,pad,shift", CASES)
def test_forward_and_backward(T, H, xt, yt, wt, residual, bias, offset, pad, shift, kind):
    d = make(T, H, xt, yt, wt, 100 + T + H, offset, pad, shift)
    norm = M.MoENorm(H, eps=1e-5, kind=KINDS[kind])
    b = d["b"] if bias else None
    y, s, mean, rstd = norm.forward(d["x"], d["w"], b, residual=d["res"] if residual else None, out_dtype=yt)
    assert y.dtype == yt and s.dtype == xt
    if residual:
        assert torch.equal(s, (d["x"].float() + d["res"].float()).to(xt))
    else:
        assert s is d["x"]
    S, W = s.double(), d["w"].double()
    ry, rm, rr = ref_forward(S, W, b.double() if bias else None, float(torch.tensor(1e-5, dtype=F32)), kind)
    xh = (S - rm) * rr
    G = gamma(H)
    mag = S.abs() + S.abs().mean(-1, keepdim=True)
    close(y, ry, 8 * G * W.abs() * rr * mag * (1 + xh.abs()) + 8 * U * (b.double().abs() if bias else 0), "y")
    if kind == "layer":
        close(mean, rm[:, 0], G * S.abs().mean(-1), "mean")
    else:
        assert mean is None
    rstd_tol = 4 * G * rr[:, 0] * (1 + rr[:, 0] * S.abs().mean(-1))
    close(rstd, rr[:, 0], rstd_tol, "rstd")

    # backward, at the saved statistics
    m64 = mean.double()[:, None] if kind == "layer" else torch.zeros_like(rm)
    dsum = d["dsum"] if residual else None
    ds, dw, db = norm.backward(d["dy"], s, d["w"], mean, rstd, dsum=dsum, bias=bias)
    rds, rdw, rdb, magd, magw, magb = ref_backward(S, W, d["dy"].double(), m64, rstd.double()[:, None], kind)
    # xhat itself is rounded: s - mean to u of |s| + |mean|
    slip = 1 + (S.abs() + m64.abs()) * rstd.double()[:, None]
    if dsum is not None:
        rds = rds + dsum.double()
    close(ds, rds, 8 * G * magd * slip + 2 * U * rds.abs() + (2 * U * dsum.double().abs() if dsum is not None else 0), "ds")
    dym = d["dy"].double().abs()
    close(dw, rdw, (T + 64) * U * (magw + (dym * slip).sum(0)), "dweight")
    assert dw.dtype == F32
    if bias:
        close(db, rdb, (T + 64) * U * magb, "dbias")
    else:
        assert db is None

    # the same inputs give the same bits
    y2, s2, mean2, rstd2 = norm.forward(d["x"], d["w"], b, residual=d["res"] if residual else None, out_dtype=yt)
    ds2, dw2, db2 = norm.backward(d["dy"], s, d["w"], mean, rstd, dsum=dsum, bias=bias)
    assert torch.equal(y, y2) and torch.equal(ds, ds2) and torch.equal(dw, dw2) and (not bias or torch.equal(db, db2))


@gpu
@pytest.mark.parametrize("H", [40, 515, 2048])
@pytest.mark.parametrize("gt", [F32, BF16])
def test_gradient_accumulation(gt, H):
    """Given buffers: overwritten, or main_grad += dw (bf16: bf16(main_grad + bf16(dw))), bit for bit the new gradient's sum."""
    d = make(65, H, BF16, BF16, F32, 3)
    norm = M.MoENorm(H)
    y, s, mean, rstd = norm.forward(d["x"], d["w"], d["b"])
    _, dw, db = norm.backward(d["dy"], s, d["w"], mean, rstd, bias=True)
    g0 = torch.randn(2, H, device="cuda").to(gt)
    w, b = g0[0].clone(), g0[1].clone()
    norm.backward(d["dy"], s, d["w"], mean, rstd, bias=True, dweight=w, dbias=b, accumulate=True)
    for got, old, new in ((w, g0[0], dw), (b, g0[1], db)):
        assert torch.equal(got, (old.float() + new.to(gt).float()).to(gt))
    norm.backward(d["dy"], s, d["w"], mean, rstd, bias=True, dweight=w, dbias=b)
    assert torch.equal(w, dw.to(gt)) and torch.equal(b, db.to(gt))


@gpu
@pytest.mark.parametrize("H", [33, 1024, 5000])
def test_nan_and_inf_stay_in_their_row(H):
    d = make(40, H, BF16, BF16, F32, 9)
    norm = M.MoENorm(H)
    y, s, mean, rstd = norm.forward(d["x"], d["w"], d["b"], residual=d["res"])
    x = d["x"].clone()
    x[3, H // 2], x[20, 0] = math.nan, math.inf
    y2, s2, mean2, rstd2 = norm.forward(x, d["w"], d["b"], residual=d["res"])
    keep = [t for t in range(40) if t not in (3, 20)]
    assert torch.equal(y[keep], y2[keep]) and torch.equal(rstd[keep], rstd2[keep])
    assert y2[3].isnan().all() and y2[20].isnan().any()
    ds, _, _ = norm.backward(d["dy"], s, d["w"], mean, rstd)
    ds2, dw2, _ = norm.backward(d["dy"], s2, d["w"], mean2, rstd2)
    assert torch.equal(ds[keep], ds2[keep]) and ds2[3].isnan().all() and dw2.isnan().all()


@gpu
def test_constant_rows_and_empty_batches():
    """A constant row has no spread: xhat is 0, y the bias, rstd 1/sqrt(eps). No rows: empty outputs, zero gradients."""
    H = 520
    norm = M.MoENorm(H, eps=1e-4)
    w, b = torch.randn(H, device="cuda"), torch.randn(H, device="cuda")
    x = torch.full((3, H), 0.5, device="cuda", dtype=BF16)
    y, _, mean, rstd = norm.forward(x, w, b, out_dtype=F32)
    assert torch.equal(y, b.expand(3, H)) and torch.equal(mean, torch.full((3,), 0.5, device="cuda"))
    assert ((rstd - 100).abs() < 100 * 4 * U + 1e-5).all()
    e = x[:0]
    y, s, mean, rstd = norm.forward(e, w, b)
    assert y.shape == (0, H)
    ds, dw, db = norm.backward(y, s, w, mean, rstd, bias=True)
    assert ds.shape == (0, H) and not dw.any() and not db.any()
    keep = dw + 3
    norm.backward(y, s, w, mean, rstd, dweight=keep, accumulate=True)
    assert torch.equal(keep, dw + 3)


@gpu
def test_in_place_sum_other_stream_and_graph():
    """sum may be the residual buffer and dx the dsum buffer; a call on another stream and its replay as a
    CUDA graph give the same bits."""
    T, H = 37, 1536
    d = make(T, H, BF16, BF16, F32, 21)
    norm = M.MoENorm(H)
    y, s, mean, rstd = norm.forward(d["x"], d["w"], d["b"], residual=d["res"])
    ds, dw, db = norm.backward(d["dy"], s, d["w"], mean, rstd, dsum=d["dsum"], bias=True)
    cfg = norm._cfg(BF16, BF16, F32)
    r, g = d["res"].clone(), d["dsum"].clone()
    y2 = torch.empty_like(y)
    M.moe_norm_forward(cfg, d["x"], d["w"], y2, d["b"], r, r, torch.empty_like(mean), torch.empty_like(rstd))
    assert torch.equal(r, s) and torch.equal(y2, y)
    dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
    ws = torch.full((M.moe_norm_backward_size(cfg, T),), 255, dtype=torch.uint8, device="cuda")
    M.moe_norm_backward(cfg, d["dy"], s, d["w"], mean, rstd, g, g, dw2, db2, workspace=ws)
    assert torch.equal(g, ds) and torch.equal(dw2, dw) and torch.equal(db2, db)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3, s3, mean3, rstd3 = norm.forward(d["x"], d["w"], d["b"], residual=d["res"], stream=side)
    ds3, dw3, _ = norm.backward(d["dy"], s3, d["w"], mean3, rstd3, dsum=d["dsum"], bias=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y3, y) and torch.equal(ds3, ds) and torch.equal(dw3, dw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, sg, mg, rg = norm.forward(d["x"], d["w"], d["b"], residual=d["res"])
        dsg, dwg, _ = norm.backward(d["dy"], sg, d["w"], mg, rg, dsum=d["dsum"], bias=True)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(yg, y) and torch.equal(dsg, ds) and torch.equal(dwg, dw)


def test_refusals():
    def status(call):
        with pytest.raises(M.MoeError) as e:
            call()
        return e.value.status

    c = lambda **kw: M.moe_norm_config(**{**dict(hidden=64, eps=1e-5, kind=0, x_type=0, y_type=0, w_type=0), **kw})  # noqa: E731
    size = lambda **kw: M.moe_norm_backward_size(c(**kw), 8)  # noqa: E731
    assert size() > 0
    for kw, want in ((dict(hidden=0), 1), (dict(hidden=32769), 2), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
                     (dict(kind=2), 1), (dict(x_type=2), 1), (dict(y_type=-1), 1), (dict(w_type=5), 1)):
        assert status(lambda: size(**kw)) == want, kw
    L = M.load()
    f = lambda cfg, T=2, x=256, xs=64, r=None, rs=0, w=256, b=None, s=None, ss=0, y=256, ys=64: L.moe_norm_forward(  # noqa: E731
        cfg, T, x, xs, r, rs, w, b, s, ss, y, ys, None, None, None)
    assert f(c(), T=0) == 0
    for kw in (dict(T=-1), dict(x=None), dict(y=None), dict(w=None), dict(xs=63), dict(ys=1), dict(r=256, rs=64),
               dict(r=256, rs=64, s=256, ss=63), dict(r=256, rs=3, s=256, ss=64), dict(x=257), dict(y=255), dict(b=1)):
        assert f(c(), **kw) == 1, kw
    assert f(c(x_type=1), x=258) == 1
    g = lambda cfg, T=2, dy=256, x=256, w=256, mean=256, rstd=256, dx=256, dw=256, gt=0, acc=0, ws=256, n=1 << 20, ld=64: L.moe_norm_backward(  # noqa: E731
        cfg, T, dy, ld, x, ld, w, mean, rstd, None, 0, dx, ld, dw, None, gt, acc, ws, n, None)
    for kw in (dict(T=-1), dict(dy=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(dx=None),
               dict(gt=2), dict(acc=2), dict(ws=None), dict(ws=264), dict(n=16), dict(ld=8), dict(dw=258), dict(mean=2)):
        assert g(c(), **kw) == 1, kw


def test_tensors_elsewhere_are_refused():
    """Tensors in host memory come back as errors before anything is launched, in any place."""
    norm = M.MoENorm(16)
    x, w, v = torch.zeros(2, 16), torch.zeros(16), torch.zeros(2)
    with pytest.raises(ValueError, match="device"):
        norm.forward(x, w)
    with pytest.raises(ValueError, match="device"):
        norm.backward(x, x, w, v, v)
    cfg = norm._cfg(F32, F32, F32)
    with pytest.raises(ValueError, match="device"):
        M.moe_norm_forward(cfg, x, w, x)
    with pytest.raises(ValueError, match="device"):
        M.moe_norm_backward(cfg, x, x, w, v, v, x)


@gpu
def test_tensors_on_two_devices_are_refused():
    norm = M.MoENorm(16)
    x, w, v, g = torch.zeros(2, 16), torch.zeros(16), torch.zeros(2), torch.zeros(16)
    X, W, V, G = (t.cuda() for t in (x, w, v, g))
    before = M.moe_launch_count()
    for args in ((x, W), (X, w), (X, W, w), (X, W, None, x)):
        with pytest.raises(ValueError, match="device"):
            norm.forward(*args)
    for args in ((x, X, W, V, V), (X, x, W, V, V), (X, X, w, V, V), (X, X, W, v, V), (X, X, W, V, v), (X, X, W, V, V, x),
                 (X, X, W, V, V, None, False, g), (X, X, W, V, V, None, True, G, g)):
        with pytest.raises(ValueError, match="device"):
            norm.backward(*args)
    cfg = norm._cfg(F32, F32, F32)
    for args in ((X, w, X), (X, W, x), (X, W, X, w), (X, W, X, None, x, X), (X, W, X, None, X, x), (X, W, X, None, None, None, v)):
        with pytest.raises(ValueError, match="device"):
            M.moe_norm_forward(cfg, *args)
    with pytest.raises(ValueError, match="device"):
        M.moe_norm_backward(cfg, X, X, W, V, V, X, None, G, None, workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    assert M.moe_launch_count() == before
    norm.forward(X, W, stream=torch.cuda.Stream())
    assert M.moe_launch_count() == before + 1
