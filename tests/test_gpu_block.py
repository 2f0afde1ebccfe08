"""The expert block (norm, router, experts, residual) against a plain fp64 implementation and its autograd.

The plain form rounds y to bf16 where the block does (with the gradient passed
through), and takes the block's choice of experts, which is checked by itself:
no expert left out may have a logit above a chosen one's by more than the
logits' error. Norms of whole tensors are compared. Forward: out is rounded to
bf16 once (2^-9 of each element), and the few elements of y that fall on the
other side of a rounding boundary move it by less: 2^-8. Backward: dhidden, dy
and (bf16 streams) dx are each rounded to bf16 once and the experts' operands
are two bf16 terms: four roundings of 2^-9 at most, each of which the norm's
projection may double: 2^-6.
"""
import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B

gpu = pytest.mark.gpu


def params(H, I, E, wr_dtype, bias, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = {"shared1": (r(2 * I, H) * 0.06).bfloat16(), "shared2": (r(H, I) * 0.06).bfloat16(),
         "fc1": (r(E, 2 * I, H) * 0.06).bfloat16(), "fc2": (r(E, H, I) * 0.06).bfloat16(),
         "norm_weight": 1 + 0.2 * r(H), "norm_bias": 0.2 * r(H) if bias else None, "router": (r(E, H) * 0.1).to(wr_dtype)}
    w = M.weights_from_combined(t["shared1"], t["shared2"], t["fc1"], t["fc2"])
    return t, M.BlockParams(t["norm_weight"], t["router"], w, norm_bias=t["norm_bias"])


def plain(t, x, residual, ids, kind, score, k, aux, z, leaves):
    """fp64 (out, s, losses, logits); leaves: t's tensors as fp64, some of them with gradients."""
    s = (x + residual) if residual is not None else x
    w, b, wr = leaves["norm_weight"], leaves["norm_bias"], leaves["router"]
    if kind == B.MOE_NORM_LAYER:
        m = s.mean(1, keepdim=True)
        h = (s - m) / torch.sqrt(((s - m) ** 2).mean(1, keepdim=True) + 1e-6)
    else:
        h = s / torch.sqrt((s ** 2).mean(1, keepdim=True) + 1e-6)
    y = h * w + (b if b is not None else 0.0)
    y = y + (y.detach().bfloat16().double() - y.detach())
    logits = y @ wr.t()
    P = torch.softmax(logits, 1) if score == B.MOE_SCORE_SOFTMAX else torch.sigmoid(logits)
    chosen = P.gather(1, ids.long())
    probs = chosen / chosen.sum(1, keepdim=True)
    Pn = P / P.sum(1, keepdim=True)
    counts = torch.bincount(ids.flatten().long(), minlength=wr.shape[0]).double()
    T, E = logits.shape
    losses = torch.stack([aux * E * ((counts / (k * T)) * Pn.mean(0)).sum(), z * (torch.logsumexp(logits, 1) ** 2).mean()])
    I = leaves["shared2"].shape[1]

    def mlp(v, fc1, fc2):
        g, u = (v @ fc1.t()).split(I, 1)
        return (torch.nn.functional.silu(g) * u) @ fc2.t()

    out = mlp(y, leaves["shared1"], leaves["shared2"])
    for e in range(E):
        at = (ids == e).nonzero()
        if len(at):
            out = out.index_add(0, at[:, 0], probs[at[:, 0], at[:, 1], None] * mlp(y[at[:, 0]], leaves["fc1"][e], leaves["fc2"][e]))
    return out, s, losses, logits


def close(a, b, tol, what):
    err = (a.double() - b).norm() / b.norm().clamp(min=1e-30)
    assert err <= tol, (what, float(err))


def check_choice(ids, logits, k):
    chosen = logits.gather(1, ids.long()).min(1).values
    rest = logits.scatter(1, ids.long(), float("-inf")).max(1).values
    assert bool((rest <= chosen + 1e-4 * logits.abs().max()).all())
    assert all(len(set(row)) == k for row in ids.tolist())


@gpu
@pytest.mark.parametrize("T,H,I,E,k,kind,score,dtype,bias,res", [
    (200, 256, 128, 16, 4, B.MOE_NORM_RMS, B.MOE_SCORE_SOFTMAX, torch.float32, False, True),
    (131, 512, 192, 24, 6, B.MOE_NORM_LAYER, B.MOE_SCORE_SIGMOID, torch.bfloat16, True, True),
    (1, 256, 128, 8, 2, B.MOE_NORM_LAYER, B.MOE_SCORE_SOFTMAX, torch.float32, True, False),
])
def test_training_step(T, H, I, E, k, kind, score, dtype, bias, res):
    t, p = params(H, I, E, torch.float32, bias, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    residual = torch.randn(T, H, generator=g, device="cuda").to(dtype) if res else None
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ds = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    aux, z = 0.02, 0.003
    block = M.MoEBlock(T, H, E, k, I, norm=kind, score=score, aux_coeff=aux, z_coeff=z)
    out, s, losses = block.forward(x, p, residual=residual)
    mg = {n: torch.zeros(*t[n].shape, device="cuda") for n in ("shared1", "shared2", "fc1", "fc2")}
    grads = M.main_grads_from_combined(mg["shared1"], mg["shared2"], mg["fc1"], mg["fc2"])
    ids = block._kept[6]
    dx, gr = block.backward(dout, grads, ds=ds)
    with pytest.raises(ValueError):
        block.backward(dout, grads)

    leaves = {n: None if v is None else v.double().requires_grad_() for n, v in t.items()}
    # s is what the stream rounds to; its gradient passes through
    if res:
        assert torch.equal(s, x + residual)
    xs = s.double().requires_grad_()
    o, ss, ls, logits = plain(t, xs, None, ids, kind, score, k, aux, z, leaves)
    check_choice(ids, logits.detach(), k)
    close(out, o.detach(), 2 ** -8, "out")
    close(losses, ls.detach(), 2 ** -8, "losses")
    ((o * dout.double()).sum() + (ss * ds.double()).sum() + ls.sum()).backward()
    close(dx, xs.grad, 2 ** -6, "dx")
    close(gr["norm_weight"], leaves["norm_weight"].grad, 2 ** -6, "norm_weight")
    if bias:
        close(gr["norm_bias"], leaves["norm_bias"].grad, 2 ** -6, "norm_bias")
    else:
        assert gr["norm_bias"] is None
    close(gr["router_weight"], leaves["router"].grad, 2 ** -6, "router")
    for n in mg:
        close(mg[n], leaves[n].grad, 2 ** -6, n)
    block.close()


@gpu
@pytest.mark.parametrize("T", [1, 5, 64])
@pytest.mark.parametrize("wr", [torch.float32, torch.bfloat16])
def test_decode_is_the_forward(T, wr):
    """decode (small batches on the decoder) and forward: the same s, and out within its one rounding to bf16."""
    H, I, E, k = 512, 128, 16, 4
    t, p = params(H, I, E, wr, False, seed=T)
    g = torch.Generator(device="cuda").manual_seed(T + 2)
    x, r = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    block = M.MoEBlock(64, H, E, k, I)
    out, s, losses = block.forward(x, p, residual=r)
    assert losses is None
    fast, s2 = block.decode(x, p, residual=r)
    assert torch.equal(s, s2)
    close(fast, out.double(), 2 ** -8, "out")
    # the decoder alone, and more tokens than it takes
    only = M.MoEBlock(0, H, E, k, I, decode_tokens=4)
    with pytest.raises(ValueError):
        only.forward(x, p)
    if T <= 4:
        assert torch.equal(only.decode(x, p, residual=r)[0], fast)
    else:
        with pytest.raises(ValueError):
            only.decode(x, p, residual=r)


@gpu
def test_two_blocks_in_a_graph():
    """Two blocks one after the other, captured once and replayed over new input."""
    T, H, I, E, k = 3, 512, 128, 16, 4
    made = [params(H, I, E, torch.float32, False, seed=40 + i) for i in range(2)]  # moe_weights are pointers: their tensors stay
    ps = [m[1] for m in made]
    block = M.MoEBlock(0, H, E, k, I)
    x = torch.randn(T, H, device="cuda").bfloat16()

    def run():
        a, s = block.decode(x, ps[0])
        return block.decode(a, ps[1], residual=s)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, s = run()
    for seed in range(3):
        x.copy_(torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        want, s2 = run()
        assert torch.equal(s, s2) and torch.equal(out, want)


def test_refuses_an_empty_block():
    with pytest.raises(ValueError):
        M.MoEBlock(0, 256, 8, 2, 128, decode_tokens=0)


@gpu
def test_gradients_of_any_layout():
    """dout with rows of a wider buffer, transposed, or one row broadcast: as the same values in compact rows. Other
    shapes, types and places are refused, and the step that waits is kept."""
    T, H, I, E, k = 33, 256, 128, 8, 2
    t, p = params(H, I, E, torch.float32, False, seed=3)
    block = M.MoEBlock(T, H, E, k, I)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    row = torch.randn(1, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()

    def step(dout):
        block.forward(x, p)
        for bad in (dout.float(), dout[:-1], dout[:, :-8], dout.cpu()):
            with pytest.raises(ValueError):
                block.backward(bad, None)
        mg = {n: torch.zeros(*t[n].shape, device="cuda") for n in ("shared1", "shared2", "fc1", "fc2")}
        dx, gr = block.backward(dout, M.main_grads_from_combined(mg["shared1"], mg["shared2"], mg["fc1"], mg["fc2"]))
        return [dx, gr["norm_weight"], gr["router_weight"], *mg.values()]

    full = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    wide = torch.zeros(T, H + 8, device="cuda").bfloat16()
    wide[:, :H] = full
    want = step(full)
    for view in (wide[:, :H], full.t().contiguous().t()):
        assert all(torch.equal(a, b) for a, b in zip(step(view), want))
    assert all(torch.equal(a, b) for a, b in zip(step(row.expand(T, H)), step(row.repeat(T, 1))))


def mx_params(H, I, E, seed):
    """params with MXFP8 experts, and (wherever a comparison needs them) their tensors."""
    t, p = params(H, I, E, torch.float32, False, seed)
    t["mx"] = [M.mxfp8_weight(m) for m in (t["fc1"][:, :I], t["fc1"][:, I:], t["fc2"])]
    p.weights.routed_gate, p.weights.routed_up, p.weights.routed_down = (M.mxfp8_view(*v) for v in t["mx"])
    return t, p


@gpu
def test_mxfp8_experts():
    """The block's steps are its parts run one by one, bit for bit, on the scales of the params that were prepared;
    with other params, or none prepared, they are refused."""
    T, H, I, E, k = 96, 256, 128, 8, 2
    sets = [mx_params(H, I, E, seed) for seed in (21, 22)]
    g = torch.Generator(device="cuda").manual_seed(23)
    x, r, dout = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    block = M.MoEBlock(T, H, E, k, I, routed_wtype=B.MOE_W_MXFP8)

    def grads(t):
        mg = {n: torch.zeros(*t[n].shape, device="cuda") for n in ("shared1", "shared2", "fc1", "fc2")}
        return mg, M.main_grads_from_combined(mg["shared1"], mg["shared2"], mg["fc1"], mg["fc2"])

    def refused(call):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.status == B.MOE_ERR_STATE

    refused(lambda: block.forward(x, sets[0][1], residual=r))
    for t, p in sets:
        block.prepare(p)
        out, s, _ = block.forward(x, p, residual=r)
        ids, counts = block._kept[6], block._kept[7]
        mg, m = grads(t)
        dx, gr = block.backward(dout, m)
        # the parts
        layer = M.MoELayer(T, H, E, k, I, routed_wtype=B.MOE_W_MXFP8)
        layer.prepare_weights(p.weights)
        y, s2, mean, rstd = block.norm.forward(x, p.norm_weight, residual=r, out_dtype=torch.bfloat16)
        logits = torch.nn.functional.linear(y.float(), p.router_weight)
        ids2, probs2, counts2, _ = block.router.forward(logits)
        assert torch.equal(ids, ids2) and torch.equal(counts, counts2) and torch.equal(s, s2)
        assert torch.equal(out, layer.forward_topk(y, ids2, probs2, p.weights))
        mg2, m2 = grads(t)
        dy, dprobs = layer.backward(dout, m2)
        dl = block.router.backward(logits, ids2, dprobs, counts=counts2)
        dx2, dw2, _ = block.norm.backward(torch.addmm(dy.float(), dl, p.router_weight), s2, p.norm_weight, mean, rstd)
        assert torch.equal(dx, dx2) and torch.equal(gr["norm_weight"], dw2) and all(torch.equal(mg[n], mg2[n]) for n in mg)
        # decoding reads the weights as they are; more tokens than the decoder takes go to the layer
        few, _ = block.decode(x[:9], p, residual=r[:9])
        scale = float(out.float().abs().max())
        assert float((few.float() - out[:9].float()).abs().max()) <= 6e-2 * scale    # the layer quantises activations
        assert torch.equal(block.decode(x, p, residual=r)[0], out)
    # the layer holds the second set's scales
    (_, p0), (t1, p1) = sets
    refused(lambda: block.forward(x, p0, residual=r))
    refused(lambda: block.decode(x, p0, residual=r))
    block.decode(x[:9], p0, residual=r[:9])
    out, _, _ = block.forward(x, p1, residual=r)
    block.prepare(p0)
    mg, m = grads(t1)
    refused(lambda: block.backward(dout, m))
    block.prepare(p1)
    dx2, _ = block.backward(dout, m)
    assert torch.equal(dx, dx2) and all(torch.equal(mg[n], mg2[n]) for n in mg)
    M.MoEBlock(0, H, E, k, I, routed_wtype=B.MOE_W_MXFP8).prepare(p0)   # nothing to prepare


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_a_captured_step_through_the_layer_keeps_its_weights(mx):
    """More tokens than the decoder takes, captured: other weights through the layer are refused from then on, the same
    ones and the decoder's are not, and replays give the captured weights' results."""
    T, H, I, E, k = 24, 256, 128, 8, 2
    made = [(mx_params(H, I, E, seed) if mx else params(H, I, E, torch.float32, False, seed)) for seed in (31, 32)]
    (_, p0), (_, p1) = made
    block = M.MoEBlock(T, H, E, k, I, decode_tokens=4, routed_wtype=B.MOE_W_MXFP8 if mx else B.MOE_W_BF16)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(33)).bfloat16()
    for p in (p1, p0):
        block.prepare(p)
        want, _ = block.decode(x, p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = block.decode(x, p0)
    few, _ = block.decode(x[:4], p1)
    for call in (lambda: block.decode(x, p1), lambda: block.forward(x, p1)) + ((lambda: block.prepare(p1),) if mx else ()):
        with pytest.raises(M.MoeError) as e:
            call()
        assert e.value.status == B.MOE_ERR_STATE
    assert torch.equal(block.decode(x, p0)[0], want)
    block.prepare(p0)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(few, block.decode(x[:4], p1)[0])


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stream_gradients_of_any_layout(dtype):
    """ds transposed, broadcast, or with rows of a wider buffer: as the same values in compact rows. One of another shape,
    type or place is refused before the experts' gradients are touched."""
    T, H, I, E, k = 20, 256, 128, 8, 2
    t, p = params(H, I, E, torch.float32, False, seed=6)
    block = M.MoEBlock(T, H, E, k, I)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, full, row = (torch.randn(n, H, generator=g, device="cuda").to(dtype) for n in (T, T, 1))
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    mg = {n: torch.zeros(*t[n].shape, device="cuda") for n in ("shared1", "shared2", "fc1", "fc2")}
    grads = M.main_grads_from_combined(mg["shared1"], mg["shared2"], mg["fc1"], mg["fc2"])

    def step(ds):
        block.forward(x, p)
        before = [m.clone() for m in mg.values()]
        other = torch.bfloat16 if dtype == torch.float32 else torch.float32
        for bad in (ds[:-1], ds[:, :-8], ds.to(other), ds.cpu()):
            with pytest.raises(ValueError):
                block.backward(dout, grads, ds=bad)
        assert all(torch.equal(a, b) for a, b in zip(before, mg.values()))
        return block.backward(dout, grads, ds=ds)[0]

    want = step(full)
    wide = torch.zeros(T, H + 8, device="cuda", dtype=dtype)  # rows on 16 bytes: sums in the same order
    wide[:, :H] = full
    assert torch.equal(step(wide[:, :H]), want) and torch.equal(step(full.t().contiguous().t()), want)
    assert torch.equal(step(row.expand(T, H)), step(row.repeat(T, 1)))
