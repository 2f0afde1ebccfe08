"""The router: the choice of experts, its probs and the balancing losses, forward and
backward, against the definition in fp64.

Tolerances. u = 2^-24. The choice compares logits, so ids and counts are equal,
not close. A score is off by the rounding of its exponent's argument (u |l - m|),
of exp and of the quotient (4 u), and of the row's sum ((E/32 + 32) u): relative
r = (E/32 + 64 + max |l - m|) u. Probs divide by another such sum: 3 r. Losses are sums over T tokens:
(T + E) u more. A gradient adds up terms whose magnitudes `mag` collects: 4 r mag.
"""
import math

import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
from mixture_experts_layer_pack_gb300 import binding as B

gpu = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
SCORES = {"softmax": B.MOE_SCORE_SOFTMAX, "sigmoid": B.MOE_SCORE_SIGMOID}


def reference(l, c, bias=None, dprobs=None, loss_grad=1.0):
    """Definition in fp64 over logits l (fp64); c: dict of E, k, score, normalise, scale, aux, z."""
    T, E, k = l.shape[0], c["E"], c["k"]
    l = l.clone().requires_grad_(True)
    free = l.detach() > -math.inf
    lf = torch.where(free, l, torch.full_like(l, -1e6))
    some = free.any(-1, keepdim=True)
    one = torch.ones_like(l[:, :1])
    score = torch.softmax(lf, -1) if c["score"] == "softmax" else torch.sigmoid(lf)
    score = torch.where(free, score, torch.zeros_like(score))
    dist = score / torch.where(some, score.sum(-1, keepdim=True), one)
    key = l.detach() if bias is None else torch.where(free, score.detach() + bias, torch.full_like(l, -math.inf))
    order = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :k]
    ok = free.gather(1, order)
    picked = score.gather(1, order)
    total = torch.where(some, picked.sum(-1, keepdim=True), one) if c["normalise"] else one
    probs = c["scale"] * picked / total
    ids = torch.where(ok, order, torch.full_like(order, -1)).int()
    counts = torch.bincount(order[ok], minlength=E)
    lse = torch.where(some[:, 0], torch.logsumexp(lf, -1), torch.zeros_like(lf[:, 0]))
    balance = c["aux"] * E * (counts.double() / (k * max(T, 1)) * dist.sum(0) / max(T, 1)).sum()
    z = c["z"] * lse.pow(2).sum() / max(T, 1)
    out = dict(ids=ids, probs=probs.detach(), counts=counts.int(), losses=torch.stack([balance, z]).detach(), lse=lse.detach())
    if dprobs is not None:
        d = torch.where(ok, dprobs, torch.zeros_like(dprobs))
        goal = (probs * d).sum() + loss_grad * (balance + z)
        out["dlogits"] = torch.autograd.grad(goal, l)[0]
        # the magnitudes that the evaluation adds up
        with torch.no_grad():
            s = d.abs() * abs(c["scale"])
            if c["normalise"]:
                s = (s + (s * picked / total).sum(-1, keepdim=True)) / total
            v = torch.zeros_like(l).scatter_add(1, order, torch.where(ok, s, torch.zeros_like(s)))
            a = (abs(loss_grad * c["aux"]) * E / (k * T * T)) * counts.double().expand(T, E)
            if c["score"] == "softmax":
                v = v + a
                mag = score * (v + (v * score).sum(-1, keepdim=True))
            else:
                mag = (v + (a + (a * dist).sum(-1, keepdim=True)) / torch.where(some, score.sum(-1, keepdim=True), one)) * score
            mag = mag + abs(loss_grad * c["z"]) * 2 / T * lse.abs()[:, None] * torch.exp(lf - lse[:, None]) * (1 + lse.abs()[:, None])
        out["mag"] = mag
    return out


def test_the_backward_of_the_definition_matches_differences():
    """Autograd of the fp64 definition against central differences, away from ties."""
    g = torch.Generator().manual_seed(3)
    for score in SCORES:
        for normalise in (False, True):
            c = dict(E=5, k=2, score=score, normalise=normalise, scale=1.5, aux=0.3, z=0.2)
            l, d = torch.randn(4, 5, generator=g, dtype=torch.float64), torch.randn(4, 2, generator=g, dtype=torch.float64)

            def goal(l):
                r = reference(l, c)
                return (r["probs"] * d).sum() + 0.7 * r["losses"].sum()

            grad, h = reference(l, c, dprobs=d, loss_grad=0.7)["dlogits"], 1e-6
            for i in range(l.numel()):
                e = torch.zeros_like(l).view(-1)
                e[i] = h
                e = e.view_as(l)
                assert abs((goal(l + e) - goal(l - e)) / (2 * h) - grad.view(-1)[i]) < 1e-7


def logits_of(T, E, xt, seed, closed=0.0, pad=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(T, E, generator=g, device="cuda") * 2
    if closed:
        l = l.masked_fill(torch.rand(T, E, generator=g, device="cuda") < closed, -math.inf)
    wide = torch.full((T * (E + pad) + shift,), math.nan, dtype=xt, device="cuda")
    v = wide[shift:].view(T, E + pad)[:, :E]
    v.copy_(l)
    return v, torch.randn(T, 32, generator=g, device="cuda")


CASES = [
    # T, E, k, type, closed, pad, shift
    (1, 1, 1, F32, 0.0, 0, 0),
    (1, 96, 6, F32, 0.0, 0, 0),
    (3, 2, 2, BF16, 0.5, 0, 0),
    (64, 8, 2, F32, 0.0, 0, 0),
    (65, 31, 5, BF16, 0.2, 1, 1),
    (200, 33, 8, F32, 0.0, 3, 1),
    (300, 96, 6, BF16, 0.0, 0, 0),
    (257, 128, 8, F32, 0.6, 0, 0),
    (40, 160, 6, BF16, 0.0, 8, 0),
    (33, 257, 32, F32, 0.9, 0, 0),
    (100, 384, 6, F32, 0.0, 0, 0),
    (20, 1000, 9, BF16, 0.0, 0, 0),
    (9, 1024, 32, F32, 0.99, 0, 0),
    (5000, 12, 3, F32, 0.3, 0, 0),
]


@gpu
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("T,E,k,xt,closed,pad,shift", CASES)
def test_forward_and_backward(T, E, k, xt, closed, pad, shift, normalise, score):
    l, d = logits_of(T, E, xt, 7 * T + E, closed, pad, shift)
    d = d[:, :k].contiguous()
    c = dict(E=E, k=k, score=score, normalise=normalise, scale=2.5, aux=0.02, z=0.003)
    router = M.MoERouter(E, k, score=SCORES[score], normalise=normalise, scale=2.5, aux_coeff=0.02, z_coeff=0.003)
    f32 = lambda v: float(torch.tensor(v, dtype=F32))  # noqa: E731
    c64 = {**c, "aux": f32(0.02), "z": f32(0.003)}
    ref = reference(l.double(), c64, dprobs=d.double(), loss_grad=0.5)
    ids, probs, counts, losses = router.forward(l)
    assert torch.equal(ids, ref["ids"]) and torch.equal(counts, ref["counts"])
    lf = l.double().masked_fill(l == -math.inf, math.nan)
    spread = (lf.nan_to_num(-100).amax(-1) - lf.nan_to_num(100).amin(-1)).abs().max()
    r = (E / 32 + 64 + float(spread)) * U
    assert ((probs.double() - ref["probs"]).abs() <= 3 * r * ref["probs"]).all()
    lse_mag = ref["lse"].abs() + 1
    assert (losses[0].double() - ref["losses"][0]).abs() <= (3 * r + (T + E) * U) * ref["losses"][0].abs() + 1e-30
    assert (losses[1].double() - ref["losses"][1]).abs() <= (3 * r + (T + E) * U) * c64["z"] * (lse_mag ** 2).mean()
    dl = router.backward(l, ids, d, counts=counts, loss_grad=0.5)
    assert dl.dtype == xt and dl.shape == l.shape
    tol = 4 * r * ref["mag"] + (2.0 ** -8 * ref["dlogits"].abs() if xt == BF16 else 0) + 1e-37
    err = (dl.double() - ref["dlogits"]).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert not dl[l == -math.inf].any()
    again = router.forward(l)
    assert all(torch.equal(a, b) for a, b in zip((ids, probs, counts, losses), again))
    assert torch.equal(dl, router.backward(l, ids, d, counts=counts, loss_grad=0.5))


@gpu
def test_ties_go_to_the_lower_id():
    E, k = 70, 9
    l = torch.zeros(4, E, device="cuda")
    l[1, 40:] = 1.0
    l[2, ::3] = -0.0                                   # equal to 0
    l[3] = torch.arange(E, device="cuda") // 10 * 0.25
    ids, *_ = M.MoERouter(E, k).forward(l)
    assert ids[0].tolist() == list(range(k)) and ids[1].tolist() == list(range(40, 40 + k))
    assert ids[2].tolist() == list(range(k)) and ids[3].tolist() == list(range(60, 60 + k))


@gpu
@pytest.mark.parametrize("score", list(SCORES))
def test_rows_without_open_experts(score):
    """No open expert: ids -1, probs 0, no gradient, nothing in the losses; one open expert: it alone."""
    E, k = 20, 4
    l = torch.full((3, E), -math.inf, device="cuda")
    l[1, 13] = -3.0
    l[2] = torch.finfo(F32).min                        # the type's lowest value is a logit like any other
    router = M.MoERouter(E, k, score=SCORES[score], normalise=True, aux_coeff=0.1, z_coeff=0.1)
    ids, probs, counts, losses = router.forward(l[:2].contiguous())
    assert ids.tolist() == [[-1] * 4, [13, -1, -1, -1]] and probs[0].tolist() == [0] * 4
    assert probs[1].tolist() == [1, 0, 0, 0] and int(counts.sum()) == 1 and counts[13] == 1
    assert torch.isfinite(losses).all()
    assert abs(float(losses[0]) - 0.1 * E / (k * 2) / 2) < 1e-6 and abs(float(losses[1]) - 0.1 * 9 / 2) < 1e-6
    d = router.backward(l[:2].contiguous(), ids, torch.ones(2, k, device="cuda"), counts=counts)
    assert torch.isfinite(d).all() and not d[0].any()
    ids, probs, *_ = M.MoERouter(E, k, score=SCORES[score], normalise=True).forward(l[2:])
    assert ids.tolist() == [[0, 1, 2, 3]]
    if score == "softmax":
        assert probs.tolist() == [[0.25] * 4]
    else:                                              # every score underflows: nothing to divide by
        assert not probs.any()


@gpu
@pytest.mark.parametrize("score", list(SCORES))
def test_nan_stays_in_its_row(score):
    l, _ = logits_of(50, 96, F32, 1)
    router = M.MoERouter(96, 6, score=SCORES[score])
    ids, probs, *_ = router.forward(l)
    bad = l.clone()
    bad[7, 30] = math.nan
    best = int(ids[7, 0])
    bad[8, best] = math.nan
    ids2, probs2, counts2, _ = router.forward(bad)
    keep = [t for t in range(50) if t not in (7, 8)]
    assert torch.equal(ids[keep], ids2[keep]) and torch.equal(probs[keep], probs2[keep])
    assert probs2[7].isnan().all() and probs2[8].isnan().all()
    assert 30 not in ids2[7].tolist() and best not in ids2[8].tolist() and int(counts2.sum()) == 300


@gpu
@pytest.mark.parametrize("score", list(SCORES))
def test_select_bias_moves_the_choice_and_not_the_probs(score):
    """Scores kept apart by more than their rounding: the order of score + bias, probs of the scores alone."""
    T, E, k = 60, 48, 5
    g = torch.Generator(device="cuda").manual_seed(4)
    l = torch.stack([torch.randperm(E, generator=g, device="cuda") for _ in range(T)]).float() * 0.1
    l[5, :40] = -math.inf
    bias = torch.linspace(-0.05, 0.04, E, device="cuda")
    c = dict(E=E, k=k, score=score, normalise=True, scale=1.0, aux=0.0, z=0.0)
    ref = reference(l.double(), c, bias=bias.double())
    router = M.MoERouter(E, k, score=SCORES[score])
    ids, probs, counts, losses = router.forward(l, select_bias=bias)
    assert losses is None
    key = torch.where(l > -math.inf, (torch.softmax(l.double(), -1) if score == "softmax" else torch.sigmoid(l.double())) + bias.double(), -1.0)
    gaps = key.sort(-1, descending=True).values[:, :k + 1]
    gaps = (gaps[:, :-1] - gaps[:, 1:]).amin(-1)
    sure = gaps > 16 * U
    assert int(sure.sum()) > 50
    assert torch.equal(ids[sure], ref["ids"][sure])
    assert ((probs.double() - ref["probs"]).abs()[sure] <= 400 * U * ref["probs"][sure]).all()


@gpu
def test_empty_batch_stream_graph_and_aliasing():
    E, k = 128, 8
    router = M.MoERouter(E, k, aux_coeff=0.01, z_coeff=0.01)
    l, d = logits_of(2000, E, F32, 11)
    d = d[:, :k].contiguous()
    ids, probs, counts, losses = router.forward(l[:0])
    assert ids.shape == (0, k) and not counts.any() and not losses.any()
    assert router.backward(l[:0], ids, d[:0]).shape == (0, E)
    ids, probs, counts, losses = router.forward(l)
    dl = router.backward(l, ids, d, counts=counts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = router.forward(l, stream=side)
    dl2 = router.backward(l, other[0], d, counts=other[2], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((ids, probs, counts, losses, dl), (*other, dl2)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = router.forward(l)
        got_d = router.backward(l, got[0], d, counts=got[2])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((ids, probs, counts, losses, dl), (*got, got_d)))
    own = l.clone()
    M.moe_router_backward(router._cfgs[F32], own, ids, d, own, counts)
    assert torch.equal(own, dl)


def test_refusals():
    c = lambda **kw: M.moe_router_config(**{**dict(num_experts=16, topk=4, score=0, normalise=1, scale=1.0, aux_coeff=0.1,  # noqa: E731
                                                   z_coeff=0.0, x_type=1), **kw})
    L = M.load()
    import ctypes
    n = ctypes.c_size_t()
    size = lambda cfg, T=4: L.moe_router_size(cfg, T, ctypes.byref(n))  # noqa: E731
    assert size(c()) == 0 and n.value > 0
    for kw, want in ((dict(num_experts=0), 1), (dict(num_experts=1025), 2), (dict(topk=0), 1), (dict(topk=17), 1),
                     (dict(num_experts=64, topk=33), 2), (dict(score=2), 1), (dict(normalise=2), 1), (dict(scale=math.inf), 1),
                     (dict(aux_coeff=math.nan), 1), (dict(z_coeff=math.inf), 1), (dict(x_type=3), 1)):
        assert size(c(**kw)) == want, kw
    assert size(c(), T=-1) == 1
    f = lambda T=2, l=256, ld=16, bias=None, ids=256, probs=256, counts=256, losses=256, ws=256, nb=1 << 20: L.moe_router_forward(  # noqa: E731
        c(), T, l, ld, bias, ids, probs, counts, losses, ws, nb, None)
    for kw in (dict(l=None), dict(ld=15), dict(ids=None), dict(probs=None), dict(counts=None), dict(ws=None), dict(ws=128),
               dict(nb=8), dict(l=258), dict(bias=2), dict(T=-1)):
        assert f(**kw) == 1, kw
    b = lambda T=2, l=256, ld=16, ids=256, dp=256, counts=256, g=1.0, dl=256, dld=16: L.moe_router_backward(  # noqa: E731
        c(), T, l, ld, ids, dp, counts, g, dl, dld, None)
    assert b(T=0) == 0
    for kw in (dict(l=None), dict(ids=None), dict(dp=None), dict(dl=None), dict(counts=None), dict(g=math.nan), dict(ld=3),
               dict(dld=15), dict(dl=257)):
        assert b(**kw) == 1, kw


def test_tensors_elsewhere_are_refused():
    """Tensors in host memory come back as errors before anything is launched."""
    router = M.MoERouter(8, 2)
    l, ids, d = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="device"):
        router.forward(l)
    with pytest.raises(ValueError, match="device"):
        router.backward(l, ids, d)
    with pytest.raises(ValueError, match="device"):
        M.moe_router_forward(router._cfgs[F32], l, ids, d)
    with pytest.raises(ValueError, match="device"):
        M.moe_router_backward(router._cfgs[F32], l, ids, d, l)


@gpu
def test_tensors_on_two_devices_are_refused():
    router = M.MoERouter(8, 2, aux_coeff=0.1)
    l, ids, d, n, b = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.zeros(8, dtype=torch.int32), torch.zeros(8)
    L, I, D, N = (t.cuda() for t in (l, ids, d, n))
    before = M.moe_launch_count()
    for args in ((l, b.cuda()), (L, b)):
        with pytest.raises(ValueError, match="device"):
            router.forward(*args)
    for args in ((l, I, D, N), (L, ids, D, N), (L, I, d, N), (L, I, D, n)):
        with pytest.raises(ValueError, match="device"):
            router.backward(*args)
    cfg = router._cfgs[F32]
    for args in ((L, ids, D), (L, I, d), (L, I, D, n), (L, I, D, N, d)):
        with pytest.raises(ValueError, match="device"):
            M.moe_router_forward(cfg, *args)
    assert M.moe_launch_count() == before


def by_definition(l, router, c, bias=None, seed=0):
    """A router's forward and backward against the definition, with the tolerances above and 2^-146 for results
    below the normal range. Returns (ids, probs)."""
    d = torch.randn(l.shape[0], c["k"], generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
    ref = reference(l.double(), c, bias=None if bias is None else bias.double(), dprobs=d.double(), loss_grad=1.0)
    ids, probs, counts, losses = router.forward(l, select_bias=bias)
    assert torch.equal(ids, ref["ids"]) and torch.equal(counts, ref["counts"])
    lf = l.double().masked_fill(l == -math.inf, math.nan)
    spread = float((lf.nan_to_num(-1e4).amax(-1) - lf.nan_to_num(1e4).amin(-1)).max())
    r, tiny = (c["E"] / 32 + 64 + spread) * U, 2.0 ** -146
    assert ((probs.double() - ref["probs"]).abs() <= 3 * r * ref["probs"] + tiny).all(), (probs, ref["probs"])
    dl = router.backward(l, ids, d, counts=counts)
    tol = 4 * r * ref["mag"] + (2.0 ** -8 * ref["dlogits"].abs() if l.dtype == BF16 else 0) + tiny
    assert ((dl.double() - ref["dlogits"]).abs() <= tol).all()
    if c["aux"] or c["z"]:
        T, z = l.shape[0], c["z"] * ((ref["lse"].abs() + 1) ** 2).mean()
        assert (losses[0].double() - ref["losses"][0]).abs() <= (3 * r + (T + c["E"]) * U) * ref["losses"][0].abs() + 1e-30
        assert (losses[1].double() - ref["losses"][1]).abs() <= (3 * r + (T + c["E"]) * U) * z
    return ids, probs


@gpu
@pytest.mark.parametrize("low", [-80.0, -88.5, -92.0, -100.0, -250.0])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_normalised_probs_of_scores_far_below_the_largest(k, low):
    """A bias that chooses experts whose softmax scores are tiny beside the row's largest: their share of each other is
    what counts, in the probs and in the gradient."""
    l = torch.tensor([[0.0, low, low - 1.5, 3.0, low - 0.25, -2.0], [low, 0.5, low + 1, 0.0, low - 4, low]], device="cuda")
    bias = torch.tensor([[-10.0, 5.0, 6.0, -10.0, 7.0, -10.0]], device="cuda")[0].contiguous()
    c = dict(E=6, k=k, score="softmax", normalise=True, scale=1.5, aux=0.0, z=0.0)
    router = M.MoERouter(6, k, normalise=True, scale=1.5)
    ids, probs = by_definition(l[:1].contiguous(), router, c, bias)
    assert ids[0].tolist() == [4, 2, 1][:k] and abs(float(probs.sum()) - 1.5) < 1e-5


@gpu
@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("low", [-60.0, -86.9, -87.5, -95.0, -120.0, -600.0])
def test_sigmoid_scores_of_low_logits(low, normalise):
    """Sigmoid scores down to fp32's smallest and below: close to the definition, and normalised by each other."""
    l = torch.tensor([[low, low - 1.0, low - 0.5, low - 3.0], [low, 2.0, low, -math.inf], [low, low, -math.inf, low - 2.0]], device="cuda")
    c = dict(E=4, k=2, score="sigmoid", normalise=normalise, scale=1.0, aux=0.0, z=0.0)
    by_definition(l, M.MoERouter(4, 2, score=SCORES["sigmoid"], normalise=normalise), c)


@gpu
@pytest.mark.parametrize("normalise", [False, True])
def test_sigmoid_gradients_of_high_logits(normalise):
    """1 - score where the score is 1 in fp32: gradients relative to their own size, not to the scores'. The last two of
    the three chosen take opposite parts of a normalised prob, so that no sum cancels: (d_i - mean) is -1, 1 and 0."""
    l = torch.tensor([[h, h, h, -math.inf] for h in (5.0, 12.0, 17.0, 30.0, 60.0, 85.0)], device="cuda")
    d = torch.tensor([[-1.0, 1.0, 0.0]] * 6, device="cuda")
    c = dict(E=4, k=3, score="sigmoid", normalise=normalise, scale=1.0, aux=0.0, z=0.0)
    ref = reference(l.double(), c, dprobs=d.double())
    router = M.MoERouter(4, 3, score=SCORES["sigmoid"], normalise=normalise)
    ids, _, counts, _ = router.forward(l)
    assert torch.equal(ids, ref["ids"])
    dl = router.backward(l, ids, d, counts=counts)
    want = torch.exp(-l[:, :1].double()) / (1 + torch.exp(-l[:, :1].double())) ** 2 * torch.tensor([-1.0, 1.0, 0.0], device="cuda").double()
    if normalise:  # share 1/3, times 1 - score alone
        want = torch.exp(-l[:, :1].double()) / (1 + torch.exp(-l[:, :1].double())) / 3 * torch.tensor([-1.0, 1.0, 0.0], device="cuda").double()
    r = (4 / 32 + 64) * U
    assert ((dl[:, :3].double() - want).abs() <= 4 * r * want.abs() + 4 * r * want.abs().amax(1, keepdim=True)).all()
    assert not dl[:, 3].any()


@gpu
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("E", [24, 200])
def test_nan_and_infinite_logits_keep_their_rows_ids_with_a_bias(score, normalise, E):
    """A NaN logit is never chosen, the row's other experts are, with NaN probs, so that the NaN reaches the token's
    result; so it is with +inf and softmax scores. Such a softmax row has no scores for the bias to move."""
    k = 4
    g = torch.Generator(device="cuda").manual_seed(8)
    l = torch.stack([torch.randperm(E, generator=g, device="cuda") for _ in range(6)]).float() * 0.05
    bias = torch.zeros(E, device="cuda")
    bias[11] = 4.0
    l[1, 5], l[2, 11], l[3, 7] = math.nan, math.nan, math.inf
    l[4, 6], l[4, 3] = math.inf, math.nan
    router = M.MoERouter(E, k, score=SCORES[score], normalise=normalise)
    ids, probs, counts, _ = router.forward(l, select_bias=bias)
    assert (ids >= 0).all() and int(counts.sum()) == 6 * k and all(len(set(r)) == k for r in ids.tolist())
    assert 5 not in ids[1].tolist() and 11 not in ids[2].tolist() and 3 not in ids[4].tolist()
    top = l.nan_to_num(nan=-math.inf, posinf=1e3).argsort(dim=-1, descending=True, stable=True)
    for t in range(6):
        rest = [e for e in top[t].tolist() if e != 11]
        want = [11] + rest[:k - 1] if t != 2 else rest[:k]
        if score == "softmax" and 1 <= t <= 4:     # no scores: by the logits alone
            want = top[t].tolist()[:k]
        assert ids[t].tolist() == want, t
    assert probs[1].isnan().all() and probs[2].isnan().all() and probs[4].isnan().all()
    assert not probs[[0, 5]].isnan().any()
    if score == "softmax":
        assert probs[3].isnan().all()
    else:
        assert float(probs[3, ids[3].tolist().index(7)]) == (1.0 if not normalise else float(probs[3].max()))
    # without a bias the same rows, by their logits
    ids, probs, counts, _ = router.forward(l)
    assert (ids >= 0).all() and ids[3, 0] == 7 and ids[4, 0] == 6 and probs[4].isnan().all()


@gpu
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T,E,k,xt", [(16384, 128, 8, F32), (7297, 70, 6, BF16), (8001, 384, 6, F32), (5003, 200, 4, BF16),
                                      (3700, 500, 8, F32), (4001, 1000, 9, BF16)])
def test_more_rows_than_the_grid_has_warps(T, E, k, xt, score):
    """A warp takes several rows, the last round uneven, some experts closed and some rows empty, with losses: forward
    and backward against the definition. Without counts the C entry gives the same choice."""
    l, _ = logits_of(T, E, xt, T + E, closed=0.2, pad=3)
    l[5], l[T - 1] = -math.inf, -math.inf
    c = dict(E=E, k=k, score=score, normalise=True, scale=2.5, aux=float(torch.tensor(0.02, dtype=F32)), z=float(torch.tensor(0.003, dtype=F32)))
    router = M.MoERouter(E, k, score=SCORES[score], scale=2.5, aux_coeff=0.02, z_coeff=0.003)
    ids, probs = by_definition(l, router, c)
    ids2, probs2 = torch.empty_like(ids), torch.empty_like(probs)
    M.moe_router_forward(router._cfgs[xt], l, ids2, probs2)
    assert torch.equal(ids, ids2) and torch.equal(probs, probs2)
    plain = M.MoERouter(E, k, score=SCORES[score], scale=2.5).forward(l)
    assert torch.equal(ids, plain[0]) and torch.equal(probs, plain[1]) and plain[3] is None
    assert torch.equal(plain[2], router.forward(l)[2])


@gpu
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T,E,k,xt", [(300, 48, 5, F32), (200, 96, 6, BF16), (120, 256, 8, F32), (5000, 384, 6, BF16)])
def test_select_bias_with_losses(T, E, k, xt, score):
    """The bias moves the choice (and so the counts), not the scores, their distribution, the losses or the gradients.
    Sums of score and bias are kept apart: scores of any size, the bias of an expert 1 more than that of the one before."""
    l, _ = logits_of(T, E, xt, 3 * T + E, closed=0.1)
    order = torch.randperm(E, generator=torch.Generator(device="cuda").manual_seed(E), device="cuda")
    bias = order.float() * 1.0 - E / 2
    l = l.clamp(max=1.0)
    l[:, ::7] -= 3.0
    c = dict(E=E, k=k, score=score, normalise=True, scale=1.5, aux=float(torch.tensor(0.02, dtype=F32)), z=float(torch.tensor(0.003, dtype=F32)))
    router = M.MoERouter(E, k, score=SCORES[score], scale=1.5, aux_coeff=0.02, z_coeff=0.003)
    ids, _ = by_definition(l, router, c, bias)
    assert not torch.equal(ids, router.forward(l)[0])
