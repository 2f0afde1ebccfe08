"""The operators of a transformer's mixture-of-experts block around the expert layer, as workloads.

Three operators, each with its plain form (elementary torch operations in fp32)
and the library's own calls:

* ``decode``: the expert layer for a few tokens (serving), ``MoEDecoder.forward_topk``
* ``norm``: the norm in front of the layer, forward and backward with the
  reduction of the weight's gradient, ``MoENorm.forward`` / ``.backward``
* ``router``: the choice of experts from the router's logits with the balancing
  losses, forward and backward, ``MoERouter.forward`` / ``.backward``

``own`` selects the side that ``run`` takes.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "fp32"
EPS = 1e-5
SKIP = 3072          # no case has this size


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dtype(name):
    return torch.bfloat16 if name == BF16 else torch.float32


# ------------------------------------------------------------------ cases
def _decode(name, T, H, I, E, k, wtype=BF16, shared=True, gate=False, limit=0.0, missing=0.0):
    return dict(name=name, op="decode", T=T, H=H, I=I, E=E, k=k, wtype=wtype, shared=shared, gate=gate, limit=limit,
                missing=missing)


def _norm(name, direction, T, H, x=BF16, y=BF16, w=BF16, kind="layer", bias=True, residual=False, pad=0):
    return dict(name=name, op="norm", direction=direction, T=T, H=H, x=x, y=y, w=w, kind=kind, bias=bias,
                residual=residual, pad=pad)


def _router(name, direction, T, E, k, x=F32, score="softmax", normalise=True, scale=1.0, losses=True, masked=0.0):
    return dict(name=name, op="router", direction=direction, T=T, E=E, k=k, x=x, score=score, normalise=normalise,
                scale=scale, losses=losses, masked=masked)


def listed():
    return [
        # one sequence being answered: the weights of k + 1 experts, once
        _decode("decode-1", 1, 2048, 1024, 96, 6),
        # a small decode batch; a few of the experts are shared by two tokens
        _decode("decode-8", 8, 2048, 1024, 96, 6),
        # a full decode batch: nearly every expert has tokens, some routes dropped
        _decode("decode-64", 64, 2048, 1024, 96, 6, missing=0.05),
        # a large model's layer in MXFP8, a handful of sequences
        _decode("decode-mxfp8-4", 4, 7168, 2048, 128, 6, wtype="mxfp8"),
        # sizes that no tile divides, clamp and output gate
        _decode("decode-odd-5", 5, 1160, 424, 10, 3, gate=True, limit=2.0, missing=0.1),
        # the norm of one decoded token
        _norm("norm-fwd-1", "forward", 1, 2048),
        # the norm of a training batch, with the residual add before it
        _norm("norm-fwd-16384", "forward", 16384, 4096, residual=True),
        # an odd width in fp32, rows of a wider buffer
        _norm("norm-bwd-odd", "backward", 777, 2051, x=F32, y=F32, w=F32, pad=5),
        # the backward pass of a training batch, the residual's gradient joined
        _norm("norm-bwd-16384", "backward", 16384, 4096, w=F32, residual=True),
        # choosing the experts of one decoded token
        _router("router-fwd-1", "forward", 1, 96, 6, losses=False),
        # a training batch's routing with the balancing losses
        _router("router-fwd-16384", "forward", 16384, 128, 8),
        # the routing's backward pass for a large expert count, sigmoid scores
        _router("router-bwd-8192", "backward", 8192, 384, 6, score="sigmoid", scale=2.5),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v != SKIP and 2 * v != SKIP:
            return v


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0), work(c)["bytes"])
    while True:
        op = rng.choice(["decode", "norm", "router"])
        if op == "decode":
            mx = rng.random() < 0.4
            step = 32 if mx else 8
            E = _spread(rng, 4, 128)
            c = _decode("", _spread(rng, 1, 64), _spread(rng, 256, 7168, step), _spread(rng, 128, 2048, step), E,
                        rng.randint(1, min(8, E)), "mxfp8" if mx else BF16, rng.random() < 0.8, False,
                        rng.choice([0.0, 0.0, 2.0]), rng.choice([0.0, 0.05, 0.3]))
            c["gate"] = c["shared"] and rng.random() < 0.3
            # the plain form gathers the routes' weights, or computes every token with every expert
            gathered = min(c["T"] * c["k"], E + c["T"]) * 3 * c["H"] * c["I"] * 6
            if gathered > 24e9 or E * 3 * c["H"] * c["I"] * 2 > 8e9:
                continue
        elif op == "norm":
            x, y = rng.choice([(BF16, BF16), (BF16, BF16), (F32, BF16), (F32, F32)])
            kind = rng.choice(["layer", "rms"])
            c = _norm("", rng.choice(["forward", "backward"]), _spread(rng, 1, 32768), _spread(rng, 64, 12288), x, y,
                      rng.choice([BF16, F32]), kind, kind == "layer" and rng.random() < 0.7, rng.random() < 0.5,
                      rng.choice([0, 0, 3, 8]))
        else:
            E = _spread(rng, 2, 512)
            k = rng.randint(1, min(8, E))
            # one normalised prob is always 1: nothing to learn from it, so nobody asks for it
            c = _router("", rng.choice(["forward", "backward"]), _spread(rng, 1, 16384), E, k,
                        rng.choice([BF16, F32]), rng.choice(["softmax", "sigmoid"]), k > 1 and rng.random() < 0.7,
                        rng.choice([1.0, 2.5]), rng.random() < 0.7, rng.choice([0.0, 0.0, 0.1]))
        if work(c)["bytes"] <= top[op]:
            del c["name"]
            return c


# ------------------------------------------------------------------ what a program has in hand
def _generator(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dev, scale=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale


def _quantise(w):
    """MXFP8 of fp32 [.., K]: E4M3 payload and E8M0 scale codes per 32 elements along K (as bytes)."""
    b = w.reshape(*w.shape[:-1], w.shape[-1] // 32, 32)
    amax = b.abs().amax(-1, keepdim=True)
    code = torch.where(amax > 0, (torch.floor(torch.log2(amax.clamp(min=1e-38))) - 8 + 127).clamp(0, 254),
                       torch.zeros_like(amax))
    q = (b * torch.exp2(127 - code)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(w.shape), code.to(torch.uint8).squeeze(-1)


def _weight(g, shape, dev, mx):
    """bf16 [E, N, K], or the MXFP8 payload and scales of it, made expert by expert."""
    if not mx:
        out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        for e in range(shape[0]):
            out[e] = _randn(g, shape[1:], dev, 0.02)
        return out
    q = torch.empty(shape, dtype=torch.uint8, device=dev)
    s = torch.empty((*shape[:-1], shape[-1] // 32), dtype=torch.uint8, device=dev)
    for e in range(shape[0]):
        q[e], s[e] = _quantise(_randn(g, shape[1:], dev, 0.02))
    return q, s


def _routing(g, T, E, k, missing, dev):
    """The router's output for T tokens: distinct experts per token, probs that sum to 1, some routes dropped."""
    logits = _randn(g, (T, E), dev, 1.5)
    top, ids = logits.topk(k, -1)
    probs = torch.softmax(top, -1)
    gone = torch.rand((T, k), generator=g, device=dev) < missing
    return ids.masked_fill(gone, -1).to(torch.int32), probs.masked_fill(gone, 0.0)


def _prepare_decode(c, g, dev):
    T, H, I, E, k = (c[n] for n in "THIEk")
    mx = c["wtype"] == "mxfp8"
    s = dict(case=c, hidden=_randn(g, (T, H), dev).bfloat16())
    s["ids"], s["probs"] = _routing(g, T, E, k, c["missing"], dev)
    s["fc1"] = _weight(g, (E, 2 * I, H), dev, mx)
    s["fc2"] = _weight(g, (E, H, I), dev, mx)
    if c["shared"]:
        s["shared_fc1"] = _randn(g, (2 * I, H), dev, 0.02).bfloat16()
        s["shared_fc2"] = _randn(g, (H, I), dev, 0.02).bfloat16()
    if c["gate"]:
        s["gate"] = _randn(g, (H,), dev, 0.02).bfloat16()
    if own:
        import mixture_experts_layer_pack_gb300 as M
        shared = (s.get("shared_fc1"), s.get("shared_fc2"))
        if mx:
            (q1, s1), (q2, s2) = s["fc1"], s["fc2"]
            s["weights"] = M.weights_from_combined_mxfp8(*shared, q1, s1, q2, s2, s.get("gate"))
        else:
            s["weights"] = M.weights_from_combined(*shared, s["fc1"], s["fc2"], s.get("gate"))
        s["layer"] = M.MoEDecoder(T, H, E, k, I, device=dev,
                                  routed_wtype=M.binding.MOE_W_MXFP8 if mx else M.binding.MOE_W_BF16,
                                  swiglu_limit=c["limit"], shared_expert=c["shared"])
    return s


def _rows(t, pad):
    """t as rows of a buffer that is `pad` elements wider."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _prepare_norm(c, g, dev):
    T, H, pad = c["T"], c["H"], c["pad"]
    xt, yt, wt = _dtype(c["x"]), _dtype(c["y"]), _dtype(c["w"])
    s = dict(case=c, x=_rows((_randn(g, (T, H), dev) + 0.25).to(xt), pad))
    s["weight"] = (1.0 + _randn(g, (H,), dev, 0.1)).to(wt)
    s["bias"] = _randn(g, (H,), dev, 0.1).to(wt) if c["bias"] else None
    if c["direction"] == "forward":
        s["residual"] = _rows(_randn(g, (T, H), dev).to(xt), pad) if c["residual"] else None
    else:
        s["dy"] = _rows(_randn(g, (T, H), dev).to(yt), pad)
        s["dsum"] = _rows(_randn(g, (T, H), dev).to(xt), pad) if c["residual"] else None
        xf = s["x"].float()       # the statistics that the forward pass saved
        mean = xf.mean(-1) if c["kind"] == "layer" else torch.zeros(T, device=dev)
        s["mean"] = mean if c["kind"] == "layer" else None
        s["rstd"] = torch.rsqrt((xf - mean[:, None]).square().mean(-1) + EPS)
    if own:
        import mixture_experts_layer_pack_gb300 as M
        s["norm"] = M.MoENorm(H, eps=EPS, kind=M.binding.MOE_NORM_LAYER if c["kind"] == "layer" else M.binding.MOE_NORM_RMS,
                              device=dev)
    return s


AUX, ZCOEFF = 0.01, 0.001


def _prepare_router(c, g, dev):
    T, E, k = c["T"], c["E"], c["k"]
    logits = _randn(g, (T, E), dev, 1.5)
    if c["masked"]:               # experts that are closed to a token
        logits = logits.masked_fill(torch.rand((T, E), generator=g, device=dev) < c["masked"], -math.inf)
    s = dict(case=c, logits=logits.to(_dtype(c["x"])))
    if c["direction"] == "backward":
        s["fwd"] = _plain_router_forward(s)
        s["dprobs"] = _randn(g, (T, k), dev)
    if own:
        import mixture_experts_layer_pack_gb300 as M
        score = M.binding.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else M.binding.MOE_SCORE_SIGMOID
        s["router"] = M.MoERouter(E, k, score=score, normalise=c["normalise"], scale=c["scale"],
                                  aux_coeff=AUX if c["losses"] else 0.0, z_coeff=ZCOEFF if c["losses"] else 0.0,
                                  device=dev)
    return s


def prepare(case, seed):
    dev = _device()
    g = _generator(seed, dev)
    return {"decode": _prepare_decode, "norm": _prepare_norm, "router": _prepare_router}[case["op"]](case, g, dev)


# ------------------------------------------------------------------ plain forms
def _plain_weight(w, at=None):
    """fp32 values of a weight (its experts `at`, if given)."""
    if isinstance(w, tuple):
        q, s = (w[0], w[1]) if at is None else (w[0][at], w[1][at])
        v = q.view(torch.float8_e4m3fn).float().reshape(*s.shape, 32)
        return (v * torch.exp2(s.float() - 127)[..., None]).reshape(q.shape)
    return (w if at is None else w[at]).float()


def _swiglu(g, u, limit):
    if limit > 0:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1 + torch.exp(-g)) * u


def _plain_decode(s):
    c = s["case"]
    I, E, T, k = c["I"], c["E"], c["T"], c["k"]
    x = s["hidden"].float()
    ids, probs = s["ids"].long(), s["probs"]
    weight = torch.where(ids >= 0, probs, torch.zeros_like(probs))
    if T * k < E:                 # the routes' weights
        at = ids.clamp(min=0).reshape(-1)
        xr = x.repeat_interleave(k, 0)
        h = torch.matmul(_plain_weight(s["fc1"], at), xr[..., None])[..., 0]
        a = _swiglu(h[:, :I], h[:, I:], c["limit"])
        y = torch.matmul(_plain_weight(s["fc2"], at), a[..., None])[..., 0]
        out = (weight[..., None] * y.reshape(T, k, -1)).sum(1)
    else:                         # every token with every expert, the others weighted 0
        h = torch.matmul(x, _plain_weight(s["fc1"]).transpose(1, 2))
        a = _swiglu(h[..., :I], h[..., I:], c["limit"])
        y = torch.matmul(a, _plain_weight(s["fc2"]).transpose(1, 2))
        at = torch.arange(E, device=x.device)
        dense = (weight[..., None] * (ids[..., None] == at)).sum(1)
        out = (dense.t()[..., None] * y).sum(0)
    if c["shared"]:
        h = x @ s["shared_fc1"].float().t()
        y = _swiglu(h[:, :I], h[:, I:], c["limit"]) @ s["shared_fc2"].float().t()
        if c["gate"]:
            y = y / (1 + torch.exp(-(x @ s["gate"].float())))[:, None]
        out = out + y
    return out.bfloat16()


def _plain_norm_forward(s):
    c = s["case"]
    x = s["x"].float()
    total = None
    if s["residual"] is not None:
        total = (x + s["residual"].float()).to(s["x"].dtype)
        x = total.float()
    mean = x.mean(-1) if c["kind"] == "layer" else None
    d = x - mean[:, None] if mean is not None else x
    rstd = torch.rsqrt(d.square().mean(-1) + EPS)
    y = d * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return dict(y=y.to(_dtype(c["y"])), total=total, mean=mean, rstd=rstd)


def _plain_norm_backward(s):
    c = s["case"]
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (x - s["mean"][:, None]) * rstd if c["kind"] == "layer" else x * rstd
    wdy = dy * s["weight"].float()
    dx = wdy - xhat * (wdy * xhat).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - wdy.mean(-1, keepdim=True)
    dx = dx * rstd
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.to(s["x"].dtype), dweight=(dy * xhat).sum(0),
                dbias=dy.sum(0) if s["bias"] is not None else None)


def _scores(l, c):
    """Scores of fp32 logits, and their distribution over the experts (zero rows where no expert is open)."""
    if c["score"] == "softmax":
        top = l.amax(-1, keepdim=True)
        p = torch.exp(l - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total > 0, total, torch.ones_like(total))
        return p, p
    sc = 1 / (1 + torch.exp(-l))
    total = sc.sum(-1, keepdim=True)
    return sc, sc / torch.where(total > 0, total, torch.ones_like(total))


def _lse(l):
    top = l.amax(-1)
    base = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    return torch.where(torch.isinf(top), torch.zeros_like(top), torch.log(torch.exp(l - base[:, None]).sum(-1)) + base)


def _plain_router_forward(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].float()
    best, ids = torch.sort(l, dim=-1, descending=True, stable=True)     # a score grows with its logit; ties to the lowest id
    open_ = best[:, :k] > -math.inf
    ids = ids[:, :k]
    sc, p = _scores(l, c)
    chosen = torch.where(open_, sc.gather(1, ids), torch.zeros_like(best[:, :k]))
    if c["normalise"]:
        total = chosen.sum(-1, keepdim=True)
        chosen = chosen / torch.where(total > 0, total, torch.ones_like(total))
    ids = torch.where(open_, ids, torch.full_like(ids, -1)).to(torch.int32)
    out = dict(ids=ids, probs=chosen * c["scale"])
    at = torch.arange(E, device=l.device, dtype=torch.int32)
    out["counts"] = (ids[..., None] == at).sum((0, 1)).to(torch.int32)
    if c["losses"]:
        balance = AUX * E / (k * T * T) * (out["counts"].float() * p.sum(0)).sum()
        out["losses"] = torch.stack([balance, ZCOEFF / T * _lse(l).square().sum()])
    return out


def _plain_router_backward(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].float()
    fwd = s["fwd"]
    sc, p = _scores(l, c)
    ids = fwd["ids"].long()
    at = ids.clamp(min=0)
    chosen = torch.where(ids >= 0, sc.gather(1, at), torch.zeros_like(fwd["probs"]))
    d = torch.where(ids >= 0, s["dprobs"] * c["scale"], torch.zeros_like(chosen))
    if c["normalise"]:
        total = chosen.sum(-1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        d = (d - (d * chosen / total).sum(-1, keepdim=True)) / total
    dsc = torch.zeros_like(l).scatter_add(1, at, d)
    dp = torch.zeros_like(l)
    if c["losses"]:
        dp = (AUX * E / (k * T * T) * fwd["counts"].float()).expand(T, E)
    if c["score"] == "softmax":
        v = dsc + dp
        dl = p * (v - (v * p).sum(-1, keepdim=True))
    else:
        total = sc.sum(-1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        dl = (dsc + (dp - (dp * p).sum(-1, keepdim=True)) / total) * sc * (1 - sc)
    if c["losses"]:
        lse = _lse(l)
        dl = dl + (2 * ZCOEFF / T) * lse[:, None] * torch.where(torch.isinf(l), torch.zeros_like(l), torch.exp(l - lse[:, None]))
    return dict(dlogits=dl.to(s["logits"].dtype))


# ------------------------------------------------------------------ one pass
def _own(s):
    c = s["case"]
    if c["op"] == "decode":
        return s["layer"].forward_topk(s["hidden"], s["ids"], s["probs"], s["weights"])
    if c["op"] == "norm":
        if c["direction"] == "forward":
            y, total, mean, rstd = s["norm"].forward(s["x"], s["weight"], s["bias"], residual=s["residual"],
                                                     out_dtype=_dtype(c["y"]))
            return dict(y=y, total=total if s["residual"] is not None else None, mean=mean, rstd=rstd)
        dx, dw, db = s["norm"].backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], dsum=s["dsum"],
                                        bias=s["bias"] is not None)
        return dict(dx=dx, dweight=dw, dbias=db)
    if c["direction"] == "forward":
        ids, probs, counts, losses = s["router"].forward(s["logits"])
        out = dict(ids=ids, probs=probs, counts=counts)
        if c["losses"]:
            out["losses"] = losses
        return out
    f = s["fwd"]
    return dict(dlogits=s["router"].backward(s["logits"], f["ids"], s["dprobs"], counts=f["counts"]))


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "decode":
        return _plain_decode(state)
    if c["op"] == "norm":
        return _plain_norm_forward(state) if c["direction"] == "forward" else _plain_norm_backward(state)
    return _plain_router_forward(state) if c["direction"] == "forward" else _plain_router_backward(state)


# ------------------------------------------------------------------ what a pass cannot do without
def _size(name):
    return 2 if name == BF16 else 4


def work(case):
    c = case
    if c["op"] == "decode":
        T, H, I, E, k = (c[n] for n in "THIEk")
        routes = T * k * (1 - c["missing"])
        active = E * (1 - (1 - k / E * (1 - c["missing"])) ** T)       # experts with a token, as expected
        per = 3 * H * I
        b = active * per * (2 if c["wtype"] == BF16 else 1 + 1 / 32) + (per * 2 if c["shared"] else 0) + 4 * T * H
        return {"bytes": b + 8 * T * k, "flops": 2 * per * (routes + (T if c["shared"] else 0))}
    if c["op"] == "norm":
        n, x, y = c["T"] * c["H"], _size(c["x"]), _size(c["y"])
        res = 1 if c["residual"] else 0
        if c["direction"] == "forward":
            return {"bytes": n * (x + y + 2 * x * res) + 8 * c["T"] + 2 * c["H"] * _size(c["w"]), "flops": 8 * n}
        return {"bytes": n * (x + y + x + x * res) + 8 * c["T"] + c["H"] * (_size(c["w"]) + 8), "flops": 14 * n}
    n = c["T"] * c["E"]
    if c["direction"] == "forward":
        return {"bytes": n * _size(c["x"]) + 8 * c["T"] * c["k"] + 4 * c["E"], "flops": 8 * n}
    return {"bytes": 2 * n * _size(c["x"]) + 8 * c["T"] * c["k"] + 4 * c["E"], "flops": 14 * n}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _exact_weight(w, e):
    if isinstance(w, tuple):
        q, s = w[0][e].view(torch.float8_e4m3fn).double(), w[1][e].double()
        return q * torch.pow(2.0, s - 127).repeat_interleave(32, -1)
    return w[e].double()


def _exact_expert(x, fc1, fc2, limit):
    gate, up = (x @ fc1.t()).chunk(2, -1)
    if limit > 0:
        gate, up = torch.minimum(gate, torch.full_like(gate, limit)), up.clamp(-limit, limit)
    return (gate * torch.sigmoid(gate) * up) @ fc2.t()


def _exact_decode(s):
    c = s["case"]
    x = s["hidden"].double()
    out = torch.zeros_like(x)
    for e in range(c["E"]):
        rows, slots = torch.nonzero(s["ids"] == e, as_tuple=True)
        if rows.numel():
            y = _exact_expert(x[rows], _exact_weight(s["fc1"], e), _exact_weight(s["fc2"], e), c["limit"])
            out.index_add_(0, rows, y * s["probs"][rows, slots].double()[:, None])
    if c["shared"]:
        y = _exact_expert(x, s["shared_fc1"].double(), s["shared_fc2"].double(), c["limit"])
        if c["gate"]:
            y = y * torch.sigmoid(x @ s["gate"].double())[:, None]
        out += y
    return out


def _exact_norm(s):
    c = s["case"]
    x = s["x"].double()
    if c["direction"] == "forward":
        total = None
        if s["residual"] is not None:
            total = x + s["residual"].double()
            x = total.to(s["x"].dtype).double()       # the stored sum is what is normalised
        mean = x.mean(-1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(x[:, :1])
        rstd = 1 / torch.sqrt((x - mean).pow(2).mean(-1, keepdim=True) + EPS)
        y = (x - mean) * rstd * s["weight"].double()
        if s["bias"] is not None:
            y = y + s["bias"].double()
        return dict(y=y, total=total, mean=mean[:, 0] if c["kind"] == "layer" else None, rstd=rstd[:, 0])
    x.requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    b = torch.zeros_like(w).requires_grad_(True)
    mean = x.mean(-1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(x[:, :1])
    y = (x - mean) / torch.sqrt((x - mean).pow(2).mean(-1, keepdim=True) + EPS) * w + b
    dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
    if s["dsum"] is not None:
        dx = dx + s["dsum"].double()
    return dict(dx=dx, dweight=dw, dbias=db if s["bias"] is not None else None)


def _exact_router(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double().requires_grad_(True)
    free = torch.isfinite(l)
    lf = torch.where(free, l, torch.full_like(l, -1e5))      # exp of it is 0 in 64 bits
    some = free.any(-1, keepdim=True)
    order = torch.argsort(l.detach(), dim=-1, descending=True, stable=True)[:, :k]
    ok = free.gather(1, order)
    score = torch.softmax(lf, -1) if c["score"] == "softmax" else torch.sigmoid(lf)
    score = torch.where(free, score, torch.zeros_like(score))
    dist = score / torch.where(some, score.sum(-1, keepdim=True), torch.ones_like(lf[:, :1]))
    picked = score.gather(1, order)
    if c["normalise"]:
        picked = picked / torch.where(some, picked.sum(-1, keepdim=True), torch.ones_like(picked[:, :1]))
    probs = c["scale"] * picked
    counts = torch.bincount(order[ok], minlength=E).double()
    balance = AUX * E * (counts / (k * T) * (dist.sum(0) / T)).sum()
    z = ZCOEFF * torch.where(some[:, 0], torch.logsumexp(lf, -1), torch.zeros_like(lf[:, 0])).pow(2).mean()
    if c["direction"] == "forward":
        out = dict(ids=None, probs=probs.detach(), counts=None)
        if c["losses"]:
            out["losses"] = torch.stack([balance, z]).detach()
        return out
    goal = (probs * s["dprobs"].double()).sum()
    if c["losses"]:
        goal = goal + balance + z
    return dict(dlogits=torch.autograd.grad(goal, l)[0])


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "norm": _exact_norm, "router": _exact_router}[case["op"]](s)
