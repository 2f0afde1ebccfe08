"""The layer for a few tokens (moe_decode) against its definition in fp64, element by element.

Tolerance, derived from the arithmetic: u = 2^-24; a dot product of n terms
accumulated in fp32 in any order by at least 32 partial sums is off by at most
G(n) = (n/32 + 40) u times the sum of its terms' magnitudes. So g and u are off by
G(H) |W||x|; a = silu(g) u by 1.1 |u| err_g + |silu(g)| err_u + 2^-19 |a| (the
activation's exp and quotient), and, as two bf16 terms, 2^-16 |a|; each expert's y by
|W_down| err_a + G(I) |W_down||a|; out adds these up with the probs (and the gate, off by
its own dot product), and rounds to bf16 once: 2^-8 |out| covers it.
Where a clamp bound lies within err_g of g its gradient does not matter: the value is continuous.
"""
import itertools
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_pack_gb300 as M
import moe_inputs as MI
from mixture_experts_layer_pack_gb300 import binding as B
from oracle import moe_oracle as O

gpu = pytest.mark.gpu
U = 2.0 ** -24


def G(n):
    return (n / 32 + 40) * U


def mx_values(q, s):
    v = q.cpu().view(torch.float8_e4m3fn).double().reshape(*s.shape, 32).to(q.device)
    return (v * torch.pow(2.0, s.double() - 127)[..., None]).reshape(q.shape)


def quantise(w):
    b = w.reshape(*w.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    code = torch.where(amax > 0, (torch.floor(torch.log2(amax.clamp(min=1e-38))) - 8 + 127).clamp(0, 254), torch.zeros_like(amax))
    q = (b * torch.exp2(127 - code)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(w.shape), code.to(torch.uint8)[..., 0]


class Layer:
    """Weights, inputs and the fp64 definition of one case."""

    def __init__(self, T, H, I, E, k, mx=False, shared=True, gate=False, limit=0.0, seed=0, missing=0.1, spread=0.02):
        g = torch.Generator(device="cuda").manual_seed(1000 + seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.T, self.H, self.I, self.E, self.k, self.mx, self.limit = T, H, I, E, k, mx, limit
        self.shared = shared
        sc = max(spread, 1 / math.sqrt(H))
        fc1, fc2 = r(E, 2 * I, H) * sc, r(E, H, I) * sc
        if mx:
            (self.q1, self.s1), (self.q2, self.s2) = quantise(fc1), quantise(fc2)
            self.fc1, self.fc2 = mx_values(self.q1, self.s1), mx_values(self.q2, self.s2)
        else:
            self.b1, self.b2 = fc1.bfloat16(), fc2.bfloat16()
            self.fc1, self.fc2 = self.b1.double(), self.b2.double()
        self.sfc1, self.sfc2 = ((r(2 * I, H) * sc).bfloat16(), (r(H, I) * sc).bfloat16()) if shared else (None, None)
        self.gate = (r(H) * sc).bfloat16() if gate else None
        self.x = r(T, H).bfloat16()
        ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(T)]) if T else torch.zeros(0, k, device="cuda")
        gone = torch.rand(T, k, generator=g, device="cuda") < missing
        self.ids = ids.masked_fill(gone, -1).int()
        self.probs = torch.rand(T, k, generator=g, device="cuda")

    def weights(self):
        if self.mx:
            return M.weights_from_combined_mxfp8(self.sfc1, self.sfc2, self.q1, self.s1, self.q2, self.s2, self.gate)
        return M.weights_from_combined(self.sfc1, self.sfc2, self.b1, self.b2, self.gate)

    def decoder(self, max_tokens=None):
        return M.MoEDecoder(max_tokens or max(self.T, 1), self.H, self.E, self.k, self.I,
                            routed_wtype=B.MOE_W_MXFP8 if self.mx else B.MOE_W_BF16, swiglu_limit=self.limit,
                            shared_expert=self.shared)

    def expert(self, x, fc1, fc2):
        """y and the bound on its error."""
        gu, mag = x @ fc1.t(), G(self.H) * (x.abs() @ fc1.abs().t())
        g, u, eg, eu = gu[:, :self.I], gu[:, self.I:], mag[:, :self.I], mag[:, self.I:]
        if self.limit:
            g, u = g.clamp(max=self.limit), u.clamp(-self.limit, self.limit)
        a = g * torch.sigmoid(g) * u
        ea = 1.1 * (u.abs() + eu) * eg + (g * torch.sigmoid(g)).abs() * eu + (2.0 ** -19 + 2.0 ** -16) * a.abs()
        return a @ fc2.t(), ea @ fc2.abs().t() + G(self.I) * (a.abs() @ fc2.abs().t())

    def reference(self, ids=None):
        x = self.x.double()
        out, tol = torch.zeros_like(x), torch.zeros_like(x)
        ids = self.ids if ids is None else ids
        for e in range(self.E):
            t, s = torch.nonzero(ids == e, as_tuple=True)
            if t.numel():
                y, err = self.expert(x[t], self.fc1[e], self.fc2[e])
                p = self.probs[t, s].double()[:, None]
                out.index_add_(0, t, p * y)
                tol.index_add_(0, t, p.abs() * (err + 4 * U * (self.k + 2) * y.abs()))
        if self.shared:
            y, err = self.expert(x, self.sfc1.double(), self.sfc2.double())
            if self.gate is not None:
                w = self.gate.double()
                gate = torch.sigmoid(x @ w)[:, None]
                eg = G(self.H) * (x.abs() @ w.abs())[:, None] * 0.25 + 2.0 ** -19 * gate
                y, err = gate * y, gate * err + eg * y.abs()
            out, tol = out + y, tol + err + 4 * U * (self.k + 2) * y.abs()
        return out, tol


def check(got, ref, tol, what=""):
    tol = tol + 2.0 ** -8 * ref.abs() + 1e-30
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), \
        f"{what}: {int((err > tol).sum())} of {err.numel()} off, worst {float((err / tol).max()):.3g} x the bound"


CASES = [
    # T, H, I, E, k, mx, shared, gate, limit
    (1, 8, 8, 1, 1, False, False, False, 0.0),
    (1, 64, 32, 4, 2, False, True, False, 0.0),
    (1, 2048, 1024, 12, 6, False, True, False, 0.0),
    (2, 24, 40, 3, 2, False, True, True, 0.5),
    (3, 520, 136, 5, 3, False, True, True, 0.0),
    (5, 1160, 424, 10, 3, False, True, True, 2.0),
    (7, 256, 64, 300, 8, False, False, False, 0.0),
    (8, 512, 256, 8, 2, False, True, False, 1.0),
    (9, 512, 264, 4, 4, False, True, False, 0.0),
    (17, 384, 200, 3, 3, False, True, True, 0.0),
    (33, 776, 88, 2, 1, False, False, False, 0.0),
    (64, 256, 128, 6, 2, False, True, True, 0.0),
    (64, 1024, 512, 40, 6, False, True, False, 0.0),
    (40, 128, 72, 64, 32, False, True, False, 0.0),
    (1, 32, 32, 1, 1, True, False, False, 0.0),
    (1, 2048, 1024, 8, 6, True, True, False, 0.0),
    (3, 96, 160, 5, 2, True, True, True, 0.5),
    (6, 1184, 416, 9, 3, True, True, False, 0.0),
    (13, 544, 96, 4, 3, True, False, False, 2.0),
    (64, 512, 224, 12, 4, True, True, True, 0.0),
    (2, 7168, 2048, 3, 2, True, True, False, 0.0),
    (11, 4096, 1408, 5, 3, False, True, False, 0.0),
    # experts with more tokens than a group, and with many; rings of few slots
    (64, 520, 264, 2, 1, False, True, False, 0.0),
    (64, 1024, 512, 4, 2, False, True, True, 0.0),
    (50, 1040, 136, 48, 32, False, True, False, 0.0),
    (64, 512, 136, 300, 32, False, True, False, 0.0),
    (10, 1160, 424, 10, 3, False, True, False, 0.0),
    (64, 1056, 224, 2, 2, True, True, False, 0.0),
    (64, 512, 160, 260, 32, True, True, False, 0.0),
    (12, 2080, 544, 20, 4, True, True, True, 1.0),
]


@gpu
@pytest.mark.parametrize("T,H,I,E,k,mx,shared,gate,limit", CASES)
def test_against_the_definition(T, H, I, E, k, mx, shared, gate, limit):
    c = Layer(T, H, I, E, k, mx, shared, gate, limit, seed=T + H)
    dec = c.decoder()
    out = dec.forward_topk(c.x, c.ids, c.probs, c.weights())
    assert dec.device_status() == B.MOE_OK
    check(out, *c.reference(), what="out")
    # the same call again, and one with other tokens in between: the same bits
    w = c.weights()
    dec.forward_topk(-c.x, c.ids.flip(0).contiguous(), c.probs, w)
    assert torch.equal(dec.forward_topk(c.x, c.ids, c.probs, w), out)


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_agrees_with_the_oracle_and_with_the_training_layer(mx):
    """The oracle of the layer (BF16 weights: its exact mode), and moe_forward_topk on the same weights, whose
    bf16 results differ by roundings (BF16 weights), or by the activations that its MXFP8 GEMMs quantise."""
    T, H, I, E, k = 24, 256, 128, 8, 3
    c = Layer(T, H, I, E, k, mx, seed=77)
    out = c.decoder().forward_topk(c.x, c.ids, c.probs, c.weights())
    layer = M.MoELayer(T, H, E, k, I, routed_wtype=B.MOE_W_MXFP8 if mx else B.MOE_W_BF16)
    w = c.weights()
    if mx:
        views = []
        for src in (c.fc1[:, :I], c.fc1[:, I:], c.fc2):
            views.append(M.mxfp8_weight(src.float().bfloat16()))   # exact: the values have 4 significant bits
        keep = views
        w.routed_gate, w.routed_up, w.routed_down = (M.mxfp8_view(*v) for v in keep)
        layer.prepare_weights(w)
    full = layer.forward_topk(c.x, c.ids, c.probs, w)
    torch.cuda.synchronize()
    scale = float(full.float().abs().max())
    assert float((out.float() - full.float()).abs().max()) <= (6e-2 if mx else 1e-2) * scale
    if not mx:
        f = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
        W = O.DenseWeights.from_combined(f(c.sfc1), f(c.sfc2), f(c.b1), f(c.b2))
        probs, rmap = np.zeros((T, E)), np.zeros((T, E), dtype=bool)
        for t in range(T):
            for s in range(k):
                if c.ids[t, s] >= 0:
                    rmap[t, int(c.ids[t, s])], probs[t, int(c.ids[t, s])] = True, float(c.probs[t, s])
        ref, _ = O.forward(f(c.x), probs, rmap, W, k, precision="exact")
        check(out, torch.from_numpy(ref).cuda(), c.reference()[1], "oracle")


@gpu
def test_inputs_of_the_seeded_workload():
    """The benchmark's seeded inputs at a reduced size, through both of the layer's routing forms."""
    T, H, E, k, I, seed = 16, 256, 12, 4, 128, MI.seed_of(2)
    r = MI.make_routing(T, E, k, seed, "topk", "second")
    w = MI.make_weights(H, I, E, seed, device=torch.device("cuda"))
    hidden, _ = MI.make_activations(T, H, seed, device=torch.device("cuda"))
    wv = M.weights_from_combined(w["shared_fc1"], w["shared_fc2"], w["routed_fc1"], w["routed_fc2"])
    dense = M.MoELayer(T, H, E, k, I).forward(hidden, torch.from_numpy(r.probs).cuda(),
                                              torch.from_numpy(r.routing_map).cuda().view(torch.uint8), wv)
    ids = np.full((T, k), -1, dtype=np.int32)
    pp = np.zeros((T, k), dtype=np.float32)
    for t in range(T):
        on = np.nonzero(r.routing_map[t])[0]
        ids[t, :len(on)], pp[t, :len(on)] = on, r.probs[t, on]
    out = M.MoEDecoder(T, H, E, k, I).forward_topk(hidden, torch.from_numpy(ids).cuda(), torch.from_numpy(pp).cuda(), wv)
    assert float((out.float() - dense.float()).abs().max()) <= 1e-2 * float(dense.float().abs().max())


@gpu
def test_routing_that_leaves_rows_empty_or_crowds_one_expert():
    c = Layer(20, 264, 104, 6, 3, seed=5)
    dec, w = c.decoder(), c.weights()
    for ids in (torch.full_like(c.ids, -1), torch.tensor([[4, -1, -1]], device="cuda").int().repeat(20, 1),
                torch.tensor([[-1, 5, 0]], device="cuda").int().repeat(20, 1)):
        c.ids = ids
        check(dec.forward_topk(c.x, ids, c.probs, w), *c.reference())
    lone = Layer(20, 264, 104, 6, 3, shared=False, seed=6)
    lone.ids[3:] = -1
    out = lone.decoder().forward_topk(lone.x, lone.ids, lone.probs, lone.weights())
    check(out, *lone.reference())
    assert not out[3:].any()


@gpu
def test_bad_ids_are_reported_and_their_rows_keep_the_shared_part():
    c = Layer(12, 128, 64, 5, 3, seed=8, missing=0.0)
    dec, w = c.decoder(), c.weights()
    good = c.ids.clone()
    bad = good.clone()
    bad[2, 1], bad[5, 0], bad[9, 2] = 5, -2, bad[9, 0]          # beyond E, below -1, twice
    out = dec.forward_topk(c.x, bad, c.probs, w)
    assert dec.device_status() == B.MOE_ERR_ROUTING and dec.device_status() == B.MOE_OK
    kept = good.clone()
    kept[[2, 5, 9]] = -1
    check(out, *c.reference(kept))
    assert torch.equal(dec.forward_topk(c.x, kept, c.probs, w), out) and dec.device_status() == B.MOE_OK


@gpu
def test_new_tables_are_refused_under_capture():
    """A table is uploaded when its pointers change: not in a graph, which would keep the upload's source. A known one is captured."""
    c = Layer(3, 256, 64, 4, 2, seed=13)
    dec = c.decoder(8)
    parts = {n: [m[e].contiguous() for e in range(4)] for n, m in (("gate", c.b1[:, :64]), ("up", c.b1[:, 64:]), ("down", c.b2))}
    w = M.set_expert_tables(c.weights(), **parts)
    out = torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(M.MoeError) as e:
            dec.forward_topk(c.x, c.ids, c.probs, w, out=out)
        kept = out + 0  # the capture goes on
    assert e.value.status == 6  # MOE_ERR_STATE
    want = dec.forward_topk(c.x, c.ids, c.probs, w)
    check(want, *c.reference())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.forward_topk(c.x, c.ids, c.probs, w, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del kept


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_strides_and_expert_tables(mx):
    """Rows of wider buffers with NaN around them, experts given one by one: the same bits."""
    T, H, I, E, k = 6, 288, 96, 7, 3
    c = Layer(T, H, I, E, k, mx, seed=12)
    dec = c.decoder(16)
    out = dec.forward_topk(c.x, c.ids, c.probs, c.weights())
    check(out, *c.reference())
    wide = torch.full((T, H + 24), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + H] = c.x
    into = torch.full((T, H + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    dec.forward_topk(wide[:, 8:8 + H], c.ids, c.probs, c.weights(), out=into[:, 3:3 + H])
    assert torch.equal(into[:, 3:3 + H], out) and (into[:, :3] == 7).all() and (into[:, 3 + H:] == 7).all()
    if mx:
        one = lambda q: [q[e].clone() for e in range(E)]  # noqa: E731
        parts = {n: (one(q), one(q), one(s), one(q)) for n, q, s in
                 (("gate", c.q1[:, :I], c.s1[:, :I]), ("up", c.q1[:, I:], c.s1[:, I:]), ("down", c.q2, c.s2))}
        w = M.set_mx_expert_tables(c.weights(), **parts)
    else:
        pad = lambda m: torch.nn.functional.pad(m, (0, 16), value=math.nan)[:, :m.shape[1]]  # noqa: E731
        parts = {n: [pad(m[e]) for e in range(E)] for n, m in (("gate", c.b1[:, :I]), ("up", c.b1[:, I:]), ("down", c.b2))}
        w = M.set_expert_tables(c.weights(), **parts)
    assert torch.equal(dec.forward_topk(c.x, c.ids, c.probs, w), out)
    # other pointers in the same table
    order = list(range(1, E)) + [0]
    moved = {n: (tuple([p[e] for e in order] for p in v) if mx else [v[e] for e in order]) for n, v in parts.items()}
    w2 = (M.set_mx_expert_tables if mx else M.set_expert_tables)(c.weights(), **moved)
    ids2 = torch.where(c.ids >= 0, (c.ids - 1) % E, c.ids)
    check(dec.forward_topk(c.x, ids2, c.probs, w2), *c.reference())


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_nan_stays_in_its_token_and_its_expert(mx):
    T, H, I, E, k = 12, 256, 96, 6, 2
    c = Layer(T, H, I, E, k, mx, seed=30, missing=0.0)
    dec, w = c.decoder(), c.weights()
    out = dec.forward_topk(c.x, c.ids, c.probs, w)
    x = c.x.clone()
    x[4, 100], x[7, 3] = math.nan, math.inf
    got = dec.forward_topk(x, c.ids, c.probs, w)
    keep = [t for t in range(T) if t not in (4, 7)]
    assert torch.equal(got[keep], out[keep]) and got[4].isnan().all() and not torch.isfinite(got[7]).any()
    # an expert's NaN weight reaches the tokens of that expert alone
    if mx:
        c.q1[3, 5, 17] = 0x7F
    else:
        c.b1[3, 5, 17] = math.nan
    got = dec.forward_topk(c.x, c.ids, c.probs, c.weights())
    hit = (c.ids == 3).any(1)
    assert hit.any() and not hit.all()
    assert torch.equal(got[~hit], out[~hit]) and got[hit].isnan().all()


@gpu
@pytest.mark.parametrize("T", [3, 20])
def test_every_e4m3_code_and_scale(T):
    """Payloads of all codes but NaN (subnormals among them) under scales from tiny to large, one row
    of subnormals alone; a scale code of 255 is NaN."""
    H, I, E, k = 512, 64, 3, 2
    c = Layer(T, H, I, E, k, True, False, seed=60, missing=0.0)
    codes = torch.tensor([v for v in range(256) if v & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    pick = lambda t, vals: vals[torch.randint(0, len(vals), t.shape, generator=g, device="cuda")]  # noqa: E731
    c.q1, c.q2 = pick(c.q1, codes), pick(c.q2, codes)
    c.q2[:, 7] = pick(c.q2[:, 7], torch.tensor([0x01, 0x81, 0x07, 0x84, 0x00, 0x80], dtype=torch.uint8, device="cuda"))
    c.s1 = pick(c.s1, torch.arange(106, 117, dtype=torch.uint8, device="cuda"))
    c.s2 = pick(c.s2, torch.arange(60, 140, dtype=torch.uint8, device="cuda"))
    c.fc1, c.fc2 = mx_values(c.q1, c.s1), mx_values(c.q2, c.s2)
    dec = c.decoder()
    out = dec.forward_topk(c.x, c.ids, c.probs, c.weights())
    check(out, *c.reference())
    assert out[:, 7].any()
    c.s2[1, 9, 1] = 255
    got = dec.forward_topk(c.x, c.ids, c.probs, c.weights())
    hit = (c.ids == 1).any(1)
    assert got[hit, 9].isnan().all() and torch.equal(got[~hit], out[~hit])
    rest = [h for h in range(H) if h != 9]
    assert torch.equal(got[:, rest], out[:, rest])


@gpu
def test_fewer_tokens_streams_graph_and_old_workspace_contents():
    c = Layer(33, 512, 160, 9, 4, seed=40)
    w = c.weights()
    dec = c.decoder(64)
    out = dec.forward_topk(c.x, c.ids, c.probs, w)
    check(out, *c.reference())
    # rows are independent of the batch that they come in, up to the order of sums
    for n in (1, 8, 20):
        part = dec.forward_topk(c.x[:n], c.ids[:n], c.probs[:n], w)
        ref, tol = c.reference()
        check(part, ref[:n], tol[:n], f"first {n}")
    # every byte of the workspace that is not the library's state may have held anything
    other = M.MoEDecoder.__new__(M.MoEDecoder)
    other.__dict__.update({n: v for n, v in dec.__dict__.items() if n not in ("handle", "workspace")})
    other.workspace = torch.full_like(dec.workspace, 255)
    other.handle = M.moe_decode_create(dec.cfg, other.workspace)
    assert torch.equal(other.forward_topk(c.x, c.ids, c.probs, w), out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = other.forward_topk(c.x, c.ids, c.probs, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dec.forward_topk(c.x, c.ids, c.probs, w)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    c.x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    check(got, *c.reference(), what="replay on new values")
    assert dec.device_status() == B.MOE_OK
    assert dec.forward_topk(c.x[:0], c.ids[:0], c.probs[:0], w).shape == (0, 512)


def test_refusals():
    def status(call):
        with pytest.raises(M.MoeError) as e:
            call()
        return e.value.status

    base = dict(max_tokens=8, hidden=64, num_experts=4, topk=2, inter=32, routed_wtype=0, swiglu_limit=0.0)
    size = lambda **kw: M.moe_decode_size(M.moe_config(**{**base, **kw}))  # noqa: E731
    assert size() > 0 and size(hidden=72, inter=40) > 0 and size(max_tokens=0) > 0
    for kw, want in ((dict(max_tokens=65), 2), (dict(max_tokens=-1), 1), (dict(hidden=60), 2), (dict(inter=12), 2),
                     (dict(routed_wtype=1, hidden=72), 2), (dict(routed_wtype=1, inter=40), 2), (dict(topk=5), 2),
                     (dict(num_experts=1025), 2), (dict(topk=0), 1), (dict(swiglu_limit=-1.0), 1), (dict(recompute_dispatch=1), 1),
                     (dict(no_shared_expert=2), 1), (dict(act_precision=3), 1), (dict(routed_wtype=2), 2), (dict(hidden=0), 1)):
        assert status(lambda: size(**kw)) == want, kw
    L = M.load()
    import ctypes
    d = ctypes.c_void_p()
    assert L.moe_decode_create(M.moe_config(**base), None, 0, ctypes.byref(d)) == 1
    assert L.moe_decode_create(M.moe_config(**base), 256, 16, ctypes.byref(d)) == 1
    assert L.moe_decode_create(M.moe_config(**base), 264, 1 << 30, ctypes.byref(d)) == 1
    assert L.moe_decode(None, 1, 256, 64, 256, 256, None, 256, 64, None) == 1
    assert L.moe_decode_status(None, None) == 1


@gpu
def test_call_refusals():
    """Arguments that a call cannot serve come back as errors before anything is launched."""
    c = Layer(4, 64, 32, 4, 2, gate=True, seed=50)
    dec = c.decoder()
    L, w = M.load(), c.weights()
    out = torch.empty_like(c.x)
    base = dict(T=4, x=c.x.data_ptr(), xs=64, ids=c.ids.data_ptr(), p=c.probs.data_ptr(), w=w, out=out.data_ptr(), os=64)

    def call(**kw):
        a = {**base, **kw}
        return L.moe_decode(dec.handle, a["T"], a["x"], a["xs"], a["ids"], a["p"], a["w"], a["out"], a["os"], None)

    before = M.moe_launch_count()
    for kw in (dict(T=5), dict(T=-1), dict(x=None), dict(x=base["x"] + 2), dict(xs=63), dict(xs=68), dict(ids=None), dict(p=None),
               dict(out=None), dict(os=63), dict(w=None), dict(ids=base["ids"] + 1)):
        assert call(**kw) == 1, kw
    for field, value in (("data", None), ("data", w.routed_up.data + 8), ("row_stride", 60), ("row_stride", 8)):
        bad = c.weights()
        setattr(bad.routed_up, field, value)
        assert call(w=bad) == 1, field
    bad = c.weights()
    bad.shared_down.data = None
    assert call(w=bad) == 1
    assert M.moe_launch_count() == before and call() == 0
    with pytest.raises(ValueError):
        dec.forward_topk(c.x.float(), c.ids, c.probs, w)
    with pytest.raises(ValueError):
        dec.forward_topk(c.x, c.ids.long(), c.probs, w)
    with pytest.raises(ValueError):
        dec.forward_topk(c.x, c.ids[:, :1], c.probs, w)


def _busy():
    """Some milliseconds of work on the current stream."""
    torch.cuda._sleep(20_000_000)


@gpu
@pytest.mark.parametrize("T", [3, 40])
def test_created_on_a_side_stream_with_work_pending(T):
    """The decoder's state is cleared after what its memory's last owner still had queued, and before the first
    call, whichever stream that is on; so is the status."""
    c = Layer(T, 512, 160, 9, 4, seed=41)
    w = c.weights()
    want = c.decoder(64).forward_topk(c.x, c.ids, c.probs, w)
    check(want, *c.reference())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    n = M.moe_decode_size(c.decoder(64).cfg)
    _busy()                                            # the default stream
    with torch.cuda.stream(side):
        old = torch.empty(n, dtype=torch.uint8, device="cuda")
        at = old.data_ptr()
        _busy()
        old.fill_(255)                                 # still to come when its memory is given away
        del old
        dec = c.decoder(64)
        assert dec.workspace.data_ptr() == at
        got = dec.forward_topk(c.x, c.ids, c.probs, w)
        assert dec.device_status() == B.MOE_OK
        bad = c.ids.clone()
        bad[0, 0] = 9
        dec.forward_topk(c.x, bad, c.probs, w)
    torch.cuda.default_stream().synchronize()
    _busy()
    assert dec.device_status(side) == B.MOE_ERR_ROUTING and dec.device_status(side) == B.MOE_OK
    with torch.cuda.stream(other):                     # at once on another stream, the default one busy
        again = dec.forward_topk(c.x, c.ids, c.probs, w)
        assert dec.device_status() == B.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)


def table_set(c, order):
    """Tables whose entry e is expert order[e], the ids that name the same experts through them, and the tables' owner."""
    E, I = c.E, c.I
    own = lambda m: [m[e].contiguous() for e in order]  # noqa: E731
    if c.mx:
        parts = {n: (own(q), own(q), own(s), own(q)) for n, q, s in
                 (("gate", c.q1[:, :I], c.s1[:, :I]), ("up", c.q1[:, I:], c.s1[:, I:]), ("down", c.q2, c.s2))}
        w = M.set_mx_expert_tables(c.weights(), **parts)
    else:
        w = M.set_expert_tables(c.weights(), **{n: own(m) for n, m in (("gate", c.b1[:, :I]), ("up", c.b1[:, I:]), ("down", c.b2))})
        parts = None
    place = torch.tensor([order.index(e) for e in range(E)], device="cuda")
    return w, torch.where(c.ids >= 0, place[c.ids.clamp(min=0).long()].int(), c.ids), parts


@gpu
@pytest.mark.parametrize("mx", [False, True])
def test_a_captured_call_keeps_its_tables(mx):
    """Calls with other tables, before and after: a replay runs with the tables that were captured; so do two sets in one graph."""
    c = Layer(4, 288, 96, 5, 2, mx, seed=14)
    ref = c.reference()
    dec = c.decoder(8)
    (wa, ia, ka), (wb, ib, kb) = table_set(c, [3, 1, 4, 0, 2]), table_set(c, [0, 4, 2, 1, 3])
    a, b = dec.forward_topk(c.x, ia, c.probs, wa), dec.forward_topk(c.x, ib, c.probs, wb)
    check(a, *ref), check(b, *ref)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    dec.forward_topk(c.x, ia, c.probs, wa)
    with torch.cuda.graph(one):
        got = dec.forward_topk(c.x, ia, c.probs, wa)
    for _ in range(2):
        assert torch.equal(dec.forward_topk(c.x, ib, c.probs, wb), b)
        got.zero_()
        one.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, a)
    with torch.cuda.graph(two):
        ga, gb = dec.forward_topk(c.x, ia, c.probs, wa), dec.forward_topk(c.x, ib, c.probs, wb)
    two.replay()
    torch.cuda.synchronize()
    assert torch.equal(ga, a) and torch.equal(gb, b)


@gpu
def test_more_table_sets_than_a_decoder_keeps():
    """The set used longest ago makes room; one that a graph reads does not: a set too many is refused."""
    c = Layer(3, 64, 32, 5, 2, seed=15)
    ref = c.reference()
    dec = c.decoder()
    sets = [table_set(c, list(p)) for p in itertools.islice(itertools.permutations(range(5)), 70)]
    call = lambda s: dec.forward_topk(c.x, s[1], c.probs, s[0])  # noqa: E731
    first = call(sets[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(sets[0])
    for _ in range(2):
        for s in sets:
            check(call(s), *ref)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, first)
    n = B.MOE_DECODE_TABLE_SETS
    assert n < 70
    for s in sets[:n]:
        call(s)
    full = torch.cuda.CUDAGraph()
    with torch.cuda.graph(full):
        outs = [call(s) for s in sets[:n]]
    with pytest.raises(M.MoeError) as e:
        call(sets[n])
    assert e.value.status == 6  # MOE_ERR_STATE
    check(call(sets[1]), *ref)
    full.replay()
    torch.cuda.synchronize()
    for o in outs:
        check(o, *ref)
    assert dec.device_status() == B.MOE_OK


@gpu
def test_tensors_on_two_devices_are_refused():
    """Tensors in host memory come back as errors before anything is launched, in any place."""
    c = Layer(3, 64, 32, 4, 2, seed=51)
    dec, w = c.decoder(), c.weights()
    out = torch.empty_like(c.x)
    before = M.moe_launch_count()
    for i in range(4):
        args = [c.x, c.ids, c.probs, w, out]
        args[i if i < 3 else 4] = args[i if i < 3 else 4].cpu()
        with pytest.raises(ValueError, match="device"):
            dec.forward_topk(*args)
        with pytest.raises(ValueError, match="device"):
            M.moe_decode(dec.handle, 3, *args)
    assert M.moe_launch_count() == before
    M.moe_decode(dec.handle, 3, c.x, c.ids, c.probs, w, out)
    check(out, *c.reference())


def overflow_case(mx, shared, finite):
    """One expert (the shared one, or expert 1) whose activation i = 3 of token 2 is 2^240, or, finite, 2^128 (1 - 2^-10):
    the largest bf16 is less, the largest fp32 more. Every other activation of that token is 0."""
    T, H, I, E, k = 5, 64, 32, 3, 1
    c = Layer(T, H, I, E, k, mx, shared, seed=70, missing=0.0)
    c.ids[:] = 1
    c.probs[:] = 0.5
    c.x[:] = 0
    c.x[2, 0], c.x[2, 40] = 2.0 ** 32, 1.0
    g, u = (2.0 ** 32, 2.0 ** 32) if finite else (2.0 ** 88, 2.0 ** 88)
    fc1, fc2 = torch.zeros(2 * I, H, device="cuda"), torch.where(torch.arange(H, device="cuda") % 3 == 0, -1.0, 1.0)[:, None].repeat(1, I)
    fc1[3, 0], fc1[I + 3, 0] = g, u
    if finite:
        fc1[I + 3, 40] = -2.0 ** 54
        fc2 *= 2.0 ** -20
    zero1, zero2 = torch.zeros_like(fc1), torch.zeros_like(fc2)
    stack = lambda m, z: torch.stack([z, z if shared else m, z])  # noqa: E731
    if mx:
        (c.q1, c.s1), (c.q2, c.s2) = quantise(stack(fc1, zero1)), quantise(stack(fc2, zero2))
        c.fc1, c.fc2 = mx_values(c.q1, c.s1), mx_values(c.q2, c.s2)
    else:
        c.b1, c.b2 = stack(fc1, zero1).bfloat16(), stack(fc2, zero2).bfloat16()
        c.fc1, c.fc2 = c.b1.double(), c.b2.double()
    if shared:
        c.sfc1, c.sfc2 = fc1.bfloat16(), fc2.bfloat16()
    return c


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("finite", [False, True])
def test_activations_past_what_bf16_holds(mx, shared, finite):
    """An activation that overflows gives the infinity that the definition's 2^240 rounds to, not NaN; one that fp32 holds
    and bf16 does not is multiplied as it is."""
    if mx and not shared:
        finite = False       # two f16 terms under a scale of their own
    c = overflow_case(mx, shared, finite)
    out = c.decoder().forward_topk(c.x, c.ids, c.probs, c.weights())
    x = c.x.double()
    fc1, fc2, p = (c.sfc1.double(), c.sfc2.double(), 1.0) if shared else (c.fc1[1], c.fc2[1], 0.5)
    gate, up = (x @ fc1.t()).chunk(2, -1)
    ref = p * ((gate * torch.sigmoid(gate) * up) @ fc2.t())
    if finite:
        assert float(ref[2].abs().max()) < 1e33
        check(out, ref, 2.0 ** -15 * ref.abs())
    else:
        assert float(ref[2].abs().min()) > 1e70
        assert torch.equal(out, ref.bfloat16()) and torch.isinf(out[2]).all()
    assert not out[[0, 1, 3, 4]].any()


@gpu
def test_two_decoders_on_two_streams():
    """Launches of two decoders that nothing orders: each has its own barrier, and all of its blocks resident."""
    c = Layer(5, 1160, 424, 10, 3, seed=42)
    w = c.weights()
    decs = [c.decoder(), c.decoder()]
    want = decs[0].forward_topk(c.x, c.ids, c.probs, w)
    check(want, *c.reference())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for d, s in zip(decs, streams):
            with torch.cuda.stream(s):
                outs.append(d.forward_topk(c.x, c.ids, c.probs, w))
    for d, s in zip(decs, streams):
        assert d.device_status(s) == B.MOE_OK
    assert all(torch.equal(o, want) for o in outs)


@gpu
def test_the_state_starts_anew_after_a_recorded_timeout():
    """A status word that says that a wait gave up, a barrier and counters as such a launch may leave them (written
    here: no wait runs out): the status is reported once, and the next call is right."""
    c = Layer(6, 520, 136, 5, 3, seed=43)
    dec, w = c.decoder(), c.weights()
    want = dec.forward_topk(c.x, c.ids, c.probs, w)
    assert dec.device_status() == B.MOE_OK
    state = dec.workspace[:4 * (2 + (520 + 15) // 16)].view(torch.int32)
    state[0] = 2                                       # the timeout bit
    state[1] = 77
    state[2:] = 3
    assert dec.device_status() == B.MOE_ERR_TIMEOUT and dec.device_status() == B.MOE_OK
    assert not state.any()
    assert torch.equal(dec.forward_topk(c.x, c.ids, c.probs, w), want) and dec.device_status() == B.MOE_OK


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,k", [(1, 4), (7, 3), (8, 4), (9, 3)])
def test_bad_ids_among_few_routes(T, k, mx):
    """Up to 32 routes are sorted by one warp: ids out of range and chosen twice, alone and beside good rows."""
    c = Layer(T, 128, 64, 5, k, mx, seed=9, missing=0.0)
    dec, w = c.decoder(), c.weights()
    good = c.ids.clone()
    for put in ([(0, 0, 5)], [(0, k - 1, -2)], [(0, 1, int(good[0, 0]))], [(T - 1, 0, 1 << 30), (0, k - 1, int(good[0, 0]))],
                [(T - 1, k - 1, -(1 << 31))], [(0, 0, -1), (0, 1, -1)]):
        bad = good.clone()
        for t, s, v in put:
            bad[t, s] = v
        out = dec.forward_topk(c.x, bad, c.probs, w)
        empty = all(v == -1 for _, _, v in put)
        assert dec.device_status() == (B.MOE_OK if empty else B.MOE_ERR_ROUTING) and dec.device_status() == B.MOE_OK
        kept = bad if empty else good.clone()
        if not empty:
            kept[[t for t, _, _ in put]] = -1
        check(out, *c.reference(kept))
        assert torch.equal(dec.forward_topk(c.x, kept, c.probs, w), out)


@gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 10, 30])
def test_no_route_and_no_shared_expert(T, mx):
    """Nothing chosen and nothing shared: rows of zeros, in a wider buffer too, and nothing beside them written; the next
    call is right."""
    c = Layer(T, 96, 64, 5, 3, mx, shared=False, seed=10, missing=0.0)
    dec, w = c.decoder(), c.weights()
    into = torch.full((T, 104), 7.0, dtype=torch.bfloat16, device="cuda")
    dec.forward_topk(c.x, torch.full_like(c.ids, -1), torch.full_like(c.probs, math.nan), w, out=into[:, :96])
    assert not into[:, :96].any() and (into[:, 96:] == 7).all() and dec.device_status() == B.MOE_OK
    check(dec.forward_topk(c.x, c.ids, c.probs, w), *c.reference())


@gpu
def test_given_up_while_a_call_on_another_stream_runs():
    """A decoder that goes away with a call pending on a stream other than the one it was made on: its memory is not
    handed out before that call has ended."""
    c = Layer(5, 512, 160, 9, 4, seed=44)
    w = c.weights()
    keep = c.decoder()
    want = keep.forward_topk(c.x, c.ids, c.probs, w)
    check(want, *c.reference())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        dec = c.decoder()
        n, at = dec.workspace.numel(), dec.workspace.data_ptr()
        with torch.cuda.stream(side):
            _busy()
            got = dec.forward_topk(c.x, c.ids, c.probs, w)
        del dec
        others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        assert all(o.data_ptr() != at for o in others)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del others
