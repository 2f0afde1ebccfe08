"""The operators of a transformer's dense blocks in 8-bit floating point, as workloads.

Numbers are held as E4M3 codes with one fp32 scale for a block of 128: along a
row, down a column (the tokens), or 128 x 128 (weights). Three operators, each
with its plain form (elementary torch operations in fp32) and the library's own calls:

* ``linear``: a linear layer, forward and backward, ``MoEFp8Linear``
* ``ffn``: the gated feed-forward network, forward, backward and a whole
  training step, ``MoEFeedForward``
* ``keep``: activations kept in 8 bits for a later backward pass and read back,
  ``fp8_quantize`` / ``fp8_dequantize``

``own`` selects the side that ``run`` takes.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "fp32"
ROW, COL, SQUARE = "row", "col", "square"
TOP, LEAST = 448.0, 2.0 ** -126      # largest E4M3 value, smallest scale


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _dtype(name):
    return torch.bfloat16 if name == BF16 else torch.float32


# ------------------------------------------------------------------ cases
def _linear(name, direction, T, K, N, grad=F32, pad=0):
    return dict(name=name, op="linear", direction=direction, T=T, K=K, N=N, grad=grad, pad=pad)


def _ffn(name, direction, T, H, I, limit=0.0, pad=0):
    return dict(name=name, op="ffn", direction=direction, T=T, H=H, I=I, limit=limit, pad=pad)


def _keep(name, block, rows, cols, x=BF16, pad=0):
    return dict(name=name, op="keep", block=block, rows=rows, cols=cols, x=x, pad=pad)


def listed():
    return [
        # a projection of one decoded token: the weights' bytes and the calls' latency
        _linear("linear-fwd-1", "forward", 1, 2048, 4096),
        # a decode batch through a large model's projection
        _linear("linear-fwd-48", "forward", 48, 7168, 2048),
        # a prefill or training batch through a large model's projection
        _linear("linear-fwd-8192", "forward", 8192, 7168, 4096),
        # sizes that no tile divides, rows of a wider buffer, a gradient in the weights' type
        _linear("linear-bwd-odd", "backward", 777, 1160, 424, grad=BF16, pad=3),
        # the backward pass of a training batch
        _linear("linear-bwd-4096", "backward", 4096, 4096, 7168),
        # a dense layer serving one sequence
        _ffn("ffn-fwd-1", "forward", 1, 7168, 2048),
        # a dense layer serving a decode batch
        _ffn("ffn-fwd-64", "forward", 64, 4096, 8192),
        # a training step of a small model with the clamp, sizes that no tile divides
        _ffn("ffn-step-odd", "step", 515, 1160, 1000, limit=2.0),
        # a training step of a dense layer four times as wide inside as outside
        _ffn("ffn-step-8192", "step", 8192, 2048, 8192),
        # a short activation kept in fp32's place, odd width
        _keep("keep-col-odd", COL, 777, 2051, x=F32, pad=5),
        # a training batch's activations kept for the weights' gradient
        _keep("keep-col-16384", COL, 16384, 7168),
        # a training batch's activations kept by rows
        _keep("keep-row-16384", ROW, 16384, 4096),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        old = top.get(c["op"], (0, 0))
        top[c["op"]] = (max(old[0], w["bytes"]), max(old[1], w["flops"]))
    while True:
        op = rng.choice(["linear", "ffn", "keep"])
        pad = rng.choice([0, 0, 3, 8])
        if op == "linear":
            c = _linear("", rng.choice(["forward", "backward"]), _spread(rng, 1, 16384), _spread(rng, 32, 8192),
                        _spread(rng, 32, 8192), rng.choice([F32, BF16]), pad)
        elif op == "ffn":
            c = _ffn("", rng.choice(["forward", "backward", "step"]), _spread(rng, 1, 16384), _spread(rng, 64, 7168),
                     _spread(rng, 64, 8192), rng.choice([0.0, 0.0, 2.0]), pad)
        else:
            c = _keep("", rng.choice([ROW, COL]), _spread(rng, 1, 32768), _spread(rng, 16, 12288),
                      rng.choice([BF16, BF16, F32]), pad)
        w = work(c)
        if w["bytes"] <= top[op][0] and w["flops"] <= top[op][1]:
            del c["name"]
            return c


# ------------------------------------------------------------------ codes with a scale for each block of 128
def _block_max(a, along_rows, along_cols):
    """Largest |a| of blocks of 128 along the given axes."""
    R, C = a.shape
    pad = torch.nn.functional.pad(a.abs(), (0, -C % 128 if along_cols else 0, 0, -R % 128 if along_rows else 0))
    if along_rows:
        pad = pad.reshape(-1, 128, pad.shape[-1]).amax(1)
    if along_cols:
        pad = pad.reshape(pad.shape[0], -1, 128).amax(-1)
    return pad


def _spread_scales(s, shape, block):
    if block != ROW:
        s = s.repeat_interleave(128, 0)[:shape[0]]
    if block != COL:
        s = s.repeat_interleave(128, 1)[:, :shape[1]]
    return s


def _quantise(x, block):
    """(codes, scales) of x [R, C]; scales [R, C/128], [R/128, C] or [R/128, C/128], rounded up."""
    x = x.float()
    amax = _block_max(x, block != ROW, block != COL)
    s = torch.maximum(amax / torch.full_like(amax, TOP), torch.full_like(amax, LEAST))
    r = torch.ones_like(s) / s
    return (x * _spread_scales(r, x.shape, block)).clamp(-TOP, TOP).to(torch.float8_e4m3fn), s


def _values(codes, s, block):
    return codes.float() * _spread_scales(s, codes.shape, block)


def _through(x, block):
    return _values(*_quantise(x, block), block)


def _as_bytes(codes):
    """The codes as uint8 rows whose stride is a multiple of 16, as the library keeps them."""
    R, C = codes.shape
    wide = torch.zeros((R, C + -C % 16), dtype=torch.uint8, device=codes.device)
    wide[:, :C] = codes.view(torch.uint8)
    return wide[:, :C]


def _kept(x, block):
    """x as the library's calls take it: (bytes, scales), the scales of row blocks as [C/128, R]."""
    codes, s = _quantise(x, block)
    return _as_bytes(codes), (s.t().contiguous() if block == ROW else s)


def _read(kept, block):
    q, s = kept
    return _values(q.contiguous().view(torch.float8_e4m3fn), s.t() if block == ROW else s, block)


# ------------------------------------------------------------------ what a program has in hand
def _generator(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dev, scale=1.0):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale


def _rows(t, pad):
    """t as rows of a buffer that is `pad` elements wider."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _activation(g, T, C, dev):
    """A normed activation: channels of different sizes, a few of them large."""
    width = torch.exp(_randn(g, (C,), dev, 0.5))
    return _randn(g, (T, C), dev) * width


def prepare(case, seed):
    c, dev = case, _device()
    g = _generator(seed, dev)
    s = dict(case=c)
    if c["op"] == "keep":
        s["x"] = _rows(_activation(g, c["rows"], c["cols"], dev).to(_dtype(c["x"])), c["pad"])
        return s
    T = c["T"]
    if c["op"] == "linear":
        s["x"] = _rows(_activation(g, T, c["K"], dev).bfloat16(), c["pad"])
        s["weight"] = _kept(_randn(g, (c["N"], c["K"]), dev, 0.02).bfloat16(), SQUARE)
        if c["direction"] == "backward":
            s["kept"] = _kept(s["x"], COL)
            s["dy"] = _rows(_randn(g, (T, c["N"]), dev).bfloat16(), c["pad"])
            s["dweight"] = torch.empty((c["N"], c["K"]), dtype=_dtype(c["grad"]), device=dev)
        if own:
            import mixture_experts_layer_pack_gb300 as M
            s["layer"] = M.MoEFp8Linear(c["K"], c["N"], device=dev)
        return s
    H, I = c["H"], c["I"]
    s["x"] = _rows(_activation(g, T, H, dev).bfloat16(), c["pad"])
    spread = 1.0 / math.sqrt(H)
    s["gate"] = _kept(_randn(g, (I, H), dev, spread).bfloat16(), SQUARE)
    s["up"] = _kept(_randn(g, (I, H), dev, spread).bfloat16(), SQUARE)
    s["down"] = _kept(_randn(g, (H, I), dev, 0.02).bfloat16(), SQUARE)
    if c["direction"] != "forward":
        s["dy"] = _rows(_randn(g, (T, H), dev).bfloat16(), c["pad"])
        s["grads"] = [torch.empty(n, dtype=torch.bfloat16, device=dev) for n in ((I, H), (I, H), (H, I))]
    if c["direction"] == "backward":       # what a forward pass over these activations keeps
        s["kept"] = (_kept(s["x"], COL), _kept(_randn(g, (T, I), dev, 1.2), ROW), _kept(_randn(g, (T, I), dev, 1.2), ROW))
    if own:
        import mixture_experts_layer_pack_gb300 as M
        s["layer"] = M.MoEFeedForward(H, I, swiglu_limit=c["limit"], device=dev)
        s["weights"] = M.FeedForwardWeights(s["gate"], s["up"], s["down"])
    return s


# ------------------------------------------------------------------ plain forms
def _plain_linear_backward(dy, weight, x, grad):
    """(dx, dW) at the kept x."""
    dx = _through(dy, ROW) @ weight
    return dx.bfloat16(), (_through(dy, COL).t() @ x).to(grad)


def _gated(g, u, limit):
    if limit > 0:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1 + torch.exp(-g)) * u


def _plain_ffn_forward(s):
    x = _through(s["x"], ROW)
    g, u = x @ _read(s["gate"], SQUARE).t(), x @ _read(s["up"], SQUARE).t()
    h = _gated(g, u, s["case"]["limit"])
    return (_through(h, ROW) @ _read(s["down"], SQUARE).t()).bfloat16(), g, u


def _plain_ffn_backward(s, x, g, u):
    """Gradients at the kept x, g and u."""
    limit = s["case"]["limit"]
    dh = _through(s["dy"], ROW) @ _read(s["down"], SQUARE)
    gc, uc = (g.clamp(max=limit), u.clamp(-limit, limit)) if limit > 0 else (g, u)
    sig = 1 / (1 + torch.exp(-gc))
    du, dg = dh * gc * sig, dh * uc * sig * (1 + gc * (1 - sig))
    if limit > 0:
        dg, du = torch.where(g > limit, torch.zeros_like(dg), dg), torch.where(u.abs() > limit, torch.zeros_like(du), du)
    h = gc * sig * uc
    dx = _through(dg, ROW) @ _read(s["gate"], SQUARE) + _through(du, ROW) @ _read(s["up"], SQUARE)
    grads = (_through(dg, COL).t() @ x, _through(du, COL).t() @ x, _through(s["dy"], COL).t() @ _through(h, COL))
    return dx.bfloat16(), [d.bfloat16() for d in grads]


def _plain(s):
    c = s["case"]
    if c["op"] == "keep":
        codes, scales = _quantise(s["x"], c["block"])
        return dict(scales=scales.t().contiguous() if c["block"] == ROW else scales, x=_values(codes, scales, c["block"]).to(_dtype(c["x"])))
    if c["op"] == "linear":
        weight = _read(s["weight"], SQUARE)
        if c["direction"] == "forward":
            return dict(y=(_through(s["x"], ROW) @ weight.t()).bfloat16())
        dx, dw = _plain_linear_backward(s["dy"], weight, _read(s["kept"], COL), _dtype(c["grad"]))
        return dict(dx=dx, dweight=dw)
    if c["direction"] == "backward":
        dx, grads = _plain_ffn_backward(s, _read(s["kept"][0], COL), _read(s["kept"][1], ROW), _read(s["kept"][2], ROW))
        return dict(dx=dx, dgate=grads[0], dup=grads[1], ddown=grads[2])
    y, g, u = _plain_ffn_forward(s)
    if c["direction"] == "forward":
        return dict(y=y)
    dx, grads = _plain_ffn_backward(s, _through(s["x"], COL), _through(g, ROW), _through(u, ROW))
    return dict(y=y, dx=dx, dgate=grads[0], dup=grads[1], ddown=grads[2])


# ------------------------------------------------------------------ one pass
def _own(s):
    import mixture_experts_layer_pack_gb300 as M
    c = s["case"]
    if c["op"] == "keep":
        block = M.MOE_B_ROW if c["block"] == ROW else M.MOE_B_COL
        q, scales = M.fp8_quantize(s["x"], block)
        return dict(scales=scales, x=M.fp8_dequantize(q, scales, block, dtype=_dtype(c["x"])))
    layer = s["layer"]
    if c["op"] == "linear":
        if c["direction"] == "forward":
            return dict(y=layer.forward(s["x"], s["weight"], keep=False)[0])
        dx, dw = layer.backward(s["dy"], s["weight"], s["kept"], dweight=s["dweight"])
        return dict(dx=dx, dweight=dw)
    if c["direction"] == "forward":
        return dict(y=layer.forward(s["x"], s["weights"], keep=False)[0])
    out, kept = {}, s.get("kept")
    if c["direction"] == "step":
        out["y"], kept = layer.forward(s["x"], s["weights"])
    dx, grads = layer.backward(s["dy"], s["weights"], kept, grads=s["grads"])
    return dict(out, dx=dx, dgate=grads[0], dup=grads[1], ddown=grads[2])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "keep":       # read, written as codes and scales, read again, written
        n, size = c["rows"] * c["cols"], 2 if c["x"] == BF16 else 4
        return {"bytes": n * (2 * size + 2 + 8 / 128), "flops": 4 * n}
    T = c["T"]
    if c["op"] == "linear":
        K, N = c["K"], c["N"]
        if c["direction"] == "forward":
            return {"bytes": 2 * T * (K + N) + K * N, "flops": 2 * T * K * N}
        return {"bytes": 2 * T * N + 3 * T * K + K * N * (1 + (4 if c["grad"] == F32 else 2)), "flops": 4 * T * K * N}
    H, I = c["H"], c["I"]
    forward = {"bytes": 4 * T * H + 3 * H * I, "flops": 6 * T * H * I}
    backward = {"bytes": 5 * T * H + 2 * T * I + 9 * H * I, "flops": 12 * T * H * I}
    if c["direction"] == "forward":
        return forward
    if c["direction"] == "backward":
        return backward
    return {"bytes": forward["bytes"] + backward["bytes"] + T * (H + 2 * I), "flops": forward["flops"] + backward["flops"]}


# ------------------------------------------------------------------ the definitions, in 64 bits
class _Exact:
    """The operators' formulas in 64 bits. A block's scale is a stored fp32 number, and a value's code is the E4M3 number
    nearest to its fp32 product with the scale's fp32 reciprocal; everything else is in 64 bits."""

    def quantised(self, x, rows, cols):
        """x's values after it is stored in blocks of `rows` x `cols`, and the blocks' scales."""
        R, C = x.shape
        down, across = torch.arange(R, device=x.device) // rows, torch.arange(C, device=x.device) // cols
        nr, nc = -(-R // rows), -(-C // cols)
        x32 = x.float()
        amax = torch.zeros((nr, C), dtype=torch.float32, device=x.device)
        amax = amax.index_reduce_(0, down, x32.abs(), "amax") if rows > 1 else x32.abs()
        if cols > 1:
            amax = torch.zeros((nc, nr), dtype=torch.float32, device=x.device).index_reduce_(0, across, amax.t().contiguous(), "amax").t()
        scale = torch.true_divide(amax.double(), 448.0).float().clamp(min=LEAST)
        each = scale[down][:, across]
        code = (x32 * torch.reciprocal(each.double()).float()).clamp(-448, 448).to(torch.float8_e4m3fn)
        return code.double() * each.double(), scale

    def stored(self, kept, rows, cols, transposed=False):
        q, scale = kept
        scale = scale.t() if transposed else scale
        R, C = q.shape
        each = scale.double()[torch.arange(R, device=q.device) // rows][:, torch.arange(C, device=q.device) // cols]
        return q.contiguous().view(torch.float8_e4m3fn).double() * each

    def ffn(self, s):
        c = s["case"]
        wg, wu, wd = (self.stored(s[n], 128, 128) for n in ("gate", "up", "down"))
        out = {}
        if c["direction"] == "backward":
            xk = self.stored(s["kept"][0], 128, 1)
            g, u = (self.stored(k, 1, 128, True) for k in s["kept"][1:])
        else:
            x = self.quantised(s["x"], 1, 128)[0]
            g, u = x @ wg.t(), x @ wu.t()
            h = self.quantised(self.gate(g, u, c["limit"]), 1, 128)[0]
            out["y"] = h @ wd.t()
            if c["direction"] == "forward":
                return out
            xk = self.quantised(s["x"], 128, 1)[0]
            g, u = self.quantised(g, 1, 128)[0], self.quantised(u, 1, 128)[0]
        g.requires_grad_(True)
        u.requires_grad_(True)
        h = self.gate(g, u, c["limit"])
        dh = self.quantised(s["dy"], 1, 128)[0] @ wd
        dg, du = torch.autograd.grad(h, (g, u), dh)
        out["dx"] = self.quantised(dg, 1, 128)[0] @ wg + self.quantised(du, 1, 128)[0] @ wu
        out["dgate"] = self.quantised(dg, 128, 1)[0].t() @ xk
        out["dup"] = self.quantised(du, 128, 1)[0].t() @ xk
        out["ddown"] = self.quantised(s["dy"], 128, 1)[0].t() @ self.quantised(h.detach(), 128, 1)[0]
        return out

    def gate(self, g, u, limit):
        if limit > 0:
            g, u = torch.clamp(g, max=limit), torch.clamp(u, min=-limit, max=limit)
        return g * torch.sigmoid(g) * u

    def linear(self, s):
        w = self.stored(s["weight"], 128, 128)
        if s["case"]["direction"] == "forward":
            return dict(y=self.quantised(s["x"], 1, 128)[0] @ w.t())
        return dict(dx=self.quantised(s["dy"], 1, 128)[0] @ w,
                    dweight=self.quantised(s["dy"], 128, 1)[0].t() @ self.stored(s["kept"], 128, 1))

    def keep(self, s):
        row = s["case"]["block"] == ROW
        x, scale = self.quantised(s["x"], *((1, 128) if row else (128, 1)))
        return dict(scales=scale.t().contiguous().double() if row else scale.double(), x=x)


def exact(case, seed):
    if work(case)["flops"] > 5e12:       # more than some 20 seconds in 64 bits
        return None
    s = prepare(case, seed)
    return getattr(_Exact(), case["op"])(s)
