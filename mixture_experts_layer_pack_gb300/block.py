"""The expert block of a transformer: norm, router, experts and the residual stream around them.

    s = x + residual            the residual stream, in x's type
    y = norm(s) w + b           bf16, the experts' input
    logits = y Wr^T             a plain library product, in Wr's type
    ids, probs = top-k(logits)  with the routes' counts and the balance and z losses
    out = experts(y, ids, probs)

``forward`` returns (out, s): the next block's norm adds them up, as this one's
added x and residual, so the stream is read and written once a block. The step
for training runs on a ``MoELayer`` and is followed by ``backward``; ``decode``
is the same function without anything kept for a backward pass: a
``MoEDecoder`` takes batches of up to ``decode_tokens`` tokens, larger ones go
to the layer.

With MXFP8 experts the layer multiplies by scales in a layout of its own, which
it holds for one set of weights: ``prepare`` converts them, before the first
forward with a set and after every change of its scales. The decoder reads the
weights as they are.

Steps may be captured into CUDA graphs. The decoder's replays keep the expert
tables that were captured with them, whatever else it decodes; the layer has one
set of tables, so a block that had a step through it captured takes no other
weights there.
"""
from __future__ import annotations

import dataclasses

from . import binding as B


@dataclasses.dataclass
class BlockParams:
    """Parameters of a block: norm_weight and norm_bias [H] (norm_bias may be None), router_weight [E,H]
    (fp32 logits from fp32, bf16 logits from bf16), select_bias [E] fp32 or None (moves the choice of
    experts only) and the experts' moe_weights, which are pointers: their tensors are the caller's to keep."""
    norm_weight: object
    router_weight: object
    weights: B.moe_weights
    norm_bias: object = None
    select_bias: object = None


class MoEBlock:
    """One expert block; one forward at a time waits for its backward."""

    def __init__(self, max_tokens, hidden, num_experts, topk, inter, device="cuda", norm=B.MOE_NORM_RMS, eps=1e-6,
                 score=B.MOE_SCORE_SOFTMAX, normalise=True, scale=1.0, aux_coeff=0.0, z_coeff=0.0,
                 routed_wtype=B.MOE_W_BF16, swiglu_limit=0.0, act_precision=None, shared_expert=True,
                 decode_tokens=B.MOE_DECODE_MAX_TOKENS):
        """max_tokens: of a training step, 0 for a block that only decodes; decode_tokens: of the decoder, 0 for none.
        The decoder is made for few tokens an expert: where experts are few, the layer is faster from some 16 tokens
        each on (64 tokens, H 4096, I 2048, 8 experts top-4: 102 us against 202), so decode_tokens may be less."""
        if max_tokens <= 0 and decode_tokens <= 0:
            raise ValueError("a block needs max_tokens, decode_tokens or both")
        self.norm = B.MoENorm(hidden, eps, norm, device=device)
        self.router = B.MoERouter(num_experts, topk, score, normalise, scale, aux_coeff, z_coeff, device=device)
        self.layer = self.decoder = None
        if max_tokens > 0:
            self.layer = B.MoELayer(max_tokens, hidden, num_experts, topk, inter, device=device, routed_wtype=routed_wtype,
                                    swiglu_limit=swiglu_limit, act_precision=act_precision, shared_expert=shared_expert)
        if decode_tokens > 0:
            self.decoder = B.MoEDecoder(decode_tokens, hidden, num_experts, topk, inter, device=device,
                                        routed_wtype=routed_wtype, swiglu_limit=swiglu_limit, shared_expert=shared_expert)
        self.decode_tokens = decode_tokens
        self._mx = routed_wtype == B.MOE_W_MXFP8
        self._kept = self._captured = None

    def prepare(self, params: BlockParams):
        """Converts the scales of params' MXFP8 experts for the layer (nothing to do for BF16 ones, or for a block that
        only decodes); on the current stream. Weights need their columnwise payloads and scales for it."""
        if self._mx and self.layer is not None:
            self._uncaptured(params)
            self.layer.prepare_weights(params.weights)

    def _uncaptured(self, p):
        """Refuses other weights than those of a captured step: its replays read the layer's tables and scales."""
        key = bytes(p.weights)
        if self._captured not in (None, key):
            raise B.MoeError(B.MOE_ERR_STATE, "MoEBlock: the layer keeps the weights of a captured step;")
        return key

    def _on_layer(self, p, call, *args):
        """call(*args) of the layer, which must not hold the scales of other weights (holding none, it says so itself)."""
        import torch
        key = self._uncaptured(p)
        if self.layer.prepared not in (None, key):
            raise B.MoeError(B.MOE_ERR_STATE, "MoEBlock: prepare(params) comes first, the layer holds other weights' scales;")
        result = call(*args)
        if torch.cuda.is_current_stream_capturing():
            self._captured = key
        return result

    def _routed(self, x, residual, p):
        import torch
        y, s, mean, rstd = self.norm.forward(x, p.norm_weight, p.norm_bias, residual=residual, out_dtype=torch.bfloat16)
        logits = torch.nn.functional.linear(y.to(p.router_weight.dtype), p.router_weight)
        return y, s, mean, rstd, logits, self.router.forward(logits, p.select_bias)

    def forward(self, x, params: BlockParams, residual=None):
        """(out [T,H] bf16, s [T,H] in x's type, losses [2] fp32 or None) of x and residual [T,H], bf16 or fp32;
        on the current stream. What backward needs is kept until it, or the next forward."""
        if self.layer is None:
            raise ValueError("the block was made for decoding only (max_tokens 0)")
        y, s, mean, rstd, logits, (ids, probs, counts, losses) = self._routed(x, residual, params)
        out = self._on_layer(params, self.layer.forward_topk, y, ids, probs, params.weights)
        self._kept = (params, y, s, mean, rstd, logits, ids, counts)
        return out, s, losses

    def backward(self, dout, main_grads: B.moe_main_grads, ds=None, loss_grad=1.0):
        """(dx, grads) for the gradients dout of out (bf16) and ds of s (x's type; None: zero), with any strides, and loss_grad of
        the losses' sum.
        dx is that of x and of residual alike. grads: norm_weight, norm_bias (None without one) and
        router_weight; the experts' are added to main_grads."""
        import torch
        if self._kept is None:
            raise ValueError("backward without a forward before it")
        p, y, s, mean, rstd, logits, ids, counts = self._kept
        if dout.shape != y.shape or dout.dtype != y.dtype or dout.device != y.device:
            raise ValueError("dout must be [T, H] bf16 on the block's device")
        if ds is not None:  # looked at before anything is added to main_grads
            if ds.shape != s.shape or ds.dtype != s.dtype or ds.device != s.device:
                raise ValueError("ds must be [T, H] of x's type on the block's device")
            if ds.stride(1) != 1 or ds.stride(0) < ds.shape[1]:
                ds = ds.contiguous()
        dy, dprobs = self._on_layer(p, self.layer.backward, dout.contiguous(), main_grads)  # the layer takes compact rows
        self._kept = None
        dlogits = self.router.backward(logits, ids, dprobs, counts=counts, loss_grad=loss_grad)
        drouter = dlogits.t() @ y.to(dlogits.dtype)
        # one rounding of the sum of both paths to y
        dy = torch.addmm(dy.to(dlogits.dtype), dlogits, p.router_weight)
        dx, dw, db = self.norm.backward(dy, s, p.norm_weight, mean, rstd, dsum=ds, bias=p.norm_bias is not None)
        return dx, {"norm_weight": dw, "norm_bias": db, "router_weight": drouter}

    def decode(self, x, params: BlockParams, residual=None):
        """(out, s) as forward's, with nothing kept; may be captured into a CUDA graph (experts given as per-expert
        tables: after one call with the same tables)."""
        small = self.decoder is not None and x.shape[0] <= self.decode_tokens
        if not small and self.layer is None:
            raise ValueError(f"the block decodes up to {self.decode_tokens} tokens")
        y, s, _, _, _, (ids, probs, _, _) = self._routed(x, residual, params)
        if small:
            return self.decoder.forward_topk(y, ids, probs, params.weights), s
        out = self._on_layer(params, self.layer.forward_topk, y, ids, probs, params.weights)
        self._kept = None  # the layer's saved state is overwritten
        return out, s

    def close(self):
        for part in (self.layer, self.decoder):
            if part is not None:
                part.close()
