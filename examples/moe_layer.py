"""A mixture-of-experts feed-forward layer on the library's operators, from router logits to the tokens.

``MoELayer`` serves one in FP8 or in 8-bit integers:

    route -> layout -> dispatch (quantizing) -> grouped GEMM -> SwiGLU -> grouped GEMM -> combine

in the contiguous layout (prompts) or the masked one (decode steps with a fixed buffer per expert; no size
on the host depends on the routing, so a step can be captured in a HIP graph).  ``train_step`` runs the
layer forward and backward: the router's weights, dispatch and combine with their gradients, the experts'
products and both of their gradients in FP8.

    python examples/moe_layer.py     # a few sizes of each, compared with the same layer in fp32
"""

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_block_scaled_gemm_amd as dg  # noqa: E402


def swiglu(h):
    gate, up = h.chunk(2, dim=-1)
    return F.silu(gate) * up


class MoELayer:
    """E experts of hidden -> 2 * inner -> hidden over a router (E, hidden); weights float32."""

    def __init__(self, router, w_in, w_out, top_k, form="fp8", bias=None, **routing):
        self.router, self.bias, self.top_k, self.form, self.routing = router, bias, top_k, form, routing
        self.experts = w_in.shape[0]
        quantize = dg.dg_quantize_per_block if form == "fp8" else dg.dg_quantize_int8_per_token
        self.w_in, self.w_out = quantize(w_in.contiguous()), quantize(w_out.contiguous())

    def route(self, x):
        return dg.dg_moe_route(x.float() @ self.router.t(), self.top_k, bias=self.bias, **self.routing)

    def experts_forward(self, q, s, layout):
        if self.form == "fp8":
            gemm = dg.dg_gemm_fp8_grouped_masked if layout.rows_per_expert else dg.dg_gemm_fp8_grouped_contiguous
            quantize = dg.dg_quantize_per_token_group
        else:
            gemm = dg.dg_gemm_int8_grouped_masked if layout.rows_per_expert else dg.dg_gemm_int8_grouped_contiguous
            quantize = dg.dg_quantize_int8_per_token
        where = layout.counts if layout.rows_per_expert else layout.m_indices
        # rows of no expert stay as they were allocated, and are never read
        h = gemm(q, s, *self.w_in, where)
        q, s = quantize(swiglu(h).contiguous())
        return gemm(q, s, *self.w_out, where)

    def __call__(self, x, rows_per_expert=0):
        """x (tokens, hidden) -> (tokens, hidden); rows_per_expert > 0: the masked layout."""
        ids, weights = self.route(x)
        layout = dg.dg_moe_layout(ids, self.experts, rows_per_expert=rows_per_expert)
        q, s = dg.dg_moe_dispatch_fp8(x, layout) if self.form == "fp8" else dg.dg_moe_dispatch_int8(x, layout)
        return dg.dg_moe_combine(self.experts_forward(q, s, layout), layout, weights=weights)


# ---- training -------------------------------------------------------------------------------------

class RouteWeights(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, routing):
        ids, weights = dg.dg_moe_route(logits, top_k, **routing)
        ctx.save_for_backward(logits, ids)
        ctx.form = {k: v for k, v in routing.items() if k in ("score", "renormalize", "scale")}
        ctx.mark_non_differentiable(ids)
        return ids, weights

    @staticmethod
    def backward(ctx, _, dweights):
        logits, ids = ctx.saved_tensors
        return dg.dg_moe_route_grad(dweights.contiguous(), logits, ids, **ctx.form), None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, layout):
        ctx.layout = layout
        return dg.dg_moe_dispatch(x, layout)

    @staticmethod
    def backward(ctx, drows):
        return dg.dg_moe_combine(drows.contiguous(), ctx.layout), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, layout):
        ctx.save_for_backward(rows, weights)
        ctx.layout = layout
        return dg.dg_moe_combine(rows, layout, weights=weights)

    @staticmethod
    def backward(ctx, dy):
        rows, weights = ctx.saved_tensors
        # rows past the last expert's take no part: zeros, so that what multiplies them stays finite
        drows, dweights = dg.dg_moe_combine_grad(dy.contiguous(), rows, ctx.layout, weights, dout=torch.zeros_like(rows))
        return drows, dweights, None


class ExpertsLinear(torch.autograd.Function):
    """rows (contiguous layout, bf16) times each expert's weight (experts, n, k) float32, in FP8."""

    @staticmethod
    def forward(ctx, rows, weight, m_indices, padded):
        w = dg.dg_quantize_per_block(weight)
        ctx.save_for_backward(rows, m_indices, *w)
        ctx.padded = padded   # rows of each expert, on the host
        d = torch.zeros((rows.shape[0], weight.shape[1]), dtype=torch.bfloat16, device=rows.device)
        return dg.dg_gemm_fp8_grouped_contiguous(*dg.dg_quantize_per_token_group(rows), *w, m_indices, d=d)

    @staticmethod
    def backward(ctx, dout):
        rows, m_indices, wq, ws = ctx.saved_tensors
        dout, used = dout.contiguous(), sum(ctx.padded)
        drows = torch.zeros_like(rows)
        dg.dg_gemm_fp8_grouped_contiguous(*dg.dg_quantize_per_token_group(dout), *dg.dg_transpose_blocks(wq, ws), m_indices,
                                          d=drows)
        dweight = dg.dg_gemm_fp8_k_grouped_row_scaled(*dg.dg_quantize_per_channel_group(dout[:used]),
                                                      *dg.dg_quantize_per_channel_group(rows[:used]), ctx.padded)
        return drows, dweight.float(), None, None


def train_step(x, router, w_in, w_out, top_k, **routing):
    """y (tokens, hidden) bf16, differentiable in x (bf16) and the float32 router, w_in and w_out."""
    ids, weights = RouteWeights.apply(x.float() @ router.t(), top_k, routing)
    layout = dg.dg_moe_layout(ids, w_in.shape[0])
    padded = [-(-int(c) // 128) * 128 for c in layout.counts.tolist()]   # the weight gradients need them on the host
    rows = Dispatch.apply(x, layout)
    h = ExpertsLinear.apply(rows, w_in, layout.m_indices, padded)
    out = ExpertsLinear.apply(swiglu(h), w_out, layout.m_indices, padded)
    return Combine.apply(out, weights, layout)


# ---- the same layer in fp32 -----------------------------------------------------------------------

def reference(x, router, w_in, w_out, ids, **routing):
    """Expert by expert, in torch, with the choice `ids` given."""
    logits = x @ router.t()
    scores = torch.softmax(logits, 1) if routing.get("score", "softmax") == "softmax" else torch.sigmoid(logits)
    chosen = scores.gather(1, ids.long())
    if routing.get("renormalize", True):
        chosen = chosen / chosen.sum(1, keepdim=True)
    chosen = chosen * routing.get("scale", 1.0)
    y = torch.zeros_like(x)
    for e in range(w_in.shape[0]):
        token, place = torch.nonzero(ids == e, as_tuple=True)
        if token.numel():
            y = y.index_add(0, token, chosen[token, place, None] * (swiglu(x[token] @ w_in[e].t()) @ w_out[e].t()))
    return y


def make(tokens, hidden, inner, experts, device, seed=0):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)
    return (r(tokens, hidden).bfloat16(), r(experts, hidden) * hidden ** -0.5, r(experts, 2 * inner, hidden) * hidden ** -0.5,
            r(experts, hidden, inner) * inner ** -0.5)


def error(got, want):
    got, want = got.detach().float(), want.detach().float()
    return float((got - want).norm() / want.norm())


def main():
    device = torch.device("cuda", 0)
    routing = dict(score="sigmoid", num_groups=4, topk_groups=2, group_top=2, scale=2.5)
    for tokens, rows in ((1, 16), (48, 64), (1000, 0)):
        x, router, w_in, w_out = make(tokens, 1024, 512, 16, device)
        for form in ("fp8", "int8"):
            layer = MoELayer(router, w_in, w_out, 4, form=form, **routing)
            ids, _ = layer.route(x)
            y = layer(x, rows_per_expert=rows)
            want = reference(x.float(), router, w_in, w_out, ids, **routing)
            print(f"{form}: {tokens} tokens, {'masked' if rows else 'contiguous'} rows: error {error(y, want):.4f}", flush=True)
    x, router, w_in, w_out = make(700, 1024, 512, 16, device)
    leaves = [t.clone().requires_grad_(True) for t in (x, router, w_in, w_out)]
    y = train_step(*leaves, 4, **routing)
    dy = torch.randn_like(y)
    y.backward(dy)
    ids, _ = dg.dg_moe_route(x.float() @ router.t(), 4, **routing)
    ref = [t.clone().float().requires_grad_(True) for t in (x, router, w_in, w_out)]
    reference(*ref, ids, **routing).backward(dy.float())
    for name, a, b in zip(("x", "router", "w_in", "w_out"), leaves, ref):
        print(f"gradient of {name}: error {error(a.grad, b.grad):.4f}", flush=True)


if __name__ == "__main__":
    main()
