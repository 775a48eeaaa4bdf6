"""Feed-forward blocks between two residual norms on the library's operators, dense and with experts.

``FeedForward`` serves one in FP8 or 8-bit integers: the norm before it writes the first product's operand, the gated
product the second one's, so that nothing is quantized in a pass of its own:

    residual norm (quantizing) -> gated product -> product

``ExpertsFeedForward`` is the mixture of experts of ``moe_layer.py`` with its two products and the activation between
them in two calls, in the contiguous layout or the masked one.  ``train_step`` runs a residual norm and a dense block
forward and backward, ``train_experts`` the rows of experts: every product and gradient of theirs in FP8.

    python examples/feed_forward.py     # a few sizes of each, compared with the same block in fp32
"""

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_block_scaled_gemm_amd as dg  # noqa: E402
import moe_layer  # noqa: E402

ACTS = {"silu": F.silu, "gelu": lambda g: F.gelu(g, approximate="tanh")}


class FeedForward:
    """hidden -> inner -> hidden behind a residual norm; w_in (2, inner, hidden) = gate, up and w_out (hidden, inner)
    float32, norm_weight float32 (hidden,) or None."""

    def __init__(self, w_in, w_out, norm_weight=None, act="silu", form="fp8"):
        self.norm_weight, self.act, self.form = norm_weight, act, form
        if form == "fp8":
            self.w_in, self.w_out = dg.dg_quantize_per_block(w_in.contiguous()), dg.dg_quantize_per_block(w_out.contiguous())
        else:
            self.w_in = dg.dg_quantize_int8_per_token(w_in.reshape(-1, w_in.shape[-1]).contiguous())
            self.w_out = dg.dg_quantize_int8_per_token(w_out.contiguous())

    def __call__(self, x, residual, gate=None, post_norm=False, scale=1.0):
        """(y, sum) (rows, hidden) from the last block's output x and the residual stream, which goes on as sum."""
        norm = dict(weight=self.norm_weight, gate=gate, post_norm=post_norm, scale=scale)
        if self.form == "fp8":
            total, q, s = dg.dg_residual_norm_fp8(x, residual, **norm)
            return dg.dg_gemm_fp8_nt(*dg.dg_gemm_fp8_gated_nt(q, s, *self.w_in, act=self.act, out="fp8"), *self.w_out), total
        total, q, s = dg.dg_residual_norm_int8(x, residual, **norm)
        pre = dg.dg_gemm_int8_nt(q, s, *self.w_in)
        return dg.dg_gemm_int8_nt(*dg.dg_gated_act_int8(pre, self.act), *self.w_out), total


class ExpertsFeedForward(moe_layer.MoELayer):
    """The mixture of experts with gated products; w_in (experts, 2 * inner, hidden) = gate | up, inner a multiple of 128."""

    def experts_forward(self, q, s, layout):
        masked = bool(layout.rows_per_expert)
        where = layout.counts if masked else layout.m_indices
        if self.form == "fp8":
            gated = dg.dg_gemm_fp8_gated_masked if masked else dg.dg_gemm_fp8_gated_contiguous
            gemm = dg.dg_gemm_fp8_grouped_masked if masked else dg.dg_gemm_fp8_grouped_contiguous
            return gemm(*gated(q, s, *self.w_in, where, out="fp8"), *self.w_out, where)
        gemm = dg.dg_gemm_int8_grouped_masked if masked else dg.dg_gemm_int8_grouped_contiguous
        # rows of no expert are skipped throughout: they stay as they were allocated, and are never read
        rows = {"masked_m" if masked else "m_indices": where}
        return gemm(*dg.dg_gated_act_int8(gemm(q, s, *self.w_in, where), **rows), *self.w_out, where)


# ---- training -------------------------------------------------------------------------------------

class ResidualNorm(torch.autograd.Function):
    """(sum, y): sum = residual + gate * x, y = weight * sum / rms(sum)."""

    @staticmethod
    def forward(ctx, x, residual, weight, gate):
        total, y = dg.dg_residual_norm(x, residual, weight=weight, gate=gate)
        ctx.save_for_backward(x, total, weight, gate)
        return total, y

    @staticmethod
    def backward(ctx, dsum, dy):
        x, total, weight, gate = ctx.saved_tensors
        g = dg.dg_residual_norm_grad(dy.contiguous(), dsum.contiguous(), x, total, weight=weight, gate=gate)
        return g.dx, g.dresidual, g.dweight, g.dgate


class GatedProducts(torch.autograd.Function):
    """rows (bf16) through w_in ([experts,] 2, inner, hidden) = gate, up and w_out ([experts,] hidden, inner), float32, in
    FP8.  Dense: rows a multiple of 16.  Experts: the contiguous layout's rows up to its last expert's, m_indices
    theirs, `padded` the rows of each expert, on the host.  The projections are kept in bf16 for the way back; what the
    second product reads is not: the activation's gradient makes it again, in the layout that the weight gradient reads."""

    @staticmethod
    def forward(ctx, rows, w_in, w_out, act, m_indices, padded):
        wi, wo = dg.dg_quantize_per_block(w_in.flatten(0, -3)), dg.dg_quantize_per_block(w_out)
        wi = (wi[0].view(w_in.shape), wi[1].view(*w_in.shape[:-2], *wi[1].shape[-2:]))
        pre = torch.empty((rows.shape[0], 2 * w_in.shape[-2]), dtype=torch.bfloat16, device=rows.device)
        q, s = dg.dg_quantize_per_token_group(rows)
        if padded is None:
            y = dg.dg_gemm_fp8_nt(*dg.dg_gemm_fp8_gated_nt(q, s, *wi, act=act, out="fp8", pre=pre), *wo)
        else:
            h = dg.dg_gemm_fp8_gated_contiguous(q, s, *wi, m_indices, act=act, out="fp8", pre=pre)
            y = dg.dg_gemm_fp8_grouped_contiguous(*h, *wo, m_indices)
        ctx.save_for_backward(rows, pre, m_indices, *wi, *wo)
        ctx.act, ctx.padded = act, padded
        return y

    @staticmethod
    def backward(ctx, dy):
        rows, pre, m_indices, wiq, wis, woq, wos = ctx.saved_tensors
        dy = dy.contiguous()
        wi = dg.dg_transpose_blocks(wiq.flatten(-3, -2), wis.flatten(-3, -2))   # inner is a multiple of 128
        wo = dg.dg_transpose_blocks(woq, wos)
        if ctx.padded is None:
            product = dg.dg_gemm_fp8_nt
            weight_grad = dg.dg_gemm_fp8_nt_row_scaled
        else:
            product = lambda *t: dg.dg_gemm_fp8_grouped_contiguous(*t, m_indices)
            weight_grad = lambda *t: dg.dg_gemm_fp8_k_grouped_row_scaled(*t, ctx.padded)
        dh = product(*dg.dg_quantize_per_token_group(dy), *wo)
        q, s, qt, st, ht, hst = dg.dg_gated_act_grad_fp8(dh, pre, ctx.act)
        drows = product(q, s, *wi)
        dw_in = weight_grad(qt, st, *dg.dg_quantize_per_channel_group(rows))
        dw_out = weight_grad(*dg.dg_quantize_per_channel_group(dy), ht, hst)
        return drows, dw_in.float().view(wiq.shape), dw_out.float(), None, None, None


def train_step(x, residual, norm_weight, gate, w_in, w_out, act="silu"):
    """(y, sum) bf16, differentiable in x, residual and gate (bf16) and the float32 norm_weight, w_in and w_out."""
    total, n = ResidualNorm.apply(x, residual, norm_weight, gate)
    return GatedProducts.apply(n, w_in, w_out, act, None, None), total


def train_experts(x, router, w_in, w_out, top_k, act="silu", **routing):
    """y (tokens, hidden) bf16 of a mixture of experts, w_in (experts, 2, inner, hidden), differentiable in x (bf16) and
    the float32 router, w_in and w_out."""
    ids, weights = moe_layer.RouteWeights.apply(x.float() @ router.t(), top_k, routing)
    layout = dg.dg_moe_layout(ids, w_in.shape[0])
    padded = [-(-int(c) // 128) * 128 for c in layout.counts.tolist()]   # the weight gradients need them on the host
    used = sum(padded)
    rows = moe_layer.Dispatch.apply(x, layout)
    out = GatedProducts.apply(rows[:used], w_in, w_out, act, layout.m_indices[:used], padded)
    return moe_layer.Combine.apply(F.pad(out, (0, 0, 0, rows.shape[0] - used)), weights, layout)


# ---- the same blocks in fp32 ----------------------------------------------------------------------

def products(x, w_in, w_out, act="silu"):
    return (ACTS[act](x @ w_in[0].t()) * (x @ w_in[1].t())) @ w_out.t()


def norm(x, residual, weight=None, gate=None, post_norm=False, scale=1.0, eps=1e-6):
    rms = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + eps)
    z = rms(x) if post_norm else x
    total = residual + scale * (z if gate is None else z * gate)
    y = rms(total)
    return total, y if weight is None else y * weight


def make(rows, hidden, inner, device, seed=0):
    """x, residual (bf16), norm weight, gate (bf16), w_in and w_out."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=device)
    return (r(rows, hidden).bfloat16(), r(rows, hidden).bfloat16(), 1 + 0.1 * r(hidden), r(hidden).bfloat16(),
            r(2, inner, hidden) * hidden ** -0.5, r(hidden, inner) * inner ** -0.5)


def main():
    device, error = torch.device("cuda", 0), moe_layer.error
    for rows in (1, 100, 2000):
        x, residual, weight, gate, w_in, w_out = make(rows, 1024, 512, device)
        total, n = norm(x.float(), residual.float(), weight, gate.float(), post_norm=True)
        for form in ("fp8", "int8"):
            y, _ = FeedForward(w_in, w_out, weight, form=form)(x, residual, gate=gate, post_norm=True)
            print(f"{form}: {rows} rows: error {error(y, products(n, w_in, w_out)):.4f}", flush=True)
    routing = dict(score="sigmoid", num_groups=4, topk_groups=2, group_top=2, scale=2.5)
    for tokens, rows in ((1, 16), (48, 64), (1000, 0)):
        x, router, w_in, w_out = moe_layer.make(tokens, 1024, 512, 16, device)
        for form in ("fp8", "int8"):
            layer = ExpertsFeedForward(router, w_in, w_out, 4, form=form, **routing)
            want = moe_layer.reference(x.float(), router, w_in, w_out, layer.route(x)[0], **routing)
            y = layer(x, rows_per_expert=rows)
            print(f"{form}: {tokens} tokens of experts, {'masked' if rows else 'contiguous'}: error {error(y, want):.4f}", flush=True)
    leaves = [t.clone().requires_grad_(True) for t in make(2000, 1024, 512, device)]
    ref = [t.detach().float().requires_grad_(True) for t in leaves]
    y, total = train_step(*leaves)
    dy = torch.randn_like(y)
    torch.autograd.backward([y, total], [dy, dy])
    want_total, n = norm(*ref[:4])
    torch.autograd.backward([products(n, *ref[4:]), want_total], [dy.float(), dy.float()])
    for name, a, b in zip(("x", "residual", "norm_weight", "gate", "w_in", "w_out"), leaves, ref):
        print(f"gradient of {name}: error {error(a.grad, b.grad):.4f}", flush=True)


if __name__ == "__main__":
    main()
