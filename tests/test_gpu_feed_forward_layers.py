"""The example's feed-forward blocks: serving in FP8 and int8, dense and with experts, and training steps, against the
same blocks in fp32.

Tolerances: an E4M3 code is within 2^-4 of its value, 2.6% in the root mean square over a binade; an int8 code within
half of amax / 127, about 1% of a normal row's rms.  In the output: activations and weights of the gate and of the up
product (4; the activation's slope times g over its value lies about 1), h and the second weights (2): 2.6% * sqrt(6) =
6.4%, 2.5% for int8.  In a gradient of the inner weights or of the rows: dy and the second weights (2), the other
projection's two roundings and the activation slope's two (4), dpre and the last operand (2): 2.6% * sqrt(8) = 7.4%.
Bounds of 1.5 times these: 0.096, 0.038, 0.11; bf16 roundings (2^-8 at most each) vanish beside them.  The residual
stream's sum is rounded once, and its reference's inputs are the same: 2^-8."""

import importlib.util
import os

import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from gpu_util import device, say

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
_spec = importlib.util.spec_from_file_location("feed_forward", _PATH)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)
moe_layer = example.moe_layer

ROUTING = [dict(score="sigmoid", num_groups=4, topk_groups=2, group_top=2, scale=2.5), dict(score="softmax", renormalize=False)]


@pytest.mark.parametrize("form,bound", [("fp8", 0.096), ("int8", 0.038)])
@pytest.mark.parametrize("rows", [1, 37, 530])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_serving(form, bound, rows, act):
    say("feed forward", form, rows, act)
    x, residual, weight, gate, w_in, w_out = example.make(rows, 512, 256, device(), seed=rows)
    block = example.FeedForward(w_in, w_out, weight, act=act, form=form)
    y, total = block(x, residual, gate=gate, post_norm=True, scale=0.5)
    want_total, n = example.norm(x.float(), residual.float(), weight, gate.float(), post_norm=True, scale=0.5)
    assert moe_layer.error(y, example.products(n, w_in, w_out, act)) < bound
    assert moe_layer.error(total, want_total) < 2 ** -8


@pytest.mark.parametrize("form,bound", [("fp8", 0.096), ("int8", 0.038)])
@pytest.mark.parametrize("tokens,rows", [(1, 16), (37, 64), (530, 0)])
@pytest.mark.parametrize("routing", ROUTING)
def test_experts_serving(form, bound, tokens, rows, routing):
    say("feed forward experts", form, tokens, rows, routing)
    x, router, w_in, w_out = moe_layer.make(tokens, 512, 256, 16, device(), seed=tokens)
    layer = example.ExpertsFeedForward(router, w_in, w_out, 4, form=form, **routing)
    ids, _ = layer.route(x)
    y = layer(x, rows_per_expert=rows)
    assert moe_layer.error(y, moe_layer.reference(x.float(), router, w_in, w_out, ids, **routing)) < bound


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_training_step(act):
    say("feed forward training", act)
    leaves = [t.clone().requires_grad_(True) for t in example.make(304, 512, 256, device(), seed=3)]
    ref = [t.detach().float().requires_grad_(True) for t in leaves]
    y, total = example.train_step(*leaves, act=act)
    g = torch.Generator(device=device()).manual_seed(1)
    dy, dsum = (torch.randn(y.shape, generator=g, device=device()).bfloat16() for _ in range(2))
    torch.autograd.backward([y, total], [dy, dsum])
    want_total, n = example.norm(*ref[:4])
    want = example.products(n, *ref[4:], act)
    torch.autograd.backward([want, want_total], [dy.float(), dsum.float()])
    assert moe_layer.error(y, want) < 0.096
    for name, a, b in zip(("x", "residual", "norm_weight", "gate", "w_in", "w_out"), leaves, ref):
        assert a.grad.dtype == a.dtype and moe_layer.error(a.grad, b.grad) < 0.11, name


@pytest.mark.parametrize("routing", ROUTING)
def test_training_experts(routing):
    say("feed forward training experts", routing)
    x, router, w_in, w_out = moe_layer.make(300, 512, 256, 8, device(), seed=5)
    leaves = [t.clone().requires_grad_(True) for t in (x, router, w_in.view(8, 2, 256, 512), w_out)]
    y = example.train_experts(*leaves, 3, **routing)
    ids, _ = dg.dg_moe_route(x.float() @ router.t(), 3, **routing)
    dy = torch.randn(y.shape, generator=torch.Generator(device=device()).manual_seed(1), device=device()).bfloat16()
    y.backward(dy)
    ref = [t.clone().float().requires_grad_(True) for t in (x, router, w_in, w_out)]
    want = moe_layer.reference(*ref, ids, **routing)
    want.backward(dy.float())
    assert moe_layer.error(y, want) < 0.096
    for name, a, b in zip(("x", "router", "w_in", "w_out"), leaves, ref):
        assert moe_layer.error(a.grad.view(b.shape), b.grad) < 0.11, name
