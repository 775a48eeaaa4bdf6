"""The example's mixture-of-experts layer: serving in FP8 and int8 and a training step, against the same
layer in fp32.

Tolerances: an E4M3 code is within 2^-4 of its value (half of 3 mantissa bits' step), uniformly spread
about 2^-4 / sqrt(3) = 3.6% in the root mean square at worst, less than that over a binade (2.6%); an int8 code
within half of amax / 127, about 1% of a normal row's rms.  Four such roundings enter a value (two
products of two quantized operands each): 2.6% * 2 = 5.2%, and 2% for int8; six enter a weight gradient of the
first product (7%).  Bounds of 1.5 times these."""

import importlib.util
import os

import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from gpu_util import device, say

pytestmark = pytest.mark.gpu

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
_spec = importlib.util.spec_from_file_location("moe_layer", _PATH)
moe_layer = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(moe_layer)

ROUTING = [dict(score="sigmoid", num_groups=4, topk_groups=2, group_top=2, scale=2.5), dict(score="softmax", renormalize=False)]


@pytest.mark.parametrize("form,bound", [("fp8", 0.08), ("int8", 0.03)])
@pytest.mark.parametrize("tokens,rows", [(1, 16), (37, 64), (530, 0)])
@pytest.mark.parametrize("routing", ROUTING)
def test_serving(form, bound, tokens, rows, routing):
    say("moe layer", form, tokens, rows, routing)
    x, router, w_in, w_out = moe_layer.make(tokens, 512, 256, 16, device(), seed=tokens)
    layer = moe_layer.MoELayer(router, w_in, w_out, 4, form=form, **routing)
    ids, _ = layer.route(x)
    y = layer(x, rows_per_expert=rows)
    assert moe_layer.error(y, moe_layer.reference(x.float(), router, w_in, w_out, ids, **routing)) < bound


@pytest.mark.parametrize("routing", ROUTING)
def test_training_step(routing):
    say("moe layer training", routing)
    x, router, w_in, w_out = moe_layer.make(300, 512, 256, 8, device(), seed=5)
    leaves = [t.clone().requires_grad_(True) for t in (x, router, w_in, w_out)]
    y = moe_layer.train_step(*leaves, 3, **routing)
    ids, _ = dg.dg_moe_route(x.float() @ router.t(), 3, **routing)
    dy = torch.randn(y.shape, generator=torch.Generator(device=device()).manual_seed(1), device=device()).bfloat16()
    y.backward(dy)
    ref = [t.clone().float().requires_grad_(True) for t in (x, router, w_in, w_out)]
    want = moe_layer.reference(*ref, ids, **routing)
    want.backward(dy.float())
    assert moe_layer.error(y, want) < 0.08
    for name, a, b in zip(("x", "router", "w_in", "w_out"), leaves, ref):
        assert moe_layer.error(a.grad, b.grad) < 0.105, name
