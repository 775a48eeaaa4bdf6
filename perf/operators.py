"""Cases and plain forms of the mixture-of-experts operators and of the 8-bit integer product.

Three operators, each in its plain form (elementary torch operations in 32 bits, rounded once at the end) and, where
``own`` is true, through the library's public calls:

* ``route``    the choice of experts for each token from its logits, and the gradient of the weights;
* ``experts``  routed tokens laid out in the rows that the grouped products read (copied, or quantized on the way), and
               the experts' results weighted back to the tokens, with the gradients of both ways;
* ``int8``     the product of 8-bit integers with one scale per token and one per output channel, from unquantized
               activations (normal form) or from codes (masked and contiguous forms).
"""

import math

import numpy as np
import torch

own = False

BLOCK = 128   # row alignment of an expert's rows in the contiguous layout
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence: the latency of a serving step's router
        dict(name="route_token", op="route", tokens=1, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, masked=0.0, dtype="bf16", grad=False),
        # the router of a long prompt: sigmoid scores with a balance bias, 4 of 8 groups kept
        dict(name="route_prompt", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, masked=0.0, dtype="f32", grad=False),
        # a training step's router, an odd number of tokens: softmax scores, some experts switched off, and the gradient
        dict(name="route_train", op="route", tokens=8191, experts=64, top_k=6, score="softmax", bias=False, groups=1,
             topk_groups=1, group_top=1, renorm=True, scale=1.0, masked=0.05, dtype="bf16", grad=True),
        # a serving step of 24 sequences over 32 experts with 256-row buffers, rows quantized to 8-bit integers
        dict(name="experts_decode", op="experts", tokens=24, top_k=4, experts=32, hidden=7168, rows=256, form="int8",
             dtype="bf16", skew=0.3, dropped=0.1, grad=False),
        # a prompt of 4096 tokens, 8 of 64 experts each (32768 rows, Zipf sizes), rows quantized to FP8
        dict(name="experts_prompt", op="experts", tokens=4096, top_k=8, experts=64, hidden=7168, rows=0, form="fp8",
             dtype="bf16", skew=1.1, dropped=0.0, grad=False),
        # a training step, an odd number of tokens: rows copied, and the gradients of both ways
        dict(name="experts_train", op="experts", tokens=4093, top_k=6, experts=64, hidden=2048, rows=0, form="copy",
             dtype="bf16", skew=0.7, dropped=0.02, grad=True),
        # one token through one projection: the weights are read once, latency counts
        dict(name="int8_token", op="int8", form="normal", m=1, n=4096, k=7168, groups=1, dtype="bf16", out="bf16"),
        # 64 sequences through the widest projection
        dict(name="int8_decode", op="int8", form="normal", m=64, n=7168, k=16384, groups=1, dtype="bf16", out="bf16"),
        # ragged in every direction, 32-bit activations and results
        dict(name="int8_ragged", op="int8", form="normal", m=777, n=2113, k=1552, groups=1, dtype="f32", out="f32"),
        # the largest dense product of the benchmark
        dict(name="int8_large", op="int8", form="normal", m=16384, n=7168, k=16384, groups=1, dtype="bf16", out="bf16"),
        # 32 experts' decode buffers of 256 rows, between none and all of them in use
        dict(name="int8_masked", op="int8", form="masked", m=256, n=4096, k=7168, groups=32, dtype="bf16", out="bf16"),
        # 4 experts' rows of a prompt in the contiguous layout, a block of them unused
        dict(name="int8_contiguous", op="int8", form="contiguous", m=4096, n=4096, k=7168, groups=4, dtype="bf16",
             out="f16"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step * 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("route", "experts", "int8"))
    if op == "route":
        score = rng.choice(("softmax", "sigmoid"))
        groups = rng.choice((1, 1, 2, 4, 8))
        per_group = _log(rng, 4, 256 // groups)
        experts = groups * per_group
        topk_groups = 1 if groups == 1 else rng.randint(1, groups)
        top_k = rng.randint(1, min(8, topk_groups * per_group))
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, top_k=top_k, score=score,
                    bias=score == "sigmoid" and rng.random() < 0.7, groups=groups, topk_groups=topk_groups,
                    group_top=rng.choice((1, 2)) if score == "sigmoid" else 1, renorm=rng.random() < 0.6,
                    scale=rng.choice((1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.1)),
                    dtype=rng.choice(("f32", "bf16", "f16")), grad=rng.random() < 0.5)
    if op == "experts":
        grad = rng.random() < 0.4
        experts, hidden, top_k = _log(rng, 2, 256), _log(rng, 128, 7168, 16), rng.randint(1, 8)
        top_k = min(top_k, experts)
        tokens = _log(rng, 1, 4096)
        rows = 0 if grad or rng.random() < 0.5 else rng.choice((32, 96, 256))
        while rows and experts * rows * hidden > 32768 * 7168:
            rows //= 2
        form = "copy" if grad else rng.choice(("copy", "fp8", "int8"))
        return dict(op=op, tokens=tokens, top_k=top_k, experts=experts, hidden=hidden, rows=rows, form=form,
                    dtype=rng.choice(("bf16", "f16", "f32")), skew=round(rng.uniform(0.0, 1.2), 2),
                    dropped=rng.choice((0.0, 0.05)), grad=grad)
    form = rng.choice(("normal", "normal", "masked", "contiguous"))
    n, k = _log(rng, 64, 16384), _log(rng, 128, 16384, 16)
    groups, m = 1, _log(rng, 1, 16384)
    if form == "masked":
        n, k = _log(rng, 64, 7168), _log(rng, 128, 7168, 16)
        groups, m = _log(rng, 2, 32), _log(rng, 1, 256)
    elif form == "contiguous":
        n, k = _log(rng, 64, 4096), _log(rng, 128, 7168, 16)
        groups, m = _log(rng, 2, 32), BLOCK * _log(rng, 2, 32)
    while 2 * m * n * k * (groups if form == "masked" else 1) > 2 * 16384 * 7168 * 16384:
        m = max(1, m // 2)
    return dict(op=op, form=form, m=m, n=n, k=k, groups=groups, dtype=rng.choice(("bf16", "f16", "f32")),
                out=rng.choice(("bf16", "f16", "f32")))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows_capacity(tokens, top_k, experts):
    """Rows that the contiguous layout of any choice of experts fits in."""
    n = tokens * top_k
    return (n + min(experts, n) * (BLOCK - 1)) // BLOCK * BLOCK


def _activations(rand, m, k, dtype):
    """N(0, 1), with one row of a hundred (one at least) 100 times larger."""
    x = rand(m, k)
    if m > 1:
        big = torch.arange(m, device=x.device) % 100 == 7 % m
        x = torch.where(big[:, None], x * 100.0, x)
    return x.to(dtype)


def _amax_scale(x, limit):
    """amax / limit over the last dimension, 1 where it is zero (a division by a tensor: each quotient is rounded once)."""
    amax = x.abs().amax(dim=-1)
    return torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, limit))


def _int8_codes(x):
    s = _amax_scale(x, 127.0)
    return torch.round(x / s.unsqueeze(-1)).to(torch.int8), s


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 2 + 1)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    st = {"case": dict(case)}
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        x = rand(t, e)
        if case["masked"]:   # experts switched off for a token; one token of 64 has none left
            off = uniform(t, e) < case["masked"]
            off |= (torch.arange(t, device=dev) % 64 == 63)[:, None]
            x = torch.where(off, torch.full_like(x, -math.inf), x)
        st["logits"] = x.to(dtype)
        st["bias"] = rand(e) * 0.1 if case["bias"] else None
        st["dweights"] = rand(t, case["top_k"]) if case["grad"] else None
    elif case["op"] == "experts":
        t, k, e, h = case["tokens"], case["top_k"], case["experts"], case["hidden"]
        rank = torch.randperm(e, generator=gen, device=dev)
        popular = -case["skew"] * torch.log1p(rank.float())
        gumbel = -torch.log(-torch.log(uniform(t, e).clamp_min(1e-20)).clamp_min(1e-20))
        ids = torch.topk(popular + gumbel, k, dim=1).indices.to(torch.int32)
        if case["dropped"]:
            ids = torch.where(uniform(t, 1) < case["dropped"], torch.full_like(ids, -1), ids)
        st["ids"] = ids.contiguous()
        w = uniform(t, k) + 0.1
        st["weights"] = w / w.sum(dim=1, keepdim=True)
        st["x"] = _activations(rand, t, h, dtype)
        rows = e * case["rows"] if case["rows"] else _rows_capacity(t, k, e)
        lead = (e, case["rows"]) if case["rows"] else (rows,)
        st["results"] = rand(rows, h).to(dtype).view(*lead, h)   # what the experts' products gave for the rows
        if case["form"] == "copy":
            st["xr"] = torch.zeros((*lead, h), dtype=dtype, device=dev)
        else:
            st["q"] = torch.zeros((*lead, h), dtype=torch.uint8 if case["form"] == "fp8" else torch.int8, device=dev)
            kb = -(-h // BLOCK)
            shape = lead if case["form"] == "int8" else (*lead[:-1], kb, -(-lead[-1] // 4) * 4)
            st["s"] = torch.zeros(shape, dtype=torch.float32, device=dev)
        if case["grad"]:
            st["dy"] = rand(t, h).to(dtype)
            st["dxr"] = rand(rows, h).to(dtype)   # the gradient of the dispatched rows
            st["dresults"] = torch.zeros((rows, h), dtype=dtype, device=dev)
    else:
        m, n, k, g = case["m"], case["n"], case["k"], case["groups"]
        w = rand(g, n, k) * 0.02
        st["b"], st["sb"] = _int8_codes(w)
        del w
        if case["form"] == "normal":
            st["b"], st["sb"] = st["b"][0], st["sb"][0]
            st["x"] = _activations(rand, m, k, dtype)
        elif case["form"] == "masked":
            st["a"], st["sa"] = _int8_codes(_activations(rand, g * m, k, dtype).float().view(g, m, k))
            st["masked_m"] = (uniform(g) * (m + 1)).to(torch.int32)
            st["d"] = torch.zeros((g, m, n), dtype=DTYPES[case["out"]], device=dev)
        else:
            st["a"], st["sa"] = _int8_codes(_activations(rand, m, k, dtype).float())
            blocks = m // BLOCK
            cut = torch.sort(uniform(blocks)).values
            expert = (cut * g).to(torch.int32).clamp(0, g - 1)
            expert[-1] = -1   # a block past the last expert's rows
            st["m_indices"] = expert.repeat_interleave(BLOCK).contiguous()
            st["d"] = torch.zeros((m, n), dtype=DTYPES[case["out"]], device=dev)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_route(st):
    c = st["case"]
    x = st["logits"].float()
    t, e, k, g = c["tokens"], c["experts"], c["top_k"], c["groups"]
    off = x == -math.inf
    if c["score"] == "softmax":
        top = x.amax(dim=1, keepdim=True)
        p = torch.where(off, torch.zeros_like(x), torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top)))
        total = p.sum(dim=1, keepdim=True)
        s = p / torch.where(total == 0, torch.ones_like(total), total)
        value = x
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
        value = s if st["bias"] is None else s + st["bias"]
        value = torch.where(off, torch.full_like(value, -math.inf), value)
    if g > 1:
        best = torch.sort(value.view(t, g, e // g), dim=2, descending=True).values[:, :, :c["group_top"]]
        of_group = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(dim=2)
        of_group = torch.where(best[:, :, 0] == -math.inf, best[:, :, 0], of_group)
        order = torch.sort(of_group, dim=1, descending=True, stable=True).indices
        place = torch.empty_like(order).scatter_(1, order, torch.arange(g, device=x.device).expand(t, g))
        kept = (place < c["topk_groups"]).repeat_interleave(e // g, dim=1)
        value = torch.where(kept, value, torch.full_like(value, -math.inf))
    found = torch.sort(value, dim=1, descending=True, stable=True)
    ids, there = found.indices[:, :k], found.values[:, :k] != -math.inf
    chosen = torch.where(there, s.gather(1, ids), torch.zeros_like(s[:, :k]))
    total = chosen.sum(dim=1, keepdim=True)
    total = torch.where(total == 0, torch.ones_like(total), total)
    w = chosen / total * c["scale"] if c["renorm"] else chosen * c["scale"]
    out = {"ids": torch.where(there, ids, torch.full_like(ids, -1)).to(torch.int32), "weights": w}
    if st["dweights"] is not None:
        dw = torch.where(there, st["dweights"], torch.zeros_like(w))
        ds = c["scale"] * ((dw - (chosen / total * dw).sum(dim=1, keepdim=True)) / total if c["renorm"] else dw)
        ds = torch.where(there, ds, torch.zeros_like(ds))
        du = torch.zeros_like(x).scatter_add_(1, ids, ds)
        dx = s * (du - (s * du).sum(dim=1, keepdim=True)) if c["score"] == "softmax" else du * s * (1.0 - s)
        out["dlogits"] = dx.to(st["logits"].dtype)
    return out


def _plain_layout(st):
    """(rows, sources, experts of the rows, counts): as elementary sorts and sums."""
    c = st["case"]
    t, k, e = c["tokens"], c["top_k"], c["experts"]
    ids = st["ids"].reshape(-1).long()
    dev, n = ids.device, ids.numel()
    key = torch.where(ids < 0, torch.full_like(ids, e), ids)
    order = torch.sort(key, stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.int64, device=dev).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(count, 0) - count
    rank = torch.empty_like(key).scatter_(0, order, torch.arange(n, device=dev)) - first[key]
    if c["rows"]:
        total = e * c["rows"]
        start = torch.arange(e + 1, device=dev) * c["rows"]
        there = (ids >= 0) & (rank < c["rows"])
        of_row = None
    else:
        total = _rows_capacity(t, k, e)
        padded = (count + BLOCK - 1) // BLOCK * BLOCK
        end = torch.cumsum(padded[:e], 0)
        start = torch.cumsum(padded, 0) - padded
        there = ids >= 0
        row = torch.arange(total, device=dev)
        of_row = torch.searchsorted(end, row, right=True)
        of_row = torch.where(of_row == e, torch.full_like(of_row, -1), of_row)
    rows = torch.where(there, start[key] + rank, torch.full_like(key, -1))
    sources = torch.full((total + 1,), -1, dtype=torch.int64, device=dev)
    sources.scatter_(0, torch.where(there, rows, torch.full_like(rows, total)), torch.arange(n, device=dev))
    return rows, sources[:total], of_row, count[:e]


def _plain_experts(st):
    c = st["case"]
    t, k, h = c["tokens"], c["top_k"], c["hidden"]
    dtype = DTYPES[c["dtype"]]
    rows, sources, of_row, count = _plain_layout(st)
    total, used = sources.numel(), sources >= 0
    written = used if of_row is None else of_row >= 0
    out = {"rows": rows.view(t, k).to(torch.int32), "counts": count.to(torch.int32)}
    if of_row is not None:
        out["m_indices"] = of_row.to(torch.int32)
    x = st["x"].float()
    xr = torch.where(used[:, None], x[sources.clamp_min(0) // k], torch.zeros((), device=x.device))
    lead = st["results"].shape[:-1]
    if c["form"] == "copy":
        out["xr"] = xr.to(dtype).view(*lead, h)
    elif c["form"] == "int8":
        q, s = _int8_codes(xr)
        out["q"] = q.view(*lead, h)
        out["s"] = torch.where(written, s, torch.zeros_like(s)).view(lead)
    else:
        kb = -(-h // BLOCK)
        grouped = torch.nn.functional.pad(xr, (0, kb * BLOCK - h)).view(total, kb, BLOCK)
        s = _amax_scale(grouped, 448.0)
        q = (grouped / s.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["q"] = q.view(total, kb * BLOCK)[:, :h].reshape(*lead, h)
        s = torch.where(written[:, None], s, torch.zeros_like(s))
        sa = torch.zeros_like(st["s"])
        sa[..., :lead[-1]] = s.view(*lead, kb).transpose(-1, -2)
        out["s"] = sa
    there = (rows >= 0).view(t, k)
    w = torch.where(there, st["weights"], torch.zeros_like(st["weights"]))
    back = st["results"].reshape(total, h)[rows.clamp_min(0)].view(t, k, h).float()
    out["y"] = (back * w.unsqueeze(-1)).sum(dim=1).to(dtype)
    if c["grad"]:
        dy = st["dy"].float()
        out["dweights"] = torch.where(there, (back * dy.unsqueeze(1)).sum(dim=2), torch.zeros_like(w))
        ws = w.reshape(-1)[sources.clamp_min(0)]
        dresults = dy[sources.clamp_min(0) // k] * ws[:, None]
        out["dresults"] = torch.where(used[:, None], dresults, torch.zeros_like(dresults)).to(dtype)
        dback = st["dxr"][rows.clamp_min(0)].view(t, k, h).float()
        out["dx"] = (dback * there.unsqueeze(-1)).sum(dim=1).to(dtype)
    return out


def _plain_int8(st):
    c = st["case"]
    dtype = DTYPES[c["out"]]
    if c["form"] == "normal":
        a, sa = _int8_codes(st["x"].float())
        d = torch.matmul(a.float(), st["b"].float().t())
        return {"d": (d * sa[:, None] * st["sb"][None, :]).to(dtype)}
    b, sb = st["b"], st["sb"]
    if c["form"] == "masked":
        d = torch.bmm(st["a"].float(), b.float().transpose(1, 2)) * st["sa"].unsqueeze(-1) * sb.unsqueeze(1)
        valid = torch.arange(c["m"], device=d.device)[None, :] < st["masked_m"][:, None]
        return {"d": torch.where(valid.unsqueeze(-1), d, torch.zeros_like(d)).to(dtype)}
    of_block = st["m_indices"].view(-1, BLOCK)[:, 0].long()
    blocks, at = of_block.numel(), of_block.clamp_min(0)
    d = torch.bmm(st["a"].float().view(blocks, BLOCK, c["k"]), b[at].float().transpose(1, 2))
    d = d * st["sa"].view(blocks, BLOCK, 1) * sb[at].unsqueeze(1)
    d = torch.where((of_block >= 0)[:, None, None], d, torch.zeros_like(d))
    return {"d": d.view(c["m"], c["n"]).to(dtype)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_route(st):
    import fp8_block_scaled_gemm_amd as dg
    c = st["case"]
    ids, w = dg.dg_moe_route(st["logits"], c["top_k"], bias=st["bias"], score=c["score"], num_groups=c["groups"],
                             topk_groups=c["topk_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                             scale=c["scale"])
    out = {"ids": ids, "weights": w}
    if st["dweights"] is not None:
        out["dlogits"] = dg.dg_moe_route_grad(st["dweights"], st["logits"], ids, score=c["score"],
                                              renormalize=c["renorm"], scale=c["scale"])
    return out


def _own_experts(st):
    import fp8_block_scaled_gemm_amd as dg
    c = st["case"]
    layout = dg.dg_moe_layout(st["ids"], c["experts"], rows_per_expert=c["rows"])
    out = {"rows": layout.rows, "counts": layout.counts}
    if not c["rows"]:
        out["m_indices"] = layout.m_indices
    if c["form"] == "copy":
        out["xr"] = dg.dg_moe_dispatch(st["x"], layout, out=st["xr"])
    elif c["form"] == "int8":
        out["q"], out["s"] = dg.dg_moe_dispatch_int8(st["x"], layout, q=st["q"], s=st["s"])
    else:
        q, out["s"] = dg.dg_moe_dispatch_fp8(st["x"], layout, q=st["q"], sa=st["s"])
        out["q"] = q.view(torch.float8_e4m3fn)
    out["y"] = dg.dg_moe_combine(st["results"], layout, weights=st["weights"])
    if c["grad"]:
        out["dresults"], out["dweights"] = dg.dg_moe_combine_grad(st["dy"], st["results"], layout, st["weights"],
                                                                  dout=st["dresults"])
        out["dx"] = dg.dg_moe_combine(st["dxr"], layout)
    return out


def _own_int8(st):
    import fp8_block_scaled_gemm_amd as dg
    c = st["case"]
    dtype = DTYPES[c["out"]]
    if c["form"] == "normal":
        return {"d": dg.dg_gemm_int8_nt_act_quant(st["x"], st["b"], st["sb"], out_dtype=dtype)}
    if c["form"] == "masked":
        return {"d": dg.dg_gemm_int8_grouped_masked(st["a"], st["sa"], st["b"], st["sb"], st["masked_m"], d=st["d"])}
    return {"d": dg.dg_gemm_int8_grouped_contiguous(st["a"], st["sa"], st["b"], st["sb"], st["m_indices"], d=st["d"])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "experts": _own_experts, "int8": _own_int8}[op](state)
    return {"route": _plain_route, "experts": _plain_experts, "int8": _plain_int8}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "route":
        t, e, k, size = case["tokens"], case["experts"], case["top_k"], BYTES[case["dtype"]]
        nbytes = t * e * size + 8 * t * k + (4 * e if case["bias"] else 0)
        if case["grad"]:
            nbytes += t * e * size + 4 * t * k
        return {"bytes": nbytes, "flops": 10 * t * e}
    if case["op"] == "experts":
        t, k, h, size = case["tokens"], case["top_k"], case["hidden"], BYTES[case["dtype"]]
        n = t * k   # rows, without the padding
        coded = {"copy": size, "int8": 1, "fp8": 1}[case["form"]]
        nbytes = 8 * n + t * h * size + n * h * coded + n * h * size + t * h * size + 4 * n
        flops = 2 * n * h
        if case["grad"]:
            nbytes += t * h * size + n * h * size + n * h * size + t * h * size + 4 * n
            flops += 5 * n * h
        return {"bytes": nbytes, "flops": flops}
    m, n, k, g = case["m"], case["n"], case["k"], case["groups"]
    rows = m
    if case["form"] == "masked":
        rows = g * m // 2   # rows in use: half of the buffers on the average
    elif case["form"] == "contiguous":
        rows = m - BLOCK
    size_in = BYTES[case["dtype"]] if case["form"] == "normal" else 1
    nbytes = rows * k * size_in + g * n * k + 4 * (rows + g * n) + rows * n * BYTES[case["out"]]
    return {"bytes": nbytes, "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_route(st):
    c = st["case"]
    x = st["logits"].double().cpu().numpy()
    t, e, k, g = c["tokens"], c["experts"], c["top_k"], c["groups"]
    ids = np.full((t, k), -1, dtype=np.int64)
    weights = np.zeros((t, k))
    dx = np.zeros((t, e))
    bias = st["bias"].double().cpu().numpy() if st["bias"] is not None else np.zeros(e)
    dw = st["dweights"].double().cpu().numpy() if st["dweights"] is not None else None
    for i in range(t):
        free = np.flatnonzero(x[i] != -np.inf)
        if not free.size:
            continue
        s = np.zeros(e)
        if c["score"] == "softmax":
            s[free] = np.exp(x[i, free] - x[i, free].max())
            s /= s.sum()
            value = x[i]
        else:
            s[free] = 1.0 / (1.0 + np.exp(-x[i, free]))
            value = s + bias
        if g > 1:
            size = e // g
            of_group = np.full(g, -np.inf)
            for j in range(g):
                mine = np.sort(value[free[free // size == j]])[::-1]
                if mine.size:
                    of_group[j] = mine[:c["group_top"]].sum()
            keep = np.argsort(-of_group, kind="stable")[:c["topk_groups"]]
            free = free[np.isin(free // size, keep)]
        pick = free[np.argsort(-value[free], kind="stable")[:k]]
        ids[i, :pick.size] = pick
        total = s[pick].sum() if c["renorm"] else 1.0
        weights[i, :pick.size] = c["scale"] * s[pick] / total
        if dw is not None:
            mine = dw[i, :pick.size]
            u = c["scale"] / total * (mine - ((s[pick] / total * mine).sum() if c["renorm"] else 0.0))
            if c["score"] == "softmax":
                dx[i] = -s * (s[pick] * u).sum()
                dx[i, pick] += s[pick] * u
            else:
                dx[i, pick] = u * s[pick] * (1.0 - s[pick])
    out = {"ids": None, "weights": torch.from_numpy(weights)}
    if dw is not None:
        out["dlogits"] = torch.from_numpy(dx)
    return out


def _exact_experts(st):
    c = st["case"]
    t, k, h, e = c["tokens"], c["top_k"], c["hidden"], c["experts"]
    ids = st["ids"].cpu().numpy()
    members = [np.flatnonzero(ids.reshape(-1) == j) for j in range(e)]
    total = st["results"].shape[:-1].numel()
    rows = np.full(t * k, -1, dtype=np.int64)
    written = np.zeros(total, dtype=bool)
    start = 0
    for j, who in enumerate(members):
        if c["rows"]:
            start, who = j * c["rows"], who[:c["rows"]]
            written[start:start + who.size] = True
        rows[who] = start + np.arange(who.size)
        if not c["rows"]:
            length = -(-who.size // BLOCK) * BLOCK
            written[start:start + length] = True
            start += length
    out = {"rows": None, "counts": None}
    if not c["rows"]:
        out["m_indices"] = None
    dev = st["x"].device
    at = torch.from_numpy(np.flatnonzero(rows >= 0)).to(dev)      # the (token, place) pairs that have a row
    row = torch.from_numpy(rows[rows >= 0]).to(dev)
    token = at // k
    x = st["x"].double()
    lead = st["results"].shape[:-1]
    if c["form"] == "copy":
        xr = torch.zeros((total, h), dtype=torch.float64, device=dev)
        xr[row] = x[token]
        out["xr"] = xr.view(*lead, h)
    else:
        width, limit = (h, 127.0) if c["form"] == "int8" else (BLOCK, 448.0)
        parts = [x[:, i:i + width].abs().amax(dim=1) for i in range(0, h, width)]
        of_token = torch.stack(parts, dim=1) / limit
        of_token = torch.where(of_token == 0, torch.ones_like(of_token), of_token)
        s = torch.zeros((total, of_token.shape[1]), dtype=torch.float64, device=dev)
        s[torch.from_numpy(np.flatnonzero(written)).to(dev)] = 1.0
        s[row] = of_token[token]
        out["q"] = None
        if c["form"] == "int8":
            out["s"] = s.view(lead)
        else:
            sa = torch.zeros(st["s"].shape, dtype=torch.float64, device=dev)
            sa[..., :lead[-1]] = s.view(*lead, -1).transpose(-1, -2)
            out["s"] = sa
    w = st["weights"].double().reshape(-1)
    results = st["results"].reshape(total, h)
    y = torch.zeros((t, h), dtype=torch.float64, device=dev)
    y.index_add_(0, token, results[row].double() * w[at][:, None])
    out["y"] = y
    if c["grad"]:
        dy = st["dy"].double()
        dweights = torch.zeros(t * k, dtype=torch.float64, device=dev)
        dweights[at] = (results[row].double() * dy[token]).sum(dim=1)
        out["dweights"] = dweights.view(t, k)
        dresults = torch.zeros((total, h), dtype=torch.float64, device=dev)
        dresults[row] = dy[token] * w[at][:, None]
        out["dresults"] = dresults
        dx = torch.zeros((t, h), dtype=torch.float64, device=dev)
        dx.index_add_(0, token, st["dxr"][row].double())
        out["dx"] = dx
    return out


def _exact_int8(st):
    c = st["case"]
    b, sb = st["b"].double(), st["sb"].double()
    if c["form"] == "normal":
        # the codes are part of the definition: fl32 scale, fl32 quotient, nearest even integer
        x = st["x"].float()
        amax = x.abs().amax(dim=1)
        sa = torch.where(amax == 0, torch.ones_like(amax), (amax.double() / 127.0).float())
        a = torch.round((x.double() / sa.double()[:, None]).float()).double()
        return {"d": a @ b.t() * (sa.double()[:, None] * sb[None, :])}
    d = torch.zeros(st["d"].shape, dtype=torch.float64, device=b.device)
    if c["form"] == "masked":
        for j, used in enumerate(st["masked_m"].tolist()):
            d[j, :used] = st["a"][j, :used].double() @ b[j].t() * (st["sa"][j, :used].double()[:, None] * sb[j][None, :])
    else:
        for j in range(c["groups"]):
            who = st["m_indices"] == j
            d[who] = st["a"][who].double() @ b[j].t() * (st["sa"][who].double()[:, None] * sb[j][None, :])
    return {"d": d}


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "int8": _exact_int8}[case["op"]](st)
