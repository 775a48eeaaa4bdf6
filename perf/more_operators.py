"""Cases and plain forms of the gated feed-forward products and of the fused residual norms.

Three operators, each in its plain form (elementary torch operations in 32 bits, rounded once at the end) and, where
``own`` is true, through the library's public calls:

* ``gated``  both projections of a gated feed-forward block from FP8 operands, the activation and the product:
             h = act(A * Bg^T) * (A * Bu^T), in its normal, contiguous-grouped and masked-grouped forms, as bf16, or as a
             whole block: h quantized on the way and multiplied by the block's last weight in FP8; with the projections' own
             values beside it where a training step keeps them;
* ``act``    the same activation and product on projections that exist already, and its backward pass: the gradient of both
             projections, or that gradient and h quantized in the layouts that the backward products read;
* ``norm``   what lies between two blocks: the norm after the first, its gate and residual scale, the residual sum and the
             norm before the second, quantized where an FP8 product follows, with the backward pass.
"""

import math

import torch

own = False

BLOCK = 128   # scale groups, weight blocks and the row alignment of the contiguous layout
E4M3_MAX = 448.0
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FP8 = torch.float8_e4m3fn
EPS = 1e-6


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence through one block: the weights are read once, latency counts
        dict(name="gated_token", op="gated", form="normal", m=1, n=2048, k=7168, groups=1, act="silu", out="block",
             pre=False),
        # ragged in every direction, the projections kept: a training step of an odd batch with the other activation
        dict(name="gated_ragged", op="gated", form="normal", m=777, n=1057, k=1552, groups=1, act="gelu", out="bf16",
             pre=True),
        # a long prompt through a wide dense block
        dict(name="gated_large", op="gated", form="normal", m=16384, n=8192, k=7168, groups=1, act="silu", out="bf16",
             pre=False),
        # 32 experts' decode buffers of 256 rows, between none and all of them in use
        dict(name="gated_masked", op="gated", form="masked", m=256, n=2048, k=7168, groups=32, act="silu", out="block",
             pre=False),
        # 8 experts' rows of a training step in the contiguous layout, a block of them unused, the projections kept
        dict(name="gated_contiguous", op="gated", form="contiguous", m=8192, n=2048, k=7168, groups=8, act="silu",
             out="block", pre=True),
        # the activation of 32 experts' decode buffers whose projections another product made
        dict(name="act_masked", op="act", form="masked", m=256, n=2048, groups=32, act="silu", out="fp8", dtype="bf16",
             grad=False),
        # the backward pass of a training step, everything that its FP8 products read in one pass over the inputs
        dict(name="act_train", op="act", form="normal", m=8192, n=2048, groups=1, act="silu", out="fp8", dtype="bf16",
             grad=True),
        # forward and backward in 32 bits on an odd batch
        dict(name="act_plain", op="act", form="normal", m=777, n=1040, groups=1, act="gelu", out="same", dtype="f32",
             grad=True),
        # one token between two blocks: latency
        dict(name="norm_token", op="norm", rows=1, hidden=7168, dtype="bf16", res="bf16", post=False, segments=0, scale=1.0,
             out="fp8", grad=False),
        # a prompt between two blocks, norms on both sides, the residual stream in 32 bits, FP8 products on both sides
        dict(name="norm_prompt", op="norm", rows=4096, hidden=7168, dtype="bf16", res="f32", post=True, segments=0, scale=0.5,
             out="fp8", grad=False),
        # a training step, an odd number of tokens: one learned gate for all of them, forward and backward
        dict(name="norm_train", op="norm", rows=8191, hidden=2048, dtype="bf16", res="bf16", post=True, segments=1, scale=1.0,
             out="same", grad=True),
        # 64 sequences of 251 tokens, each with a gate of its own, forward and backward
        dict(name="norm_segments", op="norm", rows=64 * 251, hidden=1536, dtype="f16", res="f32", post=False, segments=64,
             scale=1.0, out="same", grad=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step * 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("gated", "gated", "act", "norm"))
    act = rng.choice(("silu", "gelu"))
    if op == "gated":
        form = rng.choice(("normal", "normal", "masked", "contiguous"))
        out = rng.choice(("bf16", "block"))
        step = 16 if out == "block" else 1
        groups, m = 1, _log(rng, 1, 16384)
        n, k = _log(rng, 64, 8192, step), _log(rng, 128, 7168, 16)
        if form == "masked":
            n, groups, m = _log(rng, 64, 2048, step), _log(rng, 2, 32), _log(rng, 1, 256)
        elif form == "contiguous":
            n, groups, m = _log(rng, 64, 2048, step), _log(rng, 2, 32), BLOCK * _log(rng, 2, 64)
        return dict(op=op, form=form, m=m, n=n, k=k, groups=groups, act=act, out=out, pre=rng.random() < 0.4)
    if op == "act":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        grad = rng.random() < 0.6
        out = rng.choice(("same", "fp8"))
        if grad and out == "fp8":
            return dict(op=op, form="normal", m=_log(rng, 16, 8192, 16), n=_log(rng, 128, 4096, 128), groups=1, act=act,
                        out=out, dtype=dtype, grad=True)
        form = "normal" if grad else rng.choice(("normal", "masked", "contiguous"))
        n = _log(rng, 64, 4096, 16)
        groups, m = 1, _log(rng, 1, 8192)
        if form == "masked":
            groups, m = _log(rng, 2, 32), _log(rng, 1, 256)
        elif form == "contiguous":
            groups, m = _log(rng, 2, 32), BLOCK * _log(rng, 2, 64)
        return dict(op=op, form=form, m=m, n=n, groups=groups, act=act, out=out, dtype=dtype, grad=grad)
    grad = rng.random() < 0.5
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    segments = rng.choice((0, 1, _log(rng, 1, 64)))
    rows = max(1, _log(rng, 1, 16384) // max(1, segments)) * max(1, segments)
    if segments and rng.random() < 0.2:
        segments = rows   # a gate for each token
    return dict(op=op, rows=rows, hidden=_log(rng, 64, 7168, 16), dtype=dtype, res=rng.choice((dtype, "f32")),
                post=rng.random() < 0.5, segments=segments, scale=rng.choice((1.0, 0.5)),
                out="same" if grad else rng.choice(("same", "fp8")), grad=grad)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _amax_scale(x, limit):
    """amax / limit over the last dimension, 1 where it is zero (a division by a tensor: each quotient is rounded once)."""
    amax = x.abs().amax(dim=-1)
    return torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, limit))


def _fp8_rows(x):
    """(codes, scales (rows, ceil(k / 128))) of the 1 x 128 groups of float32 x (rows, k)."""
    rows, k = x.shape
    kb = -(-k // BLOCK)
    grouped = torch.nn.functional.pad(x, (0, kb * BLOCK - k)).view(rows, kb, BLOCK)
    s = _amax_scale(grouped, E4M3_MAX)
    q = (grouped / s.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(FP8)
    return q.view(rows, kb * BLOCK)[:, :k].contiguous(), s


def _fp8_blocks(w):
    """(codes, scales (mats, ceil(n / 128), ceil(k / 128))) of the 128 x 128 blocks of float32 w (mats, n, k)."""
    g, n, k = w.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    blocks = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(g, nb, BLOCK, kb, BLOCK)
    amax = blocks.abs().amax(dim=(2, 4))
    s = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, E4M3_MAX))
    q = (blocks / s[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(FP8)
    return q.view(g, nb * BLOCK, kb * BLOCK)[:, :n, :k].contiguous(), s


def _ld(rows):
    return -(-rows // 4) * 4


def _group_major(s, lead):
    """Scales (rows, groups) as a product reads them: (..., groups, rows rounded up to 4), zeros behind the last row."""
    rows, kb = lead[-1], s.shape[-1]
    out = torch.zeros((*lead[:-1], kb, _ld(rows)), dtype=torch.float32, device=s.device)
    out[..., :rows] = s.view(*lead, kb).transpose(-1, -2)
    return out


def _activations(rand, m, k):
    """N(0, 1), with one row of a hundred (one at least) 100 times larger."""
    x = rand(m, k)
    if m > 1:
        big = torch.arange(m, device=x.device) % 100 == 7 % m
        x = torch.where(big[:, None], x * 100.0, x)
    return x


def prepare(case, seed):
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 2 + 1)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev, dtype=torch.float32)

    def zeros(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=dev)

    st = {"case": dict(case)}
    if case["op"] == "norm":
        t, h = case["rows"], case["hidden"]
        dtype, res = DTYPES[case["dtype"]], DTYPES[case["res"]]
        st["x"] = _activations(rand, t, h).to(dtype)
        st["residual"] = (rand(t, h) * 2.0).to(res)
        st["weight"] = 1.0 + 0.1 * rand(h)
        st["post_weight"] = 1.0 + 0.1 * rand(h) if case["post"] else None
        st["gate"] = (0.5 * rand(case["segments"], h)).to(dtype) if case["segments"] else None
        if case["grad"]:
            # the backward pass reads a sum that a forward pass stored, the rounding to its type included
            st["sum"] = (st["residual"].float() + case["scale"] * st["x"].float()).to(res)
            st["dy"] = rand(t, h).to(dtype)
            st["dsum"] = rand(t, h).to(res)
        if case["out"] == "fp8":
            st["q"] = zeros((t, h), torch.uint8)
            st["s"] = zeros((-(-h // BLOCK), _ld(t)), torch.float32)
        return st

    form, m, n, g = case["form"], case["m"], case["n"], case["groups"]
    lead = (g, m) if form == "masked" else (m,)
    rows = g * m if form == "masked" else m
    st["m_indices"] = st["masked_m"] = None
    if form == "masked":
        st["masked_m"] = (uniform(g) * (m + 1)).to(torch.int32)
    elif form == "contiguous":
        expert = (torch.sort(uniform(m // BLOCK)).values * g).to(torch.int32).clamp(0, g - 1)
        expert[-1] = -1   # a block behind the last expert's rows
        st["m_indices"] = expert.repeat_interleave(BLOCK).contiguous()
    if case["op"] == "gated":
        k = case["k"]
        q, s = _fp8_rows(_activations(rand, rows, k).to(torch.bfloat16).float())
        st["a"], st["sa"] = q.view(*lead, k), _group_major(s, lead)
        experts = 1 if form == "normal" else g
        parts = [_fp8_blocks(rand(2, n, k) * 0.02) for _ in range(experts)]
        st["b"], st["sb"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        if form == "normal":
            st["b"], st["sb"] = st["b"][0], st["sb"][0]
        if case["pre"]:
            st["pre"] = zeros((*lead, 2 * n), torch.bfloat16)
        if case["out"] == "block":
            parts = [_fp8_blocks(rand(1, k, n) * 0.02) for _ in range(experts)]
            st["b_out"], st["sb_out"] = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
            if form == "normal":
                st["b_out"], st["sb_out"] = st["b_out"][0], st["sb_out"][0]
            st["y"] = zeros((*lead, k), torch.bfloat16)
    else:
        dtype = DTYPES[case["dtype"]]
        st["pre"] = (rand(*lead, 2 * n) * 1.5).to(dtype)
        if case["grad"]:
            st["dh"] = rand(*lead, n).to(dtype)
    if case["out"] == "fp8":
        st["q"] = zeros((*lead, n), torch.uint8)
        st["s"] = zeros((*lead[:-1], -(-n // BLOCK), _ld(m)), torch.float32)
    elif case["out"] != "block":
        st["h"] = zeros((*lead, n), torch.bfloat16 if case["op"] == "gated" else DTYPES[case["dtype"]])
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

GELU_C = 2.0 * math.sqrt(2.0 / math.pi)


def _plain_act(g, act):
    """g * sigmoid(g), or the tanh form of GELU: 0.5 (1 + tanh(z)) = sigmoid(2 z)."""
    z = g if act == "silu" else GELU_C * (g + 0.044715 * g * g * g)
    return g / (1.0 + torch.exp(-z))


def _plain_act_slope(g, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p * (1.0 + g * (1.0 - p))
    p = 1.0 / (1.0 + torch.exp(-GELU_C * (g + 0.044715 * g * g * g)))
    return p + g * p * (1.0 - p) * (GELU_C * (1.0 + 3.0 * 0.044715 * g * g))


def _used(st):
    """Truth values over the rows: those that the layout computes (None: all)."""
    c = st["case"]
    if c["form"] == "masked":
        return torch.arange(c["m"], device=st["masked_m"].device)[None, :] < st["masked_m"][:, None]
    return st["m_indices"] >= 0 if c["form"] == "contiguous" else None


def _only(x, used):
    return x if used is None else torch.where(used.unsqueeze(-1), x, torch.zeros_like(x))


def _plain_out(h, c, used):
    """h (float32, rows with leading dimensions) as the case's output, unused rows zero."""
    lead, n = h.shape[:-1], h.shape[-1]
    if c["out"] == "fp8":
        q, s = _fp8_rows(_only(h, used).reshape(-1, n))
        s = _only(s.view(*lead, -1), used)
        return {"q": q.view(*lead, n), "s": _group_major(s, lead)}
    return {"h": _only(h, used).to(DTYPES[c["dtype"]])}


def _spread(s, rows, k):
    """Block scales (..., rows / 128, k / 128) for each element."""
    return s.repeat_interleave(BLOCK, dim=-2)[..., :rows, :].repeat_interleave(BLOCK, dim=-1)[..., :k]


def _plain_product(a, b, st):
    """float32 a (rows with leading dimensions, k) times each row's weight in b ([groups,] n, k)."""
    c = st["case"]
    if c["form"] == "contiguous":
        of_block = st["m_indices"].view(-1, BLOCK)[:, 0].long().clamp_min(0)
        return torch.bmm(a.view(-1, BLOCK, a.shape[-1]), b[of_block].transpose(1, 2)).view(c["m"], b.shape[1])
    if c["form"] == "masked":
        return torch.bmm(a, b.transpose(1, 2))
    return torch.matmul(a, b.t())


def _plain_gated(st):
    c = st["case"]
    m, n, k = c["m"], c["n"], c["k"]
    sa = st["sa"][..., :m].transpose(-1, -2).repeat_interleave(BLOCK, dim=-1)[..., :k]
    b = (st["b"].float() * _spread(st["sb"], n, k)).flatten(-3, -2)   # gate and up rows of one expert together
    used = _used(st)
    pre = _plain_product(st["a"].float() * sa, b, st)
    h = _plain_act(pre[..., :n], c["act"]) * pre[..., n:]
    if c["out"] == "block":
        lead = h.shape[:-1]
        q, s = _fp8_rows(_only(h, used).reshape(-1, n))
        h = (q.float() * s.repeat_interleave(BLOCK, dim=1)[:, :n]).view(*lead, n)
        y = _plain_product(h, st["b_out"].float() * _spread(st["sb_out"], k, n), st)
        out = {"y": _only(y, used).to(torch.bfloat16)}
    else:
        out = {"h": _only(h, used).to(torch.bfloat16)}
    if c["pre"]:
        out["pre"] = _only(pre, used).to(torch.bfloat16)
    return out


def _plain_gated_act(st):
    c = st["case"]
    pre = st["pre"].float()
    n = c["n"]
    g, u = pre[..., :n], pre[..., n:]
    h = _plain_act(g, c["act"]) * u
    if not c["grad"]:
        return _plain_out(h, c, _used(st))
    dh = st["dh"].float()
    dpre = torch.cat((dh * u * _plain_act_slope(g, c["act"]), dh * _plain_act(g, c["act"])), dim=-1)
    if c["out"] == "same":
        return {"h": h.to(st["pre"].dtype), "dpre": dpre.to(st["pre"].dtype)}
    q, s = _fp8_rows(dpre)
    qt, stt = _fp8_rows(dpre.t())
    ht, sht = _fp8_rows(h.t())
    return {"q": q, "s": _group_major(s, (c["m"],)), "qt": qt, "st": _group_major(stt, (2 * n,)), "ht": ht,
            "sht": _group_major(sht, (n,))}


def _plain_norm(st):
    c = st["case"]
    t, h = c["rows"], c["hidden"]
    dtype, res, alpha = DTYPES[c["dtype"]], DTYPES[c["res"]], c["scale"]
    w, v = st["weight"], st["post_weight"]
    x = st["x"].float()
    gate = None
    if c["segments"]:
        gate = st["gate"].float().repeat_interleave(t // c["segments"], dim=0)

    def rms(a):
        return torch.rsqrt((a * a).mean(dim=1, keepdim=True) + EPS)

    xn = x * rms(x) if c["post"] else x
    z = xn * v if c["post"] else x
    gz = z if gate is None else z * gate
    total = st["residual"].float() + alpha * gz
    y = total * rms(total) * w
    out = {"sum": total.to(res)}
    if c["out"] == "fp8":
        out["y"], s = _fp8_rows(y)
        out["s"] = _group_major(s, (t,))
    else:
        out["y"] = y.to(dtype)
    if c["grad"]:
        u, dy = st["sum"].float(), st["dy"].float()
        rho = rms(u)
        dyw = dy * w
        du = st["dsum"].float() + rho * (dyw - u * (rho * rho) * (dyw * u).mean(dim=1, keepdim=True))
        out["dweight"] = (dy * u * rho).sum(dim=0, dtype=torch.float64).float()
        out["dresidual"] = du.to(res)
        dz = alpha * du if gate is None else alpha * du * gate
        if gate is not None:
            dgate = (alpha * du * z).view(c["segments"], -1, h)
            out["dgate"] = dgate.sum(dim=1, dtype=torch.float64).to(dtype)
        if c["post"]:
            sigma = rms(x)
            out["dpost"] = (dz * xn).sum(dim=0, dtype=torch.float64).float()
            dzv = dz * v
            dz = sigma * (dzv - x * (sigma * sigma) * (dzv * x).mean(dim=1, keepdim=True))
        out["dx"] = dz.to(dtype)
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_out(got, out):
    if out == "fp8":
        return {"q": got[0].view(FP8), "s": got[1]}
    return {"h": got}


def _own_gated(st):
    import fp8_block_scaled_gemm_amd as dg
    c = st["case"]
    operands, form = (st["a"], st["sa"], st["b"], st["sb"]), c["form"]
    where = () if form == "normal" else (st["masked_m"] if form == "masked" else st["m_indices"],)
    gated = {"normal": dg.dg_gemm_fp8_gated_nt, "masked": dg.dg_gemm_fp8_gated_masked,
             "contiguous": dg.dg_gemm_fp8_gated_contiguous}[form]
    if c["out"] == "block":
        q, s = gated(*operands, *where, act=c["act"], out="fp8", pre=st.get("pre"))
        product = {"normal": dg.dg_gemm_fp8_nt, "masked": dg.dg_gemm_fp8_grouped_masked,
                   "contiguous": dg.dg_gemm_fp8_grouped_contiguous}[form]
        out = {"y": product(q, s, st["b_out"], st["sb_out"], *where, d=st["y"])}
    else:
        out = {"h": gated(*operands, *where, act=c["act"], d=st["h"], pre=st.get("pre"))}
    if c["pre"]:
        out["pre"] = st["pre"]
    return out


def _own_gated_act(st):
    import fp8_block_scaled_gemm_amd as dg
    c = st["case"]
    if c["grad"] and c["out"] == "fp8":
        q, s, qt, stt, ht, sht = dg.dg_gated_act_grad_fp8(st["dh"], st["pre"], act=c["act"])
        return {"q": q.view(FP8), "s": s, "qt": qt.view(FP8), "st": stt, "ht": ht.view(FP8), "sht": sht}
    where = dict(m_indices=st["m_indices"], masked_m=st["masked_m"])
    if c["out"] == "fp8":
        return _own_out(dg.dg_gated_act_fp8(st["pre"], act=c["act"], q=st["q"], s=st["s"], **where), "fp8")
    out = {"h": dg.dg_gated_act(st["pre"], act=c["act"], h=st["h"], **where)}
    if c["grad"]:
        out["dpre"] = dg.dg_gated_act_grad(st["dh"], st["pre"], act=c["act"])
    return out


def _own_norm(st):
    import fp8_block_scaled_gemm_amd as dg
    c = st["case"]
    how = dict(gate=st["gate"], post_norm=c["post"], post_weight=st["post_weight"], scale=c["scale"], eps=EPS)
    if c["out"] == "fp8":
        total, q, s = dg.dg_residual_norm_fp8(st["x"], st["residual"], st["weight"], q=st["q"], s=st["s"], **how)
        return {"sum": total, "y": q.view(FP8), "s": s}
    total, y = dg.dg_residual_norm(st["x"], st["residual"], st["weight"], **how)
    out = {"sum": total, "y": y}
    if c["grad"]:
        got = dg.dg_residual_norm_grad(st["dy"], st["dsum"], st["x"], st["sum"], st["weight"], **how)
        out["dx"], out["dresidual"], out["dweight"] = got.dx, got.dresidual, got.dweight
        if c["segments"]:
            out["dgate"] = got.dgate
        if c["post"]:
            out["dpost"] = got.dpost_weight
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gated": _own_gated, "act": _own_gated_act, "norm": _own_norm}[op](state)
    return {"gated": _plain_gated, "act": _plain_gated_act, "norm": _plain_norm}[op](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        t, h, size, res = case["rows"], case["hidden"], BYTES[case["dtype"]], BYTES[case["res"]]
        gates = case["segments"] * h * size
        nbytes = t * h * (size + 2 * res) + 4 * h + (4 * h if case["post"] else 0) + gates
        nbytes += t * h + 4 * t * -(-h // BLOCK) if case["out"] == "fp8" else t * h * size
        flops = 10 * t * h
        if case["grad"]:   # dy, dsum, x and the sum in, dx and dresidual out, and the gradients of what is shared
            nbytes += t * h * (3 * size + 3 * res) + 8 * h + (8 * h if case["post"] else 0) + 2 * gates
            flops += 25 * t * h
        return {"bytes": nbytes, "flops": flops}
    m, n, g = case["m"], case["n"], case["groups"]
    rows = g * m // 2 if case["form"] == "masked" else m - BLOCK if case["form"] == "contiguous" else m
    out = rows * n + 4 * rows * -(-n // BLOCK)
    if case["op"] == "gated":
        k, experts = case["k"], 1 if case["form"] == "normal" else g
        nbytes = rows * k + 4 * rows * -(-k // BLOCK) + experts * 2 * n * k
        nbytes += 4 * rows * n if case["pre"] else 0
        if case["out"] == "block":   # the quantized h between the two products can stay on the chip
            return {"bytes": nbytes + experts * n * k + 2 * rows * k, "flops": 6 * rows * n * k}
        return {"bytes": nbytes + 2 * rows * n, "flops": 4 * rows * n * k}
    size = BYTES[case["dtype"]]
    if not case["grad"]:
        return {"bytes": 2 * rows * n * size + (out if case["out"] == "fp8" else rows * n * size), "flops": 8 * rows * n}
    if case["out"] == "fp8":
        return {"bytes": 3 * rows * n * size + 5 * rows * n + 5 * rows * n // 32, "flops": 30 * rows * n}
    return {"bytes": 2 * rows * n * size + rows * n * size + 5 * rows * n * size, "flops": 30 * rows * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_scales(h, lead, keep=None):
    """Group-major scales of float64 h (rows, n): the largest magnitude of each 128 over 448, 1 for none, 0 for unused rows."""
    rows, n = h.shape
    s = torch.stack([h[:, i:i + BLOCK].abs().amax(dim=1) for i in range(0, n, BLOCK)], dim=1) / E4M3_MAX
    s[s == 0] = 1.0
    if keep is not None:
        s[~keep.reshape(-1)] = 0.0
    out = torch.zeros((*lead[:-1], s.shape[1], _ld(lead[-1])), dtype=torch.float64, device=h.device)
    out[..., :lead[-1]] = s.view(*lead, -1).transpose(-1, -2)
    return out


def _exact_act(g, act):
    """(activation, slope) in 64 bits, by the hyperbolic tangent."""
    if act == "silu":
        half = torch.tanh(0.5 * g)
        p = 0.5 * (1.0 + half)
        return g * p, p + 0.25 * g * (1.0 - half * half)
    root = math.sqrt(2.0 / math.pi)
    th = torch.tanh(root * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * root * (1.0 + 0.134145 * g ** 2)


def _exact_product(codes, row_scales, weights, block_scales):
    """codes (m, k) with scales (m, k / 128) times weights (n, k) with block scales, 128 of k at a time."""
    m, k = codes.shape
    d = torch.zeros((m, weights.shape[0]), dtype=torch.float64, device=codes.device)
    for j, i in enumerate(range(0, k, BLOCK)):
        part = codes[:, i:i + BLOCK].double() @ weights[:, i:i + BLOCK].double().t()
        of_col = block_scales[:, j].double().repeat_interleave(BLOCK)[:weights.shape[0]]
        d += part * row_scales[:, j].double()[:, None] * of_col[None, :]
    return d


def _exact_gated(st):
    c = st["case"]
    m, n, k = c["m"], c["n"], c["k"]
    dev = st["a"].device
    lead = st["a"].shape[:-1]
    rows, row = lead.numel(), torch.arange(lead.numel(), device=dev)
    if c["form"] == "normal":
        todo = [(row, st["sa"][:, :m].t(), ...)]
    elif c["form"] == "masked":
        todo = [(row[j * m:j * m + used], st["sa"][j, :, :used].t(), j) for j, used in enumerate(st["masked_m"].tolist())]
    else:
        todo = [(row[st["m_indices"] == j], st["sa"][:, :m].t()[st["m_indices"] == j], j) for j in range(c["groups"])]
    wide = lambda width: torch.zeros((rows, width), dtype=torch.float64, device=dev)   # noqa: E731
    pre, h, y = wide(2 * n), wide(n), wide(k if c["out"] == "block" else 0)
    for who, sa, j in todo:
        codes, b, sb = st["a"].reshape(rows, k)[who], st["b"][j], st["sb"][j]
        for half in (0, 1):
            pre[who, half * n:(half + 1) * n] = _exact_product(codes, sa, b[half], sb[half])
        h[who] = _exact_act(pre[who, :n], c["act"])[0] * pre[who, n:]
        if c["out"] == "block":
            # the codes are part of the definition: the nearest E4M3 value of h over its group's scale
            mine = h[who]
            s = torch.stack([mine[:, i:i + BLOCK].abs().amax(dim=1) for i in range(0, n, BLOCK)], dim=1) / E4M3_MAX
            s[s == 0] = 1.0
            of_col = s.repeat_interleave(BLOCK, dim=1)[:, :n]
            y[who] = _exact_product((mine / of_col).float().clamp(-E4M3_MAX, E4M3_MAX).to(FP8), s, st["b_out"][j],
                                    st["sb_out"][j])
    out = {"y": y.view(*lead, k)} if c["out"] == "block" else {"h": h.view(*lead, n)}
    if c["pre"]:
        out["pre"] = pre.view(*lead, 2 * n)
    return out


def _exact_gated_act(st):
    c = st["case"]
    n, lead = c["n"], st["pre"].shape[:-1]
    pre = st["pre"].double().reshape(-1, 2 * n)
    f, slope = _exact_act(pre[:, :n], c["act"])
    h = f * pre[:, n:]
    if c["grad"]:
        dh = st["dh"].double()
        dpre = torch.cat((dh * pre[:, n:] * slope, dh * f), dim=1)
        if c["out"] == "same":
            return {"h": h, "dpre": dpre}
        return {"q": None, "s": _exact_scales(dpre, (c["m"],)), "qt": None, "st": _exact_scales(dpre.t(), (2 * n,)),
                "ht": None, "sht": _exact_scales(h.t(), (n,))}
    keep = torch.ones(h.shape[0], dtype=torch.bool, device=h.device)
    if c["form"] == "masked":
        for j, used in enumerate(st["masked_m"].tolist()):
            keep[j * c["m"] + used:(j + 1) * c["m"]] = False
    elif c["form"] == "contiguous":
        keep = st["m_indices"] != -1
    h[~keep] = 0.0
    if c["out"] == "fp8":
        return {"q": None, "s": _exact_scales(h, lead, keep)}
    return {"h": h.view(*lead, n)}


def _exact_norm(st):
    c = st["case"]
    t, h, seg = c["rows"], c["hidden"], c["segments"]
    x, r, w = st["x"].double(), st["residual"].double(), st["weight"].double()
    size = lambda a: torch.sqrt(a.square().sum(dim=1, keepdim=True) / h + EPS)   # noqa: E731
    gate = torch.ones((1, h), dtype=torch.float64, device=x.device)
    if seg:
        gate = st["gate"].double()[torch.arange(t, device=x.device) * seg // t]
    v = st["post_weight"].double() if c["post"] else torch.ones(h, dtype=torch.float64, device=x.device)
    unit = x / size(x) if c["post"] else x
    total = r + c["scale"] * gate * unit * v
    y = total / size(total) * w
    out = {"sum": total}
    if c["out"] == "fp8":
        out["y"], out["s"] = None, _exact_scales(y, (t,))
    else:
        out["y"] = y
    if c["grad"]:
        stored = st["sum"].double()
        dy, length = st["dy"].double(), size(stored)
        unit_sum = stored / length
        dunit = dy * w
        du = (dunit - unit_sum * (dunit * unit_sum).sum(dim=1, keepdim=True) / h) / length + st["dsum"].double()
        out["dweight"] = (dy * unit_sum).sum(dim=0)
        out["dresidual"] = du
        if seg:
            dgate = torch.zeros((seg, h), dtype=torch.float64, device=x.device)
            out["dgate"] = dgate.index_add_(0, torch.arange(t, device=x.device) * seg // t, c["scale"] * du * unit * v)
        dz = c["scale"] * du * gate
        if c["post"]:
            out["dpost"] = (dz * unit).sum(dim=0)
            dn = dz * v
            dz = (dn - unit * (dn * unit).sum(dim=1, keepdim=True) / h) / size(x)
        out["dx"] = dz
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"gated": _exact_gated, "act": _exact_gated_act, "norm": _exact_norm}[case["op"]](st)
