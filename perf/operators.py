"""What is measured of the serving operators with few tokens or four-bit experts.

Three kinds of case:

  few        the whole mixture-of-experts layer for 1 to 16 tokens
             (moe_layer_forward_few): bf16, FP8 with block scales, and MXFP4
             expert weights;
  roundtrip  a matrix into MXFP4 and back (moe_mxfp4_quantize,
             moe_mxfp4_dequantize): what a user runs to see what four bits
             cost a tensor before serving it;
  product    the grouped product on MXFP4 operands (moe_mxfp4_matmul): one
             linear layer over expert segments ("layers" 1), or the experts'
             FFN, whose hidden activation stays in MXFP4 between the two
             products ("layers" 2).  The activations are quantised within the
             call, the weights once beforehand.

`own` False computes the operators from elementary torch operations; `own`
True calls this repository's package.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn


def listed():
    return [
        # one decoded token through a DeepSeek-V3-shaped layer whose experts are held in four bits
        few_case("few_mxfp4_1", "mxfp4", 1, 7168, 256, 8, 2048, 1, 2048),
        # sixteen sequences decoding together through the same layer
        few_case("few_mxfp4_16", "mxfp4", 16, 7168, 256, 8, 2048, 1, 2048),
        # one decoded token, FP8 experts with 128x128 block scales
        few_case("few_fp8_1", "fp8", 1, 7168, 256, 8, 2048, 1, 2048),
        # sixteen tokens, FP8 experts: the largest call of the few-token form
        few_case("few_fp8_16", "fp8", 16, 7168, 256, 8, 2048, 1, 2048),
        # a few tokens through a fine-grained bf16 layer with two shared experts and a capacity limit
        few_case("few_bf16_5_capacity", "bf16", 5, 2048, 64, 8, 1408, 2, 1408, cf=1.25),
        # eight tokens through a Mixtral-8x7B-shaped bf16 layer (few wide experts)
        few_case("few_bf16_8_wide", "bf16", 8, 4096, 8, 2, 14336, 0, 0),
        # the smallest call: one token through the tiny layer, where latency counts
        few_case("few_bf16_1_tiny", "bf16", 1, 128, 8, 2, 256, 0, 0),
        # a ragged handful of activation rows
        {"name": "roundtrip_37", "op": "roundtrip", "rows": 37, "cols": 2080, "type": "f32"},
        # one prompt's activations, or a slice of a weight stack
        {"name": "roundtrip_16k", "op": "roundtrip", "rows": 16384, "cols": 7168, "type": "bf16"},
        # a 4096-token prompt through the 256 experts of the V3-shaped layer (32768 rows)
        {"name": "experts_prefill", "op": "product", "layers": 2, "rows": 32768, "behind": 0, "k": 7168, "n": 2048,
         "mats": 256, "segs": 256, "skew": 0.3, "out": "bf16"},
        # 128 decoding tokens, eight experts each: a few rows per expert, some experts empty
        {"name": "experts_decode", "op": "product", "layers": 2, "rows": 1024, "behind": 24, "k": 7168, "n": 2048,
         "mats": 256, "segs": 256, "skew": 1.2, "out": "bf16"},
        # a Mixtral-shaped first layer over a prompt, bound by the tensor cores; fp32 results, odd row counts
        {"name": "product_wide", "op": "product", "layers": 1, "rows": 8191, "behind": 3, "k": 4096, "n": 14336,
         "mats": 8, "segs": 8, "skew": 0.3, "out": "f32"},
    ]


def few_case(name, weights, T, d, E, K, dff, S, dffs, cf=0.0, overflow=0, bias=0):
    """One case of the few-token layer; cf: capacity factor (0: none), overflow 1: dropped slots pass the token
    through, bias 1: per-expert logit bias, 2: the same for the selection only."""
    return {"name": name, "op": "few", "weights": weights, "T": T, "d": d, "E": E, "K": K, "dff": dff, "S": S,
            "dffs": dffs, "cf": cf, "overflow": overflow, "bias": bias}


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return min(hi, max(lo, int(v) // step * step))


def draw(rng):
    kind = rng.choice(["few", "few", "few", "roundtrip", "product", "product"])
    if kind == "roundtrip":
        return {"op": "roundtrip", "rows": _log(rng, 1, 16384), "cols": _log(rng, 32, 7168, 32),
                "type": rng.choice(["f32", "bf16"])}
    if kind == "product":
        layers = rng.choice([1, 2])
        mats = _log(rng, 1, 256)
        k, n = _log(rng, 128, 7168, 128), _log(rng, 128, 2048, 128 if layers == 2 else 32)
        return {"op": "product", "layers": layers, "rows": _log(rng, 1, 16384), "behind": rng.choice([0, 0, 5, 131]),
                "k": k, "n": n, "mats": mats, "segs": _log(rng, 1, 256), "skew": rng.uniform(0.0, 1.5),
                "out": "bf16" if layers == 2 else rng.choice(["bf16", "f32"])}
    weights = rng.choice(["mxfp4", "fp8", "bf16"])
    step = 64 if weights == "bf16" else 128
    most = 2048 * 7168 * (64 if weights == "bf16" else 256)
    while True:
        d, dff, E = _log(rng, 128, 7168, step), _log(rng, 128, 8192, step), _log(rng, 2, 256)
        if E * d * dff <= most:
            break
    T, K, S = rng.randint(1, 16), rng.randint(1, min(E, 8)), rng.choice([0, 0, 1, 2])
    dffs = _log(rng, 128, 2048, step) if S else 0
    cost = {"mxfp4": 17 / 32, "fp8": 1, "bf16": 2}[weights]
    while T > 1 and _touched(E, K, T) * d * dff * cost > 1.4e9:
        T -= 1
    c = few_case(None, weights, T, d, E, K, dff, S, dffs, cf=rng.choice([0.0, 0.0, 1.0, 1.25]),
                 overflow=rng.choice([0, 1]), bias=rng.choice([0, 0, 1, 2]))
    del c["name"]
    return c


def _touched(E, K, T):
    """Expected number of experts that T tokens reach with K of E each."""
    return E * (1.0 - (1.0 - K / E) ** T)


# ------------------------------------------------------------------ inputs

def _pow2(k):
    """2^k in fp32 for integers k in [-127, 127], exactly (a library pow may be an ulp off, which decides ties)."""
    return torch.where(k > -127, (k + 127).int() << 23, 0x400000).int().view(torch.float32)


def _encode4(v):
    """(..., 32 m) fp32 -> MXFP4: codes (two per byte, the even column in the low nibble) and E8M0 scale bytes, one
    per 32: the smallest power of two with |v| / scale <= 6 (1 for zeros)."""
    b = v.unflatten(-1, (-1, 32))
    m, e = torch.frexp(b.abs().amax(-1))
    k = torch.where(m == 0, 0, (e - 3 + (m > 0.75).int()).clamp(min=-126))
    a = (b * _pow2(-k).unsqueeze(-1)).flatten(-2)
    mag = a.abs()
    code = ((mag > 0.25).byte() + (mag >= 0.75).byte() + (mag > 1.25).byte() + (mag >= 1.75).byte()
            + (mag > 2.5).byte() + (mag >= 3.5).byte() + (mag > 5.0).byte())
    code = code | (torch.signbit(a).byte() << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), (k + 127).byte()


def _encode8(w):
    """(..., 128 r, 128 c) fp32 -> e4m3 codes and one power-of-two fp32 scale per 128x128 block."""
    b = w.unflatten(-2, (-1, 128)).unflatten(-1, (-1, 128))
    m, e = torch.frexp(b.abs().amax((-3, -1)))
    s = _pow2(e - 9 + (m > 0.875).int())
    q = (b / s[..., :, None, :, None]).to(F8)
    return q.flatten(-2).flatten(-3, -2).view(torch.uint8), s


def _stack(gen, n, rows, cols, kind):
    """n weight matrices ~ N(0, 1/cols) in the layer's form: (weights, scales or None)."""
    std, dev = 1.0 / math.sqrt(cols), "cuda"
    form = {"bf16": (cols, torch.bfloat16), "fp8": (cols, torch.uint8), "mxfp4": (cols // 2, torch.uint8)}[kind]
    w = torch.empty((n, rows, form[0]), dtype=form[1], device=dev)
    s = None
    if kind == "fp8":
        s = torch.empty((n, rows // 128, cols // 128), dtype=torch.float32, device=dev)
    elif kind == "mxfp4":
        s = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (rows * cols))
    for i in range(0, n, step):
        v = torch.empty((min(step, n - i), rows, cols), device=dev).normal_(0.0, std, generator=gen)
        if kind == "bf16":
            w[i:i + step] = v
        else:
            w[i:i + step], s[i:i + step] = (_encode8 if kind == "fp8" else _encode4)(v)
    return w, s


def _few_inputs(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape, std=1.0: torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen)  # noqa: E731
    T, d, E, K, dff, S, dffs = (c[k] for k in ("T", "d", "E", "K", "dff", "S", "dffs"))
    s = {"W_r": randn(E, d, std=1.0 / math.sqrt(d)), "logit_bias": randn(E, std=0.25) if c["bias"] else None}
    # Which of two experts with equal logits wins is a matter of the last bits of a sum: tokens that
    # come near such a border are drawn again.
    x = randn(T, d).bfloat16()
    for _ in range(50):
        key = x.double() @ s["W_r"].double().T
        if c["bias"]:
            key = key + s["logit_bias"].double()
        top = key.sort(dim=-1, descending=True).values[:, :min(E, K + 1)]
        near = (top[:, :-1] - top[:, 1:]).amin(-1) < 1e-4 if top.shape[1] > 1 else torch.zeros(T, device="cuda").bool()
        if not bool(near.any()):
            break
        x = torch.where(near[:, None], randn(T, d).bfloat16(), x)
    s["x"] = x
    s["W1"], s["W1_scales"] = _stack(gen, E, dff, d, c["weights"])
    s["b1"] = randn(E, dff, std=0.1)
    s["W2"], s["W2_scales"] = _stack(gen, E, d, dff, c["weights"])
    s["b2"] = randn(E, d, std=0.1)
    for k in ("Ws1", "Ws1_scales", "bs1", "Ws2", "Ws2_scales", "bs2"):
        s[k] = None
    if S:
        s["Ws1"], s["Ws1_scales"] = _stack(gen, S, dffs, d, c["weights"])
        s["bs1"] = randn(S, dffs, std=0.1)
        s["Ws2"], s["Ws2_scales"] = _stack(gen, S, d, dffs, c["weights"])
        s["bs2"] = randn(S, d, std=0.1)
    return s


def _segment_rows(c, gen):
    """Rows of each segment: shares that fall off with the segment's (shuffled) rank to the power of the skew."""
    n = c["segs"]
    rank = torch.randperm(n, generator=gen, device="cuda").double() + 1
    p = rank ** -c["skew"]
    pick = torch.multinomial(p, c["rows"], replacement=True, generator=gen)
    return torch.bincount(pick, minlength=n)


def _product_inputs(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape, std=1.0: torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen)  # noqa: E731
    R, k, n = c["rows"] + c["behind"], c["k"], c["n"]
    rows = _segment_rows(c, gen)
    s = {"sizes": rows.tolist()}
    s["seg_offsets"] = torch.cat([rows.new_zeros(1), rows.cumsum(0)]).int()
    mats = torch.randperm(max(c["mats"], c["segs"]), generator=gen, device="cuda")[:c["segs"]] % c["mats"]
    s["seg_mat"] = mats.int()
    s["mats"] = mats.tolist()
    # activations as they come out of a normalisation: a few columns are much larger than the rest
    x = randn(R, k)
    loud = torch.rand(k, generator=gen, device="cuda") < 0.01
    s["x"] = torch.where(loud, x * 8, x).bfloat16()
    s["w1"], s["w1_scales"] = _stack(gen, c["mats"], n, k, "mxfp4")
    s["b1"] = randn(c["mats"], n, std=0.1)
    if c["layers"] == 2:
        s["w2"], s["w2_scales"] = _stack(gen, c["mats"], k, n, "mxfp4")
        s["b2"] = randn(c["mats"], k, std=0.1)
    return s


def _roundtrip_inputs(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((c["rows"], c["cols"]), device="cuda").normal_(0.0, 1.0, generator=gen)
    # blocks of very different size, and some of zeros, as in a gradient or a pruned matrix
    size = torch.randint(-12, 13, (c["rows"], c["cols"] // 32), generator=gen, device="cuda")
    x = x * _pow2(size).repeat_interleave(32, dim=1)
    x = torch.where((size == 12).repeat_interleave(32, dim=1), torch.zeros_like(x), x)
    return {"x": x if c["type"] == "f32" else x.bfloat16()}


def prepare(case, seed):
    c = case
    state = {"few": _few_inputs, "product": _product_inputs, "roundtrip": _roundtrip_inputs}[c["op"]](c, seed)
    state["case"] = c
    if own:
        _prepare_own(state)
    return state


def _prepare_own(state):
    import sparse_mixture_experts_20_b200 as M
    c = state["case"]
    state["M"] = M
    u8 = dict(dtype=torch.uint8, device="cuda")
    if c["op"] == "few":
        cfg = M.make_config(T=c["T"], d_model=c["d"], n_routed=c["E"], top_k=c["K"], d_ff=c["dff"], n_shared=c["S"],
                            d_ff_shared=c["dffs"], capacity_factor=c["cf"], overflow_mode=c["overflow"],
                            bias_mode=M.MOE_BIAS_SELECTION if c["bias"] == 2 else M.MOE_BIAS_LOGITS,
                            dtype={"bf16": M.MOE_BF16, "fp8": M.MOE_FP8_E4M3_BLOCK, "mxfp4": M.MOE_MXFP4}[c["weights"]])
        state["layer"] = M.MoELayer(cfg, {k: v for k, v in state.items() if k not in ("case", "M", "x")})
    elif c["op"] == "roundtrip":
        rows, cols = c["rows"], c["cols"]
        state["codes"], state["scales"] = torch.empty((rows, cols // 2), **u8), torch.empty((rows, cols // 32), **u8)
        state["back"] = torch.empty_like(state["x"])
    else:
        R, k, n = state["x"].shape[0], c["k"], c["n"]
        two = c["layers"] == 2
        out = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        state["a"], state["a_scales"] = torch.empty((R, k // 2), **u8), torch.empty((R, k // 32), **u8)
        # rows behind the last segment stay as they are
        state["y"] = torch.zeros((R, k if two else n), dtype=out, device="cuda")
        outs = M.MOE_BF16 if c["out"] == "bf16" else M.MOE_F32
        common = dict(rows=R, n_mats=c["mats"], n_seg=c["segs"])
        state["first"] = M.make_mxfp4_shape(n=n, k=k, activation=M.MOE_ACT_SILU, out_dtype=M.MOE_MXFP4 if two else outs,
                                            **common)
        if two:
            state["h"], state["h_scales"] = torch.empty((R, n // 2), **u8), torch.empty((R, n // 32), **u8)
            state["second"] = M.make_mxfp4_shape(n=k, k=n, activation=M.MOE_ACT_NONE, out_dtype=outs, **common)
        state["ws"] = torch.empty(M.moe_mxfp4_workspace_size(state["first"]), **u8)
        M.moe_mxfp4_workspace_init(state["first"], state["ws"])


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"few": _own_few, "product": _own_product, "roundtrip": _own_roundtrip}[op](state)
    return {"few": _plain_few, "product": _plain_product, "roundtrip": _plain_roundtrip}[op](state)


def _own_few(s):
    layer = s["layer"]
    out, f, P, loss = layer.forward_few(s["x"])
    return {"out": out, "f": f, "P": P, "loss": loss, "topk_idx": layer.topk_idx, "gates": layer.gates,
            "counts": layer.counts}


def _own_roundtrip(s):
    M = s["M"]
    M.moe_mxfp4_quantize(s["x"], s["codes"], s["scales"])
    M.moe_mxfp4_dequantize(s["codes"], s["scales"], s["back"])
    return s["back"]


def _own_product(s):
    M = s["M"]
    M.moe_mxfp4_quantize(s["x"], s["a"], s["a_scales"])
    first = (s["first"], s["a"], s["a_scales"], s["seg_offsets"], s["seg_mat"], s["w1"], s["w1_scales"], s["b1"])
    if s["case"]["layers"] == 1:
        M.moe_mxfp4_matmul(*first, s["y"], None, s["ws"])
    else:
        M.moe_mxfp4_matmul(*first, s["h"], s["h_scales"], s["ws"])
        M.moe_mxfp4_matmul(s["second"], s["h"], s["h_scales"], s["seg_offsets"], s["seg_mat"], s["w2"], s["w2_scales"],
                           s["b2"], s["y"], None, s["ws"])
    return s["y"]


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _decode4(codes, scales):
    """MXFP4 -> fp32."""
    table = torch.tensor(_E2M1, device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    s = _pow2(scales.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def _decode8(codes, scales):
    b = codes.view(F8).float().unflatten(-2, (-1, 128)).unflatten(-1, (-1, 128))
    return (b * scales[..., :, None, :, None]).flatten(-2).flatten(-3, -2)


def _weights(w, scales, kind):
    if kind == "bf16":
        return w.float()
    return _decode4(w, scales) if kind == "mxfp4" else _decode8(w, scales)


def _quant8(v):
    """Rows through e4m3 with a power-of-two scale per 128 columns, fp32 values."""
    b = v.unflatten(-1, (-1, 128))
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    s = _pow2(torch.where(m == 0, 0, e - 9 + (m > 0.875).int()))
    return ((b / s).to(F8).float() * s).flatten(-2)


def _kept(idx, c):
    """Slots within the capacity, earlier tokens first."""
    if not c["cf"]:
        return torch.ones_like(idx, dtype=torch.bool)
    C = math.ceil(c["cf"] * c["T"] * c["K"] / c["E"])
    flat = idx.flatten()
    before = torch.tril(flat[:, None] == flat[None, :], diagonal=-1).sum(1)
    return (before < C).view(idx.shape)


def _plain_few(s):
    c = s["case"]
    T, E, K, kind = c["T"], c["E"], c["K"], c["weights"]
    xf = s["x"].float()
    # the choice of experts hangs on small differences of long sums: 64 bits
    logits = s["x"].double() @ s["W_r"].double().T
    if c["bias"] == 1:
        logits = logits + s["logit_bias"].double()
    key = logits + s["logit_bias"].double() if c["bias"] == 2 else logits
    idx = key.sort(dim=-1, descending=True, stable=True).indices[:, :K]
    p = (logits - logits.amax(-1, keepdim=True)).exp()
    p = (p / p.sum(-1, keepdim=True)).float()
    gates = p.gather(1, idx)
    gates = gates / gates.sum(-1, keepdim=True)
    counts = (idx.flatten()[:, None] == torch.arange(E, device=idx.device)).sum(0)
    f, P = counts.float() / (T * K), p.mean(0)
    loss = (0.01 * E * (f * P).sum()).reshape(1)
    kept = _kept(idx, c)

    def ffn(x, e, pre):
        """x (m, d) through matrices e (m,) of a stack."""
        w1 = _weights(s[pre + "1"][e], None if kind == "bf16" else s[pre + "1_scales"][e], kind)
        bias = "b" if pre == "W" else "bs"
        h = (w1 @ x.unsqueeze(-1)).squeeze(-1) + s[bias + "1"][e]
        del w1
        h = h * torch.sigmoid(h)
        if kind == "fp8":
            h = _quant8(h)
        w2 = _weights(s[pre + "2"][e], None if kind == "bf16" else s[pre + "2_scales"][e], kind)
        return (w2 @ h.unsqueeze(-1)).squeeze(-1) + s[bias + "2"][e]

    xq = _quant8(xf) if kind == "fp8" else xf
    out = torch.empty_like(xf)
    for t in range(T):
        y = ffn(xq[t].expand(K, -1), idx[t], "W")
        g = gates[t][:, None]
        over = g * xf[t] if c["overflow"] else torch.zeros_like(y)
        out[t] = torch.where(kept[t][:, None], g * y, over).sum(0)
    for i in range(c["S"]):
        w1 = _weights(s["Ws1"][i], None if kind == "bf16" else s["Ws1_scales"][i], kind)
        h = xq @ w1.T + s["bs1"][i]
        h = h * torch.sigmoid(h)
        h = _quant8(h) if kind == "fp8" else h
        out += h @ _weights(s["Ws2"][i], None if kind == "bf16" else s["Ws2_scales"][i], kind).T + s["bs2"][i]
    return {"out": out.bfloat16(), "f": f, "P": P, "loss": loss, "topk_idx": idx.int(), "gates": gates,
            "counts": counts.int()}


def _plain_roundtrip(s):
    x = s["x"]
    return _decode4(*_encode4(x.float())).to(x.dtype)


def _plain_product(s):
    c = s["case"]
    two = c["layers"] == 2
    a = _decode4(*_encode4(s["x"].float()))
    y = torch.zeros((a.shape[0], c["k"] if two else c["n"]), device="cuda",
                    dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    o = 0
    for r, m in zip(s["sizes"], s["mats"]):
        if r:
            z = a[o:o + r] @ _decode4(s["w1"][m], s["w1_scales"][m]).T + s["b1"][m]
            z = z * torch.sigmoid(z)
            if two:
                z = _decode4(*_encode4(z)) @ _decode4(s["w2"][m], s["w2_scales"][m]).T + s["b2"][m]
            y[o:o + r] = z
        o += r
    return y


# ------------------------------------------------------------------ what it costs

def work(case):
    c = case
    if c["op"] == "roundtrip":
        n, b = c["rows"] * c["cols"], 4 if c["type"] == "f32" else 2
        return {"bytes": n * (2 * b + 2 * 17 / 32), "flops": 4 * n}
    if c["op"] == "product":
        R, k, n = c["rows"], c["k"], c["n"]
        two = c["layers"] == 2
        # segments that expect a row bring their matrix in
        p = [(i + 1) ** -c["skew"] for i in range(c["segs"])]
        total = sum(p)
        reached = min(c["mats"], sum(1 - (1 - q / total) ** R for q in p))
        weights = reached * (n * k * 17 / 32 + 4 * n)
        o = 2 if c["out"] == "bf16" else 4
        size = R * k * 2 + R * k * 17 / 32 * 2 + weights
        size += R * n * 17 / 32 * 2 + reached * (n * k * 17 / 32 + 4 * k) + R * k * o if two else R * n * o
        return {"bytes": size, "flops": 2 * R * n * k * (2 if two else 1)}
    T, d, E, K, dff, S, dffs = (c[k] for k in ("T", "d", "E", "K", "dff", "S", "dffs"))
    per = {"bf16": 2.0, "fp8": 1.0 + 4 / 16384, "mxfp4": 17 / 32}[c["weights"]]
    reached = _touched(E, K, T)
    size = (reached * dff + S * dffs) * 2 * d * per + (reached * (dff + d) + S * (dffs + d)) * 4
    size += E * d * 4 + 2 * T * d * 2
    return {"bytes": size, "flops": 4 * d * T * (K * dff + S * dffs) + 2 * T * d * E}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _two(k):
    """2^k in fp64, from its exponent field."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _value4(codes, scales):
    """MXFP4 -> fp64 by the fields of a code: sign, two exponent bits, one mantissa bit."""
    n = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.int64, device=codes.device)
    n[..., 0::2], n[..., 1::2] = (codes % 16).long(), (codes // 16).long()
    exp, man = (n // 2) % 4, (n % 2).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * _two(exp - 1))
    v = torch.where(n >= 8, -mag, mag)
    return v * _two(scales.long() - 127).repeat_interleave(32, -1)


def _nearest4(v):
    """fp64 values rounded to MXFP4 blocks of 32: to the nearest of the grid, ties to the even mantissa."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.where(top == 0, 6.0, top) / 6))
    k = torch.where(top / _two(k) > 6, k + 1, torch.where(top / _two(k - 1) <= 6, k - 1, k))
    k = torch.where(top == 0, 0.0, k.clamp(min=-126))
    a = b.abs() / _two(k)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(b) * torch.round(a / step) * step * _two(k)).reshape(v.shape)


def _nearest8(v):
    b = v.reshape(*v.shape[:-1], -1, 128)
    top = b.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.where(top == 0, 448.0, top) / 448))
    k = torch.where(top / _two(k) > 448, k + 1, torch.where(top / _two(k - 1) <= 448, k - 1, k))
    a = b / _two(k)
    e = torch.frexp(a.abs().clamp(min=2.0 ** -6)).exponent - 1
    step = _two(e - 3)
    return (torch.round(a / step) * step * _two(k)).reshape(v.shape)


def _silu(z):
    return z / (1 + torch.exp(-z))


def exact(case, seed):
    c = case
    if c["op"] == "roundtrip":
        return _nearest4(_roundtrip_inputs(c, seed)["x"].double())
    if c["op"] == "product":
        s = _product_inputs(c, seed)
        two = c["layers"] == 2
        y = torch.zeros((s["x"].shape[0], c["k"] if two else c["n"]), dtype=torch.float64, device="cuda")
        ends = s["seg_offsets"].tolist()
        for i, m in enumerate(s["seg_mat"].tolist()):
            lo, hi = ends[i], ends[i + 1]
            if hi > lo:
                h = _silu(torch.addmm(s["b1"][m].double(), _nearest4(s["x"][lo:hi].double()),
                                      _value4(s["w1"][m], s["w1_scales"][m]).T))
                if two:
                    h = torch.addmm(s["b2"][m].double(), _nearest4(h), _value4(s["w2"][m], s["w2_scales"][m]).T)
                y[lo:hi] = h
        return y
    s = _few_inputs(c, seed)
    T, E, K, kind = c["T"], c["E"], c["K"], c["weights"]

    def matrix(name, i):
        if kind == "mxfp4":
            return _value4(s[name][i], s[name + "_scales"][i])
        if kind == "fp8":
            w = s[name][i].view(F8).double()
            return w * s[name + "_scales"][i].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return s[name][i].double()

    x = s["x"].double()
    logit = torch.einsum("td,ed->te", x, s["W_r"].double())
    logit = logit + (s["logit_bias"].double() if c["bias"] == 1 else 0)
    rank = logit + (s["logit_bias"].double() if c["bias"] == 2 else 0)
    prob = torch.softmax(logit, 1)
    chosen = [sorted(range(E), key=lambda e, r=r: (-r[e], e))[:K] for r in rank.tolist()]
    counts = [sum(e in row for row in chosen) for e in range(E)]
    room = math.ceil(c["cf"] * T * K / E) if c["cf"] else T
    g = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    out = torch.zeros_like(x)
    xin = _nearest8(x) if kind == "fp8" else x
    taken = [0] * E
    rows = {}
    for t, row in enumerate(chosen):
        g[t] = prob[t, row] / prob[t, row].sum()
        for k, e in enumerate(row):
            if taken[e] < room:
                taken[e] += 1
                rows.setdefault(("W", e), []).append((t, g[t, k]))
            elif c["overflow"]:
                out[t] += g[t, k] * x[t]
    for i in range(c["S"]):
        rows["Ws", i] = [(t, 1.0) for t in range(T)]
    for (pre, e), who in rows.items():
        b = "b" if pre == "W" else "bs"
        h = _silu(xin[[t for t, _ in who]] @ matrix(pre + "1", e).T + s[b + "1"][e].double())
        y = (_nearest8(h) if kind == "fp8" else h) @ matrix(pre + "2", e).T + s[b + "2"][e].double()
        for (t, w), v in zip(who, y):
            out[t] += w * v
    f = torch.tensor(counts, dtype=torch.float64, device="cuda") / (T * K)
    return {"out": out, "f": f, "P": prob.mean(0), "loss": (0.01 * E * (f * prob.mean(0)).sum()).reshape(1),
            "topk_idx": torch.tensor(chosen, dtype=torch.int32, device="cuda"), "gates": g,
            "counts": torch.tensor(counts, dtype=torch.int32, device="cuda")}
