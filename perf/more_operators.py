"""Cases of the norm in front of a mixture-of-experts layer, of activations kept in 8 bits, and of the
experts' layer of a few tokens, with plain forms.

``run`` computes a case either in elementary torch operations in 32 bits (``own`` false) or by the
package's entry points (``own`` true); ``exact`` gives the same results from the definitions in 64 bits.

Operators:
  norm             rows + residual -> root-mean-square norm, in bf16 and in FP8 rows with scales
  norm_grad        its gradients, of the rows and of the weights
  checkpoint       bf16 rows of every expert's block -> FP8 rows with scales, or back
  checkpoint_grad  kept rows before an activation, gradient after it -> that gradient before it,
                   the activation again, and the bias gradients
  layer            few tokens and their chosen experts -> both products of each, weighted and added up
"""
import math

import torch

own = False

# ------------------------------------------------------------------------ cases


def listed():
    return [
        # one token of a serving step in front of the router: latency counts
        dict(name="norm_token", op="norm", rows=1, hidden=7168, x="bf16", residual=True, weight=True, keep=True, fp8="none"),
        # a serving step of 64 tokens that also makes the FP8 rows which the dispatch sends
        dict(name="norm_step_fp8", op="norm", rows=64, hidden=4096, x="bf16", residual=True, weight=True, keep=True, fp8="fp32"),
        # a training step: 16 ranks x 4096 tokens, bf16 rows for the router and FP8 rows for the dispatch
        dict(name="norm_train_fp8", op="norm", rows=65536, hidden=7168, x="bf16", residual=True, weight=True, keep=True, fp8="fp32"),
        # gradient on a residual stream in fp32, an odd number of rows, some of them padding
        dict(name="norm_grad_fp32", op="norm_grad", rows=1021, hidden=2048, x="fp32", through=True, masked=0.1),
        # gradient of the training step's norm
        dict(name="norm_grad_train", op="norm_grad", rows=65536, hidden=7168, x="bf16", through=True, masked=0.0),
        # 16 ranks x 512 tokens, top 8 of 64 experts: the rows before a gated activation, kept in 8 bits
        dict(name="checkpoint_keep", op="checkpoint", ranks=16, tokens=512, experts=64, topk=8, features=4096, align=1, hot=0.0,
             scales="fp32", back=False),
        # rows that travelled with packed scales, back in bf16 for the gradient of the experts' matrices
        dict(name="checkpoint_back", op="checkpoint", ranks=8, tokens=256, experts=32, topk=4, features=2048, align=16, hot=1.0,
             scales="packed", back=True),
        # the backward pass through the gated activation of the kept rows
        dict(name="checkpoint_grad_gated", op="checkpoint_grad", ranks=16, tokens=512, experts=64, topk=8, features=4096,
             align=1, hot=0.0, scales="fp32", act="swiglu", bias=True),
        # the same of a dense product with GELU, an odd number of rows
        dict(name="checkpoint_grad_gelu", op="checkpoint_grad", ranks=1, tokens=777, experts=1, topk=1, features=1024, align=1,
             hot=0.0, scales="packed", act="gelu", bias=True),
        # one token through a small layer: the least that a serving step can cost
        dict(name="layer_token_small", op="layer", tokens=1, experts=32, topk=4, hidden=1024, inner=512, act="swiglu",
             weights="bf16", bias=False, residual=False, masked=0.0),
        # one token through 8 of 256 experts with FP8 matrices
        dict(name="layer_token_fp8", op="layer", tokens=1, experts=256, topk=8, hidden=7168, inner=2048, act="swiglu",
             weights="fp8", bias=False, residual=True, masked=0.0),
        # a serving step of 64 tokens, top 8 of 64 experts: all matrices are read
        dict(name="layer_step", op="layer", tokens=64, experts=64, topk=8, hidden=4096, inner=2048, act="swiglu",
             weights="bf16", bias=False, residual=True, masked=0.0),
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of `unit`, spread over the logarithm of [lo, hi] units."""
    return unit * max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above: serving steps of one token to training steps, every type,
    activation and scale format, odd sizes among them."""
    op = rng.choice(["norm", "norm_grad", "checkpoint", "checkpoint_grad", "layer", "layer"])
    if op in ("norm", "norm_grad"):
        fp8 = rng.choice(["none", "fp32", "packed"]) if op == "norm" else "none"
        hidden = _log(rng, 1, 64, 128) if fp8 != "none" else _log(rng, 8, 1024, 8)
        x = rng.choice(["bf16", "bf16", "fp32"])
        # an amount that a power of two just holds may fall on either side of it: few rows with packed scales
        most = 500_000 // hidden if fp8 == "packed" else 200_000_000 // hidden
        rows = _log(rng, 1, max(1, min(65536, most)))
        if op == "norm":
            return dict(op=op, rows=rows, hidden=hidden, x=x, residual=rng.random() < 0.7, weight=rng.random() < 0.8,
                        keep=rng.random() < 0.7, fp8=fp8)
        return dict(op=op, rows=rows, hidden=hidden, x=x, through=rng.random() < 0.7, masked=rng.choice([0.0, 0.0, 0.1]))
    if op == "layer":
        fp8 = rng.random() < 0.4
        experts = _log(rng, 1, 256)
        hidden = _log(rng, 2, 56, 128) if fp8 else _log(rng, 32, 896, 8)
        inner = _log(rng, 1, 16, 128) if fp8 else _log(rng, 16, 256, 8)
        act = rng.choice(["swiglu", "swiglu", "silu", "gelu", "relu", "none"])
        size = hidden * inner * (3 if act == "swiglu" else 2) * (1 if fp8 else 2)
        experts = max(1, min(experts, 3_200_000_000 // size))
        return dict(op=op, tokens=_log(rng, 1, 64), experts=experts, topk=rng.randint(1, min(8, experts)), hidden=hidden,
                    inner=inner, act=act, weights="fp8" if fp8 else "bf16", bias=rng.random() < 0.4,
                    residual=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.1]))
    dense = rng.random() < 0.25
    ranks = 1 if dense else rng.choice([1, 2, 4, 8, 16])
    experts = 1 if dense else ranks * _log(rng, 1 if ranks > 4 else 4, 64 // ranks)
    topk = 1 if dense else rng.randint(1, min(8, experts))
    features = _log(rng, 1, 56, 128)
    tokens = _log(rng, 1, max(1, min(4096 if dense else 512, 200_000_000 // (features * ranks * topk))))
    c = dict(op=op, ranks=ranks, tokens=tokens, experts=experts, topk=topk, features=features,
             align=1 if dense else rng.choice([1, 1, 16, 128]), hot=0.0 if dense else rng.choice([0.0, 1.0]),
             scales=rng.choice(["fp32", "packed"]))
    if op == "checkpoint":
        return dict(c, back=rng.random() < 0.5)
    return dict(c, act=rng.choice(["swiglu", "swiglu", "silu", "gelu", "relu", "none"]), bias=rng.random() < 0.6)


# ----------------------------------------------------------------------- inputs


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _chosen(g, tokens, experts, topk, hot, masked):
    """The experts of every token with their weights: random scores, on which a few experts may be favoured."""
    score = _normal(g, tokens, experts)
    if hot:
        score += hot * (torch.rand(experts, generator=g, device="cuda") < 0.1)
    val, idx = torch.topk(score, topk, dim=-1)
    w = torch.softmax(val, dim=-1)
    if masked:
        m = torch.rand(idx.shape, generator=g, device="cuda") < masked
        idx, w = idx.masked_fill(m, -1), w.masked_fill(m, 0.0)
    return idx, w


def _blocks(idx, ranks, experts, align):
    """Every expert's block of rows as the expanded dispatch lays them out (counts, starts in the
    rank's region, regions) and the group of every row, or -1."""
    count = torch.bincount(idx.reshape(-1), minlength=experts)
    padded = (count + align - 1) // align * align
    start = torch.cat([torch.zeros_like(padded[:1]), padded.cumsum(0)])
    local = experts // ranks
    region = start[::local]
    base = torch.cat([start[:-1].reshape(ranks, local), start[local::local, None]], 1) - region[:-1, None]
    rows = idx.numel() + experts * (align - 1)
    at = torch.arange(rows, device="cuda")
    e = torch.bucketize(at, start[:-1].contiguous(), right=True) - 1
    group = torch.where(at - start[e] < count[e], e, -1)
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return {"count": i32(count.reshape(ranks, local)), "base": i32(base), "region": i32(region), "group": group}


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda").manual_seed(seed * 1_000_003 + 29)
    bf, f32 = torch.bfloat16, torch.float32
    s = {"case": c}
    if op in ("norm", "norm_grad"):
        N, H = c["rows"], c["hidden"]
        kind = f32 if c["x"] == "fp32" else bf
        # a residual stream: some columns are much larger than the others
        columns = torch.exp(0.5 * _normal(g, H))
        stream = lambda scale: (_normal(g, N, H, scale=scale) * columns).to(kind)  # noqa: E731
        weighted = op == "norm_grad" or c["weight"]
        s["weight"] = (1 + _normal(g, H, scale=0.1)).to(bf) if weighted else None
        if op == "norm":
            s["x"] = stream(0.5)
            s["residual"] = stream(2.0) if c["residual"] else None
            s["sum"] = torch.empty_like(s["x"]) if c["keep"] else None
            s["y"] = torch.empty(N, H, dtype=bf, device="cuda")
            s["codes"] = s["sf"] = None
            if c["fp8"] != "none":
                G = H // 128
                s["codes"] = torch.empty(N, H, dtype=torch.uint8, device="cuda")
                s["sf"] = torch.empty(N, G if c["fp8"] == "fp32" else (G + 3) // 4, device="cuda")
        else:
            s["sum"] = stream(2.0)
            s["d_y"] = _normal(g, N, H, scale=0.01, dtype=bf)
            s["d_sum"] = _normal(g, N, H, scale=0.01, dtype=kind) if c["through"] else None
            s["mask"] = (torch.rand(N, generator=g, device="cuda") >= c["masked"]).to(torch.uint8) if c["masked"] else None
            s["d_x"] = torch.empty_like(s["sum"])
            s["d_weight"] = torch.empty(H, device="cuda")
    elif op in ("checkpoint", "checkpoint_grad"):
        R, F = c["ranks"], c["features"]
        G = F // 128
        idx, _ = _chosen(g, R * c["tokens"], c["experts"], c["topk"], c["hot"], 0.0)
        s["lay"] = lay = _blocks(idx, R, c["experts"], c["align"])
        rows = lay["group"].numel()
        z = _normal(g, rows, F, dtype=bf)
        packed = c["scales"] == "packed"
        if op == "checkpoint" and not c["back"]:
            s["x"] = z
            s["codes"] = torch.zeros(rows, F, dtype=torch.uint8, device="cuda")
            s["sf"] = torch.zeros(rows, (G + 3) // 4 if packed else G, device="cuda")
        else:
            q, sf = _quantise(z.float(), packed)
            s["codes"], s["sf"] = q.view(torch.uint8), sf.view(f32)
            if op == "checkpoint":
                s["x"] = torch.zeros(rows, F, dtype=bf, device="cuda")
            else:
                n = F // 2 if c["act"] == "swiglu" else F
                s["d_h"] = _normal(g, rows, n, scale=0.01, dtype=bf)
                s["h"] = torch.zeros(rows, n, dtype=bf, device="cuda")
                s["d_z"] = torch.zeros(rows, F, dtype=bf, device="cuda")
                s["d_bias"] = torch.empty(c["experts"], F, device="cuda") if c["bias"] else None
    else:
        T, E, H, I = c["tokens"], c["experts"], c["hidden"], c["inner"]
        Z = 2 * I if c["act"] == "swiglu" else I
        s["idx"], s["w"] = _chosen(g, T, E, c["topk"], 0.0, c["masked"])
        s["x"] = _normal(g, T, H, dtype=bf)
        fp8 = c["weights"] == "fp8"
        for name, rows, columns in (("up", Z, H), ("down", H, I)):
            s[name] = torch.empty(E, rows, columns, dtype=torch.uint8 if fp8 else bf, device="cuda")
            s[name + "_sf"] = torch.empty(E, rows // 128, columns // 128, device="cuda") if fp8 else None
            s[name + "_bias"] = _normal(g, E, rows, scale=0.1, dtype=bf) if c["bias"] else None
            for e in range(E):
                m = _normal(g, rows, columns, scale=columns ** -0.5)
                if fp8:  # a scale for every 128 x 128
                    m = m.reshape(rows // 128, 128, columns // 128, 128)
                    sf = m.abs().amax((1, 3)) / 448
                    s[name + "_sf"][e] = sf
                    m = (m / sf[:, None, :, None]).reshape(rows, columns).to(torch.float8_e4m3fn).view(torch.uint8)
                s[name][e] = m
        s["residual"] = _normal(g, T, H, dtype=bf) if c["residual"] else None
        s["out"] = torch.empty(T, H, dtype=bf, device="cuda")
    if own:
        s["handle"] = _handle(s)
    return s


def _handle(s):
    """What a user of the package keeps beside these tensors: configuration, layout, workspace."""
    import combine_ep_get_02_gb300 as ep
    c, op = s["case"], s["case"]["op"]
    act = {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU,
           "swiglu": ep.EP_ACT_SWIGLU}[c.get("act", "none")]
    if op in ("norm", "norm_grad"):
        cfg = ep.NormConfig(rows=c["rows"], hidden=c["hidden"], eps=1e-6, sf_pack=int(c.get("fp8") == "packed"),
                            x_dtype=ep.EP_DTYPE_FP32 if c["x"] == "fp32" else ep.EP_DTYPE_BF16)
        return ep, cfg, None, ep.alloc_norm_workspace(cfg) if op == "norm_grad" else None
    if op == "layer":
        cfg = ep.LayerConfig(num_tokens=c["tokens"], num_experts=c["experts"], num_topk=c["topk"], hidden=c["hidden"],
                             inner=c["inner"], activation=act,
                             weight_dtype=ep.EP_DTYPE_FP8_E4M3 if c["weights"] == "fp8" else ep.EP_DTYPE_BF16)
        return ep, cfg, None, ep.alloc_layer_workspace(cfg)
    lay = s["lay"]
    cfg = ep.CheckpointConfig(num_ranks=c["ranks"], num_experts=c["experts"], rows=lay["group"].numel(),
                              features=c["features"], activation=act, sf_pack=int(c["scales"] == "packed"))
    layout = None if c["experts"] == 1 else ep.Layout(*[None] * 6, lay["count"], lay["base"], lay["region"])
    return ep, cfg, layout, ep.alloc_checkpoint_workspace(cfg)


# ------------------------------------------------------------------ plain forms


def _quantise(y, packed):
    """fp32 rows -> (e4m3 codes, scales per 128 columns: fp32, or powers of two as exponent bytes,
    padded to whole words)."""
    v = y.reshape(y.shape[0], -1, 128)
    amax = v.abs().amax(-1).clamp(min=1e-4)
    if not packed:
        return (v * (448 / amax)[..., None]).to(torch.float8_e4m3fn).reshape(y.shape), amax / 448
    m, e = torch.frexp(amax.double() / 448)
    e = torch.where(m > 0.5, e, e - 1)  # 2^e is the least power of two that is not below amax / 448
    q = (v * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).reshape(y.shape)
    sf = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 4))
    return q, sf.view(torch.float8_e8m0fnu)


def _values(codes, sf, packed):
    """fp32 values of FP8 rows."""
    v = codes.view(torch.float8_e4m3fn).float().reshape(codes.shape[0], -1, 128)
    scale = sf.view(torch.float8_e8m0fnu)[:, :v.shape[1]].float() if packed else sf
    return (v * scale[..., None]).reshape(codes.shape)


def _norm(s):
    c = s["case"]
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    y = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    out = [v.to(s["x"].dtype)] if c["keep"] else []
    out.append(y.to(torch.bfloat16))
    return out if c["fp8"] == "none" else [*out, *_quantise(y, c["fp8"] == "packed")]


def _norm_grad(s):
    v, d_y = s["sum"].float(), s["d_y"].float()
    q = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)
    n, t = v * q, d_y * s["weight"].float()
    d = q * (t - n * (t * n).mean(-1, keepdim=True))
    if s["d_sum"] is not None:
        d = d + s["d_sum"].float()
    dw = d_y * n
    if s["mask"] is not None:
        live = (s["mask"] != 0)[:, None]
        d, dw = torch.where(live, d, 0.0), torch.where(live, dw, 0.0)
    return d.to(s["sum"].dtype), dw.sum(0)


def _checkpoint(s):
    c = s["case"]
    packed, live = c["scales"] == "packed", (s["lay"]["group"] >= 0)[:, None]
    if c["back"]:
        return (torch.where(live, _values(s["codes"], s["sf"], packed), 0.0).to(torch.bfloat16),)
    q, sf = _quantise(s["x"].float(), packed)
    q, sf = (torch.where(live, t.view(torch.uint8) if t.dtype != torch.float32 else t, 0) for t in (q, sf))
    return q.view(torch.float8_e4m3fn), sf.view(torch.float8_e8m0fnu) if packed else sf


def _act(z, act):
    """The activation and, for a gradient t after it, the function that gives the one before it."""
    if act == "swiglu":
        a, b = z.chunk(2, -1)
        g = 1 / (1 + torch.exp(-a))
        return a * g * b, lambda t: torch.cat([t * b * g * (1 + a * (1 - g)), t * a * g], -1)
    if act == "relu":
        return torch.where(z > 0, z, 0.0), lambda t: torch.where(z > 0, t, 0.0)
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return z * g, lambda t: t * g * (1 + z * (1 - g))
    if act == "gelu":
        f = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * f, lambda t: t * (f + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    return z, lambda t: t


def _checkpoint_grad(s):
    c, group = s["case"], s["lay"]["group"]
    live = (group >= 0)[:, None]
    h, back = _act(_values(s["codes"], s["sf"], c["scales"] == "packed"), c["act"])
    d_z = torch.where(live, back(s["d_h"].float()), 0.0)
    out = [torch.where(live, h, 0.0).to(torch.bfloat16), d_z.to(torch.bfloat16)]
    if c["bias"]:
        d_bias = torch.zeros(c["experts"], c["features"], device="cuda")
        out.append(d_bias.index_add(0, group.clamp(min=0), d_z))
    return out


def _matrices(w, sf):
    """fp32 matrices [..., rows, columns] of bf16 ones, or of codes with a scale for every 128 x 128."""
    if sf is None:
        return w.float()
    v = w.view(torch.float8_e4m3fn).float()
    v = v.reshape(*w.shape[:-2], w.shape[-2] // 128, 128, w.shape[-1] // 128, 128)
    return (v * sf[..., :, None, :, None]).reshape(w.shape)


def _layer(s):
    c = s["case"]
    T, E, K, H = c["tokens"], c["experts"], c["topk"], c["hidden"]
    x, live = s["x"].float(), s["idx"] >= 0
    at, weight = s["idx"].clamp(min=0), torch.where(s["idx"] >= 0, s["w"], 0.0)
    if T * K <= E:  # the matrices of every lane's expert
        pick = lambda t: None if t is None else t[at.reshape(-1)]  # noqa: E731
        x, share = x.repeat_interleave(K, 0)[:, None], weight.reshape(-1)
    else:  # every token through every expert
        pick = lambda t: t  # noqa: E731
        x, share = x.expand(E, T, H), torch.zeros(T, E, device="cuda").scatter_add(1, at, weight).t()
    z = torch.bmm(x, _matrices(pick(s["up"]), pick(s["up_sf"])).transpose(1, 2))
    z = z if s["up_bias"] is None else z + pick(s["up_bias"]).float()[:, None]
    h = _act(z, c["act"])[0]
    y = torch.bmm(h, _matrices(pick(s["down"]), pick(s["down_sf"])).transpose(1, 2))
    y = y if s["down_bias"] is None else y + pick(s["down_bias"]).float()[:, None]
    if T * K <= E:
        out = (y.reshape(T, K, H) * share.reshape(T, K, 1)).sum(1)
    else:
        out = (y * share[..., None]).sum(0)
    return (out if s["residual"] is None else out + s["residual"].float()).to(torch.bfloat16)


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"norm": _norm, "norm_grad": _norm_grad, "checkpoint": _checkpoint, "checkpoint_grad": _checkpoint_grad,
                "layer": _layer}[op](s)
    ep, cfg, layout, ws = s["handle"]
    if op == "norm":
        ep.ep_norm(cfg, s["x"], s["residual"], s["weight"], s["sum"], s["y"], s["codes"], s["sf"])
        out = [s["sum"]] if c["keep"] else []
        out.append(s["y"])
        if c["fp8"] != "none":
            sf = s["sf"].view(torch.float8_e8m0fnu) if c["fp8"] == "packed" else s["sf"]
            out += [s["codes"].view(torch.float8_e4m3fn), sf]
        return out
    if op == "norm_grad":
        ep.ep_norm_grad(cfg, s["sum"], s["weight"], s["mask"], s["d_y"], s["d_sum"], s["d_x"], s["d_weight"], ws)
        return s["d_x"], s["d_weight"]
    if op == "checkpoint":
        if c["back"]:
            ep.ep_checkpoint_rows(cfg, layout, s["codes"], s["sf"], s["x"], ws)
            return (s["x"],)
        ep.ep_checkpoint(cfg, layout, s["x"], s["codes"], s["sf"], ws)
        sf = s["sf"].view(torch.float8_e8m0fnu) if c["scales"] == "packed" else s["sf"]
        return s["codes"].view(torch.float8_e4m3fn), sf
    if op == "checkpoint_grad":
        ep.ep_checkpoint_grad(cfg, layout, s["codes"], s["sf"], s["d_h"], s["h"], s["d_z"], s["d_bias"], ws)
        return [s["h"], s["d_z"], s["d_bias"]] if c["bias"] else [s["h"], s["d_z"]]
    ep.ep_expert_layer(cfg, s["x"], s["idx"], s["w"], s["up"], s["up_sf"], s["up_bias"], s["down"], s["down_sf"],
                       s["down_bias"], s["residual"], s["out"], ws)
    return s["out"]


# ------------------------------------------------------------- 64-bit definitions


def _scaled(y, packed):
    """What the codes and the scales stand for before the codes are rounded."""
    a = y.unflatten(-1, (-1, 128)).abs().amax(-1).clamp(min=1e-4) / 448
    if packed:
        a = torch.exp2(torch.ceil(torch.log2(a)))
    codes = y / a.repeat_interleave(128, -1)
    if packed:
        a = torch.cat([a, a.new_full((len(a), -a.shape[1] % 4), 2.0 ** -127)], 1)
    return codes, a


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    F = torch.nn.functional
    acts = {"none": lambda t: t * 1, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "swiglu": lambda t: F.silu(t[..., :t.shape[-1] // 2]) * t[..., t.shape[-1] // 2:]}
    if op == "norm":
        v = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = v * torch.rsqrt(v.square().sum(-1, keepdim=True) / c["hidden"] + 1e-6)
        y = y if s["weight"] is None else y * s["weight"].double()
        out = [v] if c["keep"] else []
        return [*out, y] if c["fp8"] == "none" else [*out, y, *_scaled(y, c["fp8"] == "packed")]
    if op == "norm_grad":  # through autograd, a part of the rows at a time
        w = s["weight"].double().requires_grad_(True)
        d_x, d_w = [], 0
        parts = lambda t: (t,) if t is None else t.split(8192)  # noqa: E731
        for i, (v, d_y) in enumerate(zip(parts(s["sum"]), parts(s["d_y"]))):
            m = 1.0 if s["mask"] is None else parts(s["mask"])[i].double()[:, None]
            v = v.double().requires_grad_(True)
            with torch.enable_grad():
                y = v * torch.rsqrt(v.square().sum(-1, keepdim=True) / c["hidden"] + 1e-6) * w * m
            gv, gw = torch.autograd.grad(y, (v, w), d_y.double())
            d_x.append(gv if s["d_sum"] is None else gv + m * parts(s["d_sum"])[i].double())
            d_w = d_w + gw
        return torch.cat(d_x), d_w
    if op == "layer":
        out = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            out += s["residual"].double()
        mat = lambda name, e: (s[name][e].double() if s[name + "_sf"] is None else  # noqa: E731
                               s[name][e].view(torch.float8_e4m3fn).double()
                               * s[name + "_sf"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1))
        for e in torch.unique(s["idx"][s["idx"] >= 0]).tolist():
            t, k = torch.nonzero(s["idx"] == e, as_tuple=True)
            z = s["x"][t].double() @ mat("up", e).T
            h = acts[c["act"]](z if s["up_bias"] is None else z + s["up_bias"][e].double())
            y = h @ mat("down", e).T
            y = y if s["down_bias"] is None else y + s["down_bias"][e].double()
            out.index_add_(0, t, y * s["w"][t, k].double()[:, None])
        return out
    group, packed = s["lay"]["group"], c["scales"] == "packed"
    live = (group >= 0).double()[:, None]
    if op == "checkpoint" and not c["back"]:
        codes, sf = _scaled(s["x"].double(), packed)
        return codes * live, torch.where(group[:, None] >= 0, sf, 2.0 ** -127 if packed else 0.0)
    v = s["codes"].view(torch.float8_e4m3fn).double() * live
    if packed:
        sf = s["sf"].view(torch.float8_e8m0fnu).double()[:, :c["features"] // 128]
    else:
        sf = s["sf"].double()
    v = v * sf.repeat_interleave(128, 1)
    if op == "checkpoint":
        return (v,)
    v.requires_grad_(True)
    with torch.enable_grad():
        h = acts[c["act"]](v)
    (d_z,) = torch.autograd.grad(h, v, s["d_h"].double() * live)
    if not c["bias"]:
        return [h.detach() * live, d_z]
    d_bias = torch.zeros(c["experts"], c["features"], dtype=torch.float64, device="cuda")
    return [h.detach() * live, d_z, d_bias.index_add_(0, group.clamp(min=0), d_z)]


# ------------------------------------------------------------------------- work


def work(case):
    c, op = case, case["op"]
    if op in ("norm", "norm_grad"):
        N, H = c["rows"], c["hidden"]
        size = 4 if c["x"] == "fp32" else 2
        if op == "norm":
            scales = {"none": 0, "fp32": 4 * (H // 128), "packed": (H // 128 + 3) // 4 * 4}[c["fp8"]]
            row = H * size * (1 + c["residual"] + c["keep"]) + 2 * H + (H + scales if c["fp8"] != "none" else 0)
            return {"bytes": N * row + (2 * H if c["weight"] else 0), "flops": 6 * N * H}
        live = int(N * (1 - c["masked"]))
        return {"bytes": N * H * size + live * H * (2 + size * (1 + c["through"])) + 6 * H, "flops": 12 * live * H}
    if op == "layer":
        T, E, K, H, I = c["tokens"], c["experts"], c["topk"], c["hidden"], c["inner"]
        size = H * I * (3 if c["act"] == "swiglu" else 2)
        used = E * (1 - (1 - K / E * (1 - c["masked"])) ** T)
        return {"bytes": int(used * size * (1 + 4 / 16384 if c["weights"] == "fp8" else 2)
                             + T * H * (6 if c["residual"] else 4) + 12 * T * K),
                "flops": int(2 * T * K * (1 - c["masked"]) * size)}
    F, rows = c["features"], c["ranks"] * c["tokens"] * c["topk"]
    kept = F + (4 * (F // 128) if c["scales"] == "fp32" else (F // 128 + 3) // 4 * 4)
    if op == "checkpoint":
        return {"bytes": rows * (kept + 2 * F), "flops": 3 * rows * F}
    n = F // 2 if c["act"] == "swiglu" else F
    return {"bytes": rows * (kept + 4 * n + 2 * F) + (4 * c["experts"] * F if c["bias"] else 0), "flops": 12 * rows * n}
