"""Cases of the router, the experts' products and the gradients around them, with plain forms.

``run`` computes a case either in elementary torch operations in 32 bits
(``own`` false) or by the package's entry points (``own`` true); ``exact`` gives
the same results from the definitions in 64 bits.

Operators:
  route         logits -> chosen experts, weights, per-expert counts, balance loss
  route_grad    gradients of the weights and of the loss -> gradient of the logits
  combine_grad  gradient of the combined tokens -> gradients of the expert outputs and weights
  product       rows grouped by expert x that expert's matrix, bias, activation, residual
  product_grad  gradients of that product's rows, matrices and biases
"""
import math

import torch

own = False

# ------------------------------------------------------------------------ cases


def listed():
    return [
        # one serving step of 64 tokens through a 256-expert router with sigmoid scores, a
        # choice bias and a limit to 4 of 8 expert groups: latency counts
        dict(name="route_step", op="route", segments=1, tokens=64, experts=256, topk=8, logits="fp32", score="sigmoid",
             bias=True, groups=8, keep=4, normalize=True, scale=2.5, masked=0.0),
        # the router of a training step: 16 ranks x 4096 tokens, top 8 of 256, a loss per rank
        dict(name="route_train", op="route", segments=16, tokens=4096, experts=256, topk=8, logits="fp32", score="softmax",
             bias=False, groups=1, keep=1, normalize=True, scale=1.0, masked=0.0),
        # gradient of a small router in bf16, with padding tokens
        dict(name="route_grad_small", op="route_grad", segments=8, tokens=128, experts=32, topk=4, logits="bf16",
             score="softmax", bias=False, groups=1, keep=1, normalize=False, scale=1.0, masked=0.1),
        # gradient of the training router
        dict(name="route_grad_train", op="route_grad", segments=16, tokens=4096, experts=256, topk=8, logits="fp32",
             score="sigmoid", bias=True, groups=8, keep=4, normalize=True, scale=2.5, masked=0.02),
        # gradient of the combine on receive rows shared by the lanes to one rank, some lanes masked
        dict(name="combine_grad_rows", op="combine_grad", ranks=16, tokens=1024, experts=256, topk=8, hidden=7168,
             expand=False, align=1, hot=0.0, masked=0.02),
        # the same on per-expert blocks, a few experts hot
        dict(name="combine_grad_expanded", op="combine_grad", ranks=64, tokens=512, experts=512, topk=8, hidden=2048,
             expand=True, align=1, hot=2.0, masked=0.0),
        # one token through a shared expert's gated product: the smallest serving call
        dict(name="product_token", op="product", ranks=1, tokens=1, experts=1, topk=1, inner=7168, outer=2048, x="bf16",
             act="swiglu", bias=False, residual=False, save=False, align=1, hot=0.0),
        # one serving step of 64 tokens, top 8 of 64 experts: the experts' matrices are what is read
        dict(name="product_step", op="product", ranks=1, tokens=64, experts=64, topk=8, inner=4096, outer=2048, x="bf16",
             act="swiglu", bias=False, residual=False, save=False, align=1, hot=0.0),
        # a prompt's or training step's up projection on rows that were dispatched in FP8 with
        # scales per 128 columns: 8192 tokens, top 8 of 64 experts
        dict(name="product_up_fp8", op="product", ranks=16, tokens=512, experts=64, topk=8, inner=7168, outer=2048, x="fp8",
             act="swiglu", bias=False, residual=False, save=False, align=1, hot=0.0),
        # a shared expert's down projection that adds the routed experts' sum: one group
        dict(name="product_down", op="product", ranks=1, tokens=4096, experts=1, topk=1, inner=2048, outer=7168, x="bf16",
             act="none", bias=True, residual=True, save=False, align=1, hot=0.0),
        # gradients of the experts' gated product, ragged groups in aligned blocks
        dict(name="product_grad_experts", op="product_grad", ranks=8, tokens=512, experts=32, topk=4, inner=2048, outer=1024,
             x="bf16", act="swiglu", bias=True, residual=False, save=True, align=16, hot=1.0),
        # gradients of a dense product with GELU
        dict(name="product_grad_dense", op="product_grad", ranks=1, tokens=4096, experts=1, topk=1, inner=4096, outer=4096,
             x="bf16", act="gelu", bias=True, residual=False, save=True, align=1, hot=0.0),
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of `unit`, spread over the logarithm of [lo, hi] units."""
    v = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return unit * (v - 1 if unit * v in (1536, 3072) else v)  # sizes of other programs' configurations


def draw(rng):
    """One more case of the ranges above: serving steps of one token to training steps,
    every score, activation, type and row layout, odd sizes among them."""
    op = rng.choice(["route", "route_grad", "combine_grad", "product", "product", "product_grad"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 2 if groups > 1 else 8, 512 // groups)
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(16, experts // groups * keep))
        segments = rng.choice([1, 1, 2, 8, 16, rng.randint(3, 24)])
        most = min(4096, 65536 * 256 // (segments * experts))
        return dict(op=op, segments=segments, tokens=_log(rng, 1, max(1, most)), experts=experts, topk=topk,
                    logits=rng.choice(["fp32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, keep=keep, normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0.0, 0.02, 0.3]))
    if op == "combine_grad":
        ranks = rng.choice([1, 2, 4, 8, 16, 32])
        experts = ranks * _log(rng, 1 if ranks > 8 else 8, 512 // ranks)
        hidden = _log(rng, 16, 896, 8)
        expand = rng.random() < 0.5
        rows = 1_000_000_000 // (2 * hidden)  # of y, at most
        topk = rng.randint(1, min(8, experts))
        tokens = _log(rng, 1, max(1, min(1024, rows // (ranks * (topk if expand else ranks)))))
        return dict(op=op, ranks=ranks, tokens=tokens, experts=experts, topk=topk, hidden=hidden, expand=expand,
                    align=rng.choice([1, 4, 128]) if expand else 1, hot=rng.choice([0.0, 1.0]), masked=rng.choice([0.0, 0.05]))
    dense = rng.random() < 0.35
    ranks = 1 if dense else rng.choice([1, 2, 4, 8, 16])
    experts = 1 if dense else ranks * _log(rng, 1 if ranks > 4 else 4, 64 // ranks)
    topk = 1 if dense else rng.randint(1, min(8, experts))
    act = rng.choice(["none", "relu", "silu", "gelu", "swiglu"])
    fp8 = op == "product" and rng.random() < 0.3
    inner = _log(rng, 2, 56, 128) if fp8 else _log(rng, 32, 896, 8)
    outer = _log(rng, 16, 512, 8)
    cost = 1_500_000_000_000 // (2 * inner * outer * (2 if act == "swiglu" else 1) * (2 if op == "product_grad" else 1))
    tokens = _log(rng, 1, max(1, min(4096 if dense else 1024, cost // (ranks * topk))))
    return dict(op=op, ranks=ranks, tokens=tokens, experts=experts, topk=topk, inner=inner, outer=outer,
                x="fp8" if fp8 else "bf16", act=act, bias=rng.random() < 0.6,
                residual=op == "product" and rng.random() < 0.4, save=op == "product_grad" or rng.random() < 0.3,
                align=1 if dense else rng.choice([1, 1, 16, 128]), hot=0.0 if dense else rng.choice([0.0, 1.0]))


# ----------------------------------------------------------------------- inputs


def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _choose(g, ranks, tokens, experts, topk, hot, masked):
    """Routing of every rank's tokens: random scores, on which a few experts may be favoured."""
    score = _normal(g, ranks, tokens, experts)
    if hot:
        score += hot * (torch.rand(experts, generator=g, device="cuda") < 0.1)
    val, idx = torch.topk(score, topk, dim=-1)
    w = torch.softmax(val, dim=-1)
    if masked:
        m = torch.rand(idx.shape, generator=g, device="cuda") < masked
        idx, w = idx.masked_fill(m, -1), w.masked_fill(m, 0.0)
    return idx, w


def _blocks(idx, ranks, experts, align):
    """Per-expert blocks of the lanes in token order, as the expanded dispatch lays them out."""
    e = idx.reshape(-1)
    count = torch.bincount(e.clamp(min=0), (e >= 0).double(), minlength=experts).long()
    padded = (count + align - 1) // align * align
    base = torch.cat([torch.zeros_like(padded[:1]), padded.cumsum(0)])  # of every block, over all ranks
    order = torch.argsort(torch.where(e >= 0, e, experts), stable=True)
    begin = torch.cat([torch.zeros_like(count[:1]), count.cumsum(0)])
    at = torch.full_like(e, -1)
    n = int(begin[-1])
    at[order[:n]] = torch.arange(n, device=e.device) - begin[e[order[:n]]] + base[e[order[:n]]]
    local = experts // ranks
    region = base[::local].contiguous()
    pos = torch.where(e >= 0, at - region[(e.clamp(min=0) // local)], -1)
    exp_base = torch.cat([base[:-1].reshape(ranks, local), base[local::local, None]], 1) - region[:-1, None]
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return {"count": i32(count.reshape(ranks, local)), "base": i32(exp_base), "region": i32(region),
            "pos": i32(pos.reshape(idx.shape)), "row": at.reshape(idx.shape), "start": base[:-1], "most": int(count.max())}


def _slots(idx, ranks, experts):
    """Receive rows of the row form: every source's running count of the tokens that reach a rank."""
    R, T, _ = idx.shape
    d = torch.where(idx >= 0, idx // (experts // ranks), ranks)
    there = torch.zeros(R, T, ranks + 1, dtype=torch.int64, device=idx.device).scatter_(2, d, 1)
    before = there.cumsum(1) - there
    slot = before.gather(2, d) + torch.arange(R, device=idx.device).reshape(R, 1, 1) * T
    slot = torch.where(idx >= 0, slot, -1)
    return {"slot": slot.to(torch.int32), "row": torch.where(idx >= 0, d * R * T + slot, -1)}


def _recv_rows(c):
    if c["op"] == "combine_grad" and not c["expand"]:
        return c["ranks"] * c["ranks"] * c["tokens"]
    return c["ranks"] * c["tokens"] * c["topk"] + c["experts"] * (c["align"] - 1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 1_000_003 + 17)
    s = {"case": c}
    if c["op"] in ("route", "route_grad"):
        N, E, K = c["segments"] * c["tokens"], c["experts"], c["topk"]
        s["logits"] = _normal(g, N, E, scale=1.5, dtype=torch.float32 if c["logits"] == "fp32" else torch.bfloat16)
        s["bias"] = _normal(g, E, scale=0.05) if c["bias"] else None
        s["mask"] = (torch.rand(N, generator=g, device="cuda") >= c["masked"]).to(torch.uint8) if c["masked"] else None
        if c["op"] == "route_grad":
            choice, weights, count, psum, valid, loss = _route(s)
            s.update(idx=choice, weights=weights, count=count, psum=psum, valid=valid, loss=loss,
                     d_weights=_normal(g, N, K, scale=0.1), d_loss=torch.full((1,), 0.01 * N, device="cuda"))
            s["d_logits"] = torch.empty_like(s["logits"])
    elif c["op"] == "combine_grad":
        R, T, E, H = c["ranks"], c["tokens"], c["experts"], c["hidden"]
        s["idx"], s["w"] = _choose(g, R, T, E, c["topk"], c["hot"], c["masked"])
        s["lay"] = _blocks(s["idx"], R, E, c["align"]) if c["expand"] else _slots(s["idx"], R, E)
        s["y"] = _normal(g, _recv_rows(c), H, dtype=torch.bfloat16)
        s["d_out"] = _normal(g, R, T, H, dtype=torch.bfloat16)
        s["d_y"] = torch.zeros_like(s["y"])
        s["d_w"] = torch.zeros(R, T, c["topk"], device="cuda")
    else:
        rows, E, I, O = _recv_rows(c), c["experts"], c["inner"], c["outer"]
        Z = 2 * O if c["act"] == "swiglu" else O
        bf = torch.bfloat16
        idx, _ = _choose(g, c["ranks"], c["tokens"], E, c["topk"], c["hot"], 0.0)
        s["lay"] = lay = _blocks(idx, c["ranks"], E, c["align"])
        # where every row stands in a batch of equal groups, for the plain form: [E, most], or past its end
        e = torch.bucketize(torch.arange(rows, device="cuda"), lay["start"], right=True) - 1
        at = torch.arange(rows, device="cuda") - lay["start"][e]
        s["live"] = at < lay["count"].reshape(-1)[e]
        s["cell"] = torch.where(s["live"], e * lay["most"] + at, 0)
        s["x"] = _normal(g, rows, I, dtype=bf)
        s["x_sf"] = None
        if c["x"] == "fp8":
            x = s["x"].float().reshape(rows, I // 128, 128)
            sf = x.abs().amax(-1, keepdim=True).clamp(min=1e-4) / 448
            s["x"], s["x_sf"] = (x / sf).reshape(rows, I).to(torch.float8_e4m3fn).view(torch.uint8), sf[..., 0].contiguous()
        s["w"] = torch.empty(E, Z, I, dtype=bf, device="cuda")
        for i in range(E):
            s["w"][i] = _normal(g, Z, I, scale=I ** -0.5, dtype=bf)
        s["b"] = _normal(g, E, Z, scale=0.1, dtype=bf) if c["bias"] else None
        s["res"] = _normal(g, rows, O, dtype=bf) if c["residual"] else None
        if c["op"] == "product":
            s["z"] = torch.zeros(rows, Z, dtype=bf, device="cuda") if c["save"] else None
            s["out"] = torch.zeros(rows, O, dtype=bf, device="cuda")
        else:
            s["z"] = _normal(g, rows, Z, dtype=bf)
            s["d_out"] = _normal(g, rows, O, dtype=bf)
            s["d_x"] = torch.zeros(rows, I, dtype=bf, device="cuda")
            s["d_w"] = torch.empty_like(s["w"])
            s["d_b"] = torch.empty(E, Z, device="cuda") if c["bias"] else None
    if own:
        s["handle"] = _handle(s)
    return s


def _handle(s):
    """What a user of the package keeps beside these tensors: configuration, layout, workspace, outputs."""
    import combine_ep_get_02_gb300 as ep
    c = s["case"]
    if c["op"] in ("route", "route_grad"):
        cfg = ep.RouteConfig(num_segments=c["segments"], num_tokens=c["tokens"], num_experts=c["experts"],
                             num_topk=c["topk"], logits_dtype=ep.EP_DTYPE_FP32 if c["logits"] == "fp32" else ep.EP_DTYPE_BF16,
                             score=ep.EP_SCORE_SOFTMAX if c["score"] == "softmax" else ep.EP_SCORE_SIGMOID,
                             num_groups=c["groups"], topk_groups=c["keep"], normalize=int(c["normalize"]), scale=c["scale"])
        out = ep.alloc_route(cfg) if c["op"] == "route" else ep.Route(
            s["idx"], s["weights"], s["count"], s["psum"], s["valid"], s["loss"])
        return ep, cfg, out, ep.alloc_route_workspace(cfg)
    lay = s["lay"]
    if c["op"] == "combine_grad":
        cfg = ep.Config(1, c["ranks"], c["experts"], c["topk"], c["tokens"], c["tokens"], c["hidden"],
                        expand=int(c["expand"]), expert_alignment=c["align"])
        layout = ep.alloc_layout(cfg)
        if c["expand"]:
            layout.exp_cnt, layout.exp_base, layout.exp_region, layout.exp_pos = (
                lay["count"], lay["base"], lay["region"], lay["pos"])
        else:
            layout.slot_map = lay["slot"]
        return ep, cfg, layout, ep.alloc_workspace(cfg)
    act = {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU,
           "swiglu": ep.EP_ACT_SWIGLU}[c["act"]]
    cfg = ep.ProductConfig(num_ranks=c["ranks"], num_experts=c["experts"], rows=s["x"].shape[0], in_features=c["inner"],
                           out_features=c["outer"], activation=act,
                           x_dtype=ep.EP_DTYPE_FP8_E4M3 if c["x"] == "fp8" else ep.EP_DTYPE_BF16)
    layout = None if c["experts"] == 1 else ep.Layout(*[None] * 6, lay["count"], lay["base"], lay["region"])
    return ep, cfg, layout, ep.alloc_product_workspace(cfg, grad=c["op"] == "product_grad")


# ------------------------------------------------------------------ plain forms


def _scores(logits, score):
    l = logits.float()
    if score == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
        return l, p, p
    s = 1.0 / (1.0 + torch.exp(-l))
    return s, s, s / s.sum(-1, keepdim=True)


def _route(s):
    c = s["case"]
    B, T, E, K, G = c["segments"], c["tokens"], c["experts"], c["topk"], c["groups"]
    pick, weight, p = _scores(s["logits"], c["score"])
    if s["bias"] is not None:
        pick = pick + s["bias"]
    if G > 1:
        in_group = pick.reshape(-1, G, E // G)
        best = torch.sort(in_group, dim=-1, descending=True, stable=True)[0]
        kept = torch.sort(best[..., 0] + best[..., 1], dim=-1, descending=True, stable=True)[1][:, :c["keep"]]
        off = torch.ones(B * T, G, dtype=torch.bool, device=pick.device).scatter_(1, kept, False)
        pick = in_group.masked_fill(off[..., None], -math.inf).reshape(-1, E)
    idx = torch.sort(pick, dim=-1, descending=True, stable=True)[1][:, :K]
    w = weight.gather(1, idx)
    if c["normalize"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * c["scale"]
    live = torch.ones(B * T, dtype=torch.bool, device=pick.device) if s["mask"] is None else s["mask"] != 0
    idx = torch.where(live[:, None], idx, -1)
    w = torch.where(live[:, None], w, 0.0)
    p = torch.where(live[:, None], p, 0.0)
    psum = p.reshape(B, T, E).sum(1)
    seg = torch.arange(B * T, device=pick.device) // T
    cell = torch.where(idx >= 0, idx + seg[:, None] * E, B * E)
    count = torch.zeros(B * E + 1, dtype=torch.int32, device=pick.device)
    count = count.index_add(0, cell.reshape(-1), torch.ones_like(cell.reshape(-1), dtype=torch.int32))[:-1].reshape(B, E)
    valid = live.reshape(B, T).sum(1).to(torch.int32)
    n = valid.clamp(min=1).float()
    loss = ((count.float() * psum).sum(1) * (E / K) / (n * n)).mean().reshape(1)
    return idx, w, count, psum, valid, loss


def _route_grad(s):
    c = s["case"]
    B, T, E, K = c["segments"], c["tokens"], c["experts"], c["topk"]
    _, weight, p = _scores(s["logits"], c["score"])
    live = s["idx"] >= 0
    at = s["idx"].clamp(min=0)
    n = s["valid"].clamp(min=1).float()
    a = s["d_loss"] * (E / (B * K)) * s["count"].float() / (n * n)[:, None]
    a = a.repeat_interleave(T, 0)
    gw = torch.where(live, s["d_weights"], 0.0) * c["scale"]
    sel = weight.gather(1, at)
    if c["normalize"]:
        q = sel / sel.sum(-1, keepdim=True)
        gl = q * (gw - (q * gw).sum(-1, keepdim=True))
        if c["score"] == "sigmoid":
            gl = gl * (1 - sel)
    elif c["score"] == "sigmoid":
        gl = gw * sel * (1 - sel)
    else:
        gl = gw * sel
    d = p * (a - (a * p).sum(-1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * (1 - weight)
    elif not c["normalize"]:
        d = d - p * gl.sum(-1, keepdim=True)
    d = d.scatter_add(1, at, gl)
    if s["mask"] is not None:
        d = torch.where((s["mask"] != 0)[:, None], d, 0.0)
    return d.to(s["logits"].dtype)


def _combine_grad(s):
    c, row = s["case"], s["lay"]["row"]
    N, K = c["ranks"] * c["tokens"], c["topk"]
    row, w = row.reshape(N, K), s["w"].reshape(N, K)
    rows = s["y"].shape[0]
    g = s["d_out"].reshape(N, -1).float()
    y = s["y"].float()[row.clamp(min=0)]
    d_w = torch.where(row >= 0, (y * g[:, None]).sum(-1), 0.0)
    to = torch.where(row >= 0, row, rows).reshape(-1)
    share = torch.zeros(rows + 1, device=g.device).index_add(0, to, w.reshape(-1))
    token = torch.full((rows + 1,), N, dtype=torch.int64, device=g.device)
    token = token.scatter(0, to, torch.arange(N, device=g.device).repeat_interleave(K))[:-1]
    g = torch.cat([g, torch.zeros_like(g[:1])])
    d_y = torch.where((token < N)[:, None], share[:-1, None] * g[token], 0.0)
    return d_y.to(s["y"].dtype), d_w.reshape(s["w"].shape)


def _gelu(z):
    return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))


def _act(z, act):
    if act == "swiglu":
        a, b = z.chunk(2, -1)
        return a / (1 + torch.exp(-a)) * b
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return _gelu(z) if act == "gelu" else z


def _d_act(z, g, act):
    if act == "swiglu":
        a, b = z.chunk(2, -1)
        t = 1 / (1 + torch.exp(-a))
        return torch.cat([g * b * t * (1 + a * (1 - t)), g * a * t], -1)
    if act == "relu":
        return torch.where(z > 0, g, 0.0)
    if act == "silu":
        t = 1 / (1 + torch.exp(-z))
        return g * t * (1 + z * (1 - t))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return g * (cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    return g


def _batch(s, t):
    """Rows as a batch of equal groups [E, most, columns], empty places zero."""
    E, most = s["case"]["experts"], s["lay"]["most"]
    to = torch.where(s["live"], s["cell"], E * most)
    out = torch.zeros(E * most + 1, t.shape[1], device=t.device)
    return out.index_copy(0, to, t.float())[:-1].reshape(E, most, -1)


def _rows(s, t):
    """The batch's rows back at their places, the rows of no group zero."""
    t = t.reshape(-1, t.shape[-1])
    return torch.where(s["live"][:, None], t[s["cell"]], 0.0)


def _product(s):
    c = s["case"]
    x = s["x"]
    if s["x_sf"] is not None:
        x = (x.view(torch.float8_e4m3fn).float().reshape(len(x), -1, 128) * s["x_sf"][..., None]).reshape(len(x), -1)
    z = torch.bmm(_batch(s, x), s["w"].float().transpose(1, 2))
    if s["b"] is not None:
        z = z + s["b"].float()[:, None]
    out = _rows(s, _act(z, c["act"]))
    if s["res"] is not None:
        out = torch.where(s["live"][:, None], out + s["res"].float(), 0.0)
    out = out.to(torch.bfloat16)
    return (out, _rows(s, z).to(torch.bfloat16)) if c["save"] else (out,)


def _product_grad(s):
    c = s["case"]
    dz = _batch(s, _d_act(s["z"].float(), s["d_out"].float(), c["act"]))
    d_x = _rows(s, torch.bmm(dz, s["w"].float()))
    d_w = torch.bmm(dz.transpose(1, 2), _batch(s, s["x"]))
    d_x, d_w = d_x.to(torch.bfloat16), d_w.to(torch.bfloat16)
    return (d_x, d_w, dz.sum(1)) if c["bias"] else (d_x, d_w)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"route": _route, "route_grad": _route_grad, "combine_grad": _combine_grad, "product": _product,
                "product_grad": _product_grad}[op](s)
    ep, cfg, kept, ws = s["handle"]
    if op == "route":
        ep.ep_route(cfg, s["logits"], s["bias"], s["mask"], kept, ws)
        return kept.topk_idx, kept.topk_weights, kept.expert_count, kept.prob_sum, kept.num_valid, kept.balance_loss
    if op == "route_grad":
        ep.ep_route_grad(cfg, s["logits"], s["mask"], kept, s["d_weights"], s["d_loss"], s["d_logits"], ws)
        return s["d_logits"]
    if op == "combine_grad":
        ep.ep_combine_grad(cfg, kept, s["y"], s["idx"], s["w"], s["d_out"], s["d_y"], s["d_w"], ws)
        return s["d_y"], s["d_w"]
    if op == "product":
        ep.ep_expert_product(cfg, kept, s["x"], s["x_sf"], s["w"], s["b"], s["res"], s["z"], s["out"], ws)
        return (s["out"], s["z"]) if s["case"]["save"] else (s["out"],)
    ep.ep_expert_product_grad(cfg, kept, s["x"], s["w"], s["z"], s["d_out"], s["d_x"], s["d_w"], s["d_b"], ws)
    return (s["d_x"], s["d_w"], s["d_b"]) if s["case"]["bias"] else (s["d_x"], s["d_w"])


# ------------------------------------------------------------- 64-bit definitions


def _exact_route(s):
    c = s["case"]
    B, T, E, K, G = c["segments"], c["tokens"], c["experts"], c["topk"], c["groups"]
    l = s["logits"].double()
    prob = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    key = (l if c["score"] == "softmax" else prob).clone()
    if s["bias"] is not None:
        key += s["bias"].double()
    if G > 1:
        g = torch.topk(key.reshape(B * T, G, E // G), 2, dim=-1)[0].sum(-1)
        allowed = torch.zeros_like(g).scatter_(1, torch.sort(g, dim=-1, descending=True, stable=True)[1][:, :c["keep"]], 1.0)
        key[allowed.repeat_interleave(E // G, 1) == 0] = -math.inf
    idx = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :K]
    w = torch.gather(prob, 1, idx)
    w = c["scale"] * (w / w.sum(1, True) if c["normalize"] else w)
    m = torch.ones(B * T, dtype=torch.float64, device=l.device) if s["mask"] is None else s["mask"].double()
    p = (prob / prob.sum(1, True)) * m[:, None]
    hit = torch.zeros(B * T, E, dtype=torch.float64, device=l.device).scatter_(1, idx, 1.0) * m[:, None]
    n = m.reshape(B, T).sum(1).clamp(min=1)
    P, f = p.reshape(B, T, E).sum(1), hit.reshape(B, T, E).sum(1)
    loss = ((f * E / (K * n[:, None])) * (P / n[:, None])).sum(1).mean()
    return None, w * m[:, None], None, P, None, loss.reshape(1)


def _exact_route_grad(s):
    """Through autograd on the weights and the loss, the choice and the counts held fixed."""
    c = s["case"]
    B, T, E, K = c["segments"], c["tokens"], c["experts"], c["topk"]
    l = s["logits"].double().requires_grad_(True)
    m = torch.ones(B * T, dtype=torch.float64, device=l.device) if s["mask"] is None else s["mask"].double()
    prob = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    w = torch.gather(prob, 1, s["idx"].clamp(min=0))
    w = c["scale"] * (w / w.sum(1, True) if c["normalize"] else w)
    n = s["valid"].double().clamp(min=1)
    P = ((prob / prob.sum(1, True)) * m[:, None]).reshape(B, T, E).sum(1)
    loss = ((s["count"].double() * E / (K * n[:, None])) * (P / n[:, None])).sum(1).mean()
    with torch.enable_grad():
        total = (w * m[:, None] * s["d_weights"].double()).sum() + loss * s["d_loss"].double()[0]
    return torch.autograd.grad(total, l)[0]


def _exact_combine_grad(s):
    c, row = s["case"], s["lay"]["row"]
    d_w = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    d_y = torch.zeros(s["y"].shape, dtype=torch.float32, device="cuda").double() if s["y"].numel() < 1 << 31 else None
    for r in range(c["ranks"]):
        g = s["d_out"][r].double()
        for k in range(c["topk"]):
            on = row[r, :, k] >= 0
            at = row[r, on, k]
            d_w[r, on, k] = (s["y"][at].double() * g[on]).sum(-1)
            if d_y is not None:
                d_y.index_add_(0, at, s["w"][r, on, k].double()[:, None] * g[on])
    return d_y, d_w


def _exact_product(s):
    c = s["case"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    pre = torch.zeros(len(out), s["w"].shape[1], dtype=torch.float64, device="cuda")
    for e, (a, n) in enumerate(zip(s["lay"]["start"].tolist(), s["lay"]["count"].reshape(-1).tolist())):
        x = s["x"][a:a + n]
        x = x.double() if s["x_sf"] is None else x.view(torch.float8_e4m3fn).double() * s["x_sf"][a:a + n].double().repeat_interleave(128, 1)
        z = x @ s["w"][e].double().T
        if s["b"] is not None:
            z = z + s["b"][e].double()
        F = torch.nn.functional
        if c["act"] == "swiglu":
            v = F.silu(z[:, :c["outer"]]) * z[:, c["outer"]:]
        else:
            v = {"none": lambda t: t, "relu": F.relu, "silu": F.silu, "gelu": F.gelu}[c["act"]](z)
        out[a:a + n] = v if s["res"] is None else v + s["res"][a:a + n].double()
        pre[a:a + n] = z
    return (out, pre) if c["save"] else (out,)


def _exact_product_grad(s):
    c = s["case"]
    F = torch.nn.functional
    d_x = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    d_w = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
    d_b = torch.zeros(s["w"].shape[:2], dtype=torch.float64, device="cuda")
    for e, (a, n) in enumerate(zip(s["lay"]["start"].tolist(), s["lay"]["count"].reshape(-1).tolist())):
        z = s["z"][a:a + n].double().requires_grad_(True)
        with torch.enable_grad():
            if c["act"] == "swiglu":
                v = F.silu(z[:, :c["outer"]]) * z[:, c["outer"]:]
            else:
                v = {"none": lambda t: t * 1, "relu": F.relu, "silu": F.silu, "gelu": F.gelu}[c["act"]](z)
        dz = torch.autograd.grad(v, z, s["d_out"][a:a + n].double())[0]
        d_x[a:a + n] = dz @ s["w"][e].double()
        d_w[e] = dz.T @ s["x"][a:a + n].double()
        d_b[e] = dz.sum(0)
    return (d_x, d_w, d_b) if c["bias"] else (d_x, d_w)


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "combine_grad": _exact_combine_grad,
            "product": _exact_product, "product_grad": _exact_product_grad}[case["op"]](s)


# ------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        N, E, K = c["segments"] * c["tokens"], c["experts"], c["topk"]
        size = 4 if c["logits"] == "fp32" else 2
        if c["op"] == "route":
            return {"bytes": N * E * size + N * K * 12 + c["segments"] * E * 8, "flops": N * E * 8}
        return {"bytes": 2 * N * E * size + N * K * 12, "flops": N * E * 12}
    if c["op"] == "combine_grad":
        lanes = c["ranks"] * c["tokens"] * c["topk"] * (1 - c["masked"])
        rows = lanes
        if not c["expand"]:  # distinct ranks of a token's lanes, were the lanes spread evenly
            rows = c["ranks"] * c["tokens"] * c["ranks"] * (1 - (1 - 1 / c["ranks"]) ** (c["topk"] * (1 - c["masked"])))
        rows = min(rows, lanes)
        H = c["hidden"]
        return {"bytes": int(c["ranks"] * c["tokens"] * H * 2 + rows * H * 4 + lanes * 20), "flops": int(lanes * H * 3)}
    rows, I, O = c["ranks"] * c["tokens"] * c["topk"], c["inner"], c["outer"]
    Z = 2 * O if c["act"] == "swiglu" else O
    used = c["experts"] if c["experts"] == 1 else c["experts"] * (1 - (1 - c["topk"] / c["experts"]) ** (c["ranks"] * c["tokens"]))
    mats = int(used * Z * I * 2)
    if c["op"] == "product":
        x = rows * I * (1 + 4 / 128) if c["x"] == "fp8" else rows * I * 2
        return {"bytes": int(x + mats + rows * O * (4 if c["residual"] else 2) + (rows * Z * 2 if c["save"] else 0)
                             + (used * Z * 2 if c["bias"] else 0)), "flops": 2 * rows * I * Z}
    return {"bytes": int(rows * (4 * I + 2 * Z + 2 * O) + mats + c["experts"] * Z * (2 * I + (4 if c["bias"] else 0))),
            "flops": 4 * rows * I * Z}
