"""The experts' products and their gradients against the 64-bit definitions."""
import math

import pytest
import torch

import _moe_reference as ref
import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu

ACTS = {"none": ep.EP_ACT_NONE, "relu": ep.EP_ACT_RELU, "silu": ep.EP_ACT_SILU, "gelu": ep.EP_ACT_GELU,
        "swiglu": ep.EP_ACT_SWIGLU}


def blocks_of(counts, R, align=1, gap=0):
    """Layout arrays and (begin, count) of blocks with these counts; `gap` rows in front of each region."""
    E, L = len(counts), len(counts) // R
    region, base, blocks, row = [], [], [], 0
    for d in range(R):
        row += gap
        region.append(row)
        at, line = 0, []
        for j in range(L):
            line.append(at)
            blocks.append((row + at, counts[d * L + j]))
            at += (counts[d * L + j] + align - 1) // align * align
        base.append(line + [at])
        row += at
    region.append(row)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lay = ep.Layout(*[None] * 6, i32(counts).reshape(R, L), i32(base), i32(region))
    return lay, blocks, row


class Case:
    def __init__(self, counts, K, N, act="none", R=1, bias=False, residual=False, align=1, gap=0, dense=False, seed=0,
                 spare=0, **cfg):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s, scale=1.0: (torch.randn(*s, device="cuda", generator=g) * scale).bfloat16()  # noqa: E731
        self.act, self.K, self.N, self.E = act, K, N, len(counts)
        if dense:
            self.lay, self.blocks, rows = None, [(0, counts[0])], counts[0]
        else:
            self.lay, self.blocks, rows = blocks_of(counts, R, align, gap)
        rows += spare
        self.rows, self.cfg = rows, ep.ProductConfig(R, self.E, rows, K, N, ACTS[act], **cfg)
        self.Z = self.cfg.z_features
        self.x = rnd(rows, K)
        self.w = rnd(self.E, self.Z, K, scale=K ** -0.5)
        self.bias = rnd(self.E, self.Z) if bias else None
        self.res = rnd(rows, N) if residual else None
        self.z_in = rnd(rows, self.Z)
        self.d_out = rnd(rows, N)
        self.live = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for a, n in self.blocks:
            self.live[a:a + n] = True
        # what no result may depend on
        for t in (self.x, self.res, self.z_in, self.d_out):
            if t is not None:
                t[~self.live] = math.nan

    def forward(self, x=None, x_sf=None, keep=True, cfg=None):
        cfg = cfg or self.cfg
        out = torch.full((self.rows, self.N), 33.0, device="cuda").bfloat16()
        z = torch.full((self.rows, self.Z), 33.0, device="cuda").bfloat16() if keep else None
        ws = ep.alloc_product_workspace(cfg)
        ep.ep_expert_product(cfg, self.lay, self.x if x is None else x, x_sf, self.w, self.bias, self.res, z, out, ws)
        assert ep.ep_check_error(ws) == ep.EP_OK
        assert (out[~self.live] == 33.0).all() and (z is None or (z[~self.live] == 33.0).all())
        return out, z

    def grads(self, d_x=True, d_w=True, d_b=True, cfg=None):
        cfg = cfg or self.cfg
        dx = torch.full_like(self.x, 33.0) if d_x else None
        dw = torch.full_like(self.w, 33.0) if d_w else None
        db = torch.full((self.E, self.Z), 33.0, device="cuda") if d_b else None
        ws = ep.alloc_product_workspace(cfg, grad=True)
        ws[256:].fill_(0xFF)  # NaN wherever the workspace is read without being written
        ep.ep_expert_product_grad(cfg, self.lay, self.x, self.w, self.z_in, self.d_out, dx, dw, db, ws)
        assert ep.ep_check_error(ws) == ep.EP_OK
        if d_x:
            assert (dx[~self.live] == 33.0).all()
        return dx, dw, db

    def check(self):
        out, z = self.forward()
        want, want_z = ref.product(self.blocks, self.x, self.w, self.bias, self.res, self.act)
        m = self.live
        # fp32 sums of K exact products (2^-20 of the sum of magnitudes at most), one rounding to
        # bf16; the activation's own error is below both
        slack = 2 ** -20 * (self.K ** 0.5 + 4)
        near(z[m], want_z[m], 2 ** -8, slack)
        near(out[m], want[m], 2 ** -8, slack * 4)

    def grad_terms(self):
        """(sum over z of (dz w)^2)^0.5 and (sum over the group's rows of (dz x)^2)^0.5."""
        tx, tw = torch.zeros_like(self.x, dtype=torch.float64), torch.zeros_like(self.w, dtype=torch.float64)
        for g, (a, n) in enumerate(self.blocks):
            z = self.z_in[a:a + n].double().requires_grad_(True)
            (dz,) = torch.autograd.grad(ref.act(z, self.act), z, self.d_out[a:a + n].double())
            tx[a:a + n] = (dz ** 2 @ self.w[g].double() ** 2).sqrt()
            tw[g] = ((dz ** 2).T @ self.x[a:a + n].double() ** 2).sqrt()
        return tx, tw

    def check_grads(self):
        dx, dw, db = self.grads()
        want = ref.product_grad(self.blocks, self.x, self.w, self.z_in, self.d_out, self.act)
        m = self.live
        # dz is rounded to bf16, 2^-9 of each term at most, with signs of their own: a sum of terms
        # t_i is off by 2^-9 (sum t_i^2)^0.5 / 3^0.5 typically, and six times 3^0.5 of that is
        # allowed (one term alone stays within it); then the result is rounded once
        tx, tw = self.grad_terms()
        near(dx[m], want[0][m], 2 ** -8, 6 * 2 ** -9 * tx[m])
        near(dw, want[1], 2 ** -8, 6 * 2 ** -9 * tw)
        near(db, want[2], 1e-5, 1e-5 * max(rms(want[2]), 1e-3) * 10)
        for g, (_, n) in enumerate(self.blocks):
            if n == 0:
                assert (dw[g] == 0).all() and (db[g] == 0).all()


def rms(t):
    return float(t.double().square().mean().sqrt()) if t.numel() else 0.0


def near(got, want, rtol, atol):
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - rtol * want.abs() - atol  # atol: a number or one per value
    assert got.numel() == 0 or float(off.max()) <= 0, f"off by {float((got - want).abs().max())}, {int((off > 0).sum())} values"


SHAPES = {
    "one_row": dict(counts=[1], K=8, N=8, dense=True),
    "one_token_wide": dict(counts=[1], K=7168, N=2048, dense=True, act="swiglu"),
    "dense_exact_tiles": dict(counts=[256], K=128, N=512, dense=True, bias=True, residual=True),
    "dense_odd": dict(counts=[131], K=200, N=264, dense=True, act="gelu", bias=True),
    "one_past": dict(counts=[129, 127, 128], K=64, N=256, act="silu", bias=True),
    "ragged_with_empty": dict(counts=[0, 3, 0, 130, 1, 0, 64, 0], K=136, N=72, R=4, act="relu", bias=True, residual=True),
    "all_empty": dict(counts=[0, 0, 0, 0], K=64, N=64, R=2, spare=5),
    "aligned": dict(counts=[5, 0, 17, 40], K=320, N=136, R=2, align=16, act="swiglu", bias=True),
    "regions_apart": dict(counts=[20, 33, 1, 64], K=72, N=8, R=4, align=4, gap=9, spare=200, act="swiglu", residual=True),
    "gated_odd": dict(counts=[70, 190], K=1000, N=200, act="swiglu", bias=True, residual=True),
    "many_experts": dict(counts=[(i * 7) % 5 for i in range(600)], K=64, N=16, R=4, act="gelu", bias=True),
    "tall": dict(counts=[2500, 10], K=256, N=328, act="silu"),
    "wide": dict(counts=[40, 300], K=2056, N=1544, act="none", bias=True),
    "many_tiles": dict(counts=[30] * 18 + [0, 60], K=264, N=2000, R=4, act="silu", bias=True, residual=True),
    "many_tiles_gated": dict(counts=[(i * 13) % 61 for i in range(24)], K=200, N=1000, act="swiglu", bias=True),
    "long_groups": dict(counts=[700, 257, 900], K=392, N=264, act="gelu", bias=True, residual=True),
    "long_groups_gated": dict(counts=[1000, 0, 513, 400], K=192, N=200, act="swiglu", R=2, align=8, bias=True),
    "long_dense": dict(counts=[1003], K=1032, N=776, dense=True, act="relu", bias=True, residual=True),
    "split_groups": dict(counts=[5, 0, 20], K=1096, N=200, act="gelu", bias=True, residual=True),
    "split_gated_rows": dict(counts=[90], K=2120, N=1104, dense=True, act="swiglu", bias=True, residual=True),
    "few_rows_each": dict(counts=[2, 8, 1, 5, 16, 3, 9, 32], K=1024, N=640, R=2, act="swiglu"),
}


@pytest.mark.parametrize("name", SHAPES)
def test_forward(name):
    Case(**SHAPES[name]).check()


@pytest.mark.parametrize("name", SHAPES)
def test_gradients(name):
    Case(**SHAPES[name]).check_grads()


@pytest.mark.parametrize("act", ACTS)
def test_every_activation(act):
    c = Case([30, 100, 7], 96, 64, act=act, bias=True, residual=True)
    c.z_in *= 3
    c.check()
    c.check_grads()


def test_most_experts():
    c = Case([1 if i % 9 == 0 else 0 for i in range(4096)], 8, 8, R=64, act="silu", bias=True)
    c.check()
    c.check_grads()


def test_gradient_against_differences():
    """The derivative along a random direction of the 64-bit forward, by central differences."""
    for act in ACTS:
        c = Case([9, 0, 20], 40, 24, act=act, bias=True, seed=5)
        _, z = ref.product(c.blocks, c.x, c.w, c.bias, None, act)
        m = c.live
        c.z_in[m] = z[m].bfloat16()
        dx, dw, db = c.grads()
        g = torch.Generator(device="cuda").manual_seed(1)
        for name in ("x", "w", "bias"):
            base = getattr(c, name).double()
            v = torch.randn(base.shape, device="cuda", generator=g, dtype=torch.float64)
            f = []
            for s in (1e-4, -1e-4):
                args = {k: getattr(c, k).double() for k in ("x", "w", "bias")}
                args[name] = base + s * v
                out, _ = ref.product(c.blocks, args["x"], args["w"], args["bias"], None, act)
                f.append(float((out[m] * c.d_out[m].double()).sum()))
            slope = (f[0] - f[1]) / 2e-4
            got = {"x": dx, "w": dw, "bias": db}[name].double()
            if name == "x":
                got, v = got[m], v[m]
            # z rounded to bf16 moves act' by 2^-9 |z|, dz and the result are rounded once each; n
            # random terms add up like n^0.5 (relu's step can also be passed by a z near zero)
            tol = 2 ** -6 * float((got * v).square().sum().sqrt())
            assert abs(slope - float((got * v).sum())) <= tol, (act, name)


def test_each_gradient_alone_and_sms():
    c = Case([50, 0, 200], 256, 136, act="swiglu", bias=True)
    dx, dw, db = c.grads()
    assert torch.equal(c.grads(True, False, False)[0][c.live], dx[c.live])
    assert torch.equal(c.grads(False, True, False)[1], dw)
    assert torch.equal(c.grads(False, False, True)[2], db)
    few = Case([50, 0, 200], 256, 136, act="swiglu", bias=True, num_sms=3)
    for a, b in zip(few.grads(), (dx, dw, db)):
        a, b = (a[c.live], b[c.live]) if a.shape == c.x.shape else (a, b)
        assert torch.equal(a, b)
    assert torch.equal(few.forward()[0], c.forward()[0])
    assert torch.equal(c.forward(keep=False)[0], c.forward()[0])


def test_bias_gradients_repeat_on_one_workspace():
    """The counters of finished tiles return to zero: the same call again, from a graph, and other sizes."""
    c = Case([700, 0, 65, 64, 900], 40, 264, act="swiglu", bias=True)
    ws = ep.alloc_product_workspace(c.cfg, grad=True)
    for other in (Case([200], 8, 1000, dense=True, act="silu"), Case([5, 130, 64], 16, 8)):  # they fit the same workspace
        want = other.grads(False, False, True)[2]
        got = torch.empty_like(want)
        ep.ep_expert_product_grad(other.cfg, other.lay, None, None, other.z_in, other.d_out, None, None, got, ws)
        assert torch.equal(got, want) and not ws[:256].any()
    want = c.grads(False, False, True)[2]
    got = [torch.empty_like(want) for _ in range(4)]
    call = lambda out: ep.ep_expert_product_grad(c.cfg, c.lay, None, None, c.z_in, c.d_out, None, None, out, ws)  # noqa: E731
    for t in got[:3]:
        call(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(got[3])
    for _ in range(2):
        got[3].fill_(7)
        graph.replay()
        for t in got:
            assert torch.equal(t, want)
    assert ep.ep_check_error(ws) == ep.EP_OK


def test_pairs_and_single_ctas_agree():
    """Long groups run on pairs of CTAs; one SM cannot: the same sums in the same order."""
    kw = dict(counts=[700, 257, 900], K=392, N=264, act="gelu", bias=True, residual=True)
    a, b = Case(**kw), Case(**kw, num_sms=1)
    for x, y in zip(a.forward(), b.forward()):
        assert torch.equal(x[a.live], y[a.live])
    for x, y in zip(a.grads(), b.grads()):
        assert torch.equal(x, y)


def test_residual_in_place():
    c = Case([100], 64, 128, dense=True, residual=True)
    want, _ = c.forward()
    out = c.res.clone()
    ws = ep.alloc_product_workspace(c.cfg)
    ep.ep_expert_product(c.cfg, None, c.x, None, c.w, None, out, None, out, ws)
    assert torch.equal(out, want)


@pytest.mark.parametrize("pack", [0, 1])
def test_fp8_rows(pack):
    """Rows and scales of an FP8 dispatch: the same as the bf16 product of bf16_rn(code * scale)."""
    c = Case([33, 0, 150, 64], 640, 200, R=2, act="swiglu", spare=17)
    g = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 256, c.x.shape, device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, codes ^ 1, codes)
    G = 5
    if pack:
        e = torch.randint(110, 125, (c.rows, 8), device="cuda", generator=g, dtype=torch.int64)
        e[0, 0] = 0  # the least scale, 2^-127
        sf = torch.exp2((e - 127).double())[:, :G]
        words = e[:, 0::4] | e[:, 1::4] << 8 | e[:, 2::4] << 16 | e[:, 3::4] << 24
        x_sf = words.to(torch.int32).view(torch.float32).contiguous()
    else:
        x_sf = torch.rand(c.rows, G, device="cuda", generator=g) * 1e-2 + 1e-3
        sf = x_sf.double()
    x = codes.view(torch.float8_e4m3fn).double() * sf.repeat_interleave(128, 1)
    cfg = ep.ProductConfig(2, 4, c.rows, 640, 200, ep.EP_ACT_SWIGLU, ep.EP_DTYPE_FP8_E4M3, pack)
    out, z = c.forward(codes, x_sf, cfg=cfg)
    want, want_z = ref.product(c.blocks, x, c.w, None, None, "swiglu")
    m = c.live
    near(z[m], want_z[m], 2 ** -8, 6 * 2 ** -9 * rms(want_z[m]) + 1e-30)
    near(out[m], want[m], 2 ** -8, 12 * 2 ** -9 * max(rms(want[m]), rms(want_z[m])) + 1e-30)


def test_no_rows():
    c = Case([1, 1], 64, 32, act="silu", bias=True)
    cfg = ep.ProductConfig(1, 2, 0, 64, 32, ep.EP_ACT_SILU)
    ws = ep.alloc_product_workspace(cfg, grad=True)
    empty = lambda n: torch.empty(0, n, device="cuda").bfloat16()  # noqa: E731
    lay, _, _ = blocks_of([0, 0], 1)
    ep.ep_expert_product(cfg, lay, empty(64), None, c.w, None, None, None, empty(32), ws)
    dw, db = torch.full_like(c.w, 5.0), torch.full((2, 32), 5.0, device="cuda")
    ep.ep_expert_product_grad(cfg, lay, empty(64), c.w, empty(32), empty(32), empty(64), dw, db, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK and (dw == 0).all() and (db == 0).all()


def test_blocks_past_the_rows_are_cut_and_reported():
    c = Case([40, 60], 64, 32)
    guard = torch.full((128, 32), 9.0, device="cuda").bfloat16()
    cfg = ep.ProductConfig(1, 2, 70, 64, 32)
    ws = ep.alloc_product_workspace(cfg)
    ep.ep_expert_product(cfg, c.lay, c.x, None, c.w, None, None, None, guard[:70], ws)
    assert ep.ep_check_error(ws) == ep.EP_ERR_OVERFLOW
    want, _ = c.forward()
    assert torch.equal(guard[:70], want[:70]) and (guard[70:] == 9.0).all()


def test_offsets_past_32_bits():
    """Outputs of more than 2^31 elements: the last block against the definition, forward and gradients."""
    rows, K, N = 300_000, 64, 8192
    lay, blocks, _ = blocks_of([rows - 300, 300], 1)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, K, device="cuda", generator=g).bfloat16()
    w = (torch.randn(2, N, K, device="cuda", generator=g) / 8).bfloat16()
    out = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    cfg = ep.ProductConfig(1, 2, rows, K, N, ep.EP_ACT_RELU)
    ws = ep.alloc_product_workspace(cfg, grad=True)
    z = torch.empty_like(out)
    ep.ep_expert_product(cfg, lay, x, None, w, None, None, z, out, ws)
    want, want_z = ref.product([(0, 300)], x[-300:], w[1:], None, None, "relu")
    near(out[-300:], want, 2 ** -8, 1e-4)
    near(z[-300:], want_z, 2 ** -8, 1e-4)
    first, _ = ref.product([(0, 200)], x[:200], w[:1], None, None, "relu")
    near(out[:200], first, 2 ** -8, 1e-4)
    out.normal_(generator=g)  # now the gradient of the output
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(2, N, device="cuda")
    ep.ep_expert_product_grad(cfg, lay, x, w, z, out, dx, dw, db, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    wx, ww, wb = ref.product_grad([(0, 300)], x[-300:], w[1:], z[-300:], out[-300:], "relu")
    # relu's dz is exact in bf16: one rounding of the result, and fp32 sums of thousands of products
    near(dx[-300:], wx, 2 ** -8, 1e-3 * rms(wx))
    near(dw[1:], ww, 2 ** -8, 1e-3 * rms(ww))
    near(db[1:], wb, 1e-5, 1e-4 * rms(wb))


def test_row_strides_that_do_not_fill_a_tile():
    """Every multiple of 8 around the tile widths, in both features."""
    for K, N in ((8, 264), (56, 8), (64, 72), (72, 120), (120, 136), (136, 248), (248, 256), (264, 56)):
        for act in ("none", "swiglu"):
            c = Case([37, 129, 5], K, N, act=act, bias=True)
            c.check()
            c.check_grads()
