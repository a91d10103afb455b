"""Rows kept in 8 bits against the definitions: the cast and the way back bit for bit, the backward pass
through the activation against 64 bits.

Error bound of the activations and their derivatives: the exponential is off by 2 + 1.2 |z| steps of 2^-23
(|z| <= 16 here, exp(-z^2/2) is small before that counts), the quotient by 2 steps, so the sigmoid by
2^-18.4 of itself, and s (1 + z (1 - s)) by less than 2^-17 (1 + |z|): FUN, relative to that and to the
factors beside it."""
import pytest
import torch

import _block_reference as ref

pytestmark = pytest.mark.gpu
FUN = 2.0 ** -17
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


@pytest.fixture(scope="module")
def ep():
    import combine_ep_get_02_gb300 as ep
    ep.lib()
    return ep


def blocks_of(ep, counts, R, align=1, slack=0):
    """(layout, [(begin, count)], rows) of experts' blocks with these counts; `slack` rows behind the last."""
    E, L = len(counts), len(counts) // R
    begin, base, region, at = [], [], [0], 0
    for e, n in enumerate(counts):
        if e % L == 0:
            start = at
        base.append(at - start)
        begin.append(at)
        at += (n + align - 1) // align * align
        if e % L == L - 1:
            base.append(at - start)
            region.append(at)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lay = ep.Layout(*[None] * 6, i32(counts), i32(base), i32(region))
    return lay, list(zip(begin, counts)), at + slack


def live_rows(blocks, rows):
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, c in blocks:
        live[a:a + c] = True
    return live


CASES = [([3], 1, 1, 0), ([0, 1, 64, 65], 2, 1, 5), ([0, 0, 0, 0], 2, 1, 7), ([200, 0, 1, 63, 130, 5, 0, 77], 4, 16, 3),
         ([1] * 40, 8, 128, 0), ([700, 31], 1, 1, 0)]


@pytest.mark.parametrize("packed", [False, True], ids=["fp32sf", "packed"])
@pytest.mark.parametrize("features", [128, 384, 1024, 1152])
@pytest.mark.parametrize("counts,R,align,slack", CASES)
def test_keep_and_back(ep, counts, R, align, slack, features, packed):
    lay, blocks, rows = blocks_of(ep, counts, R, align, slack)
    g = torch.Generator(device="cuda").manual_seed(features + rows)
    x = torch.randn(rows, features, generator=g, device="cuda")
    x[:, :64] *= torch.exp(4 * torch.randn(rows, 64, generator=g, device="cuda"))
    x = x.bfloat16()
    x[:, 128:256:7] = 0
    live, G = live_rows(blocks, rows), features // 128
    x[~live] = torch.nan
    cfg = ep.CheckpointConfig(R, len(counts), rows, features, sf_pack=int(packed))
    ws = ep.alloc_checkpoint_workspace(cfg)
    codes = torch.full((rows, features), 0x5A, dtype=torch.uint8, device="cuda")
    sf = torch.full((rows, (G + 3) // 4 if packed else G), 7.5, device="cuda")
    ep.ep_checkpoint(cfg, lay, x, codes, sf, ws)
    want, want_sf = ref.cast(x[live], packed)
    assert torch.equal(codes[live], want) and torch.equal(sf[live].view(torch.int32), want_sf.view(torch.int32))
    assert (codes[~live] == 0x5A).all() and (sf[~live] == 7.5).all()
    # within the header's bound of what was kept
    kept = ref.values(codes[live], sf[live], packed)
    err, scale = (kept - x[live].double()).abs(), ref.scales(sf[live], features, packed).double()
    assert (err <= x[live].double().abs() * (2.0 ** -4 + 2.0 ** -22) + scale * 2.0 ** -10).all()
    back = torch.full((rows, features), 3.25, dtype=torch.bfloat16, device="cuda")
    ep.ep_checkpoint_rows(cfg, lay, codes.view(torch.float8_e4m3fn), sf, back, ws)
    v = codes.view(torch.float8_e4m3fn).float() * ref.scales(sf, features, packed)
    assert torch.equal(back[live], v[live].bfloat16()) and (back[~live] == 3.25).all()
    if packed:
        assert torch.equal(back[live].double(), kept)
    assert ep.ep_check_error(ws) == ep.EP_OK and not ws[:256].any()


def test_every_code_comes_back(ep):
    """All 256 codes with scales from the least to the largest powers of two, and fp32 ones."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(255, 1)
    e = torch.arange(255, dtype=torch.uint8, device="cuda")
    words = torch.zeros(255, 4, dtype=torch.uint8, device="cuda")
    words[:, 0], words[:, 1] = e, e.flip(0)
    for packed, sf in ((1, words.view(torch.float32)), (0, torch.exp2(torch.randn(255, 2, device="cuda") * 20))):
        cfg = ep.CheckpointConfig(1, 1, 255, 256, sf_pack=packed)
        x = torch.empty(255, 256, dtype=torch.bfloat16, device="cuda")
        ep.ep_checkpoint_rows(cfg, None, codes, sf, x, ep.alloc_checkpoint_workspace(cfg))
        want = ref.values(codes, sf, packed)
        want = torch.where(want.abs() < 2.0 ** 128, want, want * torch.inf).float().bfloat16()
        nan = codes.view(torch.float8_e4m3fn).float().isnan()
        assert torch.equal(x.isnan(), nan) and torch.equal(x[~nan], want[~nan])


def test_same_as_the_dispatch_casts(ep):
    R, T, E, K, H = 2, 64, 8, 2, 384
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(R, T, H, generator=g, device="cuda").bfloat16()
    idx = torch.rand(R, T, E, generator=g, device="cuda").topk(K).indices
    w = torch.ones(R, T, K, device="cuda")
    for packed in (0, 1):
        got = []
        for fp8 in (0, 1):
            c = ep.Config(1, R, E, K, T, T, H, expand=1, recv_dtype=fp8, sf_pack=packed * fp8)
            lay, recv, ws = ep.alloc_layout(c), ep.alloc_recv(c), ep.alloc_workspace(c)
            ep.ep_get_dispatch_layout(c, idx, lay, ws)
            ep.ep_dispatch(c, lay, x, None, idx, w, recv, ws)
            got.append((lay, recv))
        rows = got[0][1].recv_x.shape[0]
        cfg = ep.CheckpointConfig(R, E, rows, H, sf_pack=packed)
        ws = ep.alloc_checkpoint_workspace(cfg)
        codes, sf = torch.empty_like(got[1][1].recv_x), torch.empty_like(got[1][1].recv_sf)
        ep.ep_checkpoint(cfg, got[0][0], got[0][1].recv_x, codes, sf, ws)
        assert torch.equal(codes, got[1][1].recv_x) and torch.equal(sf.view(torch.int32), got[1][1].recv_sf.view(torch.int32))


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("packed", [False, True], ids=["fp32sf", "packed"])
@pytest.mark.parametrize("features", [128, 640, 1024])
@pytest.mark.parametrize("counts,R,align,slack", CASES)
def test_backward(ep, counts, R, align, slack, features, packed, kind):
    lay, blocks, rows = blocks_of(ep, counts, R, align, slack)
    g = torch.Generator(device="cuda").manual_seed(features + rows)
    live, n = live_rows(blocks, rows), features // (2 if kind == "swiglu" else 1)
    x = (2 * torch.randn(rows, features, generator=g, device="cuda")).clamp(-16, 16)
    codes, sf = ref.cast(x, packed)
    d_h = torch.randn(rows, n, generator=g, device="cuda").bfloat16()
    codes[~live], d_h[~live] = 0x7F, torch.nan
    cfg = ep.CheckpointConfig(R, len(counts), rows, features, getattr(ep, f"EP_ACT_{kind.upper()}"), int(packed))
    ws = ep.alloc_checkpoint_workspace(cfg)
    h = torch.full((rows, n), 3.25, dtype=torch.bfloat16, device="cuda")
    d_z = torch.full((rows, features), 3.25, dtype=torch.bfloat16, device="cuda")
    d_bias = torch.full((len(counts), features), torch.nan, device="cuda")
    ep.ep_checkpoint_grad(cfg, lay, codes, sf, d_h, h, d_z, d_bias, ws)
    z = ref.values(codes, sf, packed)
    if not packed:  # the product of code and scale is rounded to fp32
        z = z.float().double()
    want_h, want_z, want_b = ref.checkpoint_grad(blocks, z, d_h.double(), kind)
    assert (h[~live] == 3.25).all() and (d_z[~live] == 3.25).all()
    zl, dl = z[live], d_h[live].double().abs()
    if kind == "swiglu":
        a, b = zl[:, :n].abs(), zl[:, n:].abs()
        size_h, size_z = a * b, torch.cat([dl * b * (1 + a), dl * a], 1)
    else:
        size_h, size_z = zl.abs(), dl * (1 + zl.abs())
    half = ref.HALF[torch.bfloat16]
    assert ((h[live].double() - want_h[live]).abs() <= want_h[live].abs() * half + size_h * FUN).all()
    assert ((d_z[live].double() - want_z[live]).abs() <= want_z[live].abs() * half + size_z * FUN).all()
    full = torch.zeros(rows, features, dtype=torch.float64, device="cuda")
    full[live] = size_z
    for e, (a, c) in enumerate(blocks):  # terms off by FUN, at most c + 16 additions
        bound = full[a:a + c].sum(0) * (FUN + (c + 16) * 2.0 ** -24)
        assert ((d_bias[e].double() - want_b[e]).abs() <= bound).all()
    # each output alone, the same bits
    h2, z2, b2 = torch.empty_like(h), torch.empty_like(d_z), torch.empty_like(d_bias)
    ep.ep_checkpoint_grad(cfg, lay, codes, sf, d_h, h2, None, None, ws)
    ep.ep_checkpoint_grad(cfg, lay, codes, sf, d_h, None, z2, None, ws)
    ep.ep_checkpoint_grad(cfg, lay, codes, sf, d_h, None, None, b2, ws)
    assert torch.equal(h2[live], h[live]) and torch.equal(z2[live], d_z[live]) and torch.equal(b2, d_bias)
    assert ep.ep_check_error(ws) == ep.EP_OK and not ws[:256].any()


def test_many_tiles(ep):
    """More tiles of a group than CTAs finish at once, and more groups than the header counts."""
    for counts, features in (([20000, 3], 384), ([5] * 500, 256), ([1000] * 60, 1024)):
        test_backward(ep, counts, 1, 1, 0, features, False, "swiglu")
        test_keep_and_back(ep, counts, 1, 1, 0, features, True)


def test_gradient_against_differences(ep):
    """<d_z, v> against central differences of <d_h, act(z)> in 64 bits (their own error below 1e-6 of the
    sum of magnitudes)."""
    rows, features = 64, 256
    g = torch.Generator(device="cuda").manual_seed(8)
    codes, sf = ref.cast(torch.randn(rows, features, generator=g, device="cuda"), True)
    for kind in ("silu", "gelu", "swiglu"):
        n = features // (2 if kind == "swiglu" else 1)
        d_h = torch.randn(rows, n, generator=g, device="cuda").bfloat16()
        cfg = ep.CheckpointConfig(1, 1, rows, features, getattr(ep, f"EP_ACT_{kind.upper()}"), 1)
        d_z = torch.empty(rows, features, dtype=torch.bfloat16, device="cuda")
        ep.ep_checkpoint_grad(cfg, None, codes, sf, d_h, None, d_z, None, ep.alloc_checkpoint_workspace(cfg))
        z, v = ref.values(codes, sf, True), torch.randn(rows, features, generator=g, device="cuda", dtype=torch.float64)
        f = lambda t: (ref.act(t, kind) * d_h.double()).sum()  # noqa: E731
        along = (f(z + 1e-4 * v) - f(z - 1e-4 * v)) / 2e-4
        size = (d_z.double() * v).abs().sum()
        assert abs((d_z.double() * v).sum() - along) <= size * 2.0 ** -8


def test_blocks_that_do_not_belong(ep):
    """Blocks past the rows are cut and overlapping ones left out: reported, and nothing is written outside."""
    rows, F = 100, 256
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for counts, base, region in (([90, 90], [0, 90, 180], [0, 180]), ([1 << 30, 5], [0, 50, 60], [0, 60]),
                                 ([-5, 10], [-20, 0, 10], [0, 10])):
        lay = ep.Layout(*[None] * 6, i32(counts), i32(base), i32(region))
        cfg = ep.CheckpointConfig(1, 2, rows, F, ep.EP_ACT_SWIGLU)
        ws = ep.alloc_checkpoint_workspace(cfg)
        guard = torch.full((rows + 2, F), 9.0, dtype=torch.bfloat16, device="cuda")
        codes, sf = ref.cast(torch.randn(rows, F, device="cuda"), False)
        ep.ep_checkpoint_rows(cfg, lay, codes, sf, guard[:rows], ws)
        assert ep.ep_check_error(ws) == ep.EP_ERR_OVERFLOW and (guard[rows:] == 9.0).all()
        d_h, b = torch.randn(rows, F // 2, device="cuda").bfloat16(), torch.empty(2, F, device="cuda")
        ep.ep_checkpoint_grad(cfg, lay, codes, sf, d_h, None, guard[:rows], b, ws)
        assert ep.ep_check_error(ws) == ep.EP_ERR_OVERFLOW and (guard[rows:] == 9.0).all()


def test_no_rows(ep):
    cfg = ep.CheckpointConfig(1, 1, 0, 256)
    ws, none = ep.alloc_checkpoint_workspace(cfg), torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    codes, sf, b = none.to(torch.float8_e4m3fn), torch.empty(0, 2, device="cuda"), torch.ones(1, 256, device="cuda")
    ep.ep_checkpoint(cfg, None, none, codes, sf, ws)
    ep.ep_checkpoint_rows(cfg, None, codes, sf, none, ws)
    ep.ep_checkpoint_grad(cfg, None, codes, sf, none, none, none, b, ws)
    assert (b == 0).all()
