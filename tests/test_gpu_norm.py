"""The norm with the residual's addition, its FP8 rows and its gradients against 64 bits.

Error bounds. A sum over a row is taken in a thread's chain of at most 32 terms and at most 10
pairwise steps: of squares (all positive) it is off by 42 * 2^-24 of itself, so q by 21 * 2^-24, with its
own rounding, eps' addition, s and the two products below 40 * 2^-24: ROW. A rounding to a type adds half
a step of it."""
import os
import subprocess
import sys

import pytest
import torch

import _block_reference as ref

pytestmark = pytest.mark.gpu
ROW = 40 * 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def ep():
    import combine_ep_get_02_gb300 as ep
    ep.lib()
    return ep


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows_of(g, n, h, kind, scale=1.0):
    return (torch.randn(n, h, generator=g, device="cuda") * scale).to(kind)


def config(ep, n, h, kind, **kw):
    return ep.NormConfig(rows=n, hidden=h, x_dtype=ep.EP_DTYPE_FP32 if kind is torch.float32 else ep.EP_DTYPE_BF16,
                         eps=EPS, **kw)


def assert_y(y, want):
    bound = want.abs() * (ref.HALF[torch.bfloat16] + ROW)
    assert ((y.double() - want).abs() <= bound).all()


def assert_rows(codes, sf, want, packed):
    """FP8 rows of values that are known up to ROW: a code is off by half of its step, relative 2^-4
    or 2^-10 of the scale below the normal numbers; a packed scale may be one off where the
    largest value is as near to a power of two as that."""
    H = want.shape[1]
    amax = want.reshape(len(want), -1, 128).abs().amax(-1).clamp(min=1e-4)
    got = ref.scales(sf, H, packed)[:, ::128].double()
    if packed:
        low, high = (torch.exp2(torch.ceil(torch.log2(amax * (1 + s * 2 * ROW) / 448))) for s in (-1, 1))
        assert ((got == low) | (got == high)).all()
        pad = sf.view(torch.uint8)[:, H // 128:]
        assert (pad == 0).all()
    else:
        assert ((got - amax / 448).abs() <= amax / 448 * (ROW + 2.0 ** -24)).all()
    err = (ref.values(codes, sf, packed) - want).abs()
    assert (err <= want.abs() * (2.0 ** -4 + 4 * ROW) + got.repeat_interleave(128, 1) * 2.0 ** -10).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,h", [(1, 8), (3, 24), (5, 256), (153, 264), (7, 512), (9, 520), (64, 1000), (1, 2048), (700, 2048),
                                 (152, 4096), (2, 4104), (1, 7168), (400, 7168), (3, 8192), (160, 8200), (1, 16384),
                                 (170, 16384)])
def test_norm(ep, n, h, kind):
    g = gen(n * 31 + h)
    x, r = rows_of(g, n, h, kind), rows_of(g, n, h, kind, 3.0)
    w = (1 + 0.2 * torch.randn(h, generator=g, device="cuda")).bfloat16()
    cfg = config(ep, n, h, kind)
    y, total = torch.empty(n, h, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    ep.ep_norm(cfg, x, r, w, total, y, None, None)
    assert_y(y, ref.norm(x, r, w, EPS)[2])
    assert torch.equal(total, (x.float() + r.float()).to(kind))
    again = torch.empty_like(y)  # neither residual nor weight nor sum
    ep.ep_norm(cfg, x, None, None, None, again, None, None)
    assert_y(again, ref.norm(x, None, None, EPS)[2])


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True], ids=["fp32sf", "packed"])
@pytest.mark.parametrize("n,h", [(1, 128), (33, 384), (5, 512), (200, 640), (1, 7168), (160, 7168), (4, 16384)])
def test_rows_for_the_dispatch(ep, n, h, packed, kind):
    g = gen(n * 17 + h)
    x, r, w = rows_of(g, n, h, kind), rows_of(g, n, h, kind), (1 + 0.2 * torch.randn(h, generator=g, device="cuda")).bfloat16()
    x[:, ::128] = 0
    cfg, G = config(ep, n, h, kind, sf_pack=int(packed)), h // 128
    codes = torch.full((n, h), 0xFF, dtype=torch.uint8, device="cuda")
    sf = torch.full((n, (G + 3) // 4 if packed else G), torch.nan, device="cuda")
    y = torch.empty(n, h, dtype=torch.bfloat16, device="cuda")
    ep.ep_norm(cfg, x, r, w, None, y, codes, sf)
    want = ref.norm(x, r, w, EPS)[2]
    assert_y(y, want)
    assert_rows(codes, sf, want, packed)
    only, sf2 = torch.empty(n, h, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(sf)  # without y
    ep.ep_norm(cfg, x, r, w, None, None, only, sf2)
    assert torch.equal(only.view(torch.uint8), codes) and torch.equal(sf2.view(torch.int32), sf.view(torch.int32))


def test_sum_in_place(ep):
    g = gen(3)
    for kind in (torch.bfloat16, torch.float32):
        x, r = rows_of(g, 300, 2048, kind), rows_of(g, 300, 2048, kind)
        cfg = config(ep, 300, 2048, kind)
        y, total, y2 = (torch.empty(300, 2048, dtype=t, device="cuda") for t in (torch.bfloat16, kind, torch.bfloat16))
        ep.ep_norm(cfg, x, r, None, total, y, None, None)
        for into in (0, 1):
            a, b = x.clone(), r.clone()
            ep.ep_norm(cfg, a, b, None, (a, b)[into], y2, None, None)
            assert torch.equal((a, b)[into], total) and torch.equal(y2, y) and torch.equal((b, a)[into], (r, x)[into])


@pytest.mark.parametrize("h", [256, 4096])
def test_values_at_the_ends(ep, h):
    """Rows of zeros, of values whose squares leave fp32, with NaN and infinities; their neighbours stay."""
    x = torch.randn(8, h, generator=gen(5), device="cuda")
    x[1] = 0
    x[2] *= 1e25
    x[3] = torch.finfo(torch.bfloat16).max
    x[3, 1::2] *= -1
    x[4] *= 1e-25
    x[5, 7] = torch.nan
    x[6, 7] = torch.inf
    for kind in (torch.bfloat16, torch.float32):
        v, cfg = x.to(kind), config(ep, 8, h, kind)
        y = torch.empty(8, h, dtype=torch.bfloat16, device="cuda")
        ep.ep_norm(cfg, v, None, None, None, y, None, None)
        sure = [0, 1, 2, 3, 4, 7]
        want = ref.norm(v[sure], None, None, EPS)[2]
        # row 4's results are below fp32's normal numbers: half a step of bf16's least ones, and fp32's
        assert ((y[sure].double() - want).abs() <= want.abs() * (2.0 ** -8 + ROW) + 2.0 ** -133).all()
        assert y[5].isnan().all()
        assert y[6, 7].isnan() and (y[6, :7] == 0).all() and (y[6, 8:] == 0).all()
        # gradients of the finite rows
        d_y = torch.randn(8, h, generator=gen(6), device="cuda").bfloat16()
        d_x, ws = torch.empty_like(v), ep.alloc_norm_workspace(cfg)
        ep.ep_norm_grad(cfg, v, None, None, d_y, None, d_x, None, ws)
        want, _, size, _ = ref.norm_grad(v[sure], None, None, d_y[sure], None, EPS)
        assert ((d_x[sure].double() - want).abs() <= want.abs() * ref.HALF[kind] + size * 64 * 2.0 ** -24 + 2.0 ** -133).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,h", [(1, 8), (5, 256), (153, 264), (609, 512), (9, 520), (1, 4096), (700, 2048), (2, 4104),
                                 (620, 7168), (3, 8192), (160, 8200), (1, 16384), (170, 16384), (305, 520), (1300, 1024),
                                 (2000, 1032), (306, 8200), (310, 16384)])
def test_gradients(ep, n, h, kind):
    """d_x: two sums over the row (each ROW of the sum of its terms' magnitudes) and five roundings of
    terms: 2 ROW of their magnitudes, and its own rounding. d_weight: every term off by ROW, at most
    n + 32 additions."""
    g = gen(n * 7 + h)
    s, d_y, d_sum = rows_of(g, n, h, kind, 2.0), rows_of(g, n, h, torch.bfloat16), rows_of(g, n, h, kind)
    w = (1 + 0.2 * torch.randn(h, generator=g, device="cuda")).bfloat16()
    mask = (torch.rand(n, generator=g, device="cuda") > 0.2).to(torch.uint8)
    cfg = config(ep, n, h, kind)
    ws = ep.alloc_norm_workspace(cfg)
    ws[256:] = 0xFF
    for weight, m, through in ((w, None, d_sum), (w, mask, d_sum), (None, mask, None)):
        v, dy, ds = s, d_y, through
        if m is not None:  # nothing may depend on padding
            off = (m == 0)[:, None]
            v, dy = s.masked_fill(off, torch.nan), d_y.masked_fill(off, torch.inf)
            ds = None if through is None else through.masked_fill(off, torch.nan)
        d_x, d_w = torch.full_like(s, torch.nan), torch.full((h,), torch.nan, device="cuda")
        ep.ep_norm_grad(cfg, v, weight, m, dy, ds, d_x, d_w, ws)
        want, want_w, size, size_w = ref.norm_grad(v, weight, m, dy, ds, EPS)
        assert ((d_x.double() - want).abs() <= want.abs() * ref.HALF[kind] + size * 2 * ROW).all()
        assert ((d_w.double() - want_w).abs() <= size_w * (ROW + (n + 32) * 2.0 ** -24)).all()
        first = d_x.clone(), d_w.clone()  # one output only, d_x in d_sum's place, and the same bits again
        if ds is not None:
            place = ds.clone()
            ep.ep_norm_grad(cfg, v, weight, m, dy, place, place, None, ws)
            assert torch.equal(place, first[0])
        ep.ep_norm_grad(cfg, v, weight, m.bool() if m is not None else None, dy, ds, None, d_w, ws)
        assert torch.equal(d_w, first[1])


def test_gradients_against_differences(ep):
    """<d_x, v> and <d_weight, u> against central differences of <d_y, y> in 64 bits. Their own error is a
    third derivative times 1e-8; the gradients' is half a step of fp32 and ROW of their terms."""
    n, h, g = 40, 640, gen(11)
    s, d_y = rows_of(g, n, h, torch.float32), rows_of(g, n, h, torch.bfloat16)
    w = (1 + 0.2 * torch.randn(h, generator=g, device="cuda")).bfloat16()
    cfg = config(ep, n, h, torch.float32)
    d_x, d_w = torch.empty_like(s), torch.empty(h, device="cuda")
    ep.ep_norm_grad(cfg, s, w, None, d_y, None, d_x, d_w, ep.alloc_norm_workspace(cfg))
    f = lambda a, b: (ref.norm(a, None, b, EPS)[2] * d_y.double()).sum()  # noqa: E731
    step = 1e-4
    size, size_w = ref.norm_grad(s, w, None, d_y, None, EPS)[2:]
    for seed in range(4):
        v, u = (torch.randn(*t, generator=gen(seed), device="cuda", dtype=torch.float64) for t in ((n, h), (h,)))
        along = (f(s.double() + step * v, w) - f(s.double() - step * v, w)) / (2 * step)
        assert abs((d_x.double() * v).sum() - along) <= (size * v.abs()).sum() * 4 * ROW + 1e-6 * abs(along) + 1e-5
        along = (f(s, w.double() + step * u) - f(s, w.double() - step * u)) / (2 * step)
        assert abs((d_w.double() * u).sum() - along) <= (size_w * u.abs()).sum() * (ROW + 72 * 2.0 ** -24) + 1e-5


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_values_at_the_ends_among_many_rows(ep, kind):
    """The same through the rows' ring: large values, NaN and infinities stay in their rows; a padding row
    between them is not read."""
    n, h = 700, 2048
    x = torch.randn(n, h, generator=gen(15), device="cuda")
    x[5::16] *= 1e25
    x[6::16] = 0
    x = x.to(kind)
    x[3::16, 9], x[4::16, 11] = torch.nan, torch.inf
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[7::16] = False
    x[7::16] = torch.nan
    d_y = torch.randn(n, h, generator=gen(16), device="cuda").bfloat16()
    cfg = config(ep, n, h, kind)
    d_x, ws = torch.full_like(x, 7.0), ep.alloc_norm_workspace(cfg)
    ep.ep_norm_grad(cfg, x, None, mask, d_y, None, d_x, None, ws)
    i = torch.arange(n, device="cuda") % 16
    sure = (i != 3) & (i != 4) & (i != 7)
    want, _, size, _ = ref.norm_grad(x[sure], None, None, d_y[sure], None, EPS)
    assert ((d_x[sure].double() - want).abs() <= want.abs() * ref.HALF[kind] + size * 4 * ROW + 2.0 ** -133).all()
    assert d_x[3::16].isnan().all() and (d_x[7::16] == 0).all()
    assert ep.ep_check_error(ws) == ep.EP_OK


def test_no_rows(ep):
    cfg = config(ep, 0, 1024, torch.bfloat16)
    empty = torch.empty(0, 1024, dtype=torch.bfloat16, device="cuda")
    ep.ep_norm(cfg, empty, empty, None, empty, empty, None, None)
    d_w = torch.full((1024,), 5.0, device="cuda")
    ep.ep_norm_grad(cfg, empty, None, None, empty, None, empty, d_w, ep.alloc_norm_workspace(cfg))
    assert (d_w == 0).all()


def test_past_2_31_elements(ep):
    n, h = 131_075, 16384
    x = torch.randn(16, h, generator=gen(1), device="cuda").bfloat16().repeat(n // 16 + 1, 1)[:n]
    y = torch.empty_like(x)
    cfg = config(ep, n, h, torch.bfloat16)
    ep.ep_norm(cfg, x, None, None, None, y, None, None)
    assert torch.equal(y[-16:], y[n % 16:n % 16 + 16]) and torch.equal(y[131_056:131_072], y[:16])
    assert_y(y[-20:], ref.norm(x[-20:], None, None, EPS)[2])
    d_x = torch.empty_like(x)
    ep.ep_norm_grad(cfg, x, None, None, y, None, d_x, None, ep.alloc_norm_workspace(cfg))
    want, _, size, _ = ref.norm_grad(x[-20:], None, None, y[-20:], None, EPS)
    assert ((d_x[-20:].double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2 * ROW).all()


def test_streams_and_graphs(ep):
    """On a stream of its own, and captured twice on one workspace, the graphs replayed in turn."""
    n, h, g = 300, 2048, gen(9)
    cfg = config(ep, n, h, torch.bfloat16)
    w = torch.ones(h, dtype=torch.bfloat16, device="cuda")
    ws = ep.alloc_norm_workspace(cfg)
    sets = []
    for _ in range(2):
        x, r, d_y = (rows_of(g, n, h, torch.bfloat16) for _ in range(3))
        sets.append((x, r, d_y, torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(h, device="cuda")))

    def step(x, r, d_y, total, y, d_x, d_w):
        ep.ep_norm(cfg, x, r, w, total, y, None, None)
        ep.ep_norm_grad(cfg, total, w, None, d_y, None, d_x, d_w, ws)

    side, want = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            step(*s)
            want.append([t.clone() for t in s[3:]])
    side.synchronize()
    graphs = []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(*s)
    for _ in range(3):
        for s in sets:
            for t in s[3:]:
                t.fill_(torch.nan)
        for gr in graphs:
            gr.replay()
        for s, expected in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(s[3:], expected))


def test_rows_travel_through_the_dispatch(ep):
    """The norm's FP8 rows as the dispatch's pre-cast input: every receive row holds its token's codes."""
    R, T, H, E, K = 2, 40, 256, 8, 2
    g = gen(21)
    for packed in (0, 1):
        x = rows_of(g, R * T, H, torch.bfloat16)
        cfg = config(ep, R * T, H, torch.bfloat16, sf_pack=packed)
        G = H // 128
        codes = torch.empty(R * T, H, dtype=torch.uint8, device="cuda")
        sf = torch.empty(R * T, (G + 3) // 4 if packed else G, device="cuda")
        ep.ep_norm(cfg, x, None, None, None, None, codes, sf)
        c = ep.Config(1, R, E, K, T, T, H, x_dtype=ep.EP_DTYPE_FP8_E4M3, recv_dtype=ep.EP_DTYPE_FP8_E4M3, expand=1, sf_pack=packed)
        idx = torch.rand(R, T, E, generator=g, device="cuda").topk(K).indices
        wt = torch.ones(R, T, K, device="cuda")
        lay, recv, ws = ep.alloc_layout(c), ep.alloc_recv(c), ep.alloc_workspace(c)
        ep.ep_get_dispatch_layout(c, idx, lay, ws)
        ep.ep_dispatch(c, lay, codes, sf, idx, wt, recv, ws)
        assert ep.ep_check_error(ws) == ep.EP_OK
        row = (lay.exp_pos + lay.exp_region[(idx // (E // R)).long()]).long()
        token = torch.arange(R * T, device="cuda").view(R, T, 1).expand(R, T, K)
        assert torch.equal(recv.recv_x[row.reshape(-1)], codes[token.reshape(-1)])
        assert torch.equal(recv.recv_sf.view(torch.int32)[row.reshape(-1)], sf.view(torch.int32)[token.reshape(-1)])


@pytest.mark.parametrize("n,h,kind", [(1024, 1024, 0), (700, 1640, 0), (800, 784, 2)])
def test_the_first_call_of_a_process(n, h, kind):
    """Rings of just below and just above 48 KB of shared memory, before any other call has raised a limit."""
    code = f"""
import torch, combine_ep_get_02_gb300 as ep
t = torch.bfloat16 if {kind} == 0 else torch.float32
cfg = ep.NormConfig({n}, {h}, x_dtype={kind})
s, d = (torch.randn({n}, {h}, device="cuda").to(t) for _ in range(2))
y = torch.randn({n}, {h}, device="cuda").bfloat16()
ep.ep_norm_grad(cfg, s, None, None, y, d, d, None, ep.alloc_norm_workspace(cfg))
torch.cuda.synchronize()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", code], check=True, cwd=root, timeout=300)
