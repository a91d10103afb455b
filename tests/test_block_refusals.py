"""Arguments that the norm and the rows kept in 8 bits refuse before touching the device (CPU: a call
that got as far as CUDA would answer EP_ERR_CUDA)."""
import copy
import ctypes as C
import pickle

import pytest
import torch

P = C.c_void_p
WS, A = P(0x10000), P(0x40000)


@pytest.fixture(scope="module")
def ep():
    from combine_ep_get_02_gb300 import _build
    _build.build()
    import combine_ep_get_02_gb300 as ep
    ep.lib()
    return ep


def norm_cfg(ep, **kw):
    return ep.NormConfig(**{**dict(rows=10, hidden=256), **kw})


def checkpoint_cfg(ep, **kw):
    return ep.CheckpointConfig(**{**dict(num_ranks=2, num_experts=8, rows=100, features=256), **kw})


def up(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), -1), (dict(rows=1 << 31), -2), (dict(hidden=0), -1), (dict(hidden=12), -1), (dict(hidden=-8), -1),
    (dict(hidden=16392), -2), (dict(x_dtype=1), -1), (dict(x_dtype=3), -1), (dict(sf_pack=2), -1), (dict(eps=0.0), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(eps=1e-30), -1),
])
def test_norm_configs(ep, bad, code):
    cfg = norm_cfg(ep, **bad)
    assert ep.ep_norm_workspace_bytes(cfg) == 0
    assert ep.lib().ep_norm(C.byref(cfg._c()), *[None] * 8) == code
    assert ep.lib().ep_norm_grad(C.byref(cfg._c()), *[None] * 8, 0, None) == code
    with pytest.raises(ep.EpError):
        ep.alloc_norm_workspace(cfg)


def test_norm_arguments(ep):
    L, cfg = ep.lib(), norm_cfg(ep)
    n, c = ep.ep_norm_workspace_bytes(cfg), cfg._c()
    assert n == 256 + up(4 * 608 * 256)

    def call(x=A, r=None, w=None, s=None, y=A, q=None, sf=None, cc=c):
        return L.ep_norm(C.byref(cc), x, r, w, s, y, q, sf, None)

    bad = ep.EP_ERR_INVALID_ARG
    assert call(x=None) == call(y=None) == call(q=A) == call(sf=A) == call(y=None, sf=A) == bad
    odd = P(0x40008)
    assert call(x=odd) == call(r=odd) == call(w=odd) == call(s=odd) == call(y=odd) == call(q=odd, sf=A) == bad
    assert call(q=A, sf=P(0x40002)) == bad
    assert call(q=A, sf=A, cc=norm_cfg(ep, hidden=200)._c()) == bad  # no whole groups of 128
    assert call(x=None, y=None, cc=norm_cfg(ep, rows=0)._c()) == ep.EP_OK
    assert L.ep_norm(None, *[A] * 8) == bad

    def grad(s=A, w=A, m=None, g=A, ds=None, dx=A, dw=A, ws=WS, size=n, cc=c):
        return L.ep_norm_grad(C.byref(cc), s, w, m, g, ds, dx, dw, ws, size, None)

    assert grad(ws=None) == grad(size=n - 1) == grad(ws=P(0x10010)) == ep.EP_ERR_WORKSPACE
    assert grad(s=None) == grad(g=None) == bad
    assert grad(s=odd) == grad(w=odd) == grad(g=odd) == grad(ds=odd) == grad(dx=odd) == grad(dw=P(0x40002)) == bad
    assert grad(dx=None, dw=None) == ep.EP_OK  # nothing asked for
    assert grad(dw=None, cc=norm_cfg(ep, rows=0)._c()) == ep.EP_OK


@pytest.mark.parametrize("bad,code", [
    (dict(num_ranks=0), -1), (dict(num_experts=0), -1), (dict(num_experts=9), -1), (dict(num_experts=8192), -2),
    (dict(rows=-1), -1), (dict(rows=1 << 31), -2), (dict(features=0), -1), (dict(features=64), -1), (dict(features=200), -1),
    (dict(features=1 << 22), -2), (dict(activation=5), -1), (dict(activation=-1), -1), (dict(sf_pack=2), -1),
])
def test_checkpoint_configs(ep, bad, code):
    cfg = checkpoint_cfg(ep, **bad)
    assert ep.ep_checkpoint_workspace_bytes(cfg) == 0
    c = C.byref(cfg._c())
    assert ep.lib().ep_checkpoint(c, None, None, None, None, None, 0, None) == code
    assert ep.lib().ep_checkpoint_rows(c, None, None, None, None, None, 0, None) == code
    assert ep.lib().ep_checkpoint_grad(c, None, *[None] * 6, None, 0, None) == code
    with pytest.raises(ep.EpError):
        ep.alloc_checkpoint_workspace(cfg)


def test_checkpoint_arguments(ep):
    L, cfg = ep.lib(), checkpoint_cfg(ep)
    n, c = ep.ep_checkpoint_workspace_bytes(cfg), cfg._c()
    assert n == 256 + up(4 * (100 // 64 + 8) * 256)
    lay, bad, odd = ep._Layout(*[None] * 6, A, A, A), ep.EP_ERR_INVALID_ARG, P(0x40008)
    for f in (L.ep_checkpoint, L.ep_checkpoint_rows):
        call = lambda l=lay, x=A, q=A, sf=A, ws=WS, size=n, cc=c: f(  # noqa: E731
            C.byref(cc), None if l is None else C.byref(l), x, q, sf, ws, size, None)
        assert call(ws=None) == call(size=n - 1) == call(ws=P(0x10010)) == ep.EP_ERR_WORKSPACE
        assert call(x=None) == call(q=None) == call(sf=None) == call(l=None) == call(l=ep._Layout()) == bad
        # ep_checkpoint: (x, codes, sf); ep_checkpoint_rows: (codes, sf, x)
        assert call(x=odd) == bad and call(q=P(0x40002)) == bad and call(sf=P(0x40002)) == bad
        assert call(x=None, cc=checkpoint_cfg(ep, rows=0)._c()) == ep.EP_OK

    def grad(l=lay, q=A, sf=A, g=A, h=A, dz=A, db=A, ws=WS, size=n, cc=c):
        return L.ep_checkpoint_grad(C.byref(cc), None if l is None else C.byref(l), q, sf, g, h, dz, db, ws, size, None)

    assert grad(ws=None) == grad(size=n - 1) == ep.EP_ERR_WORKSPACE
    assert grad(q=None) == grad(sf=None) == grad(g=None) == grad(l=None) == grad(l=ep._Layout(*[None] * 6, A, A)) == bad
    assert grad(q=odd) == grad(g=odd) == grad(h=odd) == grad(dz=odd) == grad(db=P(0x40002)) == grad(sf=P(0x40002)) == bad
    assert grad(h=None, dz=None, db=None) == ep.EP_OK  # nothing asked for


def test_tensors_that_a_call_would_misread(ep):
    """The binding refuses tensors by name: absent, of another type, not dense, too small, on the CPU."""
    bf, x = torch.bfloat16, torch.empty(10, 256, dtype=torch.bfloat16)
    cfg = norm_cfg(ep)
    for bad, why in ((x.float(), "float32"), (x.T, "contiguous"), (x[:9], "2304 elements"), (x, "GPU"), (None, "missing")):
        with pytest.raises(ep.EpError, match=f"ep_norm: x .*{why}"):
            ep.ep_norm(cfg, bad, None, None, None, x, None, None)
        with pytest.raises(ep.EpError, match=f"ep_norm_grad: sum .*{why}"):
            ep.ep_norm_grad(cfg, bad, None, None, x, None, x, None, torch.empty(256, dtype=torch.uint8))
        with pytest.raises(ep.EpError, match=f"ep_checkpoint: x .*{why}"):
            ep.ep_checkpoint(ep.CheckpointConfig(1, 1, 10, 256), None, bad, None, None, None)
    with pytest.raises(ep.EpError, match="x is torch.bfloat16"):
        ep.ep_norm(norm_cfg(ep, x_dtype=ep.EP_DTYPE_FP32), x, None, None, None, x, None, None)
    short = ep.Layout(*[None] * 6, *(torch.empty(2, dtype=torch.int32) for _ in range(3)))
    with pytest.raises(ep.EpError, match="exp_cnt"):
        ep.ep_checkpoint_rows(checkpoint_cfg(ep), short, torch.empty(100, 256, dtype=torch.uint8), torch.empty(100, 2),
                              torch.empty(100, 256, dtype=bf), None)


def test_configs_copy_and_pickle(ep):
    for cfg in (norm_cfg(ep, eps=1e-5), checkpoint_cfg(ep, activation=ep.EP_ACT_SWIGLU)):
        cfg._ref(), cfg._needs()
        for other in (copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
            assert other == cfg and other._sizes is None
        cfg.rows = 64  # what was kept goes with the field
        assert cfg._sizes is None and cfg._c().rows == 64
    assert checkpoint_cfg(ep, activation=ep.EP_ACT_SWIGLU).out_features == 128


def layer_cfg(ep, **kw):
    return ep.LayerConfig(**{**dict(num_tokens=4, num_experts=8, num_topk=2, hidden=256, inner=128), **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(num_tokens=-1), -1), (dict(num_tokens=65), -2), (dict(num_experts=0), -1), (dict(num_experts=4097), -2),
    (dict(num_topk=0), -1), (dict(num_topk=33), -2), (dict(hidden=0), -1), (dict(hidden=12), -1), (dict(inner=4), -1),
    (dict(hidden=1 << 21), -2), (dict(inner=1 << 21), -2), (dict(activation=5), -1), (dict(activation=-1), -1),
    (dict(weight_dtype=2), -1), (dict(weight_dtype=1, hidden=136), -1), (dict(weight_dtype=1, inner=64), -1),
    (dict(num_sms=-1), -1),
])
def test_layer_configs(ep, bad, code):
    cfg = layer_cfg(ep, **bad)
    assert ep.ep_layer_workspace_bytes(cfg) == 0
    assert ep.lib().ep_expert_layer(C.byref(cfg._c()), *[None] * 12, 0, None) == code
    with pytest.raises(ep.EpError):
        ep.alloc_layer_workspace(cfg)


def test_layer_arguments(ep):
    L, cfg = ep.lib(), layer_cfg(ep)
    n, c = ep.ep_layer_workspace_bytes(cfg), cfg._c()
    assert n == 256 + up(4 * 16) + up(4 * 4 * 2 * 128) + up(4 * 8 * 4 * 256)  # h as two terms
    five = ep.ep_layer_workspace_bytes(layer_cfg(ep, num_tokens=5))
    assert five == 256 + up(4 * 16) + up(2 * 5 * 2 * 128) + up(4 * 8 * 5 * 256)
    bad, odd, off = ep.EP_ERR_INVALID_ARG, P(0x40008), P(0x40002)

    def call(x=A, idx=A, w=A, u=A, us=None, ub=None, d=A, ds=None, db=None, r=None, out=A, ws=WS, size=n, cc=c):
        return L.ep_expert_layer(C.byref(cc), x, idx, w, u, us, ub, d, ds, db, r, out, ws, size, None)

    assert call(ws=None) == call(size=n - 1) == call(ws=P(0x10010)) == ep.EP_ERR_WORKSPACE
    assert call(x=None) == call(idx=None) == call(w=None) == call(u=None) == call(d=None) == call(out=None) == bad
    assert call(us=A) == call(ds=A) == call(us=A, ds=A) == bad  # scales of bf16 matrices
    fp8 = layer_cfg(ep, weight_dtype=1)._c()
    assert call(cc=fp8, size=1 << 30) == call(us=A, cc=fp8, size=1 << 30) == call(ds=A, cc=fp8, size=1 << 30) == bad
    for name in ("x", "u", "ub", "d", "db", "r", "out"):
        assert call(**{name: odd}) == bad
    assert call(idx=P(0x40004)) == call(w=off) == bad
    assert call(us=off, ds=A, cc=fp8, size=1 << 30) == call(us=A, ds=off, cc=fp8, size=1 << 30) == bad
    assert call(x=None, cc=layer_cfg(ep, num_tokens=0)._c()) == ep.EP_OK
    assert L.ep_expert_layer(None, *[A] * 12, n, None) == bad


def test_layer_tensors(ep):
    """The binding refuses each tensor by name before the library is called."""
    bf, cfg = torch.bfloat16, layer_cfg(ep)
    x, idx, w = torch.empty(4, 256, dtype=bf), torch.zeros(4, 2, dtype=torch.int64), torch.empty(4, 2)
    up_, down = torch.empty(8, 256, 256, dtype=bf), torch.empty(8, 256, 128, dtype=bf)
    for bad, why in ((up_.float(), "float32"), (up_[:7], "elements"), (up_.transpose(1, 2), "contiguous"), (up_, "GPU"), (None, "missing")):
        with pytest.raises(ep.EpError, match=f"ep_expert_layer: up .*{why}"):
            ep.ep_expert_layer(cfg, x, idx, w, bad, None, None, down, None, None, None, x, None)
    fp8 = layer_cfg(ep, weight_dtype=ep.EP_DTYPE_FP8_E4M3)
    with pytest.raises(ep.EpError, match="up is torch.bfloat16"):
        ep.ep_expert_layer(fp8, x, idx, w, up_, None, None, down, None, None, None, x, None)
    assert fp8._needs()[3] == 8 * 2 * 2 and fp8.z_features == 256
    cfg._ref(), cfg._needs()
    assert pickle.loads(pickle.dumps(cfg)) == cfg and copy.copy(cfg)._sizes is None
