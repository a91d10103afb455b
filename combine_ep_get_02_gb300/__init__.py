"""GB300-native MoE expert-parallel dispatch / combine on one GPU.

Thin ctypes binding over the C ABI of ``include/ep_get.h`` (``libep_get.so``,
built in-tree for sm_103a). Every step of the path runs in the library's CUDA
kernels; this module only marshals arguments: torch tensors supply device
memory and the current CUDA stream. There is no CPU fallback: if the library
is missing, importing the binding raises.

The entry points keep the C names (``ep_get_dispatch_layout``, ``ep_dispatch``,
``ep_combine``, ...). ``Config`` mirrors ``ep_config_t``; ``alloc_layout``,
``alloc_recv`` and ``alloc_workspace`` allocate correctly sized tensors.
Beside them stand the router (``ep_route`` with its balance loss), the experts'
products (``ep_expert_product``) and their gradients with the combine's.
"""
from __future__ import annotations

import ctypes as C
import dataclasses
import os

import torch

from . import _build

EP_OK, EP_ERR_INVALID_ARG, EP_ERR_UNSUPPORTED, EP_ERR_WORKSPACE, EP_ERR_CUDA, EP_ERR_BAD_TOPK, \
    EP_ERR_OVERFLOW, EP_ERR_TIMEOUT, EP_ERR_BOUNDS, EP_ERR_NONFINITE = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9
EP_DTYPE_BF16, EP_DTYPE_FP8_E4M3, EP_DTYPE_FP32 = 0, 1, 2
EP_SCORE_SOFTMAX, EP_SCORE_SIGMOID = 0, 1
EP_ACT_NONE, EP_ACT_RELU, EP_ACT_SILU, EP_ACT_GELU, EP_ACT_SWIGLU = 0, 1, 2, 3, 4

__all__ = [
    "Config", "Layout", "Recv", "EpError", "lib", "ep_workspace_bytes", "ep_recv_rows",
    "ep_workspace_init", "ep_get_dispatch_layout", "ep_get_dispatch_layout_noalloc", "ep_check_error_noalloc",
    "ep_dispatch", "ep_combine", "ep_check_error",
    "ep_dispatch_atomic", "ep_deterministic_sort",
    "ep_status_string", "ep_diag_e4m3_of_bits", "ep_diag_bf16_of_bits",
    "ep_diag_copy_fanout", "ep_diag_wait_timeout", "use_checked", "alloc_layout", "alloc_recv",
    "alloc_workspace", "config_of",
    "RouteConfig", "Route", "ProductConfig", "ep_route_workspace_bytes", "ep_product_workspace_bytes",
    "alloc_route", "alloc_route_workspace", "alloc_product_workspace", "ep_route", "ep_route_grad",
    "ep_combine_grad", "ep_expert_product", "ep_expert_product_grad",
]


class EpError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {ep_status_string(status)} ({status})")
        self.status = status


class _Config(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "num_scaleout_ranks", "num_scaleup_ranks", "num_experts", "num_topk", "num_tokens",
        "num_max_tokens_per_rank", "hidden", "x_dtype", "recv_dtype", "expand", "expert_alignment",
        "num_sms", "num_prologue_sms", "compact_recv", "zero_padding", "sf_pack", "copy_path",
        "recv_capacity")]


class _Layout(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "num_tokens_per_rank", "num_tokens_per_expert", "is_token_in_rank", "slot_map", "recv_cnt",
        "recv_psum", "exp_cnt", "exp_base", "exp_region", "exp_pos", "recv_region")]


class _Recv(C.Structure):
    _fields_ = [("recv_x", C.c_void_p), ("recv_sf", C.c_void_p), ("recv_topk_idx", C.c_void_p),
                ("recv_topk_weights", C.c_void_p), ("recv_src_metadata", C.c_void_p),
                ("recv_x_rows", C.c_int64)]


class _KeepsStruct:
    """Keeps the ctypes struct built by _c() until a field is assigned again, so
    a call reuses it instead of marshalling every field (the struct holds the
    values, and for tensors their data pointers, as of that build). Copies and
    pickles start without what is kept."""

    _struct = _reference = _sizes = _lanes = None

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_struct", "_reference", "_sizes", "_lanes")}

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_struct", None)
        object.__setattr__(self, "_reference", None)
        object.__setattr__(self, "_sizes", None)
        object.__setattr__(self, "_lanes", None)

    def _c(self):
        st = self.__dict__.get("_struct")
        if st is None:
            st = self._build_struct()
            object.__setattr__(self, "_struct", st)
        return st

    def _ref(self):
        """byref of the struct, kept as long as it is."""
        r = self.__dict__.get("_reference")
        if r is None:
            r = C.byref(self._c())
            object.__setattr__(self, "_reference", r)
        return r

    def _count(self, where: str, fields):
        """Element counts of the tensors named in `fields` ((name, dtype) pairs; -1 for None),
        refused as by _at."""
        n = []
        for name, dtype in fields:
            t = getattr(self, name)
            if t is not None:
                _at(t, dtype, 0, where, name)
            n.append(-1 if t is None else t.numel())
        return n

    def _checked(self, where: str, fields):
        """_count, kept like the struct that holds the tensors' addresses."""
        n = self.__dict__.get("_sizes")
        if n is None:
            n = self._count(where, fields)
            object.__setattr__(self, "_sizes", n)
        return n


@dataclasses.dataclass
class Config(_KeepsStruct):
    num_scaleout_ranks: int
    num_scaleup_ranks: int
    num_experts: int
    num_topk: int
    num_tokens: int
    num_max_tokens_per_rank: int
    hidden: int
    x_dtype: int = EP_DTYPE_BF16
    recv_dtype: int = EP_DTYPE_BF16
    expand: int = 0
    expert_alignment: int = 1
    num_sms: int = 0
    num_prologue_sms: int = 0
    compact_recv: int = 0
    zero_padding: int = 0
    sf_pack: int = 0
    copy_path: int = 0  # unchanged rows: 0 automatic, 1 register copies, 2 bulk copies
    recv_capacity: int = 0  # packed receive rows: rows of the receive tensors (0 = R*T*min(K,R))

    @property
    def num_ranks(self) -> int:
        return self.num_scaleout_ranks * self.num_scaleup_ranks

    def _build_struct(self) -> _Config:
        return _Config(*(int(getattr(self, f[0])) for f in _Config._fields_))


def config_of(wl, **over) -> Config:
    """Config of a workload description (attributes as in ``workloads.Workload``)."""
    c = Config(wl.n_so, wl.n_su, wl.num_experts, wl.num_topk, wl.num_tokens,
               wl.num_max_tokens_per_rank, wl.hidden,
               EP_DTYPE_FP8_E4M3 if wl.x_dtype == "fp8" else EP_DTYPE_BF16,
               EP_DTYPE_FP8_E4M3 if wl.recv_dtype == "fp8" else EP_DTYPE_BF16,
               int(bool(wl.expand)), wl.expert_alignment,
               compact_recv=int(getattr(wl, "compact", 0)),
               recv_capacity=int(getattr(wl, "recv_capacity", 0)),
               zero_padding=int(bool(getattr(wl, "zero_padding", False))),
               sf_pack=int(bool(getattr(wl, "sf_pack", False))))
    return dataclasses.replace(c, **over)


_lib = None
_checked = False


def use_checked(on: bool = True) -> None:
    """Route every later call to the bounds-checked build of the library (each
    computed row index is tested against its buffer; one outside is skipped and
    reported as EP_ERR_BOUNDS by ep_check_error), or back to the normal one."""
    global _lib, _checked
    _checked, _lib = bool(on), None


def lib():
    """The loaded library. Raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        path = _build.LIB_CHECKED if _checked else _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(path)
        P, I = C.c_void_p, C.c_int
        L.ep_workspace_bytes.restype = C.c_size_t
        L.ep_workspace_bytes.argtypes = [P]
        L.ep_recv_rows.restype = C.c_int64
        L.ep_recv_rows.argtypes = [P]
        L.ep_workspace_init.restype = I
        L.ep_workspace_init.argtypes = [P, C.c_size_t, P]
        L.ep_get_dispatch_layout.restype = I
        L.ep_get_dispatch_layout.argtypes = [P, P, P, P, C.c_size_t, P]
        L.ep_get_dispatch_layout_noalloc.restype = I
        L.ep_get_dispatch_layout_noalloc.argtypes = [P, P, P, P]
        L.ep_check_error_noalloc.restype = I
        L.ep_check_error_noalloc.argtypes = [P]
        L.ep_dispatch.restype = I
        L.ep_dispatch.argtypes = [P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_dispatch_atomic.restype = I
        L.ep_dispatch_atomic.argtypes = [P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_deterministic_sort.restype = I
        L.ep_deterministic_sort.argtypes = [P, P, P, P, P]
        L.ep_combine.restype = I
        L.ep_combine.argtypes = [P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_route_workspace_bytes.restype = C.c_size_t
        L.ep_route_workspace_bytes.argtypes = [P]
        L.ep_route.restype = I
        L.ep_route.argtypes = [P, P, P, P, P, P, C.c_size_t, P]
        L.ep_route_grad.restype = I
        L.ep_route_grad.argtypes = [P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_combine_grad.restype = I
        L.ep_combine_grad.argtypes = [P, P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_product_workspace_bytes.restype = C.c_size_t
        L.ep_product_workspace_bytes.argtypes = [P, C.c_int32]
        L.ep_expert_product.restype = I
        L.ep_expert_product.argtypes = [P, P, P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_expert_product_grad.restype = I
        L.ep_expert_product_grad.argtypes = [P, P, P, P, P, P, P, P, P, P, C.c_size_t, P]
        L.ep_check_error.restype = I
        L.ep_check_error.argtypes = [P, P]
        L.ep_status_string.restype = C.c_char_p
        L.ep_status_string.argtypes = [I]
        L.ep_diag_e4m3_of_bits.restype = I
        L.ep_diag_e4m3_of_bits.argtypes = [C.c_uint32, C.c_int64, P, P]
        L.ep_diag_bf16_of_bits.restype = I
        L.ep_diag_bf16_of_bits.argtypes = [C.c_uint32, C.c_int64, P, P]
        L.ep_diag_copy_fanout.restype = I
        L.ep_diag_copy_fanout.argtypes = [P, P, C.c_int64, I, I, I, I, I, P]
        L.ep_diag_wait_timeout.restype = I
        L.ep_diag_wait_timeout.argtypes = [P, P, I, C.c_uint32, P]
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(st: int, where: str):
    if st != EP_OK:
        raise EpError(st, where)


def ep_status_string(status: int) -> str:
    return lib().ep_status_string(int(status)).decode()


def ep_workspace_bytes(cfg: Config) -> int:
    c = cfg._c()
    return int(lib().ep_workspace_bytes(C.byref(c)))


def ep_recv_rows(cfg: Config) -> int:
    c = cfg._c()
    return int(lib().ep_recv_rows(C.byref(c)))


def ep_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().ep_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "ep_workspace_init")


@dataclasses.dataclass
class Layout(_KeepsStruct):
    num_tokens_per_rank: torch.Tensor
    num_tokens_per_expert: torch.Tensor
    is_token_in_rank: torch.Tensor
    slot_map: torch.Tensor
    recv_cnt: torch.Tensor
    recv_psum: torch.Tensor
    exp_cnt: torch.Tensor | None = None
    exp_base: torch.Tensor | None = None
    exp_region: torch.Tensor | None = None
    exp_pos: torch.Tensor | None = None
    recv_region: torch.Tensor | None = None

    def _build_struct(self) -> _Layout:
        return _Layout(*(_ptr(getattr(self, f[0])) for f in _Layout._fields_))


@dataclasses.dataclass
class Recv(_KeepsStruct):
    recv_x: torch.Tensor
    recv_sf: torch.Tensor | None
    recv_topk_idx: torch.Tensor | None
    recv_topk_weights: torch.Tensor | None
    recv_src_metadata: torch.Tensor | None

    def _build_struct(self) -> _Recv:
        return _Recv(_ptr(self.recv_x), _ptr(self.recv_sf), _ptr(self.recv_topk_idx),
                     _ptr(self.recv_topk_weights), _ptr(self.recv_src_metadata), self.recv_x.shape[0])


def alloc_workspace(cfg: Config, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of ep_workspace_bytes(cfg) bytes."""
    n = ep_workspace_bytes(cfg)
    if n == 0:
        raise EpError(EP_ERR_INVALID_ARG, "ep_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_layout(cfg: Config, device="cuda") -> Layout:
    R, E, T, K = cfg.num_ranks, cfg.num_experts, cfg.num_tokens, cfg.num_topk
    L = E // R
    i32 = dict(dtype=torch.int32, device=device)
    lay = Layout(torch.empty(R, R, **i32), torch.empty(R, E, **i32),
                 torch.empty(R, T, R, dtype=torch.uint8, device=device), torch.empty(R, T, K, **i32),
                 torch.empty(R, R, **i32), torch.empty(R, R, **i32), recv_region=torch.empty(R + 1, **i32))
    if cfg.expand:
        lay.exp_cnt = torch.empty(R, L, **i32)
        lay.exp_base = torch.empty(R, L + 1, **i32)
        lay.exp_region = torch.empty(R + 1, **i32)
        lay.exp_pos = torch.empty(R, T, K, **i32)
    return lay


def alloc_recv(cfg: Config, device="cuda", sidecars: bool = True, zero: bool = False) -> Recv:
    R, M, K, H = cfg.num_ranks, cfg.num_max_tokens_per_rank, cfg.num_topk, cfg.hidden
    rows = ep_recv_rows(cfg)
    if rows < 0:
        raise EpError(EP_ERR_INVALID_ARG, "ep_recv_rows")
    mk = torch.zeros if zero else torch.empty
    fp8 = cfg.recv_dtype == EP_DTYPE_FP8_E4M3
    recv_x = mk(rows, H, dtype=torch.uint8 if fp8 else torch.bfloat16, device=device)
    G = H // 128
    recv_sf = mk(rows, (G + 3) // 4 if cfg.sf_pack else G, dtype=torch.float32, device=device) if fp8 else None
    if not sidecars:
        return Recv(recv_x, recv_sf, None, None, None)
    # sidecar rows: one region of R*M rows per destination, or the packed rows
    side = (rows,) if cfg.compact_recv == 2 else (R, R * M)
    return Recv(recv_x, recv_sf, mk(*side, K, dtype=torch.int64, device=device),
                mk(*side, K, dtype=torch.float32, device=device),
                mk(*side, K + 2, dtype=torch.int32, device=device))


def ep_get_dispatch_layout(cfg: Config, topk_idx: torch.Tensor, layout: Layout, ws: torch.Tensor,
                           stream=None):
    c, l = cfg._c(), layout._c()
    _check(lib().ep_get_dispatch_layout(C.byref(c), _ptr(topk_idx), C.byref(l), _ptr(ws),
                                        ws.numel(), _stream(stream)), "ep_get_dispatch_layout")


def ep_get_dispatch_layout_noalloc(cfg: Config, topk_idx: torch.Tensor, layout: Layout, stream=None):
    """The layout without a caller workspace (fixed scratch inside the library)."""
    c, l = cfg._c(), layout._c()
    _check(lib().ep_get_dispatch_layout_noalloc(C.byref(c), _ptr(topk_idx), C.byref(l), _stream(stream)),
           "ep_get_dispatch_layout_noalloc")


def ep_check_error_noalloc(stream=None) -> int:
    """Synchronises the stream; returns (and clears) the status the
    allocation-free layout latched in the library's array."""
    return int(lib().ep_check_error_noalloc(_stream(stream)))


def ep_dispatch(cfg: Config, layout: Layout, x: torch.Tensor, x_sf, topk_idx: torch.Tensor,
                topk_weights: torch.Tensor, recv: Recv, ws: torch.Tensor, stream=None):
    c, l, r = cfg._c(), layout._c(), recv._c()
    _check(lib().ep_dispatch(C.byref(c), C.byref(l), _ptr(x), _ptr(x_sf), _ptr(topk_idx),
                             _ptr(topk_weights), C.byref(r), _ptr(ws), ws.numel(), _stream(stream)),
           "ep_dispatch")


def ep_dispatch_atomic(cfg: Config, x: torch.Tensor, x_sf, topk_idx: torch.Tensor,
                       topk_weights: torch.Tensor, recv: Recv, send_counters: torch.Tensor, ws: torch.Tensor,
                       stream=None):
    """Comparison path: dispatch with racing atomicAdd slots (no layout)."""
    c, r = cfg._c(), recv._c()
    _check(lib().ep_dispatch_atomic(C.byref(c), _ptr(x), _ptr(x_sf), _ptr(topk_idx), _ptr(topk_weights),
                                    C.byref(r), _ptr(send_counters), _ptr(ws), ws.numel(), _stream(stream)),
           "ep_dispatch_atomic")


def ep_deterministic_sort(cfg: Config, recv: Recv, send_counters: torch.Tensor, sorted_recv: Recv,
                          stream=None):
    """Comparison path: sort each received segment by source token into sorted_recv."""
    c, r, o = cfg._c(), recv._c(), sorted_recv._c()
    _check(lib().ep_deterministic_sort(C.byref(c), C.byref(r), _ptr(send_counters), C.byref(o),
                                       _stream(stream)), "ep_deterministic_sort")


def ep_combine(cfg: Config, layout: Layout, y: torch.Tensor, topk_idx: torch.Tensor,
               topk_weights: torch.Tensor, out: torch.Tensor, ws: torch.Tensor, stream=None):
    c, l = cfg._c(), layout._c()
    _check(lib().ep_combine(C.byref(c), C.byref(l), _ptr(y), _ptr(topk_idx), _ptr(topk_weights),
                            _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "ep_combine")


def ep_check_error(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream; returns (and clears) the latched device status."""
    return int(lib().ep_check_error(_ptr(ws), _stream(stream)))


def ep_diag_e4m3_of_bits(first: int, out: torch.Tensor, stream=None):
    _check(lib().ep_diag_e4m3_of_bits(first, out.numel(), _ptr(out), _stream(stream)),
           "ep_diag_e4m3_of_bits")


def ep_diag_bf16_of_bits(first: int, out: torch.Tensor, stream=None):
    _check(lib().ep_diag_bf16_of_bits(first, out.numel(), _ptr(out), _stream(stream)),
           "ep_diag_bf16_of_bits")


def ep_diag_copy_fanout(src: torch.Tensor, dst: torch.Tensor, rows: int, row_bytes: int, fan_num: int,
                        fan_den: int, num_sms: int = 0, method: int = 0, stream=None):
    """Row r of src goes to dst rows floor(r*num/den) .. floor((r+1)*num/den)-1;
    method 0: register loads/stores, 1: bulk copies through shared memory."""
    need = rows * fan_num // fan_den * row_bytes if fan_den > 0 else 0
    if src.numel() * src.element_size() < rows * row_bytes or dst.numel() * dst.element_size() < need:
        raise EpError(EP_ERR_INVALID_ARG, "ep_diag_copy_fanout")
    _check(lib().ep_diag_copy_fanout(_ptr(src), _ptr(dst), rows, row_bytes, fan_num, fan_den, num_sms,
                                     method, _stream(stream)), "ep_diag_copy_fanout")


def ep_diag_wait_timeout(ws: torch.Tensor, src, nbytes: int, rounds: int, stream=None):
    """Run the bulk-copy dispatch's abort sequence: a wait that runs out after
    `rounds` rounds with a load of `nbytes` from `src` in flight."""
    _check(lib().ep_diag_wait_timeout(_ptr(ws), _ptr(src), nbytes, rounds,
                                      _stream(stream)), "ep_diag_wait_timeout")


# ---- router, gradient of the combine, the experts' products ---------------------


class _RouteConfig(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "num_segments", "num_tokens", "num_experts", "num_topk", "logits_dtype", "score", "num_groups",
        "topk_groups", "normalize")] + [("scale", C.c_float)]


class _Route(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in (
        "topk_idx", "topk_weights", "expert_count", "prob_sum", "num_valid", "balance_loss")]


class _ProductConfig(C.Structure):
    _fields_ = [("num_ranks", C.c_int32), ("num_experts", C.c_int32), ("rows", C.c_int64)] + [
        (n, C.c_int32) for n in ("in_features", "out_features", "activation", "x_dtype", "sf_pack", "num_sms")]


def _refuse(where: str, name: str, t, dtype, numel: int):
    if t is None:
        why = "is missing"
    elif t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        why = f"is {t.dtype}"
    elif not t.is_contiguous():
        why = "is not contiguous"
    elif t.numel() < numel:
        why = f"has {t.numel()} elements, {numel} needed"
    else:
        why = "is not on the GPU"
    raise EpError(EP_ERR_INVALID_ARG, f"{where}: {name} {why}")


def _at(t, dtype, numel: int, where: str, name: str):
    """Address of a tensor that a call reads or writes `numel` elements of; refuses one that
    the C ABI would misread: absent, of another type, not dense, too small, not on the GPU."""
    if t is not None and t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    _refuse(where, name, t, dtype, numel)


def _maybe(t, dtype, numel: int, where: str, name: str):
    """As _at, for an argument that may be None."""
    return None if t is None else _at(t, dtype, numel, where, name)


def _space(ws, where: str):
    """Address and bytes of a workspace; refuses one that is not dense GPU memory."""
    if ws is not None and ws.is_cuda and ws.is_contiguous():
        return ws.data_ptr(), ws.nbytes
    why = "is missing" if ws is None else "is not on the GPU" if not ws.is_cuda else "is not contiguous"
    raise EpError(EP_ERR_WORKSPACE, f"{where}: the workspace {why}")


# the current stream's handle without building a Stream object; builds of torch without CUDA lack it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _raw_stream(stream):
    """The stream's handle; None: the current stream."""
    if stream is None:
        if _current_stream is None or _current_device is None:
            return torch.cuda.current_stream().cuda_stream
        return _current_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


@dataclasses.dataclass
class RouteConfig(_KeepsStruct):
    """ep_route_config_t. Softmax scores with a choice bias or groups: both act on the logits,
    not on the probabilities."""

    num_segments: int
    num_tokens: int  # per segment
    num_experts: int
    num_topk: int
    logits_dtype: int = EP_DTYPE_FP32
    score: int = EP_SCORE_SOFTMAX
    num_groups: int = 1
    topk_groups: int = 1
    normalize: int = 1
    scale: float = 1.0

    def _needs(self):
        """(logits' type, logits, lanes, statistics, segments, tokens) of a call, kept as the struct is."""
        N, B, E = self.num_segments * self.num_tokens, self.num_segments, self.num_experts
        n = (_BF16 if self.logits_dtype == EP_DTYPE_BF16 else _F32, N * E, N * self.num_topk, B * E, B, N)
        object.__setattr__(self, "_sizes", n)
        return n

    def _build_struct(self) -> _RouteConfig:
        return _RouteConfig(*(int(getattr(self, f[0])) for f in _RouteConfig._fields_[:-1]), float(self.scale))


@dataclasses.dataclass
class Route(_KeepsStruct):
    topk_idx: torch.Tensor                      # int64 [N][K]
    topk_weights: torch.Tensor                  # fp32 [N][K]
    expert_count: torch.Tensor | None = None    # int32 [B][E]
    prob_sum: torch.Tensor | None = None        # fp32 [B][E]
    num_valid: torch.Tensor | None = None       # int32 [B]
    balance_loss: torch.Tensor | None = None    # fp32 [1]

    def _build_struct(self) -> _Route:
        return _Route(*(_ptr(getattr(self, f[0])) for f in _Route._fields_))


@dataclasses.dataclass
class ProductConfig(_KeepsStruct):
    num_ranks: int
    num_experts: int
    rows: int
    in_features: int
    out_features: int
    activation: int = EP_ACT_NONE
    x_dtype: int = EP_DTYPE_BF16
    sf_pack: int = 0
    num_sms: int = 0

    @property
    def z_features(self) -> int:
        """Columns of z (and rows of each expert's matrix): twice out_features when gated."""
        return self.out_features * (2 if self.activation == EP_ACT_SWIGLU else 1)

    def _needs(self):
        """(x, x_sf, weight, bias, out, z) elements and (blocks' counts, starts, regions) of a call."""
        K, N, Z, E, rows = self.in_features, self.out_features, self.z_features, self.num_experts, self.rows
        sf = rows * ((K // 128 + 3) // 4 if self.sf_pack else K // 128)
        n = (rows * K, sf, E * Z * K, E * Z, rows * N, rows * Z, E, E + self.num_ranks, self.num_ranks + 1)
        object.__setattr__(self, "_sizes", n)
        return n

    def _build_struct(self) -> _ProductConfig:
        return _ProductConfig(*(int(getattr(self, f[0])) for f in _ProductConfig._fields_))


def ep_route_workspace_bytes(cfg: RouteConfig) -> int:
    c = cfg._c()
    return int(lib().ep_route_workspace_bytes(C.byref(c)))


def ep_product_workspace_bytes(cfg: ProductConfig, grad: bool = False) -> int:
    c = cfg._c()
    return int(lib().ep_product_workspace_bytes(C.byref(c), int(bool(grad))))


def alloc_route_workspace(cfg: RouteConfig, device="cuda") -> torch.Tensor:
    """Zero-filled workspace of ep_route_workspace_bytes(cfg) bytes."""
    n = ep_route_workspace_bytes(cfg)
    if n == 0:
        raise EpError(EP_ERR_INVALID_ARG, "ep_route_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_product_workspace(cfg: ProductConfig, grad: bool = False, device="cuda") -> torch.Tensor:
    """Workspace of ep_product_workspace_bytes(cfg, grad) bytes with a zeroed header."""
    n = ep_product_workspace_bytes(cfg, grad)
    if n == 0:
        raise EpError(EP_ERR_INVALID_ARG, "ep_product_workspace_bytes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def alloc_route(cfg: RouteConfig, device="cuda", stats: bool = True) -> Route:
    N, K = cfg.num_segments * cfg.num_tokens, cfg.num_topk
    out = Route(torch.empty(N, K, dtype=torch.int64, device=device), torch.empty(N, K, dtype=torch.float32, device=device))
    if stats:
        B, E = cfg.num_segments, cfg.num_experts
        out.expert_count = torch.empty(B, E, dtype=torch.int32, device=device)
        out.prob_sum = torch.empty(B, E, dtype=torch.float32, device=device)
        out.num_valid = torch.empty(B, dtype=torch.int32, device=device)
        out.balance_loss = torch.empty(1, dtype=torch.float32, device=device)
    return out


_ROUTE_FIELDS = (("topk_idx", _I64), ("topk_weights", _F32), ("expert_count", _I32), ("prob_sum", _F32),
                 ("num_valid", _I32), ("balance_loss", _F32))
_BLOCK_FIELDS = (("exp_cnt", _I32), ("exp_base", _I32), ("exp_region", _I32))


# what leads the combine's gradient to a lane's row: slots, compact, packed, per-expert blocks
_LANE_FIELDS = (("slot_map", _I32), ("recv_psum", _I32), ("recv_region", _I32))
_LANE_FIELDS = (*(_LANE_FIELDS[:i] for i in (1, 2, 3)), (("exp_pos", _I32), ("exp_region", _I32)))


def _too_small(where, obj, fields, need):
    for (name, dtype), n in zip(fields, need):
        t = getattr(obj, name)
        if t is not None and t.numel() < n:
            _refuse(where, name, t, dtype, n)


def _route_args(where, cfg, logits, token_mask, r):
    """What a call needs, and the addresses of the logits and the mask; refuses tensors of `r`
    that do not fit the configuration."""
    needs = cfg._sizes or cfg._needs()
    kind, NE, NK, BE, B, N = needs
    i, w, c, p, v, l = r._sizes or r._checked(where, _ROUTE_FIELDS)
    if i < NK or -1 < w < NK or -1 < c < BE or -1 < p < BE or -1 < v < B or l == 0:
        _too_small(where, r, _ROUTE_FIELDS, (NK, NK, BE, BE, B, 1))
    x = _at(logits, kind, NE, where, "logits")
    if token_mask is not None:
        token_mask = _at(token_mask, torch.bool if token_mask.dtype is torch.bool else _U8, N, where, "token_mask")
    return needs, x, token_mask


def ep_route(cfg: RouteConfig, logits: torch.Tensor, choice_bias, token_mask, out: Route, ws: torch.Tensor,
             stream=None):
    """Choose the experts of every token: logits [N][E] -> out (see Route). With
    out.balance_loss also the counts, the probability sums and the balance loss."""
    _, x, m = _route_args("ep_route", cfg, logits, token_mask, out)
    b = None if choice_bias is None else _at(choice_bias, _F32, cfg.num_experts, "ep_route", "choice_bias")
    st = (_lib or lib()).ep_route(cfg._reference or cfg._ref(), x, b, m, out._reference or out._ref(),
                                  *_space(ws, "ep_route"), _raw_stream(stream))
    if st:
        raise EpError(st, "ep_route")


def ep_route_grad(cfg: RouteConfig, logits: torch.Tensor, token_mask, route: Route, d_weights, d_loss,
                  d_logits: torch.Tensor, ws: torch.Tensor, stream=None):
    """Gradient of the logits through the weights (d_weights [N][K] or None) and the
    balance loss (d_loss [1] or None)."""
    w = "ep_route_grad"
    needs, x, m = _route_args(w, cfg, logits, token_mask, route)
    dw = None if d_weights is None else _at(d_weights, _F32, needs[2], w, "d_weights")
    dl = None if d_loss is None else _at(d_loss, _F32, 1, w, "d_loss")
    st = (_lib or lib()).ep_route_grad(cfg._reference or cfg._ref(), x, m, route._reference or route._ref(), dw, dl,
                                       _at(d_logits, needs[0], needs[1], w, "d_logits"), *_space(ws, w),
                                       _raw_stream(stream))
    if st:
        raise EpError(st, w)


def ep_combine_grad(cfg: Config, layout: Layout, y, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                    d_out: torch.Tensor, d_y, d_weights, ws: torch.Tensor, stream=None):
    """Gradient of ep_combine: d_y (rows of y) and d_weights [R][T][K]; either may be None."""
    w = "ep_combine_grad"
    N, H = cfg.num_ranks * cfg.num_tokens, cfg.hidden
    rows = cfg._sizes  # kept until a field of cfg is assigned
    if rows is None:
        rows = max(ep_recv_rows(cfg), 0)
        object.__setattr__(cfg, "_sizes", rows)
    NK, R = N * cfg.num_topk, cfg.num_ranks
    fields = _LANE_FIELDS[3 if cfg.expand else min(max(cfg.compact_recv, 0), 2)]
    kept = layout._lanes
    if kept is None or kept[0] is not fields:
        kept = (fields, layout._count(w, fields))
        object.__setattr__(layout, "_lanes", kept)
    need = (NK, R) if cfg.expand else (NK, R * R, R)
    for n, least in zip(kept[1], need):
        if -1 < n < least:
            _too_small(w, layout, fields, need)
    y = _at(y, _BF16, rows * H, w, "y") if d_weights is not None or y is not None else None
    _check((_lib or lib()).ep_combine_grad(
        cfg._reference or cfg._ref(), layout._reference or layout._ref(), y, _at(topk_idx, _I64, NK, w, "topk_idx"),
        _at(topk_weights, _F32, NK, w, "topk_weights"), _at(d_out, _BF16, N * H, w, "d_out"),
        _maybe(d_y, _BF16, rows * H, w, "d_y"), _maybe(d_weights, _F32, NK, w, "d_weights"), *_space(ws, w),
        _raw_stream(stream)), w)


def _blocks_arg(where, needs, layout):
    if layout is None:
        return None
    c, b, r = layout._sizes or layout._checked(where, _BLOCK_FIELDS)
    if -1 < c < needs[6] or -1 < b < needs[7] or -1 < r < needs[8]:
        _too_small(where, layout, _BLOCK_FIELDS, needs[6:])
    return layout._reference or layout._ref()


def ep_expert_product(cfg: ProductConfig, layout, x: torch.Tensor, x_sf, weight: torch.Tensor, bias, residual, z,
                      out: torch.Tensor, ws: torch.Tensor, stream=None):
    """out = act(x W_g^T + b_g) + residual over every expert's block of an expanded
    layout (layout None: one group of all rows); z, if given, keeps what the activation was taken of."""
    w = "ep_expert_product"
    needs = cfg._sizes or cfg._needs()
    n_x, n_sf, n_w, n_b, n_out, n_z = needs[:6]
    if cfg.x_dtype == EP_DTYPE_FP8_E4M3:
        x = _at(x, torch.float8_e4m3fn if x is not None and x.dtype is torch.float8_e4m3fn else _U8, n_x, w, "x")
        x_sf = _at(x_sf, _F32, n_sf, w, "x_sf")
    else:
        x = _at(x, _BF16, n_x, w, "x")
        x_sf = _maybe(x_sf, _F32, 0, w, "x_sf")
    st = (_lib or lib()).ep_expert_product(
        cfg._reference or cfg._ref(), _blocks_arg(w, needs, layout), x, x_sf, _at(weight, _BF16, n_w, w, "weight"),
        None if bias is None else _at(bias, _BF16, n_b, w, "bias"),
        None if residual is None else _at(residual, _BF16, n_out, w, "residual"),
        None if z is None else _at(z, _BF16, n_z, w, "z"), _at(out, _BF16, n_out, w, "out"), *_space(ws, w),
        _raw_stream(stream))
    if st:
        raise EpError(st, w)


def ep_expert_product_grad(cfg: ProductConfig, layout, x, weight, z, d_out: torch.Tensor, d_x, d_weight, d_bias,
                           ws: torch.Tensor, stream=None):
    """Gradients of ep_expert_product's rows, matrices and biases; any of the three may be None."""
    w = "ep_expert_product_grad"
    needs = cfg._sizes or cfg._needs()
    n_x, _, n_w, n_b, n_out, n_z = needs[:6]
    x = _at(x, _BF16, n_x, w, "x") if d_weight is not None or x is not None else None
    weight = _at(weight, _BF16, n_w, w, "weight") if d_x is not None or weight is not None else None
    z = _at(z, _BF16, n_z, w, "z") if cfg.activation != EP_ACT_NONE or z is not None else None
    st = (_lib or lib()).ep_expert_product_grad(
        cfg._reference or cfg._ref(), _blocks_arg(w, needs, layout), x, weight, z, _at(d_out, _BF16, n_out, w, "d_out"),
        None if d_x is None else _at(d_x, _BF16, n_x, w, "d_x"),
        None if d_weight is None else _at(d_weight, _BF16, n_w, w, "d_weight"),
        None if d_bias is None else _at(d_bias, _F32, n_b, w, "d_bias"), *_space(ws, w), _raw_stream(stream))
    if st:
        raise EpError(st, w)
