"""ctypes binding of ``liba2av.so`` (declared in ``include/a2av.h``).

Argument marshalling only: torch tensors are checked (device, dtype, shape,
contiguity) and their device pointers, together with the current CUDA stream,
are handed to the C ABI.  Every step of the data path runs in the library's
CUDA kernels; there is no CPU fallback, and loading fails loudly when the
library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

from . import build as _build

A2AV_OK = 0
A2AV_ERR_INVALID_ARG = 1
A2AV_ERR_CUDA = 2
A2AV_ERR_NO_MEMORY = 3

DEV_BAD_EXPERT = 1 << 0
DEV_WINDOW_OVERFLOW = 1 << 1
DEV_WAIT_TIMEOUT = 1 << 31

WINDOW_PACKED = 0
WINDOW_FIXED = 1
WINDOW_PADDED = 2
ORDER_SOURCE = 0  # windows in source order, each source segment sorted by expert
ORDER_EXPERT = 1  # windows grouped by local expert, sources in order inside each expert
FLAG_PACK_LSU = 1 << 0
FLAG_SPLITS_TILED = 1 << 1
FLAG_COMBINE_TMA = 1 << 2
FLAG_ROUTE_FUSED = 1 << 3
FLAG_ROUTE_WARP = 1 << 4
W_BF16 = 0  # weight types of the experts' products
W_E4M3 = 1
W_INT4 = 2
ACTIVATIONS = {None: 0, "none": 0, "swiglu": 1}
SCORES = {"softmax": 0, "sigmoid": 1}
GATE_NONE, GATE_CHANNEL, GATE_RANK, GATE_TOKEN = 0, 1, 2, 3
ROW8_TAIL = 16  # bytes behind the values of an 8-bit row: the fp32 scale and padding

# Every function the header declares, for load checks.
EXPORTED = [
    "a2av_config_check", "a2av_recv_arena_rows", "a2av_plan_create", "a2av_plan_destroy",
    "a2av_dispatch", "a2av_splits", "a2av_pack", "a2av_combine", "a2av_expert_scale",
    "a2av_read_device_status", "a2av_device_status_ptr", "a2av_plan_launches",
    "a2av_status_string", "a2av_last_error", "a2av_dispatch_static",
    "a2av_dispatch_padded", "a2av_pack_padded", "a2av_exchange_padded", "a2av_set_active_tokens",
    "a2av_route", "a2av_route_splits", "a2av_set_wait_limit", "a2av_rms_norm", "a2av_quantize_rows",
    "a2av_expert_matmul", "a2av_route_scores", "a2av_route_scores_grad", "a2av_combine_grad", "a2av_block_norm",
    "a2av_norm_scratch_bytes", "a2av_block_norm_grad",
]


class Config(ctypes.Structure):
    _fields_ = [
        ("num_ranks", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("tokens_per_rank", ctypes.c_int32),
        ("hidden", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("window_mode", ctypes.c_int32),
        ("window_rows", ctypes.c_int64),
        ("device", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("pack_ctas_per_sm", ctypes.c_int32),
        ("pack_stage_bytes", ctypes.c_int32),
        ("pack_store_lag", ctypes.c_int32),
        ("combine_ctas_per_sm", ctypes.c_int32),
        ("combine_stage_bytes", ctypes.c_int32),
        ("combine_unroll", ctypes.c_int32),
        ("recv_order", ctypes.c_int32),
    ]


class SplitsPtrs(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "send_counts", "send_offsets", "recv_counts", "recv_offsets", "recv_expert_counts",
        "recv_total", "window_base", "recv_expert_offsets")]


class A2avError(RuntimeError):
    pass


class RouteRule(ctypes.Structure):
    """How ``Plan.route_scores`` chooses experts and what their gates are (a2av_route_rule_t).

    ``score`` "softmax" (over all experts) or "sigmoid"; ``groups`` of consecutive experts, of which a token
    may choose from ``groups_kept`` (None: all), valued by their best choice or the sum of their two best
    (``group_best`` 1 or 2); ``renormalize``: gates divided by their sum; ``scale``: a factor of the gates."""

    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("groups_kept", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, score="softmax", groups=1, groups_kept=None, group_best=1, renormalize=True, scale=1.0):
        if score not in SCORES:
            raise A2avError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
        whole = []
        for name, v in (("groups", groups), ("groups_kept", groups if groups_kept is None else groups_kept),
                        ("group_best", group_best)):
            # a field would drop a fraction and what is past 32 bits
            if isinstance(v, str) or not abs(v) < 2 ** 31 or int(v) != v:
                raise A2avError(f"{name} must be a whole number of 32 bits, got {v!r}")
            whole.append(int(v))
        super().__init__(SCORES[score], *whole, int(bool(renormalize)), float(scale))


class BlockNormArgs(ctypes.Structure):
    _fields_ = [("post_weight", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("gate_kind", ctypes.c_int32), ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("eps", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(path: Optional[str] = None):
    """Load liba2av.so (declaring the C signatures).  Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise A2avError(f"{p} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(p)
    vp, i32 = ctypes.c_void_p, ctypes.c_int32
    cfgp = ctypes.POINTER(Config)
    spp = ctypes.POINTER(SplitsPtrs)
    L.a2av_config_check.argtypes = [cfgp]
    L.a2av_config_check.restype = i32
    L.a2av_recv_arena_rows.argtypes = [cfgp]
    L.a2av_recv_arena_rows.restype = ctypes.c_int64
    L.a2av_plan_create.argtypes = [cfgp, ctypes.POINTER(vp)]
    L.a2av_plan_create.restype = i32
    L.a2av_plan_destroy.argtypes = [vp]
    L.a2av_plan_destroy.restype = i32
    L.a2av_dispatch.argtypes = [vp, vp, vp, spp, vp, vp, vp]
    L.a2av_dispatch.restype = i32
    L.a2av_splits.argtypes = [vp, vp, spp, vp, vp]
    L.a2av_splits.restype = i32
    L.a2av_pack.argtypes = [vp, vp, vp, spp, vp, vp, vp]
    L.a2av_pack.restype = i32
    L.a2av_combine.argtypes = [vp, vp, vp, vp, vp, vp]
    L.a2av_combine.restype = i32
    L.a2av_expert_scale.argtypes = [vp, vp, vp, vp, vp, vp]
    L.a2av_expert_scale.restype = i32
    L.a2av_read_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, vp]
    L.a2av_read_device_status.restype = i32
    L.a2av_device_status_ptr.argtypes = [vp]
    L.a2av_device_status_ptr.restype = vp
    L.a2av_plan_launches.argtypes = [vp]
    L.a2av_plan_launches.restype = ctypes.c_int64
    L.a2av_status_string.argtypes = [i32]
    L.a2av_status_string.restype = ctypes.c_char_p
    L.a2av_last_error.argtypes = []
    L.a2av_last_error.restype = ctypes.c_char_p
    L.a2av_dispatch_static.argtypes = [cfgp, vp, vp, spp, vp, vp, vp, vp]
    L.a2av_dispatch_static.restype = i32
    L.a2av_dispatch_padded.argtypes = [vp, vp, vp, spp, vp, vp, vp, vp]
    L.a2av_dispatch_padded.restype = i32
    L.a2av_pack_padded.argtypes = [vp, vp, vp, spp, vp, vp, vp]
    L.a2av_pack_padded.restype = i32
    L.a2av_exchange_padded.argtypes = [vp, vp, vp, vp]
    L.a2av_exchange_padded.restype = i32
    L.a2av_set_active_tokens.argtypes = [vp, vp]
    L.a2av_set_active_tokens.restype = i32
    L.a2av_route.argtypes = [vp, vp, vp, vp, vp]
    L.a2av_route.restype = i32
    L.a2av_route_splits.argtypes = [vp, vp, vp, vp, spp, vp, vp]
    L.a2av_route_splits.restype = i32
    L.a2av_set_wait_limit.argtypes = [vp, ctypes.c_int64]
    L.a2av_set_wait_limit.restype = i32
    L.a2av_rms_norm.argtypes = [vp, vp, vp, vp, ctypes.c_float, vp, vp, vp, vp]
    L.a2av_rms_norm.restype = i32
    L.a2av_quantize_rows.argtypes = [vp, vp, i32, spp, vp, vp]
    L.a2av_quantize_rows.restype = i32
    L.a2av_expert_matmul.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, spp, vp]
    L.a2av_expert_matmul.restype = i32
    rulep, normp = ctypes.POINTER(RouteRule), ctypes.POINTER(BlockNormArgs)
    L.a2av_route_scores.argtypes = [vp, rulep, vp, vp, vp, vp, vp]
    L.a2av_route_scores.restype = i32
    L.a2av_route_scores_grad.argtypes = [vp, rulep, vp, vp, vp, vp, vp]
    L.a2av_route_scores_grad.restype = i32
    L.a2av_combine_grad.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    L.a2av_combine_grad.restype = i32
    L.a2av_block_norm.argtypes = [vp, normp, vp, vp, vp, vp, vp, vp]
    L.a2av_block_norm.restype = i32
    L.a2av_norm_scratch_bytes.argtypes = [vp]
    L.a2av_norm_scratch_bytes.restype = ctypes.c_int64
    L.a2av_block_norm_grad.argtypes = [vp, normp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.a2av_block_norm_grad.restype = i32
    if path is None:
        _lib = L
    return L


def _check(L, rc: int, what: str):
    if rc != A2AV_OK:
        msg = L.a2av_status_string(rc).decode()
        detail = L.a2av_last_error().decode()
        raise A2avError(f"{what}: {msg}" + (f" ({detail})" if detail else ""))


def make_config(R, E, T, H, k, window_mode="packed", window_rows=0, device=0, flags=0,
                pack_ctas_per_sm=0, pack_stage_bytes=0, pack_store_lag=0, combine_ctas_per_sm=0,
                combine_stage_bytes=0, combine_unroll=0, recv_order="source") -> Config:
    mode = {"packed": WINDOW_PACKED, "fixed": WINDOW_FIXED, "padded": WINDOW_PADDED}.get(window_mode, window_mode)
    order = {"source": ORDER_SOURCE, "expert": ORDER_EXPERT}.get(recv_order, recv_order)
    return Config(int(R), int(E), int(T), int(H), int(k), int(mode), int(window_rows), int(device),
                  int(flags), int(pack_ctas_per_sm), int(pack_stage_bytes), int(pack_store_lag),
                  int(combine_ctas_per_sm), int(combine_stage_bytes), int(combine_unroll), int(order))


class Splits:
    """Device-resident split counts/offsets of one dispatch (int32 tensors).

    ``recv_expert_offsets`` is allocated and filled only when
    ``expert_offsets`` is true (the expert-grouped receive order needs it;
    in source order it is an optional extra output of the splits kernel)."""

    NAMES = ("send_counts", "send_offsets", "recv_counts", "recv_offsets", "recv_expert_counts",
             "recv_total", "window_base", "recv_expert_offsets")

    def __init__(self, R: int, E: int, device, expert_offsets: bool = True):
        import torch

        epr = E // R
        shapes = {"send_counts": (R, E), "send_offsets": (R, E), "recv_counts": (R, R),
                  "recv_offsets": (R, R), "recv_expert_counts": (R, R, epr), "recv_total": (R,),
                  "window_base": (R,), "recv_expert_offsets": (R, R, epr)}
        self.names = self.NAMES if expert_offsets else self.NAMES[:-1]
        for n in self.NAMES:
            setattr(self, n, torch.zeros(shapes[n], dtype=torch.int32, device=device) if n in self.names else None)
        self._ptrs = SplitsPtrs(*[getattr(self, n).data_ptr() if n in self.names else None for n in self.NAMES])

    @property
    def ptrs(self) -> SplitsPtrs:
        return self._ptrs

    def to_numpy(self) -> dict:
        return {n: getattr(self, n).cpu().numpy() for n in self.names}


def _stream_ptr(stream, device):
    import torch

    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


@functools.cache
def _torch():
    """torch, which the package imports without.  (An import statement takes about as long as a check of an argument;
    this, in the calls where that counts, does not.)"""
    import torch

    return torch


def _raw_stream(index):
    """The current stream's handle by device ordinal: torch's own short way where it has one (making a
    Stream object takes longer than a small kernel)."""
    torch = _torch()
    short = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return short(index) if short else torch.cuda.current_stream(index).cuda_stream


def _width(t, name):
    """Length of a tensor's last dimension (what else it has to be, ``_p`` checks)."""
    shape = getattr(t, "shape", None)
    if not shape:
        raise A2avError(f"{name} must be a torch tensor with at least one dimension")
    return shape[-1]


class Plan:
    """A configured data plane: R emulated ranks, E experts, T tokens per rank,
    hidden H, top-k.  Owns only the library's small workspace."""

    def __init__(self, R, E, T, H, k, window_mode="packed", window_rows=0, device=None, flags=0,
                 pack_ctas_per_sm=0, pack_stage_bytes=0, pack_store_lag=0, combine_ctas_per_sm=0,
                 combine_stage_bytes=0, combine_unroll=0, recv_order="source"):
        import torch

        self.lib = load_library()
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise A2avError("a2av plans live on a CUDA device")
        self.device = dev
        self.R, self.E, self.T, self.H, self.k = int(R), int(E), int(T), int(H), int(k)
        self.window_mode = window_mode
        self.window_rows = int(window_rows)
        self.recv_order = recv_order
        self.cfg = make_config(R, E, T, H, k, window_mode, window_rows, dev.index, flags,
                               pack_ctas_per_sm, pack_stage_bytes, pack_store_lag, combine_ctas_per_sm,
                               combine_stage_bytes, combine_unroll, recv_order)
        handle = ctypes.c_void_p()
        _check(self.lib, self.lib.a2av_plan_create(ctypes.byref(self.cfg), ctypes.byref(handle)), "a2av_plan_create")
        self.handle = handle
        self.arena_rows = int(self.lib.a2av_recv_arena_rows(ctypes.byref(self.cfg)))

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            _check(self.lib, self.lib.a2av_plan_destroy(self.handle), "a2av_plan_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- tensors ------------------------------------------------------------
    def new_splits(self, expert_offsets=None) -> Splits:
        """Split arrays for this plan; ``expert_offsets`` None = only when the
        receive order needs them (the expert-grouped order)."""
        if expert_offsets is None:
            expert_offsets = self.recv_order in ("expert", ORDER_EXPERT)
        return Splits(self.R, self.E, self.device, expert_offsets=bool(expert_offsets))

    def new_buffers(self):
        """(recv [arena_rows][H] bf16, slot_map [R][T][k] int32, out [R][T][H] bf16), uninitialised."""
        import torch

        recv = torch.empty((self.arena_rows, self.H), dtype=torch.bfloat16, device=self.device)
        slot_map = torch.empty((self.R, self.T, self.k), dtype=torch.int32, device=self.device)
        out = torch.empty((self.R, self.T, self.H), dtype=torch.bfloat16, device=self.device)
        return recv, slot_map, out

    def _t(self, t, dtype, shape, name):
        import torch

        if not isinstance(t, torch.Tensor):
            raise A2avError(f"{name} must be a torch tensor")
        if t.device != self.device:
            raise A2avError(f"{name} is on {t.device}, the plan is on {self.device}")
        if t.dtype != dtype:
            raise A2avError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise A2avError(f"{name} must be contiguous")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise A2avError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        return ctypes.c_void_p(t.data_ptr())

    def _rows(self, t, name):
        import torch

        return self._t(t, torch.bfloat16, (self.arena_rows, self.H), name)

    # ---- calls ----------------------------------------------------------------
    def dispatch(self, x, topk_idx, splits: Splits, recv, slot_map, stream=None):
        import torch

        args = (self.handle, self._t(x, torch.bfloat16, (self.R, self.T, self.H), "x"),
                self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"), ctypes.byref(splits.ptrs),
                self._rows(recv, "recv"), self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
                _stream_ptr(stream, self.device))
        _check(self.lib, self.lib.a2av_dispatch(*args), "a2av_dispatch")

    def splits(self, topk_idx, splits: Splits, slot_map, stream=None):
        import torch

        _check(self.lib, self.lib.a2av_splits(
            self.handle, self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"),
            ctypes.byref(splits.ptrs), self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
            _stream_ptr(stream, self.device)), "a2av_splits")

    def pack(self, x, topk_idx, splits: Splits, recv, slot_map, stream=None):
        import torch

        _check(self.lib, self.lib.a2av_pack(
            self.handle, self._t(x, torch.bfloat16, (self.R, self.T, self.H), "x"),
            self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"), ctypes.byref(splits.ptrs),
            self._rows(recv, "recv"), self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
            _stream_ptr(stream, self.device)), "a2av_pack")

    def route(self, logits, topk_idx, gate_w, stream=None):
        """Top-k experts and softmax gates of fp32 logits [R][T][E] (a2av_route)."""
        import torch

        _check(self.lib, self.lib.a2av_route(
            self.handle, self._t(logits, torch.float32, (self.R, self.T, self.E), "logits"),
            self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"),
            self._t(gate_w, torch.float32, (self.R, self.T, self.k), "gate_w"),
            _stream_ptr(stream, self.device)), "a2av_route")

    def route_splits(self, logits, topk_idx, gate_w, splits: Splits, slot_map, stream=None):
        """Router + splits in one kernel where possible (a2av_route_splits);
        follow with ``pack`` as after ``splits``."""
        import torch

        _check(self.lib, self.lib.a2av_route_splits(
            self.handle, self._t(logits, torch.float32, (self.R, self.T, self.E), "logits"),
            self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"),
            self._t(gate_w, torch.float32, (self.R, self.T, self.k), "gate_w"), ctypes.byref(splits.ptrs),
            self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
            _stream_ptr(stream, self.device)), "a2av_route_splits")

    def set_active_tokens(self, num_tokens=None):
        """Read per-rank token counts from the int32 device tensor `num_tokens`
        [R] in every later call (None: every token takes part)."""
        import torch

        if num_tokens is None:
            self._num_tokens = None
            ptr = None
        else:
            self._t(num_tokens, torch.int32, (self.R,), "num_tokens")
            self._num_tokens = num_tokens  # keep it alive while the plan may read it
            ptr = ctypes.c_void_p(num_tokens.data_ptr())
        _check(self.lib, self.lib.a2av_set_active_tokens(self.handle, ptr), "a2av_set_active_tokens")

    def new_send_buffer(self):
        """Padded plans: the worst-case send buffer, bf16 [R*R*T*k][H] (uninitialised)."""
        import torch

        return torch.empty((self.arena_rows, self.H), dtype=torch.bfloat16, device=self.device)

    def dispatch_padded(self, x, topk_idx, splits: Splits, sendbuf, recv, slot_map, stream=None):
        import torch

        _check(self.lib, self.lib.a2av_dispatch_padded(
            self.handle, self._t(x, torch.bfloat16, (self.R, self.T, self.H), "x"),
            self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"), ctypes.byref(splits.ptrs),
            self._rows(sendbuf, "sendbuf"), self._rows(recv, "recv"),
            self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
            _stream_ptr(stream, self.device)), "a2av_dispatch_padded")

    def pack_padded(self, x, topk_idx, splits: Splits, sendbuf, slot_map, stream=None):
        import torch

        _check(self.lib, self.lib.a2av_pack_padded(
            self.handle, self._t(x, torch.bfloat16, (self.R, self.T, self.H), "x"),
            self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"), ctypes.byref(splits.ptrs),
            self._rows(sendbuf, "sendbuf"), self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
            _stream_ptr(stream, self.device)), "a2av_pack_padded")

    def exchange_padded(self, sendbuf, recv, stream=None):
        _check(self.lib, self.lib.a2av_exchange_padded(
            self.handle, self._rows(sendbuf, "sendbuf"), self._rows(recv, "recv"),
            _stream_ptr(stream, self.device)), "a2av_exchange_padded")

    def combine(self, y, gate_w, slot_map, out, stream=None):
        import torch

        _check(self.lib, self.lib.a2av_combine(
            self.handle, self._rows(y, "y"), self._t(gate_w, torch.float32, (self.R, self.T, self.k), "gate_w"),
            self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"),
            self._t(out, torch.bfloat16, (self.R, self.T, self.H), "out"),
            _stream_ptr(stream, self.device)), "a2av_combine")

    def expert_scale(self, recv, topk_idx, slot_map, y, stream=None):
        import torch

        _check(self.lib, self.lib.a2av_expert_scale(
            self.handle, self._rows(recv, "recv"), self._t(topk_idx, torch.int32, (self.R, self.T, self.k), "topk_idx"),
            self._t(slot_map, torch.int32, (self.R, self.T, self.k), "slot_map"), self._rows(y, "y"),
            _stream_ptr(stream, self.device)), "a2av_expert_scale")

    # ---- the norm in front and the experts in between ---------------------------
    def new_rows8(self, rows, K):
        """Zeroed 8-bit rows [rows][K+16] (uint8; `rows` a number or a leading
        shape): K e4m3 values, the fp32 scale, padding (``rows8_parts``)."""
        import torch

        lead = (int(rows),) if isinstance(rows, int) else tuple(rows)
        return torch.zeros(lead + (int(K) + ROW8_TAIL,), dtype=torch.uint8, device=self.device)

    def rms_norm(self, x, weight, y=None, rows8=None, residual=None, residual_out=None, eps=1e-6, stream=None):
        """Root-mean-square norm of x (+ residual) over H, times `weight`
        (a2av_rms_norm): into y (bf16) and/or rows8 (8-bit rows [R][T][H+16]),
        the sum into residual_out (which may be x or residual itself)."""
        torch = _torch()
        bf16, shape, p = torch.bfloat16, (self.R, self.T, self.H), self._p
        rc = self.lib.a2av_rms_norm(
            self.handle, p(x, bf16, shape, "x"), None if residual is None else p(residual, bf16, shape, "residual"),
            p(weight, bf16, (self.H,), "weight"), eps,
            None if residual_out is None else p(residual_out, bf16, shape, "residual_out"),
            None if y is None else p(y, bf16, shape, "y"),
            None if rows8 is None else p(rows8, torch.uint8, (self.R, self.T, self.H + ROW8_TAIL), "rows8"),
            self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_rms_norm")

    def quantize_rows(self, x, splits: Splits, rows8, stream=None):
        """8-bit rows of the live rows of an arena x [arena_rows][K] (a2av_quantize_rows)."""
        torch = _torch()
        K = _width(x, "x")
        rc = self.lib.a2av_quantize_rows(
            self.handle, self._p(x, torch.bfloat16, (self.arena_rows, K), "x"), K, self._sp(splits),
            self._p(rows8, torch.uint8, (self.arena_rows, K + ROW8_TAIL), "rows8"), self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_quantize_rows")

    def expert_matmul(self, x, w, splits: Splits, y, w_scale=None, activation=None, stream=None):
        """y[r] = act(x[r] . w[e]^T) for every live row r, e its expert (a2av_expert_matmul).

        w [E][Nw][K] bf16 with x bf16 [arena_rows][K], or float8_e4m3fn with
        w_scale fp32 [E][Nw] and x 8-bit rows [arena_rows][K+16]; y bf16
        [arena_rows][N].  activation "swiglu": Nw = 2N, gate rows then up rows."""
        torch = _torch()
        K = _width(w, "w")
        if w.dtype is torch.float8_e4m3fn:
            kind, dtype, xp = W_E4M3, w.dtype, self._p(x, torch.uint8, (self.arena_rows, K + ROW8_TAIL), "x")
        else:
            kind, dtype, xp = W_BF16, torch.bfloat16, self._p(x, torch.bfloat16, (self.arena_rows, K), "x")
        if w_scale is not None:
            w_scale = self._p(w_scale, torch.float32, w.shape[:2], "w_scale")
        self._matmul(xp, w, dtype, K, K, kind, 0, w_scale, splits, y, activation, stream)

    def expert_matmul_w4(self, x, w4, w_scale, splits: Splits, y, activation=None, stream=None):
        """``expert_matmul`` with 4-bit weights, for few rows per expert: w4 int32
        [E][Nw][K/8], w_scale bf16 [E][Nw][K/group] (``pack_weights_w4``), x bf16."""
        torch = _torch()
        K = _width(w4, "w4") * 8
        groups = max(1, _width(w_scale, "w_scale"))
        if K % groups:
            raise A2avError(f"w_scale has {groups} groups, which do not divide K = {K}")
        self._matmul(self._p(x, torch.bfloat16, (self.arena_rows, K), "x"), w4, torch.int32, K, K // 8, W_INT4,
                     K // groups, self._p(w_scale, torch.bfloat16, (*w4.shape[:2], groups), "w_scale"),
                     splits, y, activation, stream)

    def _matmul(self, x, w, w_dtype, K, w_width, kind, group, w_scale, splits, y, activation, stream):
        torch = _torch()
        act = ACTIVATIONS.get(activation, -1)
        if act < 0:
            raise A2avError(f"activation must be None or 'swiglu', got {activation!r}")
        N = _width(y, "y")
        rc = self.lib.a2av_expert_matmul(
            self.handle, x, self._p(w, w_dtype, (self.E, N << act, w_width), "w"), w_scale,
            self._p(y, torch.bfloat16, (self.arena_rows, N), "y"), K, N, kind, group, act, self._sp(splits),
            self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_expert_matmul")

    # ---- the router by scores, the gradients, the norms around a block ----------------
    def _rule(self, rule):
        if not isinstance(rule, RouteRule):
            raise A2avError("rule must be a RouteRule")
        return rule

    def route_scores(self, logits, topk_idx, gate_w, rule: RouteRule, bias=None, stream=None):
        """Experts and gates of fp32 logits [R][T][E] by ``rule`` (a2av_route_scores); ``bias`` fp32 [E]
        takes part in the choice alone."""
        torch = _torch()
        f32, p, per = torch.float32, self._p, (self.R, self.T, self.k)
        rc = self.lib.a2av_route_scores(
            self.handle, self._rule(rule), p(logits, f32, (self.R, self.T, self.E), "logits"),
            None if bias is None else p(bias, f32, (self.E,), "bias"), p(topk_idx, torch.int32, per, "topk_idx"),
            p(gate_w, f32, per, "gate_w"), self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_route_scores")

    def route_scores_grad(self, logits, topk_idx, d_gate, d_logits, rule: RouteRule, stream=None):
        """d_logits fp32 [R][T][E] from the gradient of ``route_scores``' gates (a2av_route_scores_grad)."""
        torch = _torch()
        f32, p, per, each = torch.float32, self._p, (self.R, self.T, self.k), (self.R, self.T, self.E)
        rc = self.lib.a2av_route_scores_grad(
            self.handle, self._rule(rule), p(logits, f32, each, "logits"), p(topk_idx, torch.int32, per, "topk_idx"),
            p(d_gate, f32, per, "d_gate"), p(d_logits, f32, each, "d_logits"), self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_route_scores_grad")

    def combine_grad(self, d_out, y, gate_w, slot_map, d_y=None, d_gate=None, stream=None):
        """Gradients of ``combine`` (a2av_combine_grad): d_y [arena_rows][H] bf16, live rows only (may be y
        itself), and/or d_gate fp32 [R][T][k].  y may be None without d_gate, gate_w without d_y."""
        torch = _torch()
        bf16, p, per, arena = torch.bfloat16, self._p, (self.R, self.T, self.k), (self.arena_rows, self.H)
        rc = self.lib.a2av_combine_grad(
            self.handle, p(d_out, bf16, (self.R, self.T, self.H), "d_out"), None if y is None else p(y, bf16, arena, "y"),
            None if gate_w is None else p(gate_w, torch.float32, per, "gate_w"),
            p(slot_map, torch.int32, per, "slot_map"), None if d_y is None else p(d_y, bf16, arena, "d_y"),
            None if d_gate is None else p(d_gate, torch.float32, per, "d_gate"), self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_combine_grad")

    def _gate_kind(self, gate):
        if gate is None:
            return GATE_NONE
        dim = getattr(gate, "ndim", 0)
        if dim not in (1, 2, 3):
            raise A2avError("gate must be a tensor [H], [R][H] or [R][T][H]")
        return dim

    def _gate_shape(self, kind):
        return ((self.H,), (self.R, self.H), (self.R, self.T, self.H))[kind - 1]

    def _block_norm_args(self, post_weight, gate, weight, residual_scale, branch_scale, eps):
        bf16, p, kind = _torch().bfloat16, self._p, self._gate_kind(gate)
        return kind, BlockNormArgs(
            None if post_weight is None else p(post_weight, bf16, (self.H,), "post_weight"),
            None if gate is None else p(gate, bf16, self._gate_shape(kind), "gate"),
            None if weight is None else p(weight, bf16, (self.H,), "weight"), kind, residual_scale, branch_scale, eps)

    def block_norm(self, x, residual, residual_out=None, weight=None, y=None, rows8=None, post_weight=None, gate=None,
                   residual_scale=1.0, branch_scale=1.0, eps=1e-6, stream=None):
        """Between two blocks (a2av_block_norm): x, what a block gave, normed by ``post_weight``, times ``gate``
        ([H], [R][H] or [R][T][H]) and ``branch_scale``, plus ``residual_scale`` * residual, into residual_out
        (which may be x or residual itself); that normed by ``weight`` into y (bf16) and/or rows8 (8-bit rows)."""
        torch = _torch()
        bf16, shape, p = torch.bfloat16, (self.R, self.T, self.H), self._p
        _, args = self._block_norm_args(post_weight, gate, weight, residual_scale, branch_scale, eps)
        rc = self.lib.a2av_block_norm(
            self.handle, args, p(x, bf16, shape, "x"), p(residual, bf16, shape, "residual"),
            None if residual_out is None else p(residual_out, bf16, shape, "residual_out"),
            None if y is None else p(y, bf16, shape, "y"),
            None if rows8 is None else p(rows8, torch.uint8, (self.R, self.T, self.H + ROW8_TAIL), "rows8"),
            self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_block_norm")

    def new_norm_scratch(self):
        """Scratch of ``block_norm_grad`` for this plan (uint8, uninitialised); one per call in flight."""
        torch = _torch()
        return torch.empty(int(self.lib.a2av_norm_scratch_bytes(self.handle)), dtype=torch.uint8, device=self.device)

    def block_norm_grad(self, x, residual, d_x, d_residual, weight=None, d_y=None, d_residual_out=None,
                        post_weight=None, gate=None, d_weight=None, d_post_weight=None, d_gate=None, scratch=None,
                        residual_scale=1.0, branch_scale=1.0, eps=1e-6, stream=None):
        """Gradients of ``block_norm`` from d_y and/or d_residual_out (a2av_block_norm_grad): d_x and d_residual
        bf16 [R][T][H] (which may be d_y and d_residual_out themselves), the weights' in fp32, d_gate fp32 as gate's
        shape, or bf16 for a gate [R][T][H].  ``scratch``: ``new_norm_scratch``, where a summed gradient is asked for."""
        torch = _torch()
        bf16, f32, shape, p = torch.bfloat16, torch.float32, (self.R, self.T, self.H), self._p
        kind, args = self._block_norm_args(post_weight, gate, weight, residual_scale, branch_scale, eps)
        if d_gate is not None:
            if kind == GATE_NONE:
                raise A2avError("d_gate needs gate")
            d_gate = p(d_gate, bf16 if kind == GATE_TOKEN else f32, self._gate_shape(kind), "d_gate")
        if scratch is not None:
            scratch = p(scratch, torch.uint8, (int(self.lib.a2av_norm_scratch_bytes(self.handle)),), "scratch")
        rc = self.lib.a2av_block_norm_grad(
            self.handle, args, p(x, bf16, shape, "x"), p(residual, bf16, shape, "residual"),
            None if d_y is None else p(d_y, bf16, shape, "d_y"),
            None if d_residual_out is None else p(d_residual_out, bf16, shape, "d_residual_out"),
            p(d_x, bf16, shape, "d_x"), p(d_residual, bf16, shape, "d_residual"),
            None if d_weight is None else p(d_weight, f32, (self.H,), "d_weight"),
            None if d_post_weight is None else p(d_post_weight, f32, (self.H,), "d_post_weight"),
            d_gate, scratch, self._s(stream))
        if rc:
            _check(self.lib, rc, "a2av_block_norm_grad")

    def _p(self, t, dtype, shape, name):
        """Device pointer of a tensor that is as it has to be; else ``_t`` says what is wrong.  (A torch
        dtype is one object, which nothing but a tensor has for its own.)"""
        if (getattr(t, "dtype", None) is dtype and t.shape == shape and t.is_contiguous()
                and t.device == self.device):
            return t.data_ptr()
        return self._t(t, dtype, shape, name)

    def _s(self, stream):
        return _raw_stream(self.device.index) if stream is None else stream.cuda_stream

    def _sp(self, splits):
        """The split arrays of this plan's sizes, on its device."""
        if not isinstance(splits, Splits):
            raise A2avError("splits must be a Splits")
        if splits.send_counts.shape != (self.R, self.E) or splits.send_counts.device != self.device:
            raise A2avError(f"splits were made for {tuple(splits.send_counts.shape)} on {splits.send_counts.device}, "
                            f"the plan has {(self.R, self.E)} on {self.device}")
        return splits.ptrs

    def set_wait_limit(self, polls: int = -1):
        """Main-loop poll limit of the TMA kernels' bounded waits for later
        calls (0: give up at once; negative: the default)."""
        _check(self.lib, self.lib.a2av_set_wait_limit(self.handle, int(polls)), "a2av_set_wait_limit")

    def read_status(self, clear: bool = False, stream=None) -> int:
        bits = ctypes.c_uint32(0)
        _check(self.lib, self.lib.a2av_read_device_status(self.handle, ctypes.byref(bits), int(clear),
                                                          _stream_ptr(stream, self.device)), "a2av_read_device_status")
        return int(bits.value)

    @property
    def launches(self) -> int:
        return int(self.lib.a2av_plan_launches(self.handle))


def _static_shape_checks(L, cfg, x, topk_idx, splits, recv, slot_map, dev_status, R, E, T, H, k):
    """Shapes a2av_dispatch_static's kernels rely on (the C ABI only sees
    pointers): x (R,T,H), topk_idx and slot_map (R,T,k), recv with at least
    the arena's rows of H values, a dev_status element, and split arrays
    made for R ranks and E experts.  Raises A2avError before anything is
    enqueued."""
    rc = L.a2av_config_check(ctypes.byref(cfg))
    if rc != A2AV_OK:
        raise A2avError(f"a2av_dispatch_static: invalid configuration R={R} E={E} T={T} H={H} k={k}")
    want = {"x": (x, (R, T, H)), "topk_idx": (topk_idx, (R, T, k)), "slot_map": (slot_map, (R, T, k))}
    for name, (t, shape) in want.items():
        if tuple(t.shape) != shape:
            raise A2avError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    rows = int(L.a2av_recv_arena_rows(ctypes.byref(cfg)))
    if recv.dim() != 2 or recv.shape[1] != H or recv.shape[0] < rows:
        raise A2avError(f"recv has shape {tuple(recv.shape)}, expected at least ({rows}, {H})")
    if dev_status.numel() < 1:
        raise A2avError("dev_status needs one element")
    epr = E // R
    shapes = {"send_counts": (R, E), "send_offsets": (R, E), "recv_counts": (R, R), "recv_offsets": (R, R),
              "recv_expert_counts": (R, R, epr), "recv_total": (R,), "window_base": (R,),
              "recv_expert_offsets": (R, R, epr)}
    for name in splits.names:
        t = getattr(splits, name)
        if tuple(t.shape) != shapes[name]:
            raise A2avError(f"splits.{name} has shape {tuple(t.shape)}, expected {shapes[name]} (R={R}, E={E})")
    if cfg.recv_order == ORDER_EXPERT and "recv_expert_offsets" not in splits.names:
        raise A2avError("the expert-grouped receive order needs splits.recv_expert_offsets")


def dispatch_static(x, topk_idx, splits: Splits, recv, slot_map, dev_status, R, E, T, H, k,
                    window_mode="packed", window_rows=0, flags=0, stream=None, recv_order="source"):
    """Dispatch without a plan and without any allocation (a2av_dispatch_static).

    For callers that cannot allocate device memory where they dispatch (a
    framework whose caching allocator owns all device memory, a spent
    device-memory budget, a loop that cannot take cudaMalloc's implicit
    synchronisation): the kernels' scratch lives in a static device array of
    the library (1 MiB per GPU), so shapes are bounded; ``dev_status`` is a
    caller-owned int32 device tensor of one element that receives the
    A2AV_DEV_* bits.  The first call on a device (and the first with each
    configuration) does a one-time set-up, so make it before any stream
    capture; calls that overlap on the GPU share the array and race.  Every
    shape is checked here before anything is enqueued.
    """
    import torch

    L = load_library()
    dev = x.device
    cfg = make_config(R, E, T, H, k, window_mode, window_rows, dev.index if dev.index is not None else 0, flags,
                      recv_order=recv_order)
    _static_shape_checks(L, cfg, x, topk_idx, splits, recv, slot_map, dev_status, R, E, T, H, k)
    tensors = [(x, torch.bfloat16, "x"), (topk_idx, torch.int32, "topk_idx"), (recv, torch.bfloat16, "recv"),
               (slot_map, torch.int32, "slot_map"), (dev_status, torch.int32, "dev_status")]
    tensors += [(getattr(splits, n), torch.int32, f"splits.{n}") for n in splits.names]
    for t, dt, name in tensors:
        if t.device != dev or dev.type != "cuda" or t.dtype != dt or not t.is_contiguous():
            raise A2avError(f"{name}: expected a contiguous {dt} tensor on the CUDA device of x ({dev})")
    rc = L.a2av_dispatch_static(ctypes.byref(cfg), ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(topk_idx.data_ptr()),
                                ctypes.byref(splits.ptrs), ctypes.c_void_p(recv.data_ptr()),
                                ctypes.c_void_p(slot_map.data_ptr()), ctypes.c_void_p(dev_status.data_ptr()),
                                _stream_ptr(stream, dev))
    _check(L, rc, "a2av_dispatch_static")
