"""Python binding of libmoe_layout.so: MoE token layout, dispatch and combine on GB300.

Argument marshalling only.  Every step runs in the library's CUDA kernels
(``csrc/``); PyTorch provides device memory and streams.  The entry points
mirror the C-ABI declared in ``include/moe_layout.h``:

    moe_workspace_bytes, moe_layout, moe_stats_words, moe_stats (host record,
    synchronises), moe_stats_device, moe_dispatch, moe_combine, moe_status,
    moe_status_string, moe_layout_noalloc,
    moe_relay_layout, moe_dispatch_relay, moe_combine_relay (the Mode 2 relay),
    moe_expert_groups, moe_dispatch_group, moe_combine_group (per-expert groups),
    moe_route, moe_route_groups, moe_route_backward (the router),
    moe_expert_forward, moe_expert_backward_rows, moe_expert_backward_weights
    (the experts' products), moe_expert_forward_kept, moe_expert_backward_kept
    (with pre-activations kept in 8 bits), moe_combine_backward,
    moe_quant4_row_scale_bytes, moe_quant4_weight_scale_bytes, moe_quant4_rows,
    moe_quant4_weights, moe_expert_forward4 (the experts in 4 bits),
    moe_quant8_rows, moe_quant8_weights, moe_expert_forward8 (in 8-bit integers)

``Problem``, ``Layout``, ``Routing``, ``Grouping`` and ``Experts`` are conveniences that build the C structs and
allocate the caller-owned device buffers.  If the shared library has not been
built, every call raises ``MoeLibraryMissing``; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import operator
import os
import struct
from dataclasses import dataclass, fields
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_layout.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_CUDA, MOE_ERR_BAD_IDS, MOE_ERR_ALIGN, MOE_ERR_CAPACITY, MOE_ERR_TIMEOUT = \
    0, 1, 2, 3, 4, 5, 6
MOE_NOALLOC_SCRATCH_BYTES = 2 << 20
MOE_DTYPE_BF16, MOE_DTYPE_FP8_E4M3 = 0, 1
MOE_STATUS_ID_RANGE, MOE_STATUS_ID_REPEAT, MOE_STATUS_PLACEMENT, MOE_STATUS_SRC_OFFSET = 1, 2, 4, 8
MOE_STATUS_TIMEOUT = 16
MOE_STATUS_RELAY_CAPACITY = 32
MOE_FP8_GROUP = 128
MOE_MAX_GROUPS = 64
MOE_MAX_HIDDEN = 1 << 20
MOE_STATS_HEADER_WORDS = 32
MOE_ST_STATUS = 0  # header word holding the device status bits
MOE_FAULT_WAIT_TIMEOUT = 1
MOE_MOVE_AUTO, MOE_MOVE_VECTOR, MOE_MOVE_BULK = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_LOGITS_F32, MOE_LOGITS_BF16 = 0, 1
MOE_ACT_NONE, MOE_ACT_SWIGLU = 0, 1
MOE_MAX_EXPERT_ROWS = 2 ** 31 - 512
MOE_MAX_ROUTE_GROUPS = 32
MOE_LAYOUT_AUTO, MOE_LAYOUT_SPLIT, MOE_LAYOUT_FUSED, MOE_LAYOUT_TWO_KERNELS = 0, 1, 2, 3

# Header word names in index order (include/moe_layout.h, MOE_ST_*).
STATS_HEADER = ("status", "T", "slots", "row_bytes", "max_expert_count", "argmax_expert",
                "min_expert_count", "max_rank_slots", "max_rank_tokens",
                "sum_mode0_copies", "sum_mode1_copies", "sum_mode2_copies",
                "max_src_mode1_copies", "max_src_mode2_copies", "max_recv_remote", "max_recv_relay",
                "sum_naive_bytes", "sum_mode0_bytes", "sum_mode1_bytes", "sum_mode2_bytes",
                "imbalance_ratio", "rank_imbalance", "num_hosts")
STATS_SRC = ("src_tokens", "src_copies", "src_mode0", "src_mode1", "src_mode2",
             "src_naive_bytes", "src_mode0_bytes", "src_mode1_bytes", "src_mode2_bytes")
STATS_DST = ("recv_slots", "recv_tokens", "recv_self", "recv_local", "recv_remote", "recv_relay")
EXPORTED = ("moe_workspace_bytes", "moe_layout", "moe_stats_words", "moe_stats", "moe_stats_device",
            "moe_dispatch",
            "moe_combine", "moe_status", "moe_status_string", "moe_layout_noalloc",
            "moe_move_faults", "moe_selftest_bounded_waits", "moe_dispatch_quant", "moe_swap_plan",
            "moe_relay_layout", "moe_dispatch_relay", "moe_combine_relay",
            "moe_expert_groups", "moe_dispatch_group", "moe_combine_group",
            "moe_route", "moe_route_groups", "moe_route_backward", "moe_expert_forward", "moe_expert_backward_rows",
            "moe_expert_backward_weights", "moe_expert_forward_kept", "moe_expert_backward_kept",
            "moe_combine_backward", "moe_quant4_row_scale_bytes", "moe_quant4_weight_scale_bytes",
            "moe_quant4_rows", "moe_quant4_weights", "moe_expert_forward4",
            "moe_quant8_rows", "moe_quant8_weights", "moe_expert_forward8")


class MoeLibraryMissing(RuntimeError):
    pass


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {moe_status_string(code)} (code {code})")
        self.code = code


_TUNING_FIELDS = ("dispatch_kind", "dispatch_sms", "dispatch_ctas_per_sm", "dispatch_warps", "dispatch_stages",
                  "dispatch_chunk_bytes", "combine_kind", "combine_sms", "combine_ctas_per_sm", "layout_kind")


class _TuningC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in _TUNING_FIELDS] + [("reserved", ctypes.c_int32 * 6)]


class _ProblemC(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("num_ranks", ctypes.c_int32),
                ("ranks_per_host", ctypes.c_int32), ("num_src_ranks", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("expert_to_rank", ctypes.c_void_p),
                ("src_rank_offsets", ctypes.c_void_p), ("tuning", ctypes.POINTER(_TuningC))]


@dataclass
class Tuning:
    """Launch shapes of the layout and the row movers (moe_tuning in
    include/moe_layout.h); 0 keeps the library's default.  Shapes change
    speed only, never results."""
    dispatch_kind: int = MOE_MOVE_AUTO
    dispatch_sms: int = 0
    dispatch_ctas_per_sm: int = 0
    dispatch_warps: int = 0
    dispatch_stages: int = 0
    dispatch_chunk_bytes: int = 0
    combine_kind: int = MOE_MOVE_AUTO
    combine_sms: int = 0
    combine_ctas_per_sm: int = 0
    layout_kind: int = MOE_LAYOUT_AUTO

    def c(self) -> _TuningC:
        return _TuningC(*[int(getattr(self, n)) for n in _TUNING_FIELDS])

    def as_dict(self) -> dict:
        return {n: int(getattr(self, n)) for n in _TUNING_FIELDS}

    @classmethod
    def from_env(cls, environ=None) -> "Tuning":
        """MOE_DISPATCH_KIND, MOE_DISPATCH_SMS, ... (upper-case field names
        with a MOE_ prefix; mover kinds also as "auto", "vector" or "bulk",
        the layout kind as "auto", "split", "fused" or "two_kernels")."""
        env = os.environ if environ is None else environ
        move = {"auto": MOE_MOVE_AUTO, "vector": MOE_MOVE_VECTOR, "bulk": MOE_MOVE_BULK}
        layout = {"auto": MOE_LAYOUT_AUTO, "split": MOE_LAYOUT_SPLIT, "fused": MOE_LAYOUT_FUSED,
                  "two_kernels": MOE_LAYOUT_TWO_KERNELS}
        vals = {}
        for n in _TUNING_FIELDS:
            v = env.get("MOE_" + n.upper())
            if v is not None and v != "":
                kinds = layout if n == "layout_kind" else move
                vals[n] = kinds[v.lower()] if v.lower() in kinds else int(v)
        return cls(**vals)


_LAYOUT_FIELDS = ("expert_count", "expert_offset", "rank_count", "rank_offset", "host_count",
                  "host_offset", "host_mask", "pos", "recv_src")


class _LayoutC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _LAYOUT_FIELDS] + [("stats", ctypes.c_void_p)]


class _RelayC(ctypes.Structure):
    _fields_ = [("relay_pos", ctypes.c_void_p), ("relay_src", ctypes.c_void_p), ("slot_relay", ctypes.c_void_p),
                ("capacity", ctypes.c_int64)]


class _RoutingC(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float),
                ("logits_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32 * 4)]


class _GroupingC(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("kept", ctypes.c_int32), ("top", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _ExpertsC(ctypes.Structure):
    _fields_ = [("in_cols", ctypes.c_int32), ("out_cols", ctypes.c_int32), ("act", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("weights", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libmoe_layout.so (raises MoeLibraryMissing if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise MoeLibraryMissing(f"{path} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(path)
    vp, i = ctypes.c_void_p, ctypes.c_int
    P, L = ctypes.POINTER(_ProblemC), ctypes.POINTER(_LayoutC)
    lib.moe_workspace_bytes.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_workspace_bytes.restype = i
    lib.moe_layout.argtypes = [P, vp, vp, L, vp]
    lib.moe_layout.restype = i
    lib.moe_stats_words.argtypes = [P]
    lib.moe_stats_words.restype = ctypes.c_size_t
    lib.moe_stats.argtypes = [P, L, vp, ctypes.POINTER(ctypes.c_int64), vp]
    lib.moe_stats.restype = i
    lib.moe_stats_device.argtypes = [P, vp, vp, vp]
    lib.moe_stats_device.restype = i
    lib.moe_dispatch.argtypes = [P, L, vp, vp, vp, vp, vp]
    lib.moe_dispatch.restype = i
    lib.moe_swap_plan.argtypes = [P, L, ctypes.c_int32, vp, vp, vp]
    lib.moe_swap_plan.restype = i
    lib.moe_dispatch_quant.argtypes = [P, L, vp, vp, vp, vp]
    lib.moe_dispatch_quant.restype = i
    lib.moe_combine.argtypes = [P, L, vp, vp, vp, vp]
    lib.moe_combine.restype = i
    Q = ctypes.POINTER(_RelayC)
    lib.moe_relay_layout.argtypes = [P, L, vp, Q, vp]
    lib.moe_relay_layout.restype = i
    lib.moe_dispatch_relay.argtypes = [P, L, Q, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_dispatch_relay.restype = i
    lib.moe_combine_relay.argtypes = [P, L, Q, vp, vp, vp, vp, vp]
    lib.moe_combine_relay.restype = i
    i32 = ctypes.c_int32
    lib.moe_expert_groups.argtypes = [P, i32, vp, vp]
    lib.moe_expert_groups.restype = i
    lib.moe_dispatch_group.argtypes = [P, L, vp, vp, i32, vp, vp, vp, vp, vp]
    lib.moe_dispatch_group.restype = i
    lib.moe_combine_group.argtypes = [P, L, vp, vp, i32, i32, vp, vp, vp, vp, vp]
    lib.moe_combine_group.restype = i
    G, X = ctypes.POINTER(_RoutingC), ctypes.POINTER(_ExpertsC)
    bytes_out = ctypes.POINTER(ctypes.c_size_t)
    for name, args in (("moe_route", [P, G, vp, vp, vp, vp, vp]),
                       ("moe_route_groups", [P, G, ctypes.POINTER(_GroupingC), vp, vp, vp, vp, vp]),
                       ("moe_route_backward", [P, G, vp, vp, vp, vp, vp]),
                       ("moe_combine_backward", [P, L, vp, vp, vp, vp, vp, vp]),
                       ("moe_expert_forward", [P, L, X, vp, vp, vp, vp]),
                       ("moe_expert_backward_rows", [P, L, X, vp, vp, vp, vp]),
                       ("moe_expert_backward_weights", [P, L, X, vp, vp, vp, vp]),
                       ("moe_expert_forward_kept", [P, L, X, vp, vp, vp, vp, vp]),
                       ("moe_expert_backward_kept", [P, L, X, vp, vp, vp, vp, vp, vp]),
                       ("moe_quant4_row_scale_bytes", [P, i32, bytes_out]),
                       ("moe_quant4_weight_scale_bytes", [P, X, bytes_out]),
                       ("moe_quant4_rows", [P, L, i32, vp, vp, vp, vp]),
                       ("moe_quant4_weights", [P, X, vp, vp, vp]),
                       ("moe_expert_forward4", [P, L, X, vp, vp, vp, vp, vp]),
                       ("moe_quant8_rows", [P, i32, vp, vp, vp, vp]),
                       ("moe_quant8_weights", [P, X, vp, vp, vp]),
                       ("moe_expert_forward8", [P, L, X, vp, vp, vp, vp, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = i
    lib.moe_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    lib.moe_status.restype = i
    lib.moe_layout_noalloc.argtypes = [P, vp, L, vp]
    lib.moe_layout_noalloc.restype = i
    lib.moe_move_faults.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
    lib.moe_move_faults.restype = i
    lib.moe_selftest_bounded_waits.argtypes = [ctypes.POINTER(ctypes.c_uint32), vp]
    lib.moe_selftest_bounded_waits.restype = i
    lib.moe_status_string.argtypes = [i]
    lib.moe_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


# What calls ask torch for each time, looked up once: a device's current stream without a Stream object around it, the
# current device without a look at whether CUDA is up, and whether there is one GPU, so that it need not be asked for.
_raw_stream = _get_device = _one_gpu = None


def _look_up():
    global _raw_stream, _get_device, _one_gpu
    import torch
    _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _one_gpu = torch.cuda.device_count() == 1
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is None:
            _look_up()
        return _raw_stream(0 if _one_gpu else _get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on_current_gpu(t) -> bool:
    on = t.get_device()  # -1 on the host
    return on >= 0 and on == _get_device()


@dataclass
class Problem:
    """One layer's routing problem (see include/moe_layout.h, moe_problem)."""
    num_tokens: int
    hidden: int
    topk: int
    num_experts: int
    num_ranks: int
    ranks_per_host: int
    num_src_ranks: int = 1
    dtype: int = MOE_DTYPE_BF16
    expert_to_rank: object = None      # device int32 tensor [E] or None
    src_rank_offsets: object = None    # device int32 tensor [R_src + 1] or None
    tuning: Optional[Tuning] = None    # launch shapes, or None for the defaults

    @property
    def num_hosts(self) -> int:
        return self.num_ranks // self.ranks_per_host

    @property
    def row_bytes(self) -> int:
        if self.dtype == MOE_DTYPE_FP8_E4M3:
            return self.hidden + 4 * (self.hidden // MOE_FP8_GROUP)
        return 2 * self.hidden

    def __getstate__(self):
        return {name: value for name, value in self.__dict__.items() if name != "_kept"}

    def c(self) -> _ProblemC:
        now = _PROBLEM_FIELDS(self)
        if now[8] is None and now[9] is None and now[10] is None:
            # a struct of sizes alone is kept with the fields it was made from and what it then held: it serves again
            # while the fields are the same, whoever set them, and nobody has edited it; fields that can change in place
            # (a count held in a tensor) would stay the same to a comparison, so then nothing is kept
            kept = self.__dict__.get("_kept")
            if kept is not None and kept[0] == now and bytes(kept[1]) == kept[2]:
                return kept[1]
            pc = _ProblemC(*now)
            if all(type(value) is int for value in now[:8]):
                self.__dict__["_kept"] = (now, pc, bytes(pc))
            return pc
        # the struct keeps its tuning alive for as long as it is referenced
        pc = _ProblemC(*now[:8], _ptr(now[8]), _ptr(now[9]), None)
        if now[10] is not None:
            pc._tuning = now[10].c()
            pc.tuning = ctypes.pointer(pc._tuning)
        return pc


_PROBLEM_FIELDS = operator.attrgetter(*[f.name for f in fields(Problem)])


class Layout:
    """Caller-owned device arrays of a layout (moe_layout_t)."""

    def __init__(self, problem: Problem, device="cuda", with_stats: bool = False):
        import torch
        p = problem
        i32 = dict(dtype=torch.int32, device=device)
        self.expert_count = torch.empty(p.num_experts, **i32)
        self.expert_offset = torch.empty(p.num_experts + 1, **i32)
        self.rank_count = torch.empty(p.num_ranks, **i32)
        self.rank_offset = torch.empty(p.num_ranks + 1, **i32)
        self.host_count = torch.empty(p.num_hosts, **i32)
        self.host_offset = torch.empty(p.num_hosts + 1, **i32)
        self.host_mask = torch.empty((p.num_tokens, p.num_hosts), dtype=torch.uint8, device=device)
        self.pos = torch.empty((p.num_tokens, p.topk), **i32)
        self.recv_src = torch.empty(p.num_tokens * p.topk, **i32)
        # Optional: the statistics record, written by moe_layout itself.
        self.stats = (torch.empty(moe_stats_words(p), dtype=torch.int64, device=device)
                      if with_stats else None)

    def c(self) -> _LayoutC:
        stats = getattr(self, "stats", None)
        return _LayoutC(*[getattr(self, n).data_ptr() for n in _LAYOUT_FIELDS],
                        None if stats is None else stats.data_ptr())

    def to_host(self) -> dict:
        return {n: getattr(self, n).cpu().numpy() for n in _LAYOUT_FIELDS}


class Relay:
    """Caller-owned device arrays of the Mode 2 relay rows (moe_relay_t).  The
    default capacity, T * min(k, H), holds every layout of the problem."""

    def __init__(self, problem: Problem, device="cuda", capacity: Optional[int] = None):
        import torch
        p = problem
        i32 = dict(dtype=torch.int32, device=device)
        self.capacity = p.num_tokens * min(p.topk, p.num_hosts) if capacity is None else int(capacity)
        self.relay_pos = torch.empty((p.num_tokens, p.num_hosts), **i32)
        self.relay_src = torch.empty(max(self.capacity, 1), **i32)
        self.slot_relay = torch.empty((p.num_tokens, p.topk), **i32)

    def c(self) -> _RelayC:
        return _RelayC(self.relay_pos.data_ptr(), self.relay_src.data_ptr(), self.slot_relay.data_ptr(),
                       self.capacity)


@dataclass
class Routing:
    """How the router makes its gates (moe_routing in include/moe_layout.h)."""
    score: int = MOE_SCORE_SOFTMAX
    renormalise: bool = True
    scale: float = 1.0

    def c(self, logits) -> _RoutingC:
        return _RoutingC(self.score, bool(self.renormalise), self.scale, _logits_kind(logits))


@dataclass
class Grouping:
    """Groups that limit a token's choice of experts (moe_grouping in include/moe_layout.h): the
    `kept` of `groups` whose `top` largest keys sum to most."""
    groups: int
    kept: int
    top: int = 2

    def c(self) -> _GroupingC:
        return _GroupingC(self.groups, self.kept, self.top, 0)


@dataclass
class Experts:
    """The experts of a layer (moe_experts in include/moe_layout.h): weights
    bf16 [E, W, in_cols], 4-bit codes [E, W, in_cols / 2] with their scale
    blocks, or int8 [E, W, in_cols] with fp32 scales [E, W]; W = out_cols, or
    2 * out_cols (gate rows, then up rows) with MOE_ACT_SWIGLU."""
    in_cols: int
    out_cols: int
    weights: object = None
    act: int = MOE_ACT_NONE
    scales: object = None

    @property
    def weight_rows(self) -> int:
        return 2 * self.out_cols if self.act == MOE_ACT_SWIGLU else self.out_cols

    def c(self) -> _ExpertsC:
        return _ExpertsC(self.in_cols, self.out_cols, self.act, 0, _ptr(self.weights), _ptr(self.scales))


class _Kinds(dict):
    """The torch types of names joined by "|" (of those that this torch has), looked up once."""

    def __missing__(self, kinds: str):
        import torch
        if _raw_stream is None:
            _look_up()
        found = self[kinds] = tuple(getattr(torch, n) for n in kinds.split("|") if hasattr(torch, n))
        return found


_KINDS = _Kinds()


def _logits_kind(logits) -> int:
    kind = getattr(logits, "dtype", None)
    return MOE_LOGITS_BF16 if kind is not None and kind in _KINDS["bfloat16"] else MOE_LOGITS_F32


def _take(where: str, t, kinds: str, *shape):
    """Address of a tensor argument that has to be dense, on the current GPU, of
    one of these types and (where given) of this shape."""
    kind = getattr(t, "dtype", None)
    if kind is None:  # NULL, or an object with nothing but an address
        return None if t is None else t.data_ptr()
    if kind in _KINDS[kinds] and (t.shape == shape or not shape) and t.is_contiguous() and (
            t.is_cuda if _one_gpu else _on_current_gpu(t)):
        return t.data_ptr()
    raise MoeError(MOE_ERR_INVALID, f"{where}: a dense {kinds} tensor {list(shape) or ''} on the current GPU is wanted, not "
                                    f"{t.dtype} {list(t.shape)} with strides {list(t.stride())} on {t.device}")


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def moe_status_string(code: int) -> str:
    return load_library().moe_status_string(int(code)).decode()


def moe_workspace_bytes(problem: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_bytes(ctypes.byref(problem.c()), ctypes.byref(n)),
           "moe_workspace_bytes")
    return n.value


def alloc_workspace(problem: Problem, device="cuda"):
    import torch
    return torch.empty(moe_workspace_bytes(problem), dtype=torch.uint8, device=device)


def moe_layout(problem: Problem, ids, workspace, layout: Layout, stream=None):
    _check(load_library().moe_layout(ctypes.byref(problem.c()), _ptr(ids), _ptr(workspace),
                                     ctypes.byref(layout.c()), _stream(stream)), "moe_layout")


def moe_layout_noalloc(problem: Problem, ids, layout: Layout, stream=None):
    """moe_layout without a workspace: the library's fixed device scratch is
    used instead (for callers that cannot allocate device memory).  Calls that
    may overlap on the GPU share that scratch and must be serialised."""
    _check(load_library().moe_layout_noalloc(ctypes.byref(problem.c()), _ptr(ids),
                                             ctypes.byref(layout.c()), _stream(stream)),
           "moe_layout_noalloc")


def moe_stats_words(problem: Problem) -> int:
    return int(load_library().moe_stats_words(ctypes.byref(problem.c())))


def moe_stats(problem: Problem, layout: Layout, workspace=None, stream=None):
    """The statistics record copied to host memory; synchronises the stream.
    Returns (code, record): code is what moe_status would return for the
    record's status word, record a numpy int64 array (decode_stats names its
    words).  With layout.stats set the record comes from there and the
    workspace may be None."""
    import numpy as np
    rec = np.zeros(moe_stats_words(problem), dtype=np.int64)
    rc = load_library().moe_stats(ctypes.byref(problem.c()), ctypes.byref(layout.c()), _ptr(workspace),
                                  rec.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), _stream(stream))
    # A code that the record's status word explains came from the device; any
    # other is a host-side rejection or a failed copy, and the record is empty.
    from_record = rc in (MOE_OK, MOE_ERR_BAD_IDS, MOE_ERR_CAPACITY, MOE_ERR_TIMEOUT) or (
        rc == MOE_ERR_INVALID and int(rec[0]) & (MOE_STATUS_PLACEMENT | MOE_STATUS_SRC_OFFSET))
    if not from_record:
        raise MoeError(rc, "moe_stats")
    return rc, rec


def moe_stats_device(problem: Problem, workspace, stats, stream=None):
    """The statistics record copied to a device int64 tensor, asynchronously."""
    _check(load_library().moe_stats_device(ctypes.byref(problem.c()), _ptr(workspace), _ptr(stats),
                                           _stream(stream)), "moe_stats_device")


def moe_dispatch(problem: Problem, layout: Layout, x, x_scales, recv, recv_scales, stream=None):
    _check(load_library().moe_dispatch(ctypes.byref(problem.c()), ctypes.byref(layout.c()), _ptr(x),
                                       _ptr(x_scales), _ptr(recv), _ptr(recv_scales), _stream(stream)),
           "moe_dispatch")


def moe_swap_plan(problem: Problem, layout: Layout, tau: int, new_expert_to_rank, swaps=None, stream=None):
    """Per-step intra-host expert swap plan from the layout's expert counts."""
    _check(load_library().moe_swap_plan(ctypes.byref(problem.c()), ctypes.byref(layout.c()), int(tau),
                                        _ptr(new_expert_to_rank), _ptr(swaps), _stream(stream)),
           "moe_swap_plan")


def moe_dispatch_quant(problem: Problem, layout: Layout, x_bf16, recv, recv_scales, stream=None):
    """Dispatch that converts bf16 rows to e4m3 codes + fp32 scales per 128 columns."""
    _check(load_library().moe_dispatch_quant(ctypes.byref(problem.c()), ctypes.byref(layout.c()),
                                             _ptr(x_bf16), _ptr(recv), _ptr(recv_scales), _stream(stream)),
           "moe_dispatch_quant")


def moe_combine(problem: Problem, layout: Layout, y, weights, out, stream=None):
    _check(load_library().moe_combine(ctypes.byref(problem.c()), ctypes.byref(layout.c()), _ptr(y),
                                      _ptr(weights), _ptr(out), _stream(stream)), "moe_combine")


def moe_relay_layout(problem: Problem, layout: Layout, workspace, relay: Relay, stream=None):
    """Relay rows of a layout made with this workspace."""
    _check(load_library().moe_relay_layout(ctypes.byref(problem.c()), ctypes.byref(layout.c()), _ptr(workspace),
                                           ctypes.byref(relay.c()), _stream(stream)), "moe_relay_layout")


def moe_dispatch_relay(problem: Problem, layout: Layout, relay: Relay, x, x_scales, relay_rows, relay_scales,
                       recv, recv_scales, stream=None):
    """Two-hop dispatch: x to the relay rows, then the relay rows to recv."""
    _check(load_library().moe_dispatch_relay(ctypes.byref(problem.c()), ctypes.byref(layout.c()),
                                             ctypes.byref(relay.c()), _ptr(x), _ptr(x_scales), _ptr(relay_rows),
                                             _ptr(relay_scales), _ptr(recv), _ptr(recv_scales), _stream(stream)),
           "moe_dispatch_relay")


def moe_combine_relay(problem: Problem, layout: Layout, relay: Relay, y, weights, partial, out, stream=None):
    """Two-hop combine: per-host bf16 partials, then their sum in host order."""
    _check(load_library().moe_combine_relay(ctypes.byref(problem.c()), ctypes.byref(layout.c()),
                                            ctypes.byref(relay.c()), _ptr(y), _ptr(weights), _ptr(partial),
                                            _ptr(out), _stream(stream)), "moe_combine_relay")


def moe_expert_groups(problem: Problem, num_groups: int, expert_group, stream=None):
    """Group of every expert: G contiguous runs of each rank's experts."""
    _check(load_library().moe_expert_groups(ctypes.byref(problem.c()), int(num_groups), _ptr(expert_group),
                                            _stream(stream)), "moe_expert_groups")


def moe_dispatch_group(problem: Problem, layout: Layout, ids, expert_group, group: int, x, x_scales, recv,
                       recv_scales, stream=None):
    """Dispatch of the slots whose expert is in `group`."""
    _check(load_library().moe_dispatch_group(ctypes.byref(problem.c()), ctypes.byref(layout.c()), _ptr(ids),
                                             _ptr(expert_group), int(group), _ptr(x), _ptr(x_scales), _ptr(recv),
                                             _ptr(recv_scales), _stream(stream)), "moe_dispatch_group")


def moe_combine_group(problem: Problem, layout: Layout, ids, expert_group, group: int, num_groups: int, y, weights,
                      acc, out, stream=None):
    """Combine of one expert group; the groups continue one fp32 chain per
    token through `acc` and the last writes `out`."""
    _check(load_library().moe_combine_group(ctypes.byref(problem.c()), ctypes.byref(layout.c()), _ptr(ids),
                                            _ptr(expert_group), int(group), int(num_groups), _ptr(y),
                                            _ptr(weights), _ptr(acc), _ptr(out), _stream(stream)),
           "moe_combine_group")


def moe_route(problem: Problem, routing: Routing, logits, ids, gates, bias=None, stream=None):
    """ids and gates of every token's top-k experts from logits [T, E] (fp32 or bf16)."""
    p, where = problem, "moe_route"
    _check((_lib or load_library()).moe_route(
        ctypes.byref(p.c()), ctypes.byref(routing.c(logits)),
        _take(where, logits, "float32|bfloat16", p.num_tokens, p.num_experts),
        _take(where, bias, "float32", p.num_experts), _take(where, ids, "int32", p.num_tokens, p.topk),
        _take(where, gates, "float32", p.num_tokens, p.topk), _stream(stream)), where)


# What the C structs of a routing and a grouping hold, as bytes: score, renormalise, scale, the logits' type and a grouping's fields.
_CHOICE_VALUES = struct.Struct("=i?f4i")


class _ChoiceStructs(dict):
    """References to the C structs of a routing and a grouping by the bytes of their values (0.6 us of host time a call
    less than making them; the library only reads them, and nobody else gets hold of them).  By bytes, because a field's
    object may change in place, as a tensor does, and equal ones need not be alike, as zeros are not."""

    @staticmethod
    def made(score, renormalise, scale, kind, *grouping):
        return ctypes.byref(_RoutingC(score, bool(renormalise), scale, kind)), ctypes.byref(_GroupingC(*grouping, 0))

    def __missing__(self, said: bytes):
        made = self.made(*_CHOICE_VALUES.unpack(said))
        if len(self) >= 64:
            self.clear()
        self[said] = made
        return made


_CHOICE = _ChoiceStructs()


def moe_route_groups(problem: Problem, routing: Routing, grouping: Grouping, logits, ids, gates, bias=None, stream=None):
    """moe_route with every token's choice limited to `grouping.kept` groups of experts; keys are scores (+ bias)."""
    p, where = problem, "moe_route_groups"
    values = routing.score, routing.renormalise, routing.scale, _logits_kind(logits), grouping.groups, grouping.kept, grouping.top
    try:
        choice = _CHOICE[_CHOICE_VALUES.pack(*values)]
    except (struct.error, OverflowError):  # no numbers, or past 32 bits: as the structs of the other calls take them
        choice = _CHOICE.made(*values)
    _check((_lib or load_library()).moe_route_groups(
        ctypes.byref(p.c()), *choice,
        _take(where, logits, "float32|bfloat16", p.num_tokens, p.num_experts),
        _take(where, bias, "float32", p.num_experts), _take(where, ids, "int32", p.num_tokens, p.topk),
        _take(where, gates, "float32", p.num_tokens, p.topk), _stream(stream)), where)


def moe_route_backward(problem: Problem, routing: Routing, logits, ids, dgates, dlogits, stream=None):
    """dlogits [T, E] (of the logits' type) from the gates' gradient."""
    p, where = problem, "moe_route_backward"
    at = _take(where, logits, "float32|bfloat16", p.num_tokens, p.num_experts)
    if getattr(logits, "dtype", None) != getattr(dlogits, "dtype", None):
        raise MoeError(MOE_ERR_INVALID, f"{where}: dlogits has the logits' type")
    _check((_lib or load_library()).moe_route_backward(
        ctypes.byref(p.c()), ctypes.byref(routing.c(logits)), at, _take(where, ids, "int32", p.num_tokens, p.topk),
        _take(where, dgates, "float32", p.num_tokens, p.topk),
        _take(where, dlogits, "float32|bfloat16", p.num_tokens, p.num_experts), _stream(stream)), where)


def moe_combine_backward(problem: Problem, layout: Layout, dout, y, weights, dy, dweights, stream=None):
    """Gradients of moe_combine: dy [T*k, h] and dweights [T, k] from dout [T, h]."""
    p, where = problem, "moe_combine_backward"
    slots = p.num_tokens * p.topk
    _check((_lib or load_library()).moe_combine_backward(
        ctypes.byref(p.c()), ctypes.byref(_LayoutC(pos=_take_ints(where, layout.pos, "pos", slots))),
        _take(where, dout, "bfloat16", p.num_tokens, p.hidden),
        _take(where, y, "bfloat16", slots, p.hidden), _take(where, weights, "float32", p.num_tokens, p.topk),
        _take(where, dy, "bfloat16", slots, p.hidden), _take(where, dweights, "float32", p.num_tokens, p.topk),
        _stream(stream)), where)


def _take_ints(where: str, t, name: str, size: int):
    """Address of a layout's array: dense int32 on the current GPU, `size` long at least."""
    kind = getattr(t, "dtype", None)
    if kind is None:  # an object with nothing but an address
        return t.data_ptr()
    if t.numel() >= size and kind is _KINDS["int32"][0] and t.is_contiguous() and (
            t.is_cuda if _one_gpu else _on_current_gpu(t)):
        return t.data_ptr()
    raise MoeError(MOE_ERR_INVALID, f"{where}: the layout's {name} has to be dense int32 on the current GPU, {size} values "
                                    f"or more, not {t.dtype} {list(t.shape)} with strides {list(t.stride())} on {t.device}")


def _groups(where: str, p: Problem, layout) -> _LayoutC:
    """The two layout arrays that the experts' calls read (the struct's first two fields)."""
    return _LayoutC(_take_ints(where, layout.expert_count, "expert_count", p.num_experts),
                    _take_ints(where, layout.expert_offset, "expert_offset", p.num_experts + 1))


def _take_weights(where: str, p: Problem, x: Experts):
    _take(where, x.weights, "bfloat16", p.num_experts, x.weight_rows, x.in_cols)
    return ctypes.byref(x.c())


def moe_expert_forward(problem: Problem, layout: Layout, experts: Experts, rows, out, pre=None, stream=None):
    """out [T*k, out_cols] = every receive row times its expert's weights, gated
    with MOE_ACT_SWIGLU (pre [T*k, W] then receives what the gate is made of)."""
    p, x, where = problem, experts, "moe_expert_forward"
    slots = p.num_tokens * p.topk
    _check((_lib or load_library()).moe_expert_forward(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), _take_weights(where, p, x),
        _take(where, rows, "bfloat16", slots, x.in_cols), _take(where, pre, "bfloat16", slots, x.weight_rows),
        _take(where, out, "bfloat16", slots, x.out_cols), _stream(stream)), where)


def moe_expert_backward_rows(problem: Problem, layout: Layout, experts: Experts, dout, drows, pre=None, stream=None):
    """drows [T*k, in_cols] = dout [T*k, W] times the experts' weights; with
    pre [T*k, 2 * in_cols] (the rows were its gated halves) drows is pre's gradient."""
    p, x, where = problem, experts, "moe_expert_backward_rows"
    slots, wide = p.num_tokens * p.topk, x.in_cols * (1 if pre is None else 2)
    _check((_lib or load_library()).moe_expert_backward_rows(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), _take_weights(where, p, x),
        _take(where, dout, "bfloat16", slots, x.weight_rows), _take(where, pre, "bfloat16", slots, wide),
        _take(where, drows, "bfloat16", slots, wide), _stream(stream)), where)


def moe_expert_backward_weights(problem: Problem, layout: Layout, experts: Experts, rows, dout, dweights, stream=None):
    """dweights [E, W, in_cols] = per expert, the sum of dout[r]^T rows[r] over its rows."""
    p, x, where = problem, experts, "moe_expert_backward_weights"
    slots = p.num_tokens * p.topk
    _check((_lib or load_library()).moe_expert_backward_weights(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), ctypes.byref(x.c()),
        _take(where, rows, "bfloat16", slots, x.in_cols), _take(where, dout, "bfloat16", slots, x.weight_rows),
        _take(where, dweights, "bfloat16", p.num_experts, x.weight_rows, x.in_cols), _stream(stream)), where)


def moe_expert_forward_kept(problem: Problem, layout: Layout, experts: Experts, rows, out, kept, scales, stream=None):
    """moe_expert_forward with MOE_ACT_SWIGLU that keeps pre in 8 bits: e4m3 codes [T*k, 2 * out_cols] (uint8 or
    float8_e4m3fn) and e8m0 scales [T*k, 2, ceil(out_cols / 32)] (uint8 or float8_e8m0fnu)."""
    p, x, where = problem, experts, "moe_expert_forward_kept"
    slots = p.num_tokens * p.topk
    _check((_lib or load_library()).moe_expert_forward_kept(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), _take_weights(where, p, x),
        _take(where, rows, "bfloat16", slots, x.in_cols), _take(where, out, "bfloat16", slots, x.out_cols),
        _take(where, kept, "uint8|float8_e4m3fn", slots, 2 * x.out_cols),
        _take(where, scales, "uint8|float8_e8m0fnu", slots, 2, -(-x.out_cols // 32)), _stream(stream)), where)


def moe_expert_backward_kept(problem: Problem, layout: Layout, experts: Experts, dout, kept, scales, drows, act=None,
                             stream=None):
    """drows [T*k, 2 * in_cols]: the gradient of the (g, u) that was kept, from dout [T*k, W] of the product whose rows
    were silu(g) * u; act [T*k, in_cols] receives those rows made anew."""
    p, x, where = problem, experts, "moe_expert_backward_kept"
    slots = p.num_tokens * p.topk
    _check((_lib or load_library()).moe_expert_backward_kept(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), _take_weights(where, p, x),
        _take(where, dout, "bfloat16", slots, x.weight_rows),
        _take(where, kept, "uint8|float8_e4m3fn", slots, 2 * x.in_cols),
        _take(where, scales, "uint8|float8_e8m0fnu", slots, 2, -(-x.in_cols // 32)),
        _take(where, drows, "bfloat16", slots, 2 * x.in_cols), _take(where, act, "bfloat16", slots, x.in_cols),
        _stream(stream)), where)


def moe_quant4_row_scale_bytes(problem: Problem, cols: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_quant4_row_scale_bytes(ctypes.byref(problem.c()), int(cols), ctypes.byref(n)),
           "moe_quant4_row_scale_bytes")
    return n.value


def moe_quant4_weight_scale_bytes(problem: Problem, experts: Experts) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_quant4_weight_scale_bytes(ctypes.byref(problem.c()), ctypes.byref(experts.c()),
                                                        ctypes.byref(n)), "moe_quant4_weight_scale_bytes")
    return n.value


# The sizes again, without a call into the library (a test holds them together).

def _row_scale_bytes(p: Problem, cols: int) -> int:
    return (p.num_tokens * p.topk // 128 + p.num_experts) * -(-cols // 128) * 512


def _weight_scale_bytes(p: Problem, x: Experts) -> int:
    per = 64 if x.act == MOE_ACT_SWIGLU else 128
    return p.num_experts * -(-x.out_cols // per) * -(-x.in_cols // 128) * 512


def _take_bytes(where: str, t, size: int):
    """Address of a dense uint8 tensor of at least `size` bytes."""
    at = _take(where, t, "uint8")
    if hasattr(t, "numel") and t.numel() < size:
        raise MoeError(MOE_ERR_INVALID, f"{where}: {size} bytes of scale blocks are wanted, not {t.numel()}")
    return at


def moe_quant4_rows(problem: Problem, layout: Layout, rows, codes, scales, stream=None):
    """Receive rows bf16 [T*k, cols] to 4-bit codes [T*k, cols / 2] and scale blocks."""
    p, where = problem, "moe_quant4_rows"
    shape = getattr(codes, "shape", ())
    if len(shape) != 2:
        raise MoeError(MOE_ERR_INVALID, f"{where}: codes are [T*k, cols / 2], not {list(shape)}")
    slots, cols = p.num_tokens * p.topk, 2 * int(shape[1])
    _check((_lib or load_library()).moe_quant4_rows(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), cols, _take(where, rows, "bfloat16", slots, cols),
        _take(where, codes, "uint8", slots, cols // 2),
        _take_bytes(where, scales, _row_scale_bytes(p, cols)), _stream(stream)), where)


def moe_quant4_weights(problem: Problem, experts: Experts, codes, scales, stream=None):
    """The experts' bf16 weights to 4-bit codes [E, W, in_cols / 2] and scale blocks."""
    p, x, where = problem, experts, "moe_quant4_weights"
    _check((_lib or load_library()).moe_quant4_weights(
        ctypes.byref(p.c()), _take_weights(where, p, x),
        _take(where, codes, "uint8", p.num_experts, x.weight_rows, x.in_cols // 2),
        _take_bytes(where, scales, _weight_scale_bytes(p, x)), _stream(stream)), where)


def moe_expert_forward4(problem: Problem, layout: Layout, experts: Experts, codes, scales, out, pre=None, stream=None):
    """moe_expert_forward from 4-bit rows (moe_quant4_rows) and 4-bit weights (experts.weights,
    experts.scales of moe_quant4_weights); out and pre are bf16."""
    p, x, where = problem, experts, "moe_expert_forward4"
    slots = p.num_tokens * p.topk
    _take(where, x.weights, "uint8", p.num_experts, x.weight_rows, x.in_cols // 2)
    if x.scales is not None:
        _take_bytes(where, x.scales, _weight_scale_bytes(p, x))
    _check((_lib or load_library()).moe_expert_forward4(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), ctypes.byref(x.c()),
        _take(where, codes, "uint8", slots, x.in_cols // 2),
        _take_bytes(where, scales, _row_scale_bytes(p, x.in_cols)),
        _take(where, pre, "bfloat16", slots, x.weight_rows), _take(where, out, "bfloat16", slots, x.out_cols),
        _stream(stream)), where)


def moe_quant8_rows(problem: Problem, rows, codes, scales, stream=None):
    """Receive rows bf16 [T*k, cols] to 8-bit integers [T*k, cols] and one fp32 scale a row."""
    p, where = problem, "moe_quant8_rows"
    shape = getattr(codes, "shape", ())
    if len(shape) != 2:
        raise MoeError(MOE_ERR_INVALID, f"{where}: codes are [T*k, cols], not {list(shape)}")
    slots, cols = p.num_tokens * p.topk, int(shape[1])
    _check((_lib or load_library()).moe_quant8_rows(
        ctypes.byref(p.c()), cols, _take(where, rows, "bfloat16", slots, cols), _take(where, codes, "int8", slots, cols),
        _take(where, scales, "float32", slots), _stream(stream)), where)


def moe_quant8_weights(problem: Problem, experts: Experts, codes, scales, stream=None):
    """The experts' bf16 weights to 8-bit integers [E, W, in_cols] and fp32 scales [E, W]."""
    p, x, where = problem, experts, "moe_quant8_weights"
    _check((_lib or load_library()).moe_quant8_weights(
        ctypes.byref(p.c()), _take_weights(where, p, x),
        _take(where, codes, "int8", p.num_experts, x.weight_rows, x.in_cols),
        _take(where, scales, "float32", p.num_experts, x.weight_rows), _stream(stream)), where)


def moe_expert_forward8(problem: Problem, layout: Layout, experts: Experts, codes, scales, out, pre=None, stream=None):
    """moe_expert_forward from 8-bit integer rows (moe_quant8_rows) and weights (experts.weights,
    experts.scales of moe_quant8_weights); out and pre are bf16."""
    p, x, where = problem, experts, "moe_expert_forward8"
    slots = p.num_tokens * p.topk
    _take(where, x.weights, "int8", p.num_experts, x.weight_rows, x.in_cols)
    _take(where, x.scales, "float32", p.num_experts, x.weight_rows)
    _check((_lib or load_library()).moe_expert_forward8(
        ctypes.byref(p.c()), ctypes.byref(_groups(where, p, layout)), ctypes.byref(x.c()),
        _take(where, codes, "int8", slots, x.in_cols), _take(where, scales, "float32", slots),
        _take(where, pre, "bfloat16", slots, x.weight_rows), _take(where, out, "bfloat16", slots, x.out_cols),
        _stream(stream)), where)


def moe_status(workspace, stream=None):
    """Synchronises the stream; returns (code, status_bits)."""
    bits = ctypes.c_uint32(0)
    rc = load_library().moe_status(_ptr(workspace), ctypes.byref(bits), _stream(stream))
    return rc, bits.value


def moe_move_faults(stream=None) -> int:
    """Synchronises the stream; returns and clears the row movers' fault bits."""
    bits = ctypes.c_uint32(0)
    _check(load_library().moe_move_faults(ctypes.byref(bits), _stream(stream)), "moe_move_faults")
    return bits.value


def moe_selftest_bounded_waits(stream=None) -> int:
    """Runs the bounded-wait self-test; returns its bits (0xF = all good)."""
    bits = ctypes.c_uint32(0)
    _check(load_library().moe_selftest_bounded_waits(ctypes.byref(bits), _stream(stream)),
           "moe_selftest_bounded_waits")
    return bits.value


def decode_stats(problem: Problem, stats_host) -> dict:
    """Names the words of a statistics record copied to the host (numpy int64)."""
    import numpy as np
    s = np.asarray(stats_host, dtype=np.int64)
    out = {}
    for i, n in enumerate(STATS_HEADER):
        out[n] = int(s[i])
    for n in ("imbalance_ratio", "rank_imbalance"):
        out[n] = float(np.array([out[n]], np.int64).view(np.float64)[0])
    base = MOE_STATS_HEADER_WORDS
    rs, r = problem.num_src_ranks, problem.num_ranks
    for i, n in enumerate(STATS_SRC):
        out[n] = s[base + i * rs: base + (i + 1) * rs].copy()
    base += len(STATS_SRC) * rs
    for i, n in enumerate(STATS_DST):
        out[n] = s[base + i * r: base + (i + 1) * r].copy()
    return out
