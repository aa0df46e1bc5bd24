"""Python binding of libmoe_dispatch.so (MoE routing, token dispatch, expert
products and combine on MI355X / gfx950).

Argument marshalling only: every step runs in the library's HIP kernels on the
caller's current torch stream. Torch tensors supply device memory; bf16 rows
may be passed as torch.bfloat16, torch.int16 or torch.uint16 tensors (the bits
are what matter). There is no CPU fallback: if the library is missing or the
tensors are not on a GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch  # loads the HIP runtime the library binds to; must come first

try:  # the costly part of a small call in C++ (csrc/binding.cpp); without it: slower
    from . import _binding as _fast
except ImportError:
    _fast = None

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_dispatch.so")

MOE_OK = 0
MOE_ERR_ARG = -1
MOE_ERR_HIP = -2
ERRBIT_BAD_ID = 1
ERRBIT_RANK_CAP = 2
ERRBIT_EXPERT_CAP = 4
ERRBIT_BAD_LOGIT = 8
ERRBIT_BAD_SEQ = 16

EXPORTS = ("moe_abi_version", "moe_status_string", "moe_dispatch_layout",
           "moe_dispatch_layout_noalloc", "moe_layout_workspace_bytes", "moe_dispatch_pack",
           "moe_permute_by_expert", "moe_combine", "moe_combine_rank_partial",
           "moe_combine_ranks", "moe_dispatch_pack_mxfp8", "moe_permute_by_expert_mxfp8",
           "moe_dispatch_pack_mxfp4", "moe_permute_by_expert_mxfp4",
           "moe_dispatch_pack_nvfp4", "moe_permute_by_expert_nvfp4",
           "moe_dispatch", "moe_dispatch_quantised", "moe_route", "moe_route_backward",
           "moe_balance_loss", "moe_balance_workspace_bytes", "moe_expert_product",
           "moe_norm", "moe_norm_backward", "moe_norm_workspace_bytes", "moe_quantise_rows",
           "moe_int8_product",
           "moe_testing_set_layout_form",
           "moe_testing_set_layout_match",
           "moe_testing_set_dispatch_fused", "moe_testing_time_next_launch")


ABI_VERSION = 9

# Quantised wire formats: name -> (code bits per value, values per scale byte).
WIRE_FORMATS = {"mxfp8": (8, 32), "mxfp4": (4, 32), "nvfp4": (4, 16)}
WIRE_CODES = {"mxfp8": 1, "mxfp4": 2, "nvfp4": 3}  # moe_dispatch_quantised's format

LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ROW_TYPES = (torch.bfloat16, torch.int16, torch.uint16)  # of the expert products' rows
SCORINGS = {"softmax": 0, "sigmoid": 1}
ACTS = {None: 0, "none": 0, "swiglu": 1}
NORM_TYPES = {torch.float32: 0, torch.bfloat16: 1}  # of a norm's stream and weight
NORM_FORMATS = {None: 0, "int8": 4, "mxfp8": 1}


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("R", ctypes.c_int32), ("k", ctypes.c_int32), ("align", ctypes.c_int32),
                ("block", ctypes.c_int32)]

    def __init__(self, T=0, H=8, E=1, R=1, k=1, align=1, block=0):
        super().__init__(T, H, E, R, k, align, block)


class MoeError(RuntimeError):
    pass


_lib = None
_address = None  # the C++ module's, once lib() has found that it fits
# its functions, in the order of its bind() and built_for()
_FAST_CALLS = ("moe_norm", "moe_norm_backward", "moe_quantise_rows", "moe_int8_product")


# arguments' types as the C++ module's built_for() names them
_KINDS = {ctypes.c_void_p: "p", ctypes.POINTER(MoeShape): "p", ctypes.c_int: "i",
          ctypes.c_int64: "q", ctypes.c_size_t: "n", ctypes.c_float: "f"}


def _fits(module, L) -> bool:
    """Whether the C++ module was compiled for this torch, this version of the library
    and the signatures declared here."""
    want = (ABI_VERSION, str(torch.__version__),
            *("".join(_KINDS.get(t, "?") for t in getattr(L, name).argtypes)
              for name in _FAST_CALLS))
    return hasattr(module, "built_for") and module.built_for() == want


def lib():
    """Load the library (once) and declare its signatures."""
    global _lib, _fast, _address
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MoeError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    for name in EXPORTS:
        if not hasattr(L, name):
            raise MoeError(f"{LIB_PATH} does not export {name}")
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    shp = ctypes.POINTER(MoeShape)
    L.moe_abi_version.restype = ctypes.c_int
    L.moe_abi_version.argtypes = []
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [ctypes.c_int]
    L.moe_dispatch_layout.restype = ctypes.c_int
    L.moe_dispatch_layout.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp,
                                      vp]
    L.moe_dispatch_layout_noalloc.restype = ctypes.c_int
    L.moe_dispatch_layout_noalloc.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_layout_workspace_bytes.restype = ctypes.c_size_t
    L.moe_layout_workspace_bytes.argtypes = [shp]
    L.moe_dispatch_pack.restype = ctypes.c_int
    L.moe_dispatch_pack.argtypes = [shp, vp, vp, vp, vp, i64, vp, vp]
    L.moe_permute_by_expert.restype = ctypes.c_int
    L.moe_permute_by_expert.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, i64, vp,
                                        vp]
    L.moe_combine.restype = ctypes.c_int
    L.moe_combine.argtypes = [shp, vp, vp, vp, i64, vp, vp, vp, vp]
    L.moe_combine_rank_partial.restype = ctypes.c_int
    L.moe_combine_rank_partial.argtypes = [shp, vp, vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp]
    L.moe_combine_ranks.restype = ctypes.c_int
    L.moe_combine_ranks.argtypes = [shp, vp, vp, i64, vp, vp, vp, vp]
    L.moe_dispatch_pack_mxfp8.restype = ctypes.c_int
    L.moe_dispatch_pack_mxfp8.argtypes = [shp, vp, vp, vp, vp, vp, i64, vp, vp]
    L.moe_permute_by_expert_mxfp8.restype = ctypes.c_int
    L.moe_permute_by_expert_mxfp8.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp,
                                              vp, i64, vp, vp]
    L.moe_dispatch_pack_mxfp4.restype = ctypes.c_int
    L.moe_dispatch_pack_mxfp4.argtypes = L.moe_dispatch_pack_mxfp8.argtypes
    L.moe_permute_by_expert_mxfp4.restype = ctypes.c_int
    L.moe_permute_by_expert_mxfp4.argtypes = L.moe_permute_by_expert_mxfp8.argtypes
    L.moe_dispatch_pack_nvfp4.restype = ctypes.c_int
    L.moe_dispatch_pack_nvfp4.argtypes = L.moe_dispatch_pack_mxfp8.argtypes
    L.moe_permute_by_expert_nvfp4.restype = ctypes.c_int
    L.moe_permute_by_expert_nvfp4.argtypes = L.moe_permute_by_expert_mxfp8.argtypes
    L.moe_dispatch.restype = ctypes.c_int
    L.moe_dispatch.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, i64,
                               vp, ctypes.c_size_t, vp, vp]
    L.moe_dispatch_quantised.restype = ctypes.c_int
    L.moe_dispatch_quantised.argtypes = [shp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                         vp, vp, i64, vp, vp, vp, i64, vp, ctypes.c_size_t, vp,
                                         vp]
    L.moe_route.restype = ctypes.c_int
    L.moe_route.argtypes = [shp, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp]
    L.moe_route_backward.restype = ctypes.c_int
    L.moe_route_backward.argtypes = [shp, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp,
                                     ctypes.c_int, vp, vp, vp]
    L.moe_balance_loss.restype = ctypes.c_int
    L.moe_balance_loss.argtypes = [shp, vp, ctypes.c_int, vp, vp, vp, ctypes.c_int, vp, vp, vp,
                                   vp, vp, ctypes.c_size_t, vp, vp]
    L.moe_balance_workspace_bytes.restype = ctypes.c_size_t
    L.moe_balance_workspace_bytes.argtypes = [shp, ctypes.c_int]
    L.moe_expert_product.restype = ctypes.c_int
    L.moe_expert_product.argtypes = [shp, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp,
                                     i64, vp, vp, vp, vp, vp, vp]
    ci, sz = ctypes.c_int, ctypes.c_size_t
    L.moe_norm.restype = ci
    L.moe_norm.argtypes = [shp, ci, vp, vp, vp, ci, vp, ctypes.c_float, vp, ci, vp, vp, vp, vp]
    L.moe_norm_backward.restype = ci
    L.moe_norm_backward.argtypes = [shp, ci, vp, vp, vp, ci, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_norm_workspace_bytes.restype = sz
    L.moe_norm_workspace_bytes.argtypes = [shp]
    L.moe_quantise_rows.restype = ci
    L.moe_quantise_rows.argtypes = [shp, vp, vp, i64, vp, vp, vp, vp]
    L.moe_int8_product.restype = ci
    L.moe_int8_product.argtypes = [shp, ci, ci, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp]
    L.moe_testing_set_dispatch_fused.restype = ctypes.c_int
    L.moe_testing_set_dispatch_fused.argtypes = [ctypes.c_int]
    L.moe_testing_set_layout_form.restype = ctypes.c_int
    L.moe_testing_set_layout_form.argtypes = [ctypes.c_int]
    L.moe_testing_set_layout_match.restype = ctypes.c_int
    L.moe_testing_set_layout_match.argtypes = [ctypes.c_int]
    L.moe_testing_time_next_launch.restype = ctypes.c_int
    L.moe_testing_time_next_launch.argtypes = [vp, vp]
    if L.moe_abi_version() != ABI_VERSION:
        raise MoeError(f"{LIB_PATH} has ABI version {L.moe_abi_version()}, this binding "
                       f"expects {ABI_VERSION}: rebuild with __graft_entry__.build()")
    if _fast is not None and _fits(_fast, L):
        _fast.bind(*(ctypes.cast(getattr(L, name), ctypes.c_void_p).value
                     for name in _FAST_CALLS))
        _address = _fast.address
    else:
        _fast = _address = None
    _lib = L
    return L


def _entry(name: str):
    """A function of the library, through the C++ module where it is there."""
    L = lib()
    return getattr(L if _fast is None else _fast, name)


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        msg = lib().moe_status_string(status).decode()
        raise MoeError(f"{what} failed: {msg} ({status})")


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoeError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise MoeError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor | None, name: str, shape: tuple | None = None,
          min_numel: int | None = None) -> None:
    """Checks a tensor against the shape of the call before its pointer goes to
    the library, which cannot see buffer lengths: `shape` exactly, or at least
    `min_numel` elements. Raises MoeError."""
    if t is None:
        return
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise MoeError(f"{name} has shape {tuple(t.shape)}, the call needs {tuple(shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise MoeError(f"{name} has {t.numel()} elements, the call needs at least {min_numel}")


def _rows(t: torch.Tensor, name: str, width: int) -> int:
    """Rows of a row buffer [rows, width]; raises MoeError on another width."""
    if t.dim() != 2 or t.shape[1] != width:
        raise MoeError(f"{name} has shape {tuple(t.shape)}, the call needs [rows, {width}]")
    return t.shape[0]


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _i32(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.int32:
        raise MoeError(f"expected int32, got {t.dtype}")
    return t


def _check_err(t: torch.Tensor | None) -> None:
    """The device error word: None, or an int32 tensor of at least one element
    (the kernels OR 4 bytes into its first element)."""
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1):
        raise MoeError(f"err must be an int32 tensor of at least 1 element, got {t.dtype} "
                       f"with {t.numel()}")


def _err(t: torch.Tensor | None):
    _check_err(t)
    return _ptr(t)


def _rows16(t: torch.Tensor) -> torch.Tensor:
    if t.element_size() != 2:
        raise MoeError(f"expected a 16-bit row tensor, got {t.dtype}")
    return t


@dataclass
class Shape:
    T: int
    H: int
    E: int
    R: int
    k: int
    align: int = 1  # expert runs padded to a multiple of align rows
    block: int = 0  # > 0: a fixed block of rows per expert (masked layout)

    def c(self) -> MoeShape:
        return MoeShape(self.T, self.H, self.E, self.R, self.k, self.align, self.block)

    @property
    def cap_rank(self) -> int:
        """Worst-case rank-buffer rows: T * min(k, R)."""
        return self.T * min(self.k, self.R)

    @property
    def cap_expert(self) -> int:
        """Worst-case expert-buffer rows: T*k + E*(align-1), or E*block."""
        if self.block > 0:
            return self.E * self.block
        return self.T * self.k + self.E * (self.align - 1)


def layout_workspace_bytes(shape: "Shape") -> int:
    """moe_layout_workspace_bytes: scratch the two-launch layout needs (0: none)."""
    return int(lib().moe_layout_workspace_bytes(ctypes.byref(shape.c())))


def layout(topk_ids: torch.Tensor, E: int, R: int, H: int = 8, *, align: int = 1,
           block: int = 0, err=None, out: dict | None = None,
           workspace: torch.Tensor | None = None) -> dict:
    """moe_dispatch_layout: counts, offsets, token_rank_slot [T,R], pair_row [T,k].
    `workspace` (a device tensor of at least layout_workspace_bytes bytes)
    selects the two-launch layout; without it every workgroup counts all ids."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    shape = Shape(T, H, E, R, k, align, block)
    _check_err(err)
    if out is not None:
        for key, want in (("rank_counts", (R,)), ("rank_offsets", (R + 1,)),
                          ("expert_counts", (E,)), ("expert_offsets", (E + 1,)),
                          ("token_rank_slot", (T, R)), ("pair_row", (T, k))):
            _need(out[key], key, want)
            if out[key].dtype != torch.int32:
                raise MoeError(f"{key} must be int32, got {out[key].dtype}")
    if out is None:
        out = dict(
            rank_counts=torch.empty(R, dtype=torch.int32, device=dev),
            rank_offsets=torch.empty(R + 1, dtype=torch.int32, device=dev),
            expert_counts=torch.empty(E, dtype=torch.int32, device=dev),
            expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            token_rank_slot=torch.empty((T, R), dtype=torch.int32, device=dev),
            pair_row=torch.empty((T, k), dtype=torch.int32, device=dev),
        )
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().moe_dispatch_layout(
        ctypes.byref(shape.c()), _ptr(_i32(topk_ids)), _ptr(_i32(out["rank_counts"])),
        _ptr(_i32(out["rank_offsets"])), _ptr(_i32(out["expert_counts"])),
        _ptr(_i32(out["expert_offsets"])), _ptr(_i32(out["token_rank_slot"])),
        _ptr(_i32(out["pair_row"])), _ptr(workspace), ws_bytes,
        _err(err), _stream(dev))
    _check(st, "moe_dispatch_layout")
    return out


def layout_noalloc(topk_ids: torch.Tensor, E: int, R: int, H: int = 8, *, align: int = 1,
                   block: int = 0, err=None, out: dict) -> dict:
    """moe_dispatch_layout_noalloc: the layout into caller-provided `out`
    tensors (the same keys as layout()), its workspace the library's static
    array on the current device; this call allocates nothing."""
    T, k = topk_ids.shape
    shape = Shape(T, H, E, R, k, align, block)
    _check_err(err)
    for key, want in (("rank_counts", (R,)), ("rank_offsets", (R + 1,)),
                      ("expert_counts", (E,)), ("expert_offsets", (E + 1,)),
                      ("token_rank_slot", (T, R)), ("pair_row", (T, k))):
        _need(out[key], key, want)
        if out[key].dtype != torch.int32:
            raise MoeError(f"{key} must be int32, got {out[key].dtype}")
    st = lib().moe_dispatch_layout_noalloc(
        ctypes.byref(shape.c()), _ptr(_i32(topk_ids)), _ptr(out["rank_counts"]),
        _ptr(out["rank_offsets"]), _ptr(out["expert_counts"]), _ptr(out["expert_offsets"]),
        _ptr(out["token_rank_slot"]), _ptr(out["pair_row"]), _err(err),
        _stream(topk_ids.device))
    _check(st, "moe_dispatch_layout_noalloc")
    return out


def pack(hidden: torch.Tensor, token_rank_slot: torch.Tensor, E: int, k: int, rank_buf,
         rank_src_token, *, err=None) -> None:
    """moe_dispatch_pack into caller-provided rank_buf [cap_rank, H] and
    rank_src_token [cap_rank]."""
    _check_err(err)
    T, H = hidden.shape
    R = token_rank_slot.shape[1]
    _need(token_rank_slot, "token_rank_slot", (T, R))
    cap = _rows(rank_buf, "rank_buf", H)
    _need(rank_src_token, "rank_src_token", min_numel=cap)
    shape = Shape(T, H, E, R, k)
    st = lib().moe_dispatch_pack(
        ctypes.byref(shape.c()), _ptr(_rows16(hidden)), _ptr(_i32(token_rank_slot)),
        _ptr(_rows16(rank_buf)), _ptr(_i32(rank_src_token)), rank_buf.shape[0], _err(err),
        _stream(hidden.device))
    _check(st, "moe_dispatch_pack")


def permute(rank_buf, rank_src_token, rank_offsets, topk_ids, pair_row, E: int, expert_buf,
            expert_src_pair, *, expert_counts=None, expert_offsets=None, align: int = 1,
            block: int = 0, err=None) -> None:
    """moe_permute_by_expert into caller-provided expert_buf [cap_expert, H].
    A padded (align > 1) or blocked (block > 0) layout needs the layout's
    expert_counts and expert_offsets, to mark its padding rows."""
    _check_err(err)
    T, k = topk_ids.shape
    H = rank_buf.shape[1]
    R = rank_offsets.shape[0] - 1
    _need(pair_row, "pair_row", (T, k))
    cap_r = _rows(rank_buf, "rank_buf", H)
    _need(rank_src_token, "rank_src_token", min_numel=cap_r)
    cap_e = _rows(expert_buf, "expert_buf", H)
    _need(expert_src_pair, "expert_src_pair", min_numel=cap_e)
    _need(expert_counts, "expert_counts", (E,))
    _need(expert_offsets, "expert_offsets", (E + 1,))
    shape = Shape(T, H, E, R, k, align, block)
    st = lib().moe_permute_by_expert(
        ctypes.byref(shape.c()), _ptr(_rows16(rank_buf)), _ptr(_i32(rank_src_token)),
        _ptr(_i32(rank_offsets)), _ptr(_i32(topk_ids)), _ptr(_i32(pair_row)),
        _ptr(None if expert_counts is None else _i32(expert_counts)),
        _ptr(None if expert_offsets is None else _i32(expert_offsets)),
        rank_buf.shape[0], _ptr(_rows16(expert_buf)), _ptr(_i32(expert_src_pair)),
        expert_buf.shape[0], _err(err), _stream(rank_buf.device))
    _check(st, "moe_permute_by_expert")


def dispatch_all(hidden, topk_ids, E: int, R: int, out: dict, rank_buf, rank_src_token,
                 expert_buf, expert_src_pair, *, align: int = 1, block: int = 0,
                 workspace: torch.Tensor | None = None, err=None) -> None:
    """moe_dispatch: layout, pack and permute in one call (one kernel launch
    for up to 256 tokens with k in {1, 2, 4, 6, 8}, up to 64
    for another k; else the layout and one pack-and-permute kernel), into
    the caller's tensors: `out`
    holds the layout's outputs (the keys of layout()), rank_buf [cap_rank, H],
    rank_src_token [cap_rank], expert_buf [cap_expert, H], expert_src_pair
    [cap_expert]."""
    _check_err(err)
    T, k = topk_ids.shape
    H = hidden.shape[1]
    _need(hidden, "hidden", (T, H))
    for key, want in (("rank_counts", (R,)), ("rank_offsets", (R + 1,)),
                      ("expert_counts", (E,)), ("expert_offsets", (E + 1,)),
                      ("token_rank_slot", (T, R)), ("pair_row", (T, k))):
        _need(out[key], key, want)
        _i32(out[key])
    cap_r = _rows(rank_buf, "rank_buf", H)
    _need(rank_src_token, "rank_src_token", min_numel=cap_r)
    cap_e = _rows(expert_buf, "expert_buf", H)
    _need(expert_src_pair, "expert_src_pair", min_numel=cap_e)
    shape = Shape(T, H, E, R, k, align, block)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().moe_dispatch(
        ctypes.byref(shape.c()), _ptr(_rows16(hidden)), _ptr(_i32(topk_ids)),
        _ptr(out["rank_counts"]), _ptr(out["rank_offsets"]), _ptr(out["expert_counts"]),
        _ptr(out["expert_offsets"]), _ptr(out["token_rank_slot"]), _ptr(out["pair_row"]),
        _ptr(_rows16(rank_buf)), _ptr(_i32(rank_src_token)), rank_buf.shape[0],
        _ptr(_rows16(expert_buf)), _ptr(_i32(expert_src_pair)), expert_buf.shape[0],
        _ptr(workspace), ws_bytes, _err(err), _stream(hidden.device))
    _check(st, "moe_dispatch")


def _bytes(t: torch.Tensor) -> torch.Tensor:
    if t.element_size() != 1 or not t.is_contiguous():
        raise MoeError(f"expected a contiguous 8-bit tensor, got {t.dtype}")
    return t


def _wire(fmt) -> tuple:
    """A wire format name (or the bits 8 / 4 of an MX format) -> (name, code
    bits per value, values per scale byte)."""
    name = {8: "mxfp8", 4: "mxfp4"}.get(fmt, fmt)
    if name not in WIRE_FORMATS:
        raise MoeError(f"unknown wire format {fmt!r}: one of {sorted(WIRE_FORMATS)}")
    return (name,) + WIRE_FORMATS[name]


def pack_mx(fmt, hidden: torch.Tensor, token_rank_slot: torch.Tensor, E: int, k: int,
            rank_q, rank_scale, rank_src_token, *, err=None) -> None:
    """moe_dispatch_pack_mxfp8 / _mxfp4 / _nvfp4 (fmt "mxfp8", "mxfp4",
    "nvfp4", or the bits 8 / 4 of an MX format): quantise each hidden row once
    and pack it once per distinct rank into rank_q [cap_rank, H*bits/8] (uint8
    codes) and rank_scale [cap_rank, H/block] (uint8 scales)."""
    name, bits, blk = _wire(fmt)
    _check_err(err)
    T, H = hidden.shape
    R = token_rank_slot.shape[1]
    _need(token_rank_slot, "token_rank_slot", (T, R))
    cap = _rows(rank_q, "rank_q", H * bits // 8)
    _need(rank_scale, "rank_scale", (cap, H // blk))
    _need(rank_src_token, "rank_src_token", min_numel=cap)
    shape = Shape(T, H, E, R, k)
    fn = getattr(lib(), f"moe_dispatch_pack_{name}")
    st = fn(ctypes.byref(shape.c()), _ptr(_rows16(hidden)), _ptr(_i32(token_rank_slot)),
            _ptr(_bytes(rank_q)), _ptr(_bytes(rank_scale)), _ptr(_i32(rank_src_token)),
            rank_q.shape[0], _err(err), _stream(hidden.device))
    _check(st, f"moe_dispatch_pack_{name}")


def dispatch_all_mx(fmt, hidden, topk_ids, E: int, R: int, out: dict, rank_q, rank_scale,
                    rank_src_token, expert_q, expert_scale, expert_src_pair, *, align: int = 1,
                    block: int = 0, workspace: torch.Tensor | None = None, err=None) -> None:
    """moe_dispatch_quantised: layout, quantise-and-pack and permute of the
    quantised rows in one call (one kernel launch for a decode-sized batch, else
    the layout and one quantise-pack-and-permute kernel, as dispatch_all), into
    the caller's tensors: `out` holds the layout's outputs,
    rank_q [cap_rank, H*bits/8] and rank_scale [cap_rank, H/block] (uint8),
    rank_src_token [cap_rank], expert_q / expert_scale / expert_src_pair
    likewise with cap_expert rows."""
    name, bits, blk = _wire(fmt)
    _check_err(err)
    T, k = topk_ids.shape
    H = hidden.shape[1]
    _need(hidden, "hidden", (T, H))
    for key, want in (("rank_counts", (R,)), ("rank_offsets", (R + 1,)),
                      ("expert_counts", (E,)), ("expert_offsets", (E + 1,)),
                      ("token_rank_slot", (T, R)), ("pair_row", (T, k))):
        _need(out[key], key, want)
        _i32(out[key])
    cap_r = _rows(rank_q, "rank_q", H * bits // 8)
    _need(rank_scale, "rank_scale", (cap_r, H // blk))
    _need(rank_src_token, "rank_src_token", min_numel=cap_r)
    cap_e = _rows(expert_q, "expert_q", H * bits // 8)
    _need(expert_scale, "expert_scale", (cap_e, H // blk))
    _need(expert_src_pair, "expert_src_pair", min_numel=cap_e)
    shape = Shape(T, H, E, R, k, align, block)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().moe_dispatch_quantised(
        ctypes.byref(shape.c()), WIRE_CODES[name], _ptr(_rows16(hidden)), _ptr(_i32(topk_ids)),
        _ptr(out["rank_counts"]), _ptr(out["rank_offsets"]), _ptr(out["expert_counts"]),
        _ptr(out["expert_offsets"]), _ptr(out["token_rank_slot"]), _ptr(out["pair_row"]),
        _ptr(_bytes(rank_q)), _ptr(_bytes(rank_scale)), _ptr(_i32(rank_src_token)),
        rank_q.shape[0], _ptr(_bytes(expert_q)), _ptr(_bytes(expert_scale)),
        _ptr(_i32(expert_src_pair)), expert_q.shape[0], _ptr(workspace), ws_bytes, _err(err),
        _stream(hidden.device))
    _check(st, "moe_dispatch_quantised")


def pack_mxfp8(*args, **kw) -> None:
    pack_mx("mxfp8", *args, **kw)


def pack_mxfp4(*args, **kw) -> None:
    pack_mx("mxfp4", *args, **kw)


def pack_nvfp4(*args, **kw) -> None:
    pack_mx("nvfp4", *args, **kw)


def permute_mx(fmt, rank_q, rank_scale, rank_src_token, rank_offsets, topk_ids, pair_row,
               E: int, expert_q, expert_scale, expert_src_pair, *, expert_counts=None,
               expert_offsets=None, align: int = 1, block: int = 0, err=None) -> None:
    """moe_permute_by_expert_mxfp8 / _mxfp4 / _nvfp4: the codes and scales of
    each rank-buffer row to the rows of its token's experts on that rank."""
    name, bits, blk = _wire(fmt)
    _check_err(err)
    T, k = topk_ids.shape
    H = rank_q.shape[1] * 8 // bits
    R = rank_offsets.shape[0] - 1
    _need(pair_row, "pair_row", (T, k))
    cap_r = rank_q.shape[0]
    _need(rank_scale, "rank_scale", (cap_r, H // blk))
    _need(rank_src_token, "rank_src_token", min_numel=cap_r)
    cap_e = _rows(expert_q, "expert_q", rank_q.shape[1])
    _need(expert_scale, "expert_scale", (cap_e, H // blk))
    _need(expert_src_pair, "expert_src_pair", min_numel=cap_e)
    _need(expert_counts, "expert_counts", (E,))
    _need(expert_offsets, "expert_offsets", (E + 1,))
    shape = Shape(T, H, E, R, k, align, block)
    fn = getattr(lib(), f"moe_permute_by_expert_{name}")
    st = fn(ctypes.byref(shape.c()), _ptr(_bytes(rank_q)), _ptr(_bytes(rank_scale)),
            _ptr(_i32(rank_src_token)), _ptr(_i32(rank_offsets)), _ptr(_i32(topk_ids)),
            _ptr(_i32(pair_row)), _ptr(None if expert_counts is None else _i32(expert_counts)),
            _ptr(None if expert_offsets is None else _i32(expert_offsets)), rank_q.shape[0],
            _ptr(_bytes(expert_q)), _ptr(_bytes(expert_scale)), _ptr(_i32(expert_src_pair)),
            expert_q.shape[0], _err(err), _stream(rank_q.device))
    _check(st, f"moe_permute_by_expert_{name}")


def permute_mxfp8(*args, **kw) -> None:
    permute_mx("mxfp8", *args, **kw)


def permute_mxfp4(*args, **kw) -> None:
    permute_mx("mxfp4", *args, **kw)


def permute_nvfp4(*args, **kw) -> None:
    permute_mx("nvfp4", *args, **kw)


def combine(expert_out, pair_row, topk_weights, E: int, R: int, out, *, out_f32=None,
            err=None) -> None:
    """moe_combine: out [T, H] bf16 (and optionally out_f32 [T, H] float32)."""
    _check_err(err)
    T, k = pair_row.shape
    H = out.shape[1]
    if topk_weights.dtype != torch.float32:
        raise MoeError("topk_weights must be float32")
    if out_f32 is not None and out_f32.dtype != torch.float32:
        raise MoeError("out_f32 must be float32")
    _need(topk_weights, "topk_weights", (T, k))
    _need(out, "out", (T, H))
    _need(out_f32, "out_f32", (T, H))
    _rows(expert_out, "expert_out", H)
    shape = Shape(T, H, E, R, k)
    st = lib().moe_combine(
        ctypes.byref(shape.c()), _ptr(_rows16(expert_out)), _ptr(_i32(pair_row)),
        _ptr(topk_weights), expert_out.shape[0], _ptr(_rows16(out)), _ptr(out_f32), _err(err),
        _stream(out.device))
    _check(st, "moe_combine")


def combine_rank_partial(expert_out, rank_src_token, rank_offsets, topk_ids, pair_row,
                         topk_weights, E: int, partial, *, partial_f32=None, err=None) -> None:
    """moe_combine_rank_partial: one bf16 partial row per rank-buffer row into
    caller-provided partial [cap_rank, H] (and optionally partial_f32)."""
    _check_err(err)
    T, k = topk_ids.shape
    H = partial.shape[1]
    R = rank_offsets.shape[0] - 1
    if topk_weights.dtype != torch.float32:
        raise MoeError("topk_weights must be float32")
    if partial_f32 is not None and partial_f32.dtype != torch.float32:
        raise MoeError("partial_f32 must be float32")
    _need(pair_row, "pair_row", (T, k))
    _need(topk_weights, "topk_weights", (T, k))
    cap_r = _rows(partial, "partial", H)
    _need(partial_f32, "partial_f32", (cap_r, H))
    _need(rank_src_token, "rank_src_token", min_numel=cap_r)
    _rows(expert_out, "expert_out", H)
    shape = Shape(T, H, E, R, k)
    st = lib().moe_combine_rank_partial(
        ctypes.byref(shape.c()), _ptr(_rows16(expert_out)), _ptr(_i32(rank_src_token)),
        _ptr(_i32(rank_offsets)), _ptr(_i32(topk_ids)), _ptr(_i32(pair_row)),
        _ptr(topk_weights), expert_out.shape[0], partial.shape[0], _ptr(_rows16(partial)),
        _ptr(partial_f32), _err(err), _stream(partial.device))
    _check(st, "moe_combine_rank_partial")


def combine_ranks(partial, token_rank_slot, E: int, k: int, out, *, out_f32=None,
                  err=None) -> None:
    """moe_combine_ranks: out [T, H] = sum over ranks of the token's partial rows."""
    _check_err(err)
    T, R = token_rank_slot.shape
    H = out.shape[1]
    if out_f32 is not None and out_f32.dtype != torch.float32:
        raise MoeError("out_f32 must be float32")
    _need(out, "out", (T, H))
    _need(out_f32, "out_f32", (T, H))
    _rows(partial, "partial", H)
    shape = Shape(T, H, E, R, k)
    st = lib().moe_combine_ranks(
        ctypes.byref(shape.c()), _ptr(_rows16(partial)), _ptr(_i32(token_rank_slot)),
        partial.shape[0], _ptr(_rows16(out)), _ptr(out_f32), _err(err), _stream(out.device))
    _check(st, "moe_combine_ranks")


class Router(ctypes.Structure):
    """moe_router_t: how the router scores, chooses and weighs. scoring
    "softmax" or "sigmoid"; renorm: the weights are the chosen scores over
    their sum; scale: a factor on them; groups / top_groups: the experts come
    from the best top_groups of `groups` equal groups (sigmoid only)."""
    _fields_ = [("scoring", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("scale", ctypes.c_float), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32)]

    def __init__(self, scoring: str = "softmax", renorm: bool = True, scale: float = 1.0,
                 groups: int = 1, top_groups: int = 1):
        if scoring not in SCORINGS:
            raise MoeError(f"unknown scoring {scoring!r}: one of {sorted(SCORINGS)}")
        super().__init__(SCORINGS[scoring], 1 if renorm else 0, scale, groups, top_groups)


# The raw stream and device of the caller's context, without the objects that
# torch.cuda.current_stream() makes at every call (2 us of a 9 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _current_stream(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _current_device() -> int:
    return _raw_device() if _raw_device is not None else torch.cuda.current_device()


@functools.lru_cache(maxsize=1024)
def _sizes(T: int, H: int, E: int, k: int) -> MoeShape:
    """The shape structure of a call (only ever read by the library)."""
    return MoeShape(T, H, E, 1, k)


def _dev(t: torch.Tensor | None, name: str, dtype, shape: tuple, device) -> int | None:
    """The address of a tensor of exactly this type and shape, contiguous and
    on `device`; None for None. Raises MoeError."""
    if t is None:
        return None
    if _address is not None:
        at = _address(t, dtype, device.index, shape)
        if at is not None:
            return at  # else what is wrong is found below
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise MoeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise MoeError(f"{name} has shape {tuple(t.shape)}, the call needs {shape}")
    if t.device != device:
        raise MoeError(f"{name} is on {t.device}, the call needs {device}: all tensors must be "
                       "on one GPU")
    raise MoeError(f"{name} must be contiguous")


def _dev_err(t: torch.Tensor | None, device) -> int | None:
    """The address of the device error word (see _check_err)."""
    if t is None:
        return None
    _check_err(t)
    return _dev(t, "err", torch.int32, t.shape, device)


def _logits(logits: torch.Tensor, device) -> int:
    """The type code of a [T, E] tensor of router logits on a GPU."""
    code = LOGIT_TYPES.get(logits.dtype)
    if code is None or logits.dim() != 2:
        raise MoeError("logits must be [T, E] of float32, bfloat16 or float16, got "
                       f"{tuple(logits.shape)} of {logits.dtype}")
    if device.type != "cuda":
        raise MoeError("tensors must be on the GPU")
    return code


def _call(fn, name: str, device, *args) -> None:
    """One library call on the current stream of the tensors' device, which is
    made current for it."""
    if device.index != _current_device():
        with torch.cuda.device(device):
            st = fn(*args, _current_stream(device))
    else:
        st = fn(*args, _current_stream(device))
    if st != MOE_OK:
        _check(st, name)


def route(logits: torch.Tensor, k: int, router: Router, topk_ids, topk_weights, *, bias=None,
          token_mask=None, err=None) -> None:
    """moe_route: the k experts of every token and their weights into
    topk_ids [T, k] int32 and topk_weights [T, k] float32, from logits [T, E]
    (float32, bfloat16 or float16); bias [E] float32 is added to the choice's
    scores (sigmoid only); token_mask [T] bool or uint8: tokens with 0 get no
    expert. The outputs are what layout() / dispatch_all() and combine() take."""
    dev = logits.device
    code = _logits(logits, dev)
    T, E = logits.shape
    if token_mask is not None and token_mask.dtype == torch.bool:
        token_mask = token_mask.view(torch.uint8)
    _call(lib().moe_route, "moe_route", dev, _sizes(T, 8, E, k), ctypes.byref(router), code,
          _dev(logits, "logits", logits.dtype, (T, E), dev),
          _dev(bias, "bias", torch.float32, (E,), dev),
          _dev(token_mask, "token_mask", torch.uint8, (T,), dev),
          _dev(topk_ids, "topk_ids", torch.int32, (T, k), dev),
          _dev(topk_weights, "topk_weights", torch.float32, (T, k), dev), _dev_err(err, dev))


def route_backward(logits: torch.Tensor, topk_ids, router: Router, d_logits, *, d_weights=None,
                   balance: tuple | None = None, err=None) -> None:
    """moe_route_backward: the gradient of the logits into d_logits [T, E] (the
    logits' type), from d_weights [T, k] float32 (the gradient of route()'s
    weights), from the balance losses, or from both: `balance` is (d_loss [S]
    float32, expert_counts [S, E], token_counts [S], seq_offsets [S + 1] or
    None), with the counts balance_loss() gave."""
    dev = logits.device
    code = _logits(logits, dev)
    T, E = logits.shape
    if topk_ids.dim() != 2:
        raise MoeError(f"topk_ids has shape {tuple(topk_ids.shape)}, the call needs [T, k]")
    k = topk_ids.shape[1]
    i32, f32 = torch.int32, torch.float32
    S, d_loss, counts, tokens, offsets = 0, None, None, None, None
    if d_weights is None and balance is None:
        raise MoeError("give d_weights, balance or both")
    if balance is not None:
        d_loss, counts, tokens, offsets = balance
        S = d_loss.numel()
        d_loss = _dev(d_loss, "d_loss", f32, (S,), dev)
        counts = _dev(counts, "expert_counts", i32, (S, E), dev)
        tokens = _dev(tokens, "token_counts", i32, (S,), dev)
        offsets = _dev(offsets, "seq_offsets", i32, (S + 1,), dev)
    _call(lib().moe_route_backward, "moe_route_backward", dev, _sizes(T, 8, E, k),
          ctypes.byref(router), code, _dev(logits, "logits", logits.dtype, (T, E), dev),
          _dev(topk_ids, "topk_ids", i32, (T, k), dev),
          _dev(d_weights, "d_weights", f32, (T, k), dev), d_loss, counts, tokens, offsets, S,
          _dev(d_logits, "d_logits", logits.dtype, (T, E), dev), _dev_err(err, dev))


def balance_workspace_bytes(T: int, E: int, k: int, sequences: int = 1) -> int:
    """moe_balance_workspace_bytes: scratch that balance_loss() needs, for this
    many tokens, experts and sequences or fewer."""
    return int(lib().moe_balance_workspace_bytes(_sizes(T, 8, E, k), sequences))


def balance_loss(logits: torch.Tensor, topk_ids, router: Router, loss, expert_counts,
                 token_counts, score_mean, *, workspace, seq_offsets=None, err=None) -> None:
    """moe_balance_loss: the balance loss of each of S sequences into loss [S]
    float32, with expert_counts [S, E] int32 (pairs per expert), token_counts
    [S] int32 and score_mean [S, E] float32. seq_offsets [S + 1] int32, or None
    for one sequence of all tokens; workspace: a device tensor of at least
    balance_workspace_bytes bytes."""
    dev = logits.device
    code = _logits(logits, dev)
    T, E = logits.shape
    if topk_ids.dim() != 2:
        raise MoeError(f"topk_ids has shape {tuple(topk_ids.shape)}, the call needs [T, k]")
    if workspace is None:
        raise MoeError("balance_loss needs a workspace of balance_workspace_bytes bytes")
    k, S = topk_ids.shape[1], loss.numel()
    i32, f32 = torch.int32, torch.float32
    _call(lib().moe_balance_loss, "moe_balance_loss", dev, _sizes(T, 8, E, k),
          ctypes.byref(router), code, _dev(logits, "logits", logits.dtype, (T, E), dev),
          _dev(topk_ids, "topk_ids", i32, (T, k), dev),
          _dev(seq_offsets, "seq_offsets", i32, (S + 1,), dev), S,
          _dev(loss, "loss", f32, (S,), dev),
          _dev(expert_counts, "expert_counts", i32, (S, E), dev),
          _dev(token_counts, "token_counts", i32, (S,), dev),
          _dev(score_mean, "score_mean", f32, (S, E), dev),
          _dev(workspace, "workspace", workspace.dtype, workspace.shape, dev),
          workspace.numel() * workspace.element_size(), _dev_err(err, dev))


def expert_product(fmt: str, rows: torch.Tensor, expert_counts, expert_offsets, T: int, k: int,
                   w_q, w_scale, out, *, act: str | None = None, factor=None, err=None) -> None:
    """moe_expert_product: the rows [cap, H] (bf16) of the expert-grouped
    buffer times their experts' 4-bit weights into out [cap, N] bf16, or
    [cap, N / 2] with act "swiglu". fmt "mxfp4" or "nvfp4"; w_q [E, N, H / 2]
    and w_scale [E, N, H / 32 or H / 16] uint8; factor [E] float32 multiplies
    an expert's products; the launch is laid out for T * k rows in use (other
    numbers cost time, no rows). expert_counts [E] and expert_offsets [E + 1]
    are the layout's, or those of the experts [a, b) of it with their weights:
    counts[a:b], offsets[a:b + 1], and best a T of their share of the rows."""
    if fmt not in ("mxfp4", "nvfp4"):
        raise MoeError(f"unknown weight format {fmt!r}: mxfp4 or nvfp4")
    if act not in ACTS:
        raise MoeError(f"unknown activation {act!r}: one of {sorted(a for a in ACTS if a)}")
    dev = rows.device
    if dev.type != "cuda":
        raise MoeError("tensors must be on the GPU")
    if rows.dim() != 2 or w_q.dim() != 3:
        raise MoeError("rows must be [cap, H] and w_q [E, N, H / 2]")
    cap, H = rows.shape
    E, N, _ = w_q.shape
    code = ACTS[act]
    u8, i32 = torch.uint8, torch.int32
    if rows.dtype not in ROW_TYPES or out.dtype not in ROW_TYPES:
        raise MoeError(f"rows and out must be bf16 (or its bits), got {rows.dtype} and {out.dtype}")
    _call(lib().moe_expert_product, "moe_expert_product", dev, _sizes(T, H, E, k), N,
          WIRE_CODES[fmt], code, _dev(rows, "rows", rows.dtype, (cap, H), dev),
          _dev(expert_counts, "expert_counts", i32, (E,), dev),
          _dev(expert_offsets, "expert_offsets", i32, (E + 1,), dev), cap,
          _dev(w_q, "w_q", u8, (E, N, H // 2), dev),
          _dev(w_scale, "w_scale", u8, (E, N, H // WIRE_FORMATS[fmt][1]), dev),
          _dev(factor, "factor", torch.float32, (E,), dev),
          _dev(out, "out", out.dtype, (cap, N // 2 if code else N), dev), _dev_err(err, dev))


def _norm_type(t: torch.Tensor, name: str) -> int:
    code = NORM_TYPES.get(t.dtype)
    if code is None:
        raise MoeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def norm(x: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6, residual=None, sum=None,
         out=None, fmt: str | None = None, q=None, q_scale=None, inv_rms=None) -> None:
    """moe_norm: the root-mean-square norm of x [T, H] bf16, or of x + residual,
    times weight [H] (float32 or bfloat16). residual and sum [T, H] are float32 or
    bfloat16, sum the rounded x + residual (it may be the residual itself). The
    result goes to out [T, H] bf16, to codes, or to both: fmt "int8" with q
    [T, H] int8 and q_scale [T] float32, or "mxfp8" with q [T, H] and q_scale
    [T, H / 32] uint8. inv_rms [T] float32 is what norm_backward() needs."""
    dev = x.device
    if dev.type != "cuda":
        raise MoeError("tensors must be on the GPU")
    if fmt not in NORM_FORMATS:
        raise MoeError(f"unknown format {fmt!r}: int8 or mxfp8")
    if x.dim() != 2 or x.dtype not in ROW_TYPES:
        raise MoeError(f"x must be [T, H] of bf16 (or its bits), got {tuple(x.shape)} of {x.dtype}")
    if (residual is None) != (sum is None):
        raise MoeError("give residual and sum, or neither")
    if (fmt is None) != (q is None) or (fmt is None) != (q_scale is None):
        raise MoeError("q and q_scale go with a format")
    if out is None and q is None:
        raise MoeError("give out, q or both")
    T, H = x.shape
    bf16, f32 = torch.bfloat16, torch.float32
    stream = bf16 if residual is None else residual.dtype
    code = 1 if residual is None else _norm_type(residual, "residual")
    kind, scales = (torch.int8, (T,)) if fmt == "int8" else (torch.uint8, (T, H // 32))
    _call(_entry("moe_norm"), "moe_norm", dev, _sizes(T, H, 1, 1), code,
          _dev(x, "x", x.dtype, (T, H), dev), _dev(residual, "residual", stream, (T, H), dev),
          _dev(sum, "sum", stream, (T, H), dev), _norm_type(weight, "weight"),
          _dev(weight, "weight", weight.dtype, (H,), dev), eps,
          _dev(out, "out", bf16 if out is None or out.dtype not in ROW_TYPES else out.dtype,
               (T, H), dev), NORM_FORMATS[fmt], _dev(q, "q", kind, (T, H), dev),
          _dev(q_scale, "q_scale", f32 if fmt == "int8" else kind, scales, dev),
          _dev(inv_rms, "inv_rms", f32, (T,), dev))


def norm_workspace_bytes(T: int, H: int) -> int:
    """moe_norm_workspace_bytes: scratch that norm_backward() needs for the
    weight's gradient, for this many tokens or fewer."""
    return int(lib().moe_norm_workspace_bytes(_sizes(T, H, 1, 1)))


def norm_backward(d_out: torch.Tensor, sum: torch.Tensor, inv_rms, weight, *, d_sum=None,
                  d_x=None, d_residual=None, d_weight=None, workspace=None) -> None:
    """moe_norm_backward: from d_out [T, H] bf16 (the gradient of norm()'s
    result), sum and inv_rms as norm() wrote them (sum: x where there was no
    residual) and d_sum [T, H] (the gradient that reaches the sum from elsewhere,
    of the sum's type), the gradient of x and the residual into d_x [T, H] bf16
    and d_residual [T, H] of the sum's type, and the weight's into d_weight [H]
    float32 (with workspace: a device tensor of norm_workspace_bytes bytes)."""
    dev = d_out.device
    if dev.type != "cuda":
        raise MoeError("tensors must be on the GPU")
    if d_out.dim() != 2 or d_out.dtype not in ROW_TYPES:
        raise MoeError("d_out must be [T, H] of bf16 (or its bits), got "
                       f"{tuple(d_out.shape)} of {d_out.dtype}")
    if d_x is None and d_residual is None and d_weight is None:
        raise MoeError("give d_x, d_residual or d_weight")
    if d_weight is not None and workspace is None:
        raise MoeError("d_weight needs a workspace of norm_workspace_bytes bytes")
    T, H = d_out.shape
    code, stream, f32 = _norm_type(sum, "sum"), sum.dtype, torch.float32
    room = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call(_entry("moe_norm_backward"), "moe_norm_backward", dev, _sizes(T, H, 1, 1), code,
          _dev(d_out, "d_out", d_out.dtype, (T, H), dev), _dev(sum, "sum", stream, (T, H), dev),
          _dev(inv_rms, "inv_rms", f32, (T,), dev), _norm_type(weight, "weight"),
          _dev(weight, "weight", weight.dtype, (H,), dev),
          _dev(d_sum, "d_sum", stream, (T, H), dev),
          _dev(d_x, "d_x", torch.bfloat16 if d_x is None or d_x.dtype not in ROW_TYPES
               else d_x.dtype, (T, H), dev),
          _dev(d_residual, "d_residual", stream, (T, H), dev),
          _dev(d_weight, "d_weight", f32, (H,), dev),
          None if workspace is None else _dev(workspace, "workspace", workspace.dtype,
                                              workspace.shape, dev), room)


def quantise_rows(rows: torch.Tensor, q, scale, *, pair_row=None, err=None) -> None:
    """moe_quantise_rows: rows [cap, H] bf16 to q [cap, H] int8 with scale [cap]
    float32: the rows that pair_row [T, k] (the layout's) names, or all of them."""
    dev = rows.device
    if dev.type != "cuda":
        raise MoeError("tensors must be on the GPU")
    if rows.dim() != 2 or rows.dtype not in ROW_TYPES:
        raise MoeError(f"rows must be [cap, H] of bf16 (or its bits), got {tuple(rows.shape)} of "
                       f"{rows.dtype}")
    cap, H = rows.shape
    T, k = cap, 1
    if pair_row is not None:
        if pair_row.dim() != 2:
            raise MoeError(f"pair_row has shape {tuple(pair_row.shape)}, the call needs [T, k]")
        T, k = pair_row.shape
    _call(_entry("moe_quantise_rows"), "moe_quantise_rows", dev, _sizes(T, H, k, k),
          _dev(rows, "rows", rows.dtype, (cap, H), dev),
          _dev(pair_row, "pair_row", torch.int32, (T, k), dev), cap,
          _dev(q, "q", torch.int8, (cap, H), dev),
          _dev(scale, "scale", torch.float32, (cap,), dev), _dev_err(err, dev))


def int8_product(rows: torch.Tensor, row_scale, w_q, w_scale, out, *, act: str | None = None,
                 expert_counts=None, expert_offsets=None, T: int | None = None, k: int = 1,
                 err=None) -> None:
    """moe_int8_product: rows [cap, H] int8 with row_scale [cap] float32 times
    weights w_q [E, N, H] int8 with w_scale [E, N] float32 into out [cap, N] bf16,
    or [cap, N / 2] with act "swiglu". With expert_counts [E] and expert_offsets
    [E + 1] (the layout's, or those of a slice of its experts, as for
    expert_product()) the rows are the expert-grouped buffer's, and T * k of them
    are in use as far as the host knows; without, the first T * k rows have the one
    expert. Without T it is all rows."""
    if act not in ACTS:
        raise MoeError(f"unknown activation {act!r}: one of {sorted(a for a in ACTS if a)}")
    dev = rows.device
    if dev.type != "cuda":
        raise MoeError("tensors must be on the GPU")
    if rows.dim() != 2 or w_q.dim() != 3:
        raise MoeError("rows must be [cap, H] and w_q [E, N, H]")
    if (expert_counts is None) != (expert_offsets is None):
        raise MoeError("give expert_counts and expert_offsets, or neither")
    cap, H = rows.shape
    E, N, _ = w_q.shape
    code = ACTS[act]
    i8, i32, f32 = torch.int8, torch.int32, torch.float32
    if T is None:
        T, k = cap, 1
    if out.dtype not in ROW_TYPES:
        raise MoeError(f"out must be bf16 (or its bits), got {out.dtype}")
    _call(_entry("moe_int8_product"), "moe_int8_product", dev, _sizes(T, H, E, k), N, code,
          _dev(rows, "rows", i8, (cap, H), dev), _dev(row_scale, "row_scale", f32, (cap,), dev),
          _dev(expert_counts, "expert_counts", i32, (E,), dev),
          _dev(expert_offsets, "expert_offsets", i32, (E + 1,), dev), cap,
          _dev(w_q, "w_q", i8, (E, N, H), dev), _dev(w_scale, "w_scale", f32, (E, N), dev),
          _dev(out, "out", out.dtype, (cap, N // 2 if code else N), dev), _dev_err(err, dev))


def time_next_launch(start: "torch.cuda.Event | None", stop: "torch.cuda.Event | None") -> None:
    """moe_testing_time_next_launch: the library's next kernel launch records
    `start` as it begins and `stop` as it ends (a measurement hook; both events
    must have been recorded once, so that they exist). None, None disarms."""
    if (start is None) != (stop is None):
        raise MoeError("give both events or neither")
    if start is not None and not (start.cuda_event and stop.cuda_event):
        raise MoeError("record both events once before arming them")
    st = lib().moe_testing_time_next_launch(
        None if start is None else ctypes.c_void_p(start.cuda_event),
        None if stop is None else ctypes.c_void_p(stop.cuda_event))
    _check(st, "moe_testing_time_next_launch")


class Buffers:
    """Every buffer of one dispatch + combine pass, allocated once for a shape
    at worst-case size (Shape.cap_rank and Shape.cap_expert rows)."""

    def __init__(self, shape: Shape, device, row_dtype=torch.bfloat16, want_f32: bool = False):
        T, H, E, R, k = shape.T, shape.H, shape.E, shape.R, shape.k
        d = device
        i32 = torch.int32
        self.shape = shape
        self.rank_counts = torch.empty(R, dtype=i32, device=d)
        self.rank_offsets = torch.empty(R + 1, dtype=i32, device=d)
        self.expert_counts = torch.empty(E, dtype=i32, device=d)
        self.expert_offsets = torch.empty(E + 1, dtype=i32, device=d)
        self.token_rank_slot = torch.empty((T, R), dtype=i32, device=d)
        self.pair_row = torch.empty((T, k), dtype=i32, device=d)
        self.rank_buf = torch.empty((shape.cap_rank, H), dtype=row_dtype, device=d)
        self.rank_src_token = torch.empty(shape.cap_rank, dtype=i32, device=d)
        self.expert_buf = torch.empty((shape.cap_expert, H), dtype=row_dtype, device=d)
        self.expert_src_pair = torch.empty(shape.cap_expert, dtype=i32, device=d)
        self.out = torch.empty((T, H), dtype=row_dtype, device=d)
        self.out_f32 = torch.empty((T, H), dtype=torch.float32, device=d) if want_f32 else None
        self.err = torch.zeros(1, dtype=i32, device=d)
        ws = layout_workspace_bytes(shape)
        self.workspace = torch.empty(max(ws, 4) // 4, dtype=i32, device=d) if ws else None

    def layout_dict(self) -> dict:
        return dict(rank_counts=self.rank_counts, rank_offsets=self.rank_offsets,
                    expert_counts=self.expert_counts, expert_offsets=self.expert_offsets,
                    token_rank_slot=self.token_rank_slot, pair_row=self.pair_row)


def dispatch(buf: Buffers, hidden, topk_ids) -> None:
    """Layout, pack and permute into `buf` (three library calls, no host sync)."""
    s = buf.shape
    layout(topk_ids, s.E, s.R, s.H, align=s.align, block=s.block, err=buf.err,
           out=buf.layout_dict(), workspace=buf.workspace)
    pack(hidden, buf.token_rank_slot, s.E, s.k, buf.rank_buf, buf.rank_src_token, err=buf.err)
    permute(buf.rank_buf, buf.rank_src_token, buf.rank_offsets, topk_ids, buf.pair_row, s.E,
            buf.expert_buf, buf.expert_src_pair, expert_counts=buf.expert_counts,
            expert_offsets=buf.expert_offsets, align=s.align, block=s.block, err=buf.err)


def combine_into(buf: Buffers, expert_out, topk_weights) -> None:
    s = buf.shape
    combine(expert_out, buf.pair_row, topk_weights, s.E, s.R, buf.out, out_f32=buf.out_f32,
            err=buf.err)
