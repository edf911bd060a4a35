"""ctypes binding of libbitffn_moe.so (include/bitffn_moe.h).

Argument marshalling only: tensors are checked for device, dtype and shape,
their data pointers and the current HIP stream are passed to the C ABI, and
any output tensor the caller did not supply is allocated with torch.  Every
step of the computation runs in the library's kernels.  There is no fallback:
if the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os
from typing import NamedTuple, Optional

import torch

LIB_NAME = "libbitffn_moe.so"
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), LIB_NAME)

MOE_OK, MOE_EINVAL, MOE_EALIGN, MOE_EFORMAT, MOE_ENOSPC, MOE_EHIP = 0, -1, -2, -3, -4, -5
FMT_Q2S, FMT_Q2SM, FMT_Q3G = 1, 2, 3
DTYPE_F32, DTYPE_BF16 = 0, 1
MAX_MX_OUT = 65536   # rows of the weight matrix of a 4-bit product (MOE_MAX_MX_OUT)

# every symbol the header declares, with its ctypes signature
_c_int, _c_i64, _c_sz, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p


class MoeLayerC(ctypes.Structure):
    _fields_ = [
        ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("fmt", ctypes.c_int32), ("n_slots", ctypes.c_int32),
        ("shared_slot", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("slot_bytes", ctypes.c_int64), ("pool", ctypes.c_void_p),
    ]


class MoeStackLayerC(ctypes.Structure):
    _fields_ = [
        ("pool", ctypes.c_void_p), ("slot_bytes", ctypes.c_int64),
        ("n_slots", ctypes.c_int32), ("fmt", ctypes.c_int32),
        ("shared_slot", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("slot_of_expert", ctypes.c_void_p), ("logits", ctypes.c_void_p),
        ("addend", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("idx", ctypes.c_void_p), ("w", ctypes.c_void_p), ("slot", ctypes.c_void_p),
        ("miss_expert", ctypes.c_void_p), ("miss_pair", ctypes.c_void_p),
        ("n_miss", ctypes.c_void_p),
    ]


class Mxfp4C(ctypes.Structure):
    _fields_ = [
        ("n_mats", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
    ]


_MXP = ctypes.POINTER(Mxfp4C)
_LP = ctypes.POINTER(MoeLayerC)
_SLP = ctypes.POINTER(MoeStackLayerC)
SIGNATURES = {
    "moe_abi_version": (_c_int, []),
    "moe_status_str": (ctypes.c_char_p, [_c_int]),
    "moe_last_hip_error": (_c_int, []),
    "moe_slot_bytes": (_c_i64, [_c_int, _c_int, _c_int]),
    "moe_router_logits": (_c_int, [_vp, _c_int, _c_int, _vp, _c_int, _vp, _vp]),
    "moe_route_topk": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "moe_lookup_workspace_bytes": (_c_sz, [_c_int, _c_int, _c_int]),
    "moe_cache_lookup": (_c_int, [_vp, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp, _vp,
                                  _c_sz, _vp]),
    "moe_decode_workspace_bytes": (_c_sz, [_LP, _c_int]),
    "moe_expert_ffn_decode": (_c_int, [_LP, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _c_sz, _vp]),
    "moe_decode_layer": (_c_int, [_LP, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _c_sz, _vp]),
    "moe_decode_layer_noalloc": (_c_int, [_LP, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _vp, _vp, _vp]),
    "moe_decode_stack_workspace_bytes": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "moe_decode_stack": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _SLP, _vp,
                                  _vp, _c_sz, _vp]),
    "moe_decode_misses": (_c_int, [_LP, _vp, _c_int, _vp, _vp, _vp, _vp, _c_int, _vp, _vp,
                                   _c_sz, _vp]),
    "moe_decode_misses_phases": (_c_int, [_LP, _vp, _c_int, _vp, _vp, _vp, _vp, _c_int, _vp,
                                          _vp, _c_sz, _c_int, _vp]),
    "moe_decode_layer_tiers": (_c_int, [_LP, _LP, _vp, _c_int, _vp, _c_int, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _vp, _c_sz, _vp]),
    "moe_cache_count": (_c_int, [_vp, _c_int, _c_int, _vp, _vp]),
    "moe_cache_plan": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _c_int, _vp, _c_int, _c_int,
                                _c_int, _vp, _vp, _vp]),
    "moe_cache_fill": (_c_int, [_LP, _LP, _vp, _vp, _c_int, _vp]),
    "moe_cache_commit": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _vp]),
    "moe_stage_layer": (_c_int, [_LP, _vp, _LP, _vp, _vp, _c_sz, _vp]),
    "moe_prefill_workspace_bytes": (_c_sz, [_LP, _c_int]),
    "moe_expert_ffn_prefill": (_c_int, [_LP, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _c_sz, _vp]),
    "moe_combine": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_group_workspace_bytes": (_c_sz, [_c_int, _c_int]),
    "moe_group_pairs": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_sz, _vp]),
    "moe_mxfp4_quantize": (_c_int, [_vp, _c_int, _c_i64, _c_int, _vp, _vp, _vp]),
    "moe_mxfp4_dequantize": (_c_int, [_vp, _vp, _c_i64, _c_int, _vp, _c_int, _vp]),
    "moe_mxfp4_linear": (_c_int, [_MXP, _MXP, _vp, _vp, _c_int, _c_i64, _vp, _c_int, _vp]),
    "moe_mxfp4_gate_up": (_c_int, [_MXP, _MXP, _vp, _vp, _c_int, _c_i64, _vp, _c_int, _vp]),
    "moe_mxfp4_ffn_decode_workspace_bytes": (_c_sz, [_c_int, _c_int, _c_int]),
    "moe_mxfp4_ffn_decode": (_c_int, [_MXP, _MXP, _c_int, _vp, _c_int, _c_int, _vp, _vp, _vp, _vp,
                                      _c_sz, _vp]),
    "moe_route_balance_workspace_bytes": (_c_sz, [_c_int, _c_int, _c_int]),
    "moe_route_balance": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, _c_sz, _vp]),
    "moe_route_backward": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _c_int, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _vp, _vp]),
}

_lib = None


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{LIB_NAME} is not built; run `python -m bit_expert_ffn_top_amd.build`")
        handle = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = lib().moe_status_str(status).decode()
        if status == MOE_EHIP:
            msg += f" (hip error {lib().moe_last_hip_error()})"
        super().__init__(f"{what}: {msg} [{status}]")
        self.status = status


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shape(t: torch.Tensor, shape, name: str):
    """t must have exactly this shape (None: any extent).  Checked before the
    device checks, so that a wrong size is reported as such."""
    got = t.shape
    if len(got) == len(shape):
        for a, s in zip(got, shape):
            if a != s and s is not None:
                break
        else:
            return t
    parts = ["*" if s is None else str(s) for s in shape]
    want = "(" + ", ".join(parts) + ("," if len(parts) == 1 else "") + ")"
    raise ValueError(f"{name}: shape {want} expected, got {tuple(got)}")


def _at_least(t: torch.Tensor, n: int, name: str):
    if t.numel() < n:
        raise ValueError(f"{name}: at least {n} elements expected, got {t.numel()}")
    return t


@dataclasses.dataclass
class MoeLayer:
    """One layer's packed expert pool in device memory."""
    d_model: int
    d_ff: int
    n_experts: int
    top_k: int
    fmt: int
    pool: torch.Tensor            # uint8 [n_slots, slot_bytes] on the device
    shared_slot: int = -1

    def c_struct(self) -> MoeLayerC:
        _dev(self.pool, torch.uint8, "pool")
        n_slots, sb = self.pool.shape
        return MoeLayerC(self.d_model, self.d_ff, self.n_experts, self.top_k, self.fmt,
                         n_slots, self.shared_slot, 0, sb, self.pool.data_ptr())


def abi_version() -> int:
    return lib().moe_abi_version()


def slot_bytes(fmt: int, d_model: int, d_ff: int) -> int:
    v = lib().moe_slot_bytes(fmt, d_model, d_ff)
    _check(int(v) if v < 0 else 0, "moe_slot_bytes")
    return int(v)


def router_logits(x: torch.Tensor, w: torch.Tensor, logits=None, stream=None):
    """logits [T, E] = x [T, d] (fp32) times the bf16 router weights w [E, d]."""
    _dev(_shape(x, (None, None), "x"), torch.float32, "x")
    T, d = x.shape
    _dev(_shape(w, (None, d), "w"), torch.bfloat16, "w")
    E = w.shape[0]
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _dev(_shape(logits, (T, E), "logits"), torch.float32, "logits")
    _check(lib().moe_router_logits(_ptr(x), T, d, _ptr(w), E, _ptr(logits), _stream(stream)),
           "moe_router_logits")
    return logits


def route_topk(logits: torch.Tensor, k: int, idx=None, w=None, stream=None):
    _shape(logits, (None, None), "logits")
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    if idx is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _dev(_shape(idx, (T, k), "idx"), torch.int32, "idx")
    _dev(_shape(w, (T, k), "w"), torch.float32, "w")
    _check(lib().moe_route_topk(_ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream(stream)),
           "moe_route_topk")
    return idx, w


def lookup_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(lib().moe_lookup_workspace_bytes(T, k, E))


def cache_lookup(idx: torch.Tensor, slot_of_expert: torch.Tensor, slot=None, miss_expert=None,
                 miss_pair=None, n_miss=None, ws=None, want_pairs=True, stream=None):
    _shape(idx, (None, None), "idx")
    _shape(slot_of_expert, (None,), "slot_of_expert")
    _dev(idx, torch.int32, "idx")
    _dev(slot_of_expert, torch.int32, "slot_of_expert")
    T, k = idx.shape
    E = slot_of_expert.shape[0]
    dev = idx.device
    n = T * k
    slot = torch.empty((T, k), dtype=torch.int32, device=dev) if slot is None else slot
    miss_expert = torch.full((max(n, 1),), -1, dtype=torch.int32, device=dev) if miss_expert is None else miss_expert
    if want_pairs and miss_pair is None:
        miss_pair = torch.full((max(n, 1),), -1, dtype=torch.int32, device=dev)
    n_miss = torch.zeros((4,), dtype=torch.int32, device=dev) if n_miss is None else n_miss
    _dev(_shape(slot, (T, k), "slot"), torch.int32, "slot")
    _dev(_at_least(miss_expert, n, "miss_expert"), torch.int32, "miss_expert")
    if miss_pair is not None:
        _dev(_at_least(miss_pair, n, "miss_pair"), torch.int32, "miss_pair")
    _dev(_at_least(n_miss, 2, "n_miss"), torch.int32, "n_miss")
    need = lookup_workspace_bytes(T, k, E)
    if need and ws is None:
        ws = torch.empty((need,), dtype=torch.uint8, device=dev)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().moe_cache_lookup(_ptr(idx), T, k, _ptr(slot_of_expert), E, _ptr(slot),
                                  _ptr(miss_expert), _ptr(miss_pair), _ptr(n_miss), _ptr(ws),
                                  ws_bytes, _stream(stream)), "moe_cache_lookup")
    return slot, miss_expert, miss_pair, n_miss


def decode_workspace_bytes(layer: MoeLayer, T: int) -> int:
    L = layer.c_struct()
    return int(lib().moe_decode_workspace_bytes(ctypes.byref(L), T))


def expert_ffn_decode(layer: MoeLayer, x, idx, slot, w, y=None, ws=None, stream=None):
    _dev(_shape(x, (None, layer.d_model), "x"), torch.float32, "x")
    T = x.shape[0]
    for name, t, dt in (("idx", idx, torch.int32), ("slot", slot, torch.int32),
                        ("w", w, torch.float32)):
        _dev(_shape(t, (T, layer.top_k), name), dt, name)
    L = layer.c_struct()
    if y is None:
        y = torch.empty_like(x)
    _dev(_shape(y, tuple(x.shape), "y"), torch.float32, "y")
    if ws is None:
        ws = torch.empty((decode_workspace_bytes(layer, T),), dtype=torch.uint8, device=x.device)
    _check(lib().moe_expert_ffn_decode(ctypes.byref(L), _ptr(x), T, _ptr(idx), _ptr(slot),
                                       _ptr(w), _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_expert_ffn_decode")
    return y


def decode_layer(layer: MoeLayer, x, logits, slot_of_expert, idx=None, w=None, slot=None,
                 miss_expert=None, miss_pair=None, n_miss=None, y=None, ws=None,
                 want_pairs=True, stream=None):
    """Route, look up and run one decode layer (moe_decode_layer).
    Returns (y, idx, w, slot, miss_expert, miss_pair, n_miss)."""
    _dev(_shape(x, (None, layer.d_model), "x"), torch.float32, "x")
    T = x.shape[0]
    k = layer.top_k
    _dev(_shape(logits, (T, layer.n_experts), "logits"), torch.float32, "logits")
    _dev(_shape(slot_of_expert, (layer.n_experts,), "slot_of_expert"), torch.int32,
         "slot_of_expert")
    dev = x.device
    n = T * k
    idx = torch.empty((T, k), dtype=torch.int32, device=dev) if idx is None else idx
    w = torch.empty((T, k), dtype=torch.float32, device=dev) if w is None else w
    slot = torch.empty((T, k), dtype=torch.int32, device=dev) if slot is None else slot
    if miss_expert is None:
        miss_expert = torch.full((n,), -1, dtype=torch.int32, device=dev)
    if want_pairs and miss_pair is None:
        miss_pair = torch.full((n,), -1, dtype=torch.int32, device=dev)
    n_miss = torch.zeros((4,), dtype=torch.int32, device=dev) if n_miss is None else n_miss
    y = torch.empty_like(x) if y is None else y
    for name, t, dt in (("idx", idx, torch.int32), ("w", w, torch.float32),
                        ("slot", slot, torch.int32)):
        _dev(_shape(t, (T, k), name), dt, name)
    _dev(_at_least(miss_expert, n, "miss_expert"), torch.int32, "miss_expert")
    if miss_pair is not None:
        _dev(_at_least(miss_pair, n, "miss_pair"), torch.int32, "miss_pair")
    _dev(_at_least(n_miss, 2, "n_miss"), torch.int32, "n_miss")
    _dev(_shape(y, tuple(x.shape), "y"), torch.float32, "y")
    L = layer.c_struct()
    if ws is _NO_WS:   # moe_decode_layer_noalloc: the library's own scratch
        _check(lib().moe_decode_layer_noalloc(ctypes.byref(L), _ptr(x), T, _ptr(logits),
                                              _ptr(slot_of_expert), _ptr(idx), _ptr(w),
                                              _ptr(slot), _ptr(miss_expert), _ptr(miss_pair),
                                              _ptr(n_miss), _ptr(y), _stream(stream)),
               "moe_decode_layer_noalloc")
        return y, idx, w, slot, miss_expert, miss_pair, n_miss
    if ws is None:
        ws = torch.empty((decode_workspace_bytes(layer, T),), dtype=torch.uint8, device=dev)
    _check(lib().moe_decode_layer(ctypes.byref(L), _ptr(x), T, _ptr(logits),
                                  _ptr(slot_of_expert), _ptr(idx), _ptr(w), _ptr(slot),
                                  _ptr(miss_expert), _ptr(miss_pair), _ptr(n_miss), _ptr(y),
                                  _ptr(ws), ws.numel(), _stream(stream)), "moe_decode_layer")
    return y, idx, w, slot, miss_expert, miss_pair, n_miss


_NO_WS = object()


def decode_layer_noalloc(layer: MoeLayer, x, logits, slot_of_expert, idx=None, w=None, slot=None,
                         miss_expert=None, miss_pair=None, n_miss=None, y=None, want_pairs=True,
                         stream=None):
    """decode_layer through moe_decode_layer_noalloc (no workspace: the
    library's own scratch array).  Outputs not given are allocated here, by
    torch; pass every output to allocate nothing."""
    return decode_layer(layer, x, logits, slot_of_expert, idx=idx, w=w, slot=slot,
                        miss_expert=miss_expert, miss_pair=miss_pair, n_miss=n_miss, y=y,
                        ws=_NO_WS, want_pairs=want_pairs, stream=stream)


def decode_stack_workspace_bytes(d_model, d_ff, n_experts, top_k, T) -> int:
    return int(lib().moe_decode_stack_workspace_bytes(d_model, d_ff, n_experts, top_k, T))


def new_stack_workspace(layers, T: int, device=None):
    """A workspace for decode_stack over layers of the shape of layers[0]."""
    L0 = layers[0]
    nb = decode_stack_workspace_bytes(L0.d_model, L0.d_ff, L0.n_experts, L0.top_k, T)
    if nb == 0:
        raise ValueError("decode_stack: sizes out of range")
    return torch.empty((nb,), dtype=torch.uint8, device=L0.pool.device if device is None else device)


def decode_stack(layers, x, logits, tables, addends=None, ys=None, routing=False, ws=None,
                 stream=None):
    """Decode / verify through a stack of layers in one call (moe_decode_stack).

    layers: list of MoeLayer (same d_model, d_ff, n_experts, top_k; formats may
    differ); x fp32 [T, d_model]; logits fp32 [L, T, E] (or a list of [T, E]);
    tables: list of int32 [E] slot tables; addends: None or fp32 [L, T, d]
    (entry 0 unused).  ys: fp32 [L, T, d] outputs (allocated if None), or
    fp32 [T, d] for the last layer's output only.  With routing=True also
    returns idx, w, slot [L, T, k], miss_expert, miss_pair [L, T*k] and
    n_miss [L, 4].  Returns a dict."""
    nl = len(layers)
    if nl < 1:
        raise ValueError("decode_stack: at least one layer")
    L0 = layers[0]
    d, f, E, k = L0.d_model, L0.d_ff, L0.n_experts, L0.top_k
    for Lx in layers:
        if (Lx.d_model, Lx.d_ff, Lx.n_experts, Lx.top_k) != (d, f, E, k):
            raise ValueError("decode_stack: every layer needs the same d_model, d_ff, n_experts, top_k")
    _dev(_shape(x, (None, d), "x"), torch.float32, "x")
    T = x.shape[0]
    dev = x.device
    if len(logits) != nl or len(tables) != nl:
        raise ValueError("decode_stack: one logits tensor and one table per layer")
    for l in range(nl):
        _dev(_shape(logits[l], (T, E), f"logits[{l}]"), torch.float32, f"logits[{l}]")
        _dev(_shape(tables[l], (E,), f"tables[{l}]"), torch.int32, f"tables[{l}]")
    if addends is not None:
        if len(addends) != nl:
            raise ValueError("decode_stack: one addend per layer")
        for l in range(nl):
            _dev(_shape(addends[l], (T, d), f"addends[{l}]"), torch.float32, f"addends[{l}]")
    if ys is None:
        ys = torch.empty((nl, T, d), dtype=torch.float32, device=dev)
    last_only = ys.dim() == 2
    _dev(_shape(ys, (T, d) if last_only else (nl, T, d), "ys"), torch.float32, "ys")
    out = {"y": ys}
    if routing:
        # per-layer rows padded to 16 bytes (every pointer must be 16-byte aligned)
        n = T * k
        pad = (n + 3) // 4 * 4

        def rows(dtype, fill):
            buf = torch.full((nl, pad), fill, dtype=dtype, device=dev)
            return buf[:, :n]

        out["idx"] = rows(torch.int32, 0).unflatten(1, (T, k))
        out["w"] = rows(torch.float32, 0).unflatten(1, (T, k))
        out["slot"] = rows(torch.int32, 0).unflatten(1, (T, k))
        out["miss_expert"] = rows(torch.int32, -1)
        out["miss_pair"] = rows(torch.int32, -1)
        out["n_miss"] = torch.zeros((nl, 4), dtype=torch.int32, device=dev)
    if ws is None:
        ws = new_stack_workspace(layers, T)
    _dev(ws, torch.uint8, "ws")
    arr = (MoeStackLayerC * nl)()
    for l, Lx in enumerate(layers):
        _dev(Lx.pool, torch.uint8, "pool")
        n_slots, sb = Lx.pool.shape
        c = arr[l]
        c.pool, c.slot_bytes, c.n_slots, c.fmt = Lx.pool.data_ptr(), sb, n_slots, Lx.fmt
        c.shared_slot, c.reserved = Lx.shared_slot, 0
        c.slot_of_expert, c.logits = tables[l].data_ptr(), logits[l].data_ptr()
        c.addend = addends[l].data_ptr() if (addends is not None and l > 0) else None
        if last_only:
            c.y = ys.data_ptr() if l + 1 == nl else None
        else:
            c.y = ys[l].data_ptr()
        if routing:
            c.idx, c.w, c.slot = (out["idx"][l].data_ptr(), out["w"][l].data_ptr(),
                                  out["slot"][l].data_ptr())
            c.miss_expert, c.miss_pair = out["miss_expert"][l].data_ptr(), out["miss_pair"][l].data_ptr()
            c.n_miss = out["n_miss"][l].data_ptr()
    _check(lib().moe_decode_stack(d, f, E, k, T, nl, arr, _ptr(x), _ptr(ws), ws.numel(),
                                  _stream(stream)), "moe_decode_stack")
    out["ws"] = ws
    return out


@dataclasses.dataclass
class HostTier:
    """A layer's experts in pinned host memory that the GPU reads directly
    (the tier the GPU cache's misses are computed from)."""
    d_model: int
    d_ff: int
    n_experts: int
    top_k: int
    fmt: int
    pool: torch.Tensor            # uint8 [n_slots, slot_bytes], pinned host (or device) memory

    def __post_init__(self):
        if self.pool.dtype != torch.uint8 or self.pool.dim() != 2 or not self.pool.is_contiguous():
            raise ValueError("host tier pool: contiguous uint8 [n_slots, slot_bytes] expected")
        if not (self.pool.is_cuda or self.pool.is_pinned()):
            raise ValueError("host tier pool: pinned host memory or device memory expected")

    def c_struct(self) -> MoeLayerC:
        n_slots, sb = self.pool.shape
        return MoeLayerC(self.d_model, self.d_ff, self.n_experts, self.top_k, self.fmt,
                         n_slots, -1, 0, sb, self.pool.data_ptr())


MISSES_READ, MISSES_JOIN = 1, 2   # phases of moe_decode_misses_phases


def decode_misses(tier: HostTier, x, idx, slot, w, host_slot_of_expert, y, max_rank=None,
                  ws=None, stream=None, phases=MISSES_READ | MISSES_JOIN):
    """Add the missed pairs of a decode step, computed from the host tier,
    into y (moe_decode_misses).  y holds the GPU part on entry.  Returns y.
    phases: MISSES_READ (the products into ws; y, w unused and may be None),
    MISSES_JOIN (y += the products in ws; x may be None), or both
    (moe_decode_misses_phases)."""
    T = (x if x is not None else y).shape[0]
    k = tier.top_k
    read, join = bool(phases & MISSES_READ), bool(phases & MISSES_JOIN)
    checks = [(idx, (T, k), torch.int32, "idx"), (slot, (T, k), torch.int32, "slot"),
              (host_slot_of_expert, (tier.n_experts,), torch.int32, "host_slot_of_expert")]
    if read or x is not None:
        checks.append((x, (T, tier.d_model), torch.float32, "x"))
    if join:
        checks += [(w, (T, k), torch.float32, "w"), (y, (T, tier.d_model), torch.float32, "y")]
    for t, shp, dt, name in checks:   # every shape first, then the devices and types
        _shape(t, shp, name)
    for t, shp, dt, name in checks:
        _dev(t, dt, name)
    r = k if max_rank is None else int(max_rank)
    L = tier.c_struct()
    if ws is None:
        ws = torch.empty((int(lib().moe_decode_workspace_bytes(ctypes.byref(L), T)),),
                         dtype=torch.uint8, device=idx.device)
    _check(lib().moe_decode_misses_phases(ctypes.byref(L), _ptr(x), T, _ptr(idx), _ptr(slot),
                                          _ptr(w), _ptr(host_slot_of_expert), r, _ptr(y),
                                          _ptr(ws), ws.numel(), int(phases), _stream(stream)),
           "moe_decode_misses_phases")
    return y


def decode_layer_tiers(layer: MoeLayer, tier: HostTier, x, logits, slot_of_expert,
                       host_slot_of_expert, max_rank=None, idx=None, w=None, slot=None,
                       miss_expert=None, miss_pair=None, n_miss=None, y=None, ws=None,
                       want_pairs=True, stream=None):
    """Route, look up and run one decode layer with the misses read from the
    host tier in the same launch (moe_decode_layer_tiers).
    Returns (y, idx, w, slot, miss_expert, miss_pair, n_miss)."""
    _shape(x, (None, layer.d_model), "x")
    T = x.shape[0]
    k = layer.top_k
    checks = [(x, torch.float32, "x"),
              (_shape(logits, (T, layer.n_experts), "logits"), torch.float32, "logits"),
              (_shape(slot_of_expert, (layer.n_experts,), "slot_of_expert"), torch.int32,
               "slot_of_expert"),
              (_shape(host_slot_of_expert, (tier.n_experts,), "host_slot_of_expert"),
               torch.int32, "host_slot_of_expert")]
    for t, dt, name in checks:   # every shape above first, then the devices and types
        _dev(t, dt, name)
    dev = x.device
    n = T * k
    idx = torch.empty((T, k), dtype=torch.int32, device=dev) if idx is None else idx
    w = torch.empty((T, k), dtype=torch.float32, device=dev) if w is None else w
    slot = torch.empty((T, k), dtype=torch.int32, device=dev) if slot is None else slot
    if miss_expert is None:
        miss_expert = torch.full((n,), -1, dtype=torch.int32, device=dev)
    if want_pairs and miss_pair is None:
        miss_pair = torch.full((n,), -1, dtype=torch.int32, device=dev)
    n_miss = torch.zeros((4,), dtype=torch.int32, device=dev) if n_miss is None else n_miss
    y = torch.empty_like(x) if y is None else y
    for name, t, dt in (("idx", idx, torch.int32), ("w", w, torch.float32),
                        ("slot", slot, torch.int32)):
        _dev(_shape(t, (T, k), name), dt, name)
    _dev(_at_least(miss_expert, n, "miss_expert"), torch.int32, "miss_expert")
    if miss_pair is not None:
        _dev(_at_least(miss_pair, n, "miss_pair"), torch.int32, "miss_pair")
    _dev(_at_least(n_miss, 2, "n_miss"), torch.int32, "n_miss")
    _dev(_shape(y, tuple(x.shape), "y"), torch.float32, "y")
    if ws is None:
        ws = torch.empty((decode_workspace_bytes(layer, T),), dtype=torch.uint8, device=dev)
    r = k if max_rank is None else int(max_rank)
    L, H = layer.c_struct(), tier.c_struct()
    _check(lib().moe_decode_layer_tiers(ctypes.byref(L), ctypes.byref(H),
                                        _ptr(host_slot_of_expert), r, _ptr(x), T, _ptr(logits),
                                        _ptr(slot_of_expert), _ptr(idx), _ptr(w), _ptr(slot),
                                        _ptr(miss_expert), _ptr(miss_pair), _ptr(n_miss),
                                        _ptr(y), _ptr(ws), ws.numel(), _stream(stream)),
           "moe_decode_layer_tiers")
    return y, idx, w, slot, miss_expert, miss_pair, n_miss


def cache_count(idx, counts, stream=None):
    """counts[e] += uses of expert e in idx (moe_cache_count).  counts: int32
    tensor viewed as uint32 [E]."""
    _dev(idx, torch.int32, "idx")
    _dev(_shape(counts, (None,), "counts"), torch.int32, "counts")
    _check(lib().moe_cache_count(_ptr(idx), idx.numel(), counts.numel(), _ptr(counts),
                                 _stream(stream)), "moe_cache_count")
    return counts


def cache_plan(counts, slot_of_expert, expert_of_slot, shared_slot, host_slot_of_expert,
               host_n_slots, max_swaps, decay_shift=1, swaps=None, n_swaps=None, stream=None):
    """Plan up to max_swaps swaps, updating the tables and decaying the
    counts in place (moe_cache_plan).  Returns (swaps [max_swaps, 4], n_swaps [4])."""
    E = counts.numel()
    for t, name in ((counts, "counts"), (slot_of_expert, "slot_of_expert"),
                    (host_slot_of_expert, "host_slot_of_expert")):
        _shape(t, (E,), name)
    _shape(expert_of_slot, (None,), "expert_of_slot")
    for t, name in ((counts, "counts"), (slot_of_expert, "slot_of_expert"),
                    (expert_of_slot, "expert_of_slot"), (host_slot_of_expert, "host_slot_of_expert")):
        _dev(t, torch.int32, name)
    dev = counts.device
    swaps = torch.full((max_swaps, 4), -1, dtype=torch.int32, device=dev) if swaps is None else swaps
    n_swaps = torch.zeros((4,), dtype=torch.int32, device=dev) if n_swaps is None else n_swaps
    _dev(_shape(swaps, (max_swaps, 4), "swaps"), torch.int32, "swaps")
    _dev(_at_least(n_swaps, 1, "n_swaps"), torch.int32, "n_swaps")
    _check(lib().moe_cache_plan(_ptr(counts), counts.numel(), _ptr(slot_of_expert),
                                _ptr(expert_of_slot), expert_of_slot.numel(), shared_slot,
                                _ptr(host_slot_of_expert), host_n_slots, max_swaps, decay_shift,
                                _ptr(swaps), _ptr(n_swaps), _stream(stream)), "moe_cache_plan")
    return swaps, n_swaps


def cache_fill(layer: MoeLayer, tier: HostTier, swaps, n_swaps, stream=None):
    """Copy the planned experts from the host tier into the cache's slots
    (moe_cache_fill)."""
    _dev(_shape(swaps, (None, 4), "swaps"), torch.int32, "swaps")
    _dev(_at_least(n_swaps, 1, "n_swaps"), torch.int32, "n_swaps")
    L, H = layer.c_struct(), tier.c_struct()
    _check(lib().moe_cache_fill(ctypes.byref(L), ctypes.byref(H), _ptr(swaps), _ptr(n_swaps),
                                swaps.shape[0], _stream(stream)), "moe_cache_fill")


def cache_commit(slot_of_expert, swaps, n_swaps, stream=None):
    """Make the admitted experts visible in the slot table (moe_cache_commit)."""
    _dev(_shape(slot_of_expert, (None,), "slot_of_expert"), torch.int32, "slot_of_expert")
    _dev(_shape(swaps, (None, 4), "swaps"), torch.int32, "swaps")
    _dev(_at_least(n_swaps, 1, "n_swaps"), torch.int32, "n_swaps")
    _check(lib().moe_cache_commit(_ptr(slot_of_expert), slot_of_expert.numel(), _ptr(swaps),
                                  _ptr(n_swaps), swaps.shape[0], _stream(stream)),
           "moe_cache_commit")


def stage_layer(cache: MoeLayer, slot_of_expert, tier: HostTier, host_slot_of_expert, staging,
                stream=None):
    """Copy every expert of the layer into `staging` in expert order
    (moe_stage_layer).  slot_of_expert / host_slot_of_expert: host int32
    arrays [n_experts]; staging: device uint8 [(n_experts + 1), slot_bytes].
    Returns the MoeLayer that reads the staged pool."""
    import numpy as np
    soe = np.ascontiguousarray(np.asarray(slot_of_expert, dtype=np.int32))
    hs = np.ascontiguousarray(np.asarray(host_slot_of_expert, dtype=np.int32))
    for a, name in ((soe, "slot_of_expert"), (hs, "host_slot_of_expert")):
        if a.shape != (cache.n_experts,):
            raise ValueError(f"{name}: shape ({cache.n_experts},) expected, got {a.shape}")
    _dev(staging, torch.uint8, "staging")
    C, H = cache.c_struct(), tier.c_struct()
    _check(lib().moe_stage_layer(ctypes.byref(C), soe.ctypes.data, ctypes.byref(H), hs.ctypes.data,
                                 _ptr(staging), staging.numel(), _stream(stream)),
           "moe_stage_layer")
    return MoeLayer(cache.d_model, cache.d_ff, cache.n_experts, cache.top_k, cache.fmt, staging,
                    cache.n_experts if cache.shared_slot >= 0 else -1)


def prefill_workspace_bytes(layer: MoeLayer, T: int) -> int:
    L = layer.c_struct()
    return int(lib().moe_prefill_workspace_bytes(ctypes.byref(L), T))


def expert_ffn_prefill(layer: MoeLayer, x_bf16, idx, slot, out_pairs=None, pair_pos=None,
                       expert_offsets=None, out_shared=None, with_shared=True, ws=None,
                       stream=None):
    _dev(_shape(x_bf16, (None, layer.d_model), "x_bf16"), torch.bfloat16, "x_bf16")
    T, d = x_bf16.shape
    k = layer.top_k
    _dev(_shape(idx, (T, k), "idx"), torch.int32, "idx")
    _dev(_shape(slot, (T, k), "slot"), torch.int32, "slot")
    dev = x_bf16.device
    if out_pairs is None:
        out_pairs = torch.empty((T * k, d), dtype=torch.float32, device=dev)
    if pair_pos is None:
        pair_pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    if expert_offsets is None:
        expert_offsets = torch.empty((layer.n_experts + 1,), dtype=torch.int32, device=dev)
    if with_shared and layer.shared_slot >= 0 and out_shared is None:
        out_shared = torch.empty((T, d), dtype=torch.float32, device=dev)
    if not with_shared:
        out_shared = None
    if ws is None:
        ws = torch.empty((prefill_workspace_bytes(layer, T),), dtype=torch.uint8, device=dev)
    _dev(_shape(out_pairs, (T * k, d), "out_pairs"), torch.float32, "out_pairs")
    _dev(_shape(pair_pos, (T, k), "pair_pos"), torch.int32, "pair_pos")
    _dev(_shape(expert_offsets, (layer.n_experts + 1,), "expert_offsets"), torch.int32,
         "expert_offsets")
    if out_shared is not None:
        _dev(_shape(out_shared, (T, d), "out_shared"), torch.float32, "out_shared")
    _dev(ws, torch.uint8, "ws")
    L = layer.c_struct()
    _check(lib().moe_expert_ffn_prefill(ctypes.byref(L), _ptr(x_bf16), T, _ptr(idx), _ptr(slot),
                                        _ptr(out_pairs), _ptr(pair_pos), _ptr(expert_offsets),
                                        _ptr(out_shared), _ptr(ws), ws.numel(),
                                        _stream(stream)), "moe_expert_ffn_prefill")
    return out_pairs, pair_pos, expert_offsets, out_shared


def combine(x, rows, pair_pos, w, shared=None, y=None, stream=None):
    if x.dtype == torch.float32:
        x_dtype = DTYPE_F32
    elif x.dtype == torch.bfloat16:
        x_dtype = DTYPE_BF16
    else:
        raise ValueError("x must be float32 or bfloat16")
    _dev(_shape(x, (None, None), "x"), x.dtype, "x")
    T, d = x.shape
    k = pair_pos.shape[1] if pair_pos is not None else 0
    if k:
        _dev(_shape(pair_pos, (T, k), "pair_pos"), torch.int32, "pair_pos")
        _dev(_shape(w, (T, k), "w"), torch.float32, "w")
        _dev(_shape(rows, (None, d), "rows"), torch.float32, "rows")
    if shared is not None:
        _dev(_shape(shared, (T, d), "shared"), torch.float32, "shared")
    if y is None:
        y = torch.empty((T, d), dtype=torch.float32, device=x.device)
    _dev(_shape(y, (T, d), "y"), torch.float32, "y")
    _check(lib().moe_combine(_ptr(x), x_dtype, T, d, k, _ptr(rows), _ptr(pair_pos), _ptr(w),
                             _ptr(shared), _ptr(y), _stream(stream)), "moe_combine")
    return y


# --- microscaled 4-bit floats and the router's losses ---------------------------
#
# These calls run on the device of their tensors (which must be one device);
# outputs and workspaces that they allocate come from the memory of the stream
# they are given, so that a buffer given back there is not used elsewhere before
# the call is done with it.


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _same_device(what, tensors):
    """The device of the tensors (None entries passed over), which must be one."""
    first, at = None, -1
    for t in tensors:
        if t is not None:
            if first is None:
                first, at = t, t.get_device()
            elif t.get_device() != at:
                raise ValueError(f"{what}: tensors on {first.device} and {t.device}, one device expected")
    return first.device


def _on_stream(fn):
    """For fn(dev, handle, ...) -> run(what, stream, tensors, ...): the tensors'
    one device and the handle of the stream (the device's current one if None),
    with both current while fn allocates and launches.  A stream of another
    device is refused."""
    def run(what, stream, tensors, *args):
        dev = _same_device(what, tensors)
        if stream is None and dev.index == torch.cuda.current_device():
            return fn(dev, _raw_stream(dev.index), *args)
        with torch.cuda.device(dev):
            s = torch.cuda.current_stream() if stream is None else stream
            if s.device != dev:
                raise ValueError(f"{what}: the stream belongs to {s.device}, the tensors to {dev}")
            with torch.cuda.stream(s):
                return fn(dev, s.cuda_stream, *args)
    return run


def _float_dtype(dtype, name):
    if dtype == torch.float32:
        return DTYPE_F32
    if dtype == torch.bfloat16:
        return DTYPE_BF16
    raise ValueError(f"{name} must be float32 or bfloat16, got {dtype}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _int32(value, name):
    """value as one of the library's 32-bit integers, which ctypes would cut to
    its low bits if it were larger."""
    i = int(value)
    if i != value or not -0x80000000 <= i <= 0x7FFFFFFF:
        raise ValueError(f"{name}: a 32-bit integer expected, got {value}")
    return i


def _sizes(what, *extents):
    """The same for the extents of tensors (not negative): one check of all."""
    for n in extents:
        if n >> 31:
            raise ValueError(f"{what}: sizes that fit 32-bit integers expected, got {n}")


def _scratch(need, ws, dev):
    """(address, bytes, tensor to keep until the launch) of a workspace."""
    if ws is None:
        if need == 0:
            return None, 0, None
        ws = torch.empty((need,), dtype=torch.uint8, device=dev)
    return ws.data_ptr(), ws.numel(), ws


@dataclasses.dataclass
class Mxfp4:
    """Microscaled 4-bit floats: codes uint8 [..., rows, cols / 2] and scales
    uint8 [..., rows, cols / 32] of one matrix or, with a leading dimension, of
    several (the layout of moe_mxfp4)."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        """(matrices, rows, cols)"""
        c = self.codes.shape
        return (1 if len(c) == 2 else c[0], c[-2], 2 * c[-1])

    def check(self, name):
        """The shape, after a check that codes and scales belong together."""
        c, s = self.codes.shape, self.scales.shape
        n = len(c)
        if n in (2, 3) and (c[0] | c[-2] | c[-1]) >> 30:   # cols is twice the last one
            _sizes(name, c[0], c[-2], 2 * c[-1])
        if n == len(s) and 2 <= n <= 3 and c[-1] == 16 * s[-1] and c[-2] == s[-2] and c[0] == s[0]:
            return (1 if n == 2 else c[0], c[-2], 2 * c[-1])
        if n not in (2, 3):
            raise ValueError(f"{name}.codes: shape (rows, cols / 2) or (matrices, rows, cols / 2) "
                             f"expected, got {tuple(c)}")
        cols = 2 * c[-1]
        if cols % 32:
            raise ValueError(f"{name}.codes: cols a multiple of 32 expected, got {cols}")
        _shape(self.scales, tuple(c[:-1]) + (cols // 32,), f"{name}.scales")
        return self.shape

    def on_device(self, name):
        for t, part in ((self.codes, "codes"), (self.scales, "scales")):
            if not (t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous()):
                _dev(t, torch.uint8, f"{name}.{part}")
        return self

    def c_struct(self, shape=None) -> Mxfp4C:
        """shape: the shape, where it is known already."""
        n, rows, cols = shape or self.shape
        return Mxfp4C(n, rows, cols, 0, self.codes.data_ptr(), self.scales.data_ptr())


def group_workspace_bytes(T: int, E: int) -> int:
    return int(lib().moe_group_workspace_bytes(_int32(T, "T"), _int32(E, "E")))


@_on_stream
def _group_pairs(dev, stream, idx, T, k, E, offsets, pair_pos, row_pair, ws):
    if offsets is None:
        offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    if pair_pos is None:
        pair_pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    if row_pair is None:
        row_pair = torch.empty((T * k,), dtype=torch.int32, device=dev)
    wp, wn, keep = _scratch(group_workspace_bytes(T, E), ws, dev)
    _check(lib().moe_group_pairs(idx.data_ptr(), T, k, E, offsets.data_ptr(), pair_pos.data_ptr(),
                                 row_pair.data_ptr(), wp, wn, stream), "moe_group_pairs")
    return offsets, pair_pos, row_pair


def group_pairs(idx, n_experts, offsets=None, pair_pos=None, row_pair=None, ws=None, stream=None):
    """Group the pairs of idx [T, k] by expert (moe_group_pairs).
    Returns (offsets [E + 1], pair_pos [T, k], row_pair [T * k])."""
    _shape(idx, (None, None), "idx")
    T, k = idx.shape
    E = _int32(n_experts, "n_experts")
    _sizes("idx", T, k)
    for t, shp, name in ((offsets, (E + 1,), "offsets"), (pair_pos, (T, k), "pair_pos"),
                         (row_pair, (T * k,), "row_pair")):
        if t is not None:
            _dev(_shape(t, shp, name), torch.int32, name)
    _dev(idx, torch.int32, "idx")
    if ws is not None:
        _dev(ws, torch.uint8, "ws")
    return _group_pairs("group_pairs", stream, (idx, offsets, pair_pos, row_pair, ws),
                        idx, T, k, E, offsets, pair_pos, row_pair, ws)


@_on_stream
def _quantize(dev, stream, x, dtype, lead, cols, out):
    if out is None:
        out = Mxfp4(torch.empty(lead + (cols // 2,), dtype=torch.uint8, device=dev),
                    torch.empty(lead + (cols // 32,), dtype=torch.uint8, device=dev))
    _check(lib().moe_mxfp4_quantize(x.data_ptr(), dtype, math.prod(lead), cols, out.codes.data_ptr(),
                                    out.scales.data_ptr(), stream), "moe_mxfp4_quantize")
    return out


def mxfp4_quantize(x, out: Optional[Mxfp4] = None, stream=None) -> Mxfp4:
    """x [rows, cols] or [matrices, rows, cols] (fp32 or bf16) as microscaled
    4-bit floats (moe_mxfp4_quantize)."""
    if x.dim() not in (2, 3):
        raise ValueError(f"x: 2 or 3 dimensions expected, got {tuple(x.shape)}")
    cols = x.shape[-1]
    if cols % 32:
        raise ValueError(f"x: a last dimension that is a multiple of 32 expected, got {cols}")
    _sizes("x", cols)
    dtype = _float_dtype(x.dtype, "x")
    lead = tuple(x.shape[:-1])
    if out is not None:
        _shape(out.codes, lead + (cols // 2,), "out.codes")
        _shape(out.scales, lead + (cols // 32,), "out.scales")
        out.on_device("out")
    _dev(x, x.dtype, "x")
    return _quantize("mxfp4_quantize", stream,
                     (x,) if out is None else (x, out.codes, out.scales), x, dtype, lead, cols, out)


@_on_stream
def _dequantize(dev, stream, q, shape, y, dtype, y_dtype):
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=dev)
    _check(lib().moe_mxfp4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), math.prod(shape[:-1]),
                                      shape[-1], y.data_ptr(), y_dtype, stream),
           "moe_mxfp4_dequantize")
    return y


def mxfp4_dequantize(q: Mxfp4, dtype=torch.float32, y=None, stream=None):
    """The values of q in fp32 or bf16, shape [..., rows, cols]
    (moe_mxfp4_dequantize)."""
    q.check("q")
    y_dtype = _float_dtype(dtype if y is None else y.dtype, "y")
    shape = tuple(q.codes.shape[:-1]) + (2 * q.codes.shape[-1],)
    if y is not None:
        _dev(_shape(y, shape, "y"), y.dtype, "y")
    q.on_device("q")
    return _dequantize("mxfp4_dequantize", stream, (q.codes, q.scales, y), q, shape, y, dtype, y_dtype)


@_on_stream
def _product(dev, stream, name, A, W, offsets, row_src, src_div, R, n_out, y, dtype, y_dtype):
    if y is None:
        y = torch.empty((R, n_out), dtype=dtype, device=dev)
    _check(getattr(lib(), name)(ctypes.byref(A), ctypes.byref(W), _addr(offsets), _addr(row_src),
                                src_div, R, y.data_ptr(), y_dtype, stream), name)
    return y


def _mx_product(what, gated, a, w, offsets, row_src, src_div, y, dtype, stream):
    na, ma, K = a_shape = a.check("a")
    G, N, Kw = w_shape = w.check("w")
    if na != 1:
        raise ValueError(f"{what}: a holds one matrix, got {na}")
    if K != Kw:
        raise ValueError(f"{what}: a has {K} columns, w {Kw}")
    if N > MAX_MX_OUT:
        raise ValueError(f"w: at most {MAX_MX_OUT} rows expected, got {N}")
    if offsets is not None:
        _shape(offsets, (G + 1,), "offsets")
    elif G != 1:
        raise ValueError(f"{what}: offsets are needed with {G} matrices")
    if row_src is not None:
        _shape(row_src, (None,), "row_src")
    R = ma if row_src is None else row_src.shape[0]
    if gated and N % 2:
        raise ValueError(f"{what}: an even number of rows of w expected, got {N}")
    n_out = N // 2 if gated else N
    src_div = _int32(src_div, "src_div")
    y_dtype = _float_dtype(dtype if y is None else y.dtype, "y")
    if y is not None:
        _dev(_shape(y, (R, n_out), "y"), y.dtype, "y")
    if offsets is not None:
        _dev(offsets, torch.int32, "offsets")
    if row_src is not None:
        _dev(row_src, torch.int32, "row_src")
    a.on_device("a")
    w.on_device("w")
    return _product(what, stream, (a.codes, a.scales, w.codes, w.scales, offsets, row_src, y),
                    f"moe_{what}", a.c_struct(a_shape), w.c_struct(w_shape), offsets, row_src, src_div, R, n_out,
                    y, dtype, y_dtype)


def mxfp4_linear(a: Mxfp4, w: Mxfp4, offsets=None, row_src=None, src_div=1, y=None,
                 dtype=torch.float32, stream=None):
    """y[r] = a[src(r)] . w[g]^T for the rows r of group g (moe_mxfp4_linear).

    a [rows, K]; w [G, N, K] (or [N, K]), N a multiple of 16 and at most 65536
    (a larger matrix goes in slices of its rows); offsets int32 [G + 1] bounds of the
    groups (None: one group); row_src int32 [R] with src(r) = row_src[r] //
    src_div (None: r).  Returns y [R, N] in dtype; rows of no group are left as
    they were (undefined in a y allocated here)."""
    return _mx_product("mxfp4_linear", False, a, w, offsets, row_src, src_div, y, dtype, stream)


def mxfp4_gate_up(a: Mxfp4, w: Mxfp4, offsets=None, row_src=None, src_div=1, h=None,
                  dtype=torch.bfloat16, stream=None):
    """h[r] = silu(gate) * up of the product with w [G, 2 F, K], gate rows even,
    up rows odd, 2 F a multiple of 64 and at most 65536 (moe_mxfp4_gate_up).
    Returns h [R, F]; arguments as mxfp4_linear."""
    return _mx_product("mxfp4_gate_up", True, a, w, offsets, row_src, src_div, h, dtype, stream)


def mxfp4_ffn_decode_workspace_bytes(T: int, k: int, d_ff: int) -> int:
    return int(lib().moe_mxfp4_ffn_decode_workspace_bytes(_int32(T, "T"), _int32(k, "k"), _int32(d_ff, "d_ff")))


@_on_stream
def _mx_decode(dev, stream, GU, D, shared_slot, x, T, d, k, f, slot, w, y, ws):
    if y is None:
        y = torch.empty((T, d), dtype=torch.float32, device=dev)
    wp, wn, keep = _scratch(lib().moe_mxfp4_ffn_decode_workspace_bytes(T, k, f), ws, dev)
    _check(lib().moe_mxfp4_ffn_decode(ctypes.byref(GU), ctypes.byref(D), shared_slot,
                                      x.data_ptr(), T, k, slot.data_ptr(), w.data_ptr(),
                                      y.data_ptr(), wp, wn, stream), "moe_mxfp4_ffn_decode")
    return y


def mxfp4_ffn_decode(gate_up: Mxfp4, down: Mxfp4, x, slot, w, shared_slot=-1, y=None, ws=None,
                     stream=None):
    """Decode / verify FFN of T = 1..4 tokens over 4-bit experts
    (moe_mxfp4_ffn_decode).  gate_up [n, 2 F, d], down [n, d, F]; x fp32 [T, d];
    slot int32 and w fp32 [T, k].  Returns y fp32 [T, d]."""
    n, f2, d = gate_up.check("gate_up")
    if down.check("down") != (n, d, f2 // 2) or f2 % 2:
        raise ValueError(f"down: (matrices, rows, cols) = {(n, d, f2 // 2)} expected, got {down.shape}")
    _shape(x, (None, d), "x")
    T = x.shape[0]
    _shape(slot, (T, None), "slot")
    k = slot.shape[1]
    _shape(w, (T, k), "w")
    _sizes("mxfp4_ffn_decode", T, k)
    shared_slot = _int32(shared_slot, "shared_slot")
    if y is not None:
        _dev(_shape(y, (T, d), "y"), torch.float32, "y")
    if ws is not None:
        _dev(ws, torch.uint8, "ws")
    _dev(x, torch.float32, "x")
    _dev(slot, torch.int32, "slot")
    _dev(w, torch.float32, "w")
    gate_up.on_device("gate_up")
    down.on_device("down")
    return _mx_decode("mxfp4_ffn_decode", stream,
                      (x, slot, w, gate_up.codes, gate_up.scales, down.codes, down.scales, y, ws),
                      gate_up.c_struct((n, f2, d)), down.c_struct((n, d, f2 // 2)), shared_slot, x, T, d, k,
                      f2 // 2, slot, w, y, ws)


class RouteBalance(NamedTuple):
    """What route_balance returns, per sequence."""
    balance: torch.Tensor     # fp32 [S]
    z: torch.Tensor           # fp32 [S]
    counts: torch.Tensor      # int32 [S, E]
    prob_sum: torch.Tensor    # fp32 [S, E]
    n_tokens: torch.Tensor    # int32 [S]


def _balance_args(logits, idx, seq_offsets, mask):
    """Shapes first, then devices and types.  Returns (T, E, k, S)."""
    _shape(logits, (None, None), "logits")
    T, E = logits.shape
    _shape(idx, (T, None), "idx")
    if seq_offsets is not None:
        _shape(seq_offsets, (None,), "seq_offsets")
        if seq_offsets.shape[0] < 2:
            raise ValueError("seq_offsets: at least 2 elements expected")
    k, S = idx.shape[1], 1 if seq_offsets is None else seq_offsets.shape[0] - 1
    _sizes("logits, idx, seq_offsets", T, E, k, S)
    if mask is not None:
        _shape(mask, (T,), "mask")
        if mask.dtype not in (torch.uint8, torch.bool):
            raise ValueError(f"mask must be uint8 or bool, got {mask.dtype}")
    _dev(logits, torch.float32, "logits")
    _dev(idx, torch.int32, "idx")
    if seq_offsets is not None:
        _dev(seq_offsets, torch.int32, "seq_offsets")
    if mask is not None:
        _dev(mask, mask.dtype, "mask")
    return T, E, k, S


def route_balance_workspace_bytes(T: int, E: int, n_seq: int) -> int:
    return int(lib().moe_route_balance_workspace_bytes(_int32(T, "T"), _int32(E, "E"), _int32(n_seq, "n_seq")))


@_on_stream
def _route_balance(dev, stream, logits, idx, T, E, k, seq_offsets, S, mask, out, ws):
    if out is None:
        f32, i32 = torch.float32, torch.int32
        out = RouteBalance(torch.empty((S,), dtype=f32, device=dev), torch.empty((S,), dtype=f32, device=dev),
                           torch.empty((S, E), dtype=i32, device=dev),
                           torch.empty((S, E), dtype=f32, device=dev), torch.empty((S,), dtype=i32, device=dev))
    wp, wn, keep = _scratch(lib().moe_route_balance_workspace_bytes(T, E, S), ws, dev)
    balance, z, counts, prob_sum, n_tokens = out
    _check(lib().moe_route_balance(logits.data_ptr(), idx.data_ptr(), T, E, k, _addr(seq_offsets), S,
                                   _addr(mask), balance.data_ptr(), z.data_ptr(), counts.data_ptr(),
                                   prob_sum.data_ptr(), n_tokens.data_ptr(), wp, wn, stream),
           "moe_route_balance")
    return out


def route_balance(logits, idx, seq_offsets=None, mask=None, out: Optional[RouteBalance] = None,
                  ws=None, stream=None) -> RouteBalance:
    """The router's balance and z losses, per-expert counts and probability
    sums, per sequence (moe_route_balance).  logits fp32 [T, E], idx int32
    [T, k], seq_offsets int32 [S + 1] (None: one sequence of all rows), mask
    uint8 or bool [T] (0: the row takes no part)."""
    T, E, k, S = _balance_args(logits, idx, seq_offsets, mask)
    if out is not None:
        want = (((S,), torch.float32), ((S,), torch.float32), ((S, E), torch.int32),
                ((S, E), torch.float32), ((S,), torch.int32))
        for t, (shp, dt), name in zip(out, want, RouteBalance._fields):
            _dev(_shape(t, shp, name), dt, name)
    if ws is not None:
        _dev(ws, torch.uint8, "ws")
    return _route_balance("route_balance", stream, (logits, idx, seq_offsets, mask, ws) + (out or ()),
                          logits, idx, T, E, k, seq_offsets, S, mask, out, ws)


@_on_stream
def _route_backward(dev, stream, logits, idx, T, E, k, seq_offsets, S, mask, counts, n_tokens,
                    g_balance, g_z, w, dw, dlogits):
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=torch.float32, device=dev)
    _check(lib().moe_route_backward(logits.data_ptr(), idx.data_ptr(), T, E, k, _addr(seq_offsets), S,
                                    _addr(mask), _addr(counts), _addr(n_tokens), _addr(g_balance),
                                    _addr(g_z), _addr(w), _addr(dw), dlogits.data_ptr(), stream),
           "moe_route_backward")
    return dlogits


def route_backward(logits, idx, counts=None, n_tokens=None, g_balance=None, g_z=None, w=None,
                   dw=None, seq_offsets=None, mask=None, dlogits=None, stream=None):
    """Gradient of the router's logits from those of the two losses (g_balance,
    g_z fp32 [S]) and of the routing weights (dw fp32 [T, k], with w as
    route_topk gave it) (moe_route_backward).  counts and n_tokens as
    route_balance returns them.  Returns dlogits fp32 [T, E]."""
    T, E, k, S = _balance_args(logits, idx, seq_offsets, mask)
    checks = ((counts, (S, E), torch.int32, "counts"), (n_tokens, (S,), torch.int32, "n_tokens"),
              (g_balance, (S,), torch.float32, "g_balance"), (g_z, (S,), torch.float32, "g_z"),
              (w, (T, k), torch.float32, "w"), (dw, (T, k), torch.float32, "dw"),
              (dlogits, (T, E), torch.float32, "dlogits"))
    for t, shp, dt, name in checks:
        if t is not None:
            _dev(_shape(t, shp, name), dt, name)
    return _route_backward("route_backward", stream,
                           (logits, idx, seq_offsets, mask, counts, n_tokens, g_balance, g_z, w, dw, dlogits),
                           logits, idx, T, E, k, seq_offsets, S, mask, counts, n_tokens, g_balance, g_z,
                           w, dw, dlogits)
