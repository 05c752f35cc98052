"""Routed mixture-of-experts FFN layer for AMD MI355X (gfx950).

A thin ctypes binding over ``libcoli_moe.so`` -- the C ABI declared in
``include/coli_moe.h``.  Every step of the layer runs in the library's HIP
kernels; this module only marshals arguments (device pointers taken from
torch tensors, sizes, the current HIP stream) and turns error codes into
exceptions.  PyTorch provides device memory and streams, nothing else.

The entry points keep the C names:

  coli_moe_workspace_bytes(shape, int4=False) -> int
  coli_moe_route(shape, x, w_router, bias, routing, ws, stream=None)
  coli_moe_ffn(shape, x, routing, weights, y, residual=None, y_bf16=None, ws, stream=None)
  coli_moe_ffn_int4(shape, x, routing, weights_int4, y, residual=None, y_bf16=None, ws, stream=None)
  coli_moe_dense_workspace_bytes(shape) -> int
  coli_moe_dense_ffn(shape, x, dense_weights, y, residual=None, y_bf16=None, ws, stream=None)
  coli_moe_bank_fill(shape, host_tensors, bank_tensors, experts=None, int4=False, group=32,
                     copy_stream, wait_event=None, ready_event=None)
  coli_moe_bank_acquire(compute_stream, ready_event) / coli_moe_bank_release(compute_stream, free_event)
  coli_index_topk_workspace_bytes(rows, L, k) -> int
  coli_index_topk(scores, k, idx, tail=0, lens=None, ws=None, stream=None)
  coli_kv_append(shape, k_new, v_new, cache, start=None, stream=None)
  coli_kv_attn_workspace_bytes(shape, idx_k=0, acc=False) -> int
  coli_kv_attn(shape, q, cache, out, scale, idx=None, acc_in=None, acc_out=None, lse=None, ws, stream=None)
  coli_kv_evict(shape, cache, acc, k, new_table, new_lens, kept, tail=0, new_acc=None, stream=None)
  coli_kv_attn_shared_workspace_bytes(shape, n_groups) -> int
  coli_kv_attn_shared(shape, q, cache, out, scale, shared, group_start, lse=None, ws, stream=None)
  coli_kv_plan(shape, table, lens, want, ring, state, start, slot, pos, shared=None, new_lens=None,
               new_state=None, stream=None)
  coli_rope_freqs(rot, base=10000.0, scaling="plain", factor=1.0, length=4096) -> (freq, amp)
  coli_kv_rope(shape, q, k, v, q_out, pos=None, rope=None, norm=None, k_out=None, pool_k=None, pool_v=None,
               slot=None, stream=None)
  coli_moe_status_str(code) -> str

If the library has not been built the import still works, but every call
raises ``ColiError`` -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcoli_moe.so")

COLI_F32, COLI_BF16 = 0, 1
STATUS_NAMES = {0: "COLI_OK", 1: "COLI_E_NULL", 2: "COLI_E_SHAPE", 3: "COLI_E_DTYPE",
                4: "COLI_E_ALIGN", 5: "COLI_E_WORKSPACE", 6: "COLI_E_DEVICE",
                7: "COLI_E_LAUNCH", 8: "COLI_E_ALIAS", 9: "COLI_E_MEMORY"}
EXPORTED = ("coli_moe_workspace_bytes", "coli_moe_route", "coli_moe_ffn", "coli_moe_ffn_int4",
            "coli_moe_route_timed", "coli_moe_ffn_timed", "coli_moe_ffn_int4_timed",
            "coli_moe_dense_workspace_bytes", "coli_moe_dense_ffn",
            "coli_moe_bank_fill", "coli_moe_bank_acquire", "coli_moe_bank_release",
            "coli_index_topk_workspace_bytes", "coli_index_topk", "coli_moe_ffn_noalloc",
            "coli_kv_append", "coli_kv_attn_workspace_bytes", "coli_kv_attn", "coli_kv_evict",
            "coli_kv_plan", "coli_rope_freqs", "coli_kv_rope",
            "coli_kv_attn_shared_workspace_bytes", "coli_kv_attn_shared",
            "coli_moe_status_str", "coli_moe_version")
ROUTE_STAGES = ("router", "topk", "perm")
FFN_STAGES = ("gate_up", "down", "combine")


class ColiError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {STATUS_NAMES.get(code, code)}"
        try:
            msg += f" ({coli_moe_status_str(code)})"
        except Exception:   # library missing: keep the code only
            pass
        super().__init__(msg)


class CShape(C.Structure):
    _fields_ = [("T", C.c_int32), ("D", C.c_int32), ("E", C.c_int32), ("K", C.c_int32),
                ("F", C.c_int32), ("dtype", C.c_int32)]


class CRouting(C.Structure):
    _fields_ = [("ids", C.c_void_p), ("w", C.c_void_p), ("count", C.c_void_p),
                ("offset", C.c_void_p), ("perm", C.c_void_p), ("inv", C.c_void_p)]


class CWeights(C.Structure):
    _fields_ = [("gate", C.c_void_p), ("up", C.c_void_p), ("down", C.c_void_p),
                ("s_gate", C.c_void_p), ("s_up", C.c_void_p), ("s_down", C.c_void_p)]


class CWeightsInt4(C.Structure):
    _fields_ = [("gate_q", C.c_void_p), ("up_q", C.c_void_p), ("down_q", C.c_void_p),
                ("gate_s", C.c_void_p), ("up_s", C.c_void_p), ("down_s", C.c_void_p),
                ("group", C.c_int32),
                ("s_gate", C.c_void_p), ("s_up", C.c_void_p), ("s_down", C.c_void_p)]


class CDenseWeights(C.Structure):
    _fields_ = [("gate", C.c_void_p), ("up", C.c_void_p), ("down", C.c_void_p)]


class CKvShape(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("B", "Hq", "Hkv", "Dk", "Dv", "page", "n_pages", "max_pages", "dtype")]


class CKvCache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("table", C.c_void_p), ("lens", C.c_void_p)]


class CQkNorm(C.Structure):
    _fields_ = [("q_w", C.c_void_p), ("k_w", C.c_void_p), ("width", C.c_int32), ("eps", C.c_float)]


class CRope(C.Structure):
    _fields_ = [("freq", C.c_void_p), ("rot", C.c_int32), ("rot_at", C.c_int32), ("interleaved", C.c_int32), ("amp", C.c_float)]


_lib = None


def lib():
    """Load libcoli_moe.so (raises ColiError-like RuntimeError if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                               "(there is no fallback implementation)")
        L = C.CDLL(LIB_PATH)
        vp, sz = C.c_void_p, C.c_size_t
        sp = C.POINTER(CShape)
        L.coli_moe_workspace_bytes.restype = sz
        L.coli_moe_workspace_bytes.argtypes = [sp, C.c_int]
        L.coli_moe_route.restype = C.c_int
        L.coli_moe_route.argtypes = [sp, vp, vp, vp, C.POINTER(CRouting), vp, sz, vp]
        L.coli_moe_ffn.restype = C.c_int
        L.coli_moe_ffn.argtypes = [sp, vp, C.POINTER(CRouting), C.POINTER(CWeights), vp, vp, vp,
                                   vp, sz, vp]
        L.coli_moe_ffn_int4.restype = C.c_int
        L.coli_moe_ffn_int4.argtypes = [sp, vp, C.POINTER(CRouting), C.POINTER(CWeightsInt4),
                                        vp, vp, vp, vp, sz, vp]
        ev = C.POINTER(C.c_void_p)
        L.coli_moe_route_timed.restype = C.c_int
        L.coli_moe_route_timed.argtypes = L.coli_moe_route.argtypes + [ev, C.c_int32]
        L.coli_moe_ffn_timed.restype = C.c_int
        L.coli_moe_ffn_timed.argtypes = L.coli_moe_ffn.argtypes + [ev, C.c_int32]
        L.coli_moe_ffn_int4_timed.restype = C.c_int
        L.coli_moe_ffn_int4_timed.argtypes = L.coli_moe_ffn_int4.argtypes + [ev, C.c_int32]
        L.coli_moe_dense_workspace_bytes.restype = sz
        L.coli_moe_dense_workspace_bytes.argtypes = [sp]
        L.coli_moe_dense_ffn.restype = C.c_int
        L.coli_moe_dense_ffn.argtypes = [sp, vp, C.POINTER(CDenseWeights), vp, vp, vp, vp, sz, vp]
        L.coli_moe_bank_fill.restype = C.c_int
        L.coli_moe_bank_fill.argtypes = [sp, C.c_int32, C.c_int32, C.POINTER(C.c_void_p),
                                         C.POINTER(C.c_void_p), C.POINTER(C.c_int32), C.c_int32,
                                         vp, vp, vp]
        L.coli_moe_bank_acquire.restype = C.c_int
        L.coli_moe_bank_acquire.argtypes = [vp, vp]
        L.coli_moe_bank_release.restype = C.c_int
        L.coli_moe_bank_release.argtypes = [vp, vp]
        L.coli_index_topk_workspace_bytes.restype = sz
        L.coli_index_topk_workspace_bytes.argtypes = [C.c_int32, C.c_int32, C.c_int32]
        L.coli_index_topk.restype = C.c_int
        L.coli_index_topk.argtypes = [vp, C.c_int32, C.c_int32, C.c_int64, vp, C.c_int32, C.c_int32,
                                      vp, vp, sz, vp]
        L.coli_moe_ffn_noalloc.restype = C.c_int
        L.coli_moe_ffn_noalloc.argtypes = [sp, vp, C.POINTER(CRouting), C.POINTER(CWeights), vp, vp,
                                           vp, vp]
        kp, cp, i32, i64 = C.POINTER(CKvShape), C.POINTER(CKvCache), C.c_int32, C.c_int64
        L.coli_kv_append.restype = C.c_int
        L.coli_kv_append.argtypes = [kp, vp, vp, i32, vp, cp, vp]
        L.coli_kv_attn_workspace_bytes.restype = sz
        L.coli_kv_attn_workspace_bytes.argtypes = [kp, i32, i32]
        L.coli_kv_attn.restype = C.c_int
        L.coli_kv_attn.argtypes = [kp, vp, cp, C.c_float, vp, i32, vp, vp, i64, vp, vp, vp, sz, vp]
        L.coli_kv_evict.restype = C.c_int
        L.coli_kv_evict.argtypes = [kp, cp, vp, i64, i32, i32, vp, i32, vp, vp, vp, i64, vp]
        L.coli_kv_plan.restype = C.c_int
        L.coli_kv_plan.argtypes = [kp] + [vp] * 9 + [i32, vp, vp, vp]
        L.coli_kv_attn_shared_workspace_bytes.restype = sz
        L.coli_kv_attn_shared_workspace_bytes.argtypes = [kp, i32]
        L.coli_kv_attn_shared.restype = C.c_int
        L.coli_kv_attn_shared.argtypes = [kp, vp, cp, C.c_float, vp, vp, i32, vp, vp, vp, sz, vp]
        f64 = C.c_double
        L.coli_rope_freqs.restype = C.c_int
        L.coli_rope_freqs.argtypes = [i32, f64, i32, f64, f64, C.POINTER(f64), C.POINTER(C.c_float)]
        L.coli_kv_rope.restype = C.c_int
        L.coli_kv_rope.argtypes = [kp, i32, vp, i64, vp, i64, vp, i64, C.POINTER(CQkNorm), C.POINTER(CRope)] + [vp] * 7
        L.coli_moe_status_str.restype = C.c_char_p
        L.coli_moe_status_str.argtypes = [C.c_int]
        L.coli_moe_version.restype = C.c_int32
        L.coli_moe_version.argtypes = []
        _lib = L
    return _lib


# ---------------------------------------------------------------------------
# argument containers
# ---------------------------------------------------------------------------

@dataclass
class Shape:
    T: int
    D: int
    E: int
    K: int
    F: int
    dtype: int = COLI_BF16

    def c(self) -> CShape:
        return CShape(self.T, self.D, self.E, self.K, self.F, self.dtype)


def _ptr(t) -> Optional[int]:
    """Device pointer of a tensor (None stays NULL; ints pass through)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the C ABI must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        # the current stream's handle alone (a Stream object around it costs 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


@dataclass
class Routing:
    """Routing tensors (device, int32 / fp32), see coli_moe_routing."""
    ids: object
    w: object
    count: object
    offset: object
    perm: object
    inv: object

    @staticmethod
    def empty(T: int, E: int, K: int, device="cuda"):
        import torch
        i32 = dict(dtype=torch.int32, device=device)
        return Routing(ids=torch.empty((T, K), **i32),
                       w=torch.empty((T, K), dtype=torch.float32, device=device),
                       count=torch.empty(E, **i32), offset=torch.empty(E + 1, **i32),
                       perm=torch.empty(T * K, **i32), inv=torch.empty(T * K, **i32))

    def c(self) -> CRouting:
        return CRouting(*[_ptr(getattr(self, k)) for k in
                          ("ids", "w", "count", "offset", "perm", "inv")])


@dataclass
class Weights:
    gate: object
    up: object
    down: object
    s_gate: object
    s_up: object
    s_down: object

    def c(self) -> CWeights:
        return CWeights(*[_ptr(getattr(self, k)) for k in
                          ("gate", "up", "down", "s_gate", "s_up", "s_down")])


@dataclass
class WeightsInt4:
    gate_q: object
    up_q: object
    down_q: object
    gate_s: object
    up_s: object
    down_s: object
    group: int
    s_gate: object
    s_up: object
    s_down: object

    def c(self) -> CWeightsInt4:
        return CWeightsInt4(_ptr(self.gate_q), _ptr(self.up_q), _ptr(self.down_q),
                            _ptr(self.gate_s), _ptr(self.up_s), _ptr(self.down_s), self.group,
                            _ptr(self.s_gate), _ptr(self.s_up), _ptr(self.s_down))


def _check(code: int, where: str):
    if code != 0:
        raise ColiError(code, where)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def coli_moe_status_str(code: int) -> str:
    return lib().coli_moe_status_str(code).decode()


def coli_moe_version() -> int:
    return lib().coli_moe_version()


def coli_moe_workspace_bytes(shape: Shape, int4: bool = False) -> int:
    cs = shape.c()
    return lib().coli_moe_workspace_bytes(C.byref(cs), 1 if int4 else 0)


def _nbytes(ws, ws_bytes):
    if ws_bytes is not None:
        return ws_bytes
    return ws.numel() * ws.element_size() if ws is not None else 0


def _events(events):
    """A list of hipEvent_t handles (ints) -> (void** array, count); None -> (None, 0)."""
    if not events:
        return None, 0
    arr = (C.c_void_p * len(events))(*events)
    return arr, len(events)


def coli_moe_route(shape: Shape, x, w_router, bias, routing: Routing, ws, ws_bytes=None,
                   stream=None, events=None) -> None:
    """Route T tokens; ``events`` (hipEvent_t handles) selects the timed variant."""
    cs, cr = shape.c(), routing.c()
    args = [C.byref(cs), _ptr(x), _ptr(w_router), _ptr(bias), C.byref(cr), _ptr(ws),
            _nbytes(ws, ws_bytes), _stream(stream)]
    if events:
        _check(lib().coli_moe_route_timed(*args, *_events(events)), "coli_moe_route_timed")
    else:
        _check(lib().coli_moe_route(*args), "coli_moe_route")


def coli_moe_ffn(shape: Shape, x, routing: Routing, weights: Weights, y, residual=None,
                 y_bf16=None, ws=None, ws_bytes=None, stream=None, events=None) -> None:
    cs, cr, cw = shape.c(), routing.c(), weights.c()
    args = [C.byref(cs), _ptr(x), C.byref(cr), C.byref(cw), _ptr(residual), _ptr(y),
            _ptr(y_bf16), _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)]
    if events:
        _check(lib().coli_moe_ffn_timed(*args, *_events(events)), "coli_moe_ffn_timed")
    else:
        _check(lib().coli_moe_ffn(*args), "coli_moe_ffn")


def coli_moe_ffn_int4(shape: Shape, x, routing: Routing, weights: WeightsInt4, y, residual=None,
                      y_bf16=None, ws=None, ws_bytes=None, stream=None, events=None) -> None:
    cs, cr, cw = shape.c(), routing.c(), weights.c()
    args = [C.byref(cs), _ptr(x), C.byref(cr), C.byref(cw), _ptr(residual), _ptr(y),
            _ptr(y_bf16), _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)]
    if events:
        _check(lib().coli_moe_ffn_int4_timed(*args, *_events(events)), "coli_moe_ffn_int4_timed")
    else:
        _check(lib().coli_moe_ffn_int4(*args), "coli_moe_ffn_int4")


# ---------------------------------------------------------------------------
# dense FFN layers, the expert bank, index selection
# ---------------------------------------------------------------------------

@dataclass
class DenseWeights:
    gate: object
    up: object
    down: object

    def c(self) -> CDenseWeights:
        return CDenseWeights(_ptr(self.gate), _ptr(self.up), _ptr(self.down))


def coli_moe_dense_workspace_bytes(shape: Shape) -> int:
    cs = shape.c()
    return lib().coli_moe_dense_workspace_bytes(C.byref(cs))


def coli_moe_dense_ffn(shape: Shape, x, weights: DenseWeights, y, residual=None, y_bf16=None,
                       ws=None, ws_bytes=None, stream=None) -> None:
    cs, cw = shape.c(), weights.c()
    _check(lib().coli_moe_dense_ffn(C.byref(cs), _ptr(x), C.byref(cw), _ptr(residual), _ptr(y),
                                    _ptr(y_bf16), _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)),
           "coli_moe_dense_ffn")


def _event_handle(ev, record_on=None):
    """torch.cuda.Event (or a raw hipEvent_t int, or None) -> handle.

    torch creates an event's handle when it is first recorded.  An event the
    library will record (record_on = that stream) is recorded there once
    first, which creates it; an event to wait for that was never recorded has
    nothing to wait for and is passed as NULL."""
    if ev is None or isinstance(ev, int):
        return ev
    if ev.cuda_event == 0:
        if record_on is None:
            return None
        ev.record(record_on)
    return ev.cuda_event


def coli_moe_bank_fill(shape: Shape, host, bank, experts=None, int4: bool = False, group: int = 32,
                       copy_stream=None, wait_event=None, ready_event=None) -> None:
    """Copy the listed experts (host ints; None = all) of `host` tensors (pinned) into `bank`."""
    n_t = 6 if int4 else 3
    if len(host) != n_t or len(bank) != n_t:
        raise ValueError(f"{n_t} tensors expected")
    cs = shape.c()
    h = (C.c_void_p * n_t)(*[_ptr(t) for t in host])
    b = (C.c_void_p * n_t)(*[_ptr(t) for t in bank])
    if experts is None:
        ex, n = None, 0
    else:
        ex = (C.c_int32 * len(experts))(*[int(e) for e in experts])
        n = len(experts)
    import torch
    cstream = copy_stream if copy_stream is not None else torch.cuda.current_stream()
    _check(lib().coli_moe_bank_fill(C.byref(cs), 1 if int4 else 0, group, h, b, ex, n,
                                    _stream(cstream), _event_handle(wait_event),
                                    _event_handle(ready_event, cstream)), "coli_moe_bank_fill")


def coli_moe_bank_acquire(compute_stream, ready_event) -> None:
    _check(lib().coli_moe_bank_acquire(_stream(compute_stream), _event_handle(ready_event)),
           "coli_moe_bank_acquire")


def coli_moe_bank_release(compute_stream, free_event) -> None:
    import torch
    cstream = compute_stream if compute_stream is not None else torch.cuda.current_stream()
    _check(lib().coli_moe_bank_release(_stream(cstream), _event_handle(free_event, cstream)),
           "coli_moe_bank_release")


def coli_index_topk_workspace_bytes(rows: int, L: int, k: int) -> int:
    return lib().coli_index_topk_workspace_bytes(rows, L, k)


def coli_index_topk(scores, k: int, idx, tail: int = 0, lens=None, ws=None, ws_bytes=None,
                    stream=None, L: Optional[int] = None, ld: Optional[int] = None) -> None:
    """scores: fp32 [rows][ld] device tensor (L columns used); idx: int32 [rows][k]."""
    rows = scores.shape[0]
    ld = scores.stride(0) if ld is None else ld
    L = scores.shape[1] if L is None else L
    _check(lib().coli_index_topk(scores.data_ptr(), rows, L, ld, _ptr(lens), k, tail, _ptr(idx),
                                 _ptr(ws), _nbytes(ws, ws_bytes), _stream(stream)),
           "coli_index_topk")


# ---------------------------------------------------------------------------
# the paged key-value cache
# ---------------------------------------------------------------------------

@dataclass(frozen=True)
class KvShape:
    """Sizes of a paged cache and of the calls on it, see coli_kv_shape."""
    B: int
    Hq: int
    Hkv: int
    Dk: int
    Dv: int
    page: int
    n_pages: int
    max_pages: int
    dtype: int = COLI_BF16

    def __getstate__(self):
        # a copy forms its own C form
        return {n: v for n, v in self.__dict__.items() if n != "_ref"}

    def c(self) -> CKvShape:
        return CKvShape(self.B, self.Hq, self.Hkv, self.Dk, self.Dv, self.page, self.n_pages, self.max_pages,
                        self.dtype)


@dataclass(frozen=True)
class KvCache:
    """The pools, the page table and the lengths (device tensors), see
    coli_kv_cache.  v None: a latent cache.  A handle that a program makes once
    and uses in every step; its tensors are written in place (lens and table
    change from step to step)."""
    k: object
    v: object
    table: object
    lens: object

    def __getstate__(self):
        # a copy holds the tensors and not what calls have formed from them
        return {n: v for n, v in self.__dict__.items() if n != "_handles"}

    def c(self) -> CKvCache:
        return CKvCache(_ptr(self.k), _ptr(self.v), _ptr(self.table), _ptr(self.lens))


def _kv_arg(where: str, at: int, name: str, t, dtype, size) -> Optional[int]:
    """Address of an argument (None: none).  The C ABI takes addresses only, so types, sizes, order and device numbers
    are checked here."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != size:
        raise ValueError(f"{where}: {name} must be {dtype} {list(size)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != at:
        raise ValueError(f"{where}: {name} is on {t.device}, the cache on device {at}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")
    return t.data_ptr()


def _shape_ref(shape: KvShape):
    """Reference to a shape's C form, formed once (a shape's fields do not change)."""
    ref = shape.__dict__.get("_ref")
    if ref is None:
        ref = C.byref(shape.c())
        object.__setattr__(shape, "_ref", ref)
    return ref


def _kv_handles(where: str, shape: KvShape, cache: KvCache):
    """The C forms of a shape and a cache and what calls on them share: (shape, cache, dtype, device number, torch).
    Checked and formed once for a pair of handles, and kept in the cache's until a tensor's memory, type, sizes or order
    is another one (its methods can change them in place)."""
    kept = cache.__dict__.get("_handles")
    k, v, table, lens = cache.k, cache.v, cache.table, cache.lens
    now = (k.data_ptr(), k.dtype, k.shape, k.is_contiguous(), table.data_ptr(), table.dtype, table.shape, table.is_contiguous(),
           lens.data_ptr(), lens.dtype, lens.shape, lens.is_contiguous(),
           None if v is None else (v.data_ptr(), v.dtype, v.shape, v.is_contiguous()))
    if kept is not None and kept[0] is shape and kept[2] == now:
        return kept[1]
    import torch
    dt, i32, at = torch.float32 if shape.dtype == COLI_F32 else torch.bfloat16, torch.int32, k.get_device()
    pool = (shape.n_pages, shape.Hkv, shape.page)
    c = CKvCache(_kv_arg(where, at, "cache.k", k, dt, pool + (shape.Dk,)), _kv_arg(where, at, "cache.v", v, dt, pool + (shape.Dv,)),
                 _kv_arg(where, at, "cache.table", table, i32, (shape.B, shape.max_pages)),
                 _kv_arg(where, at, "cache.lens", lens, i32, (shape.B,)))
    if k.device.type != "cuda":
        raise ValueError(f"{where}: the cache must be on a GPU, not on {k.device}")
    got = (C.byref(shape.c()), C.byref(c), dt, at, torch)
    object.__setattr__(cache, "_handles", (shape, got, now))
    return got


def _kv_call(torch, where: str, at: int, stream, *args) -> None:
    """The library's function with the cache's device as the current one, on its current stream where `stream` is None."""
    f = getattr(lib(), where)
    if torch._C._cuda_getDevice() == at:          # (the cache is on a GPU: the runtime is up)
        code = f(*args, torch._C._cuda_getCurrentRawStream(at) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(at):
            code = f(*args, _stream(stream))
    if code:
        _check(code, where)


def coli_kv_append(shape: KvShape, k_new, v_new, cache: KvCache, start=None, stream=None) -> None:
    """k_new [rows][Hkv][Dk], v_new [rows][Hkv][Dv] (None for a latent cache); start int32 [B + 1] or None."""
    me = "coli_kv_append"
    cs, cc, dt, at, torch = _kv_handles(me, shape, cache)
    rows, H = k_new.shape[0], shape.Hkv
    _kv_call(torch, me, at, stream, cs, _kv_arg(me, at, "k_new", k_new, dt, (rows, H, shape.Dk)),
             _kv_arg(me, at, "v_new", v_new, dt, (rows, H, shape.Dv)), rows,
             _kv_arg(me, at, "start", start, torch.int32, (shape.B + 1,)), cc)


def coli_kv_attn_workspace_bytes(shape: KvShape, idx_k: int = 0, acc: bool = False) -> int:
    cs = shape.c()
    return lib().coli_kv_attn_workspace_bytes(C.byref(cs), idx_k, 1 if acc else 0)


def coli_kv_attn(shape: KvShape, q, cache: KvCache, out, scale: float, idx=None, acc_in=None, acc_out=None, lse=None,
                 ws=None, ws_bytes=None, stream=None) -> None:
    """q [B][Hq][Dk], out [B][Hq][Dv], lse fp32 [B][Hq], idx int32 [B][idx_k], acc fp32 [B][Hkv][ld]."""
    me = "coli_kv_attn"
    cs, cc, dt, at, torch = _kv_handles(me, shape, cache)
    B, Hq, H, f32 = shape.B, shape.Hq, shape.Hkv, torch.float32
    ld = 0 if acc_out is None else acc_out.shape[-1]
    idx_k = 0 if idx is None else idx.shape[-1]
    # an empty tensor has no address, and without one the argument would count as absent
    if (idx is not None and idx_k == 0) or (acc_out is not None and ld == 0):
        raise ValueError("coli_kv_attn: idx and acc_out must not be empty")
    if ws is not None and ws.get_device() != at:
        raise ValueError(f"coli_kv_attn: ws is on {ws.device}, the cache on device {at}")
    _kv_call(torch, me, at, stream, cs, _kv_arg(me, at, "q", q, dt, (B, Hq, shape.Dk)), cc, scale,
             _kv_arg(me, at, "idx", idx, torch.int32, (B, idx_k)), idx_k, _kv_arg(me, at, "acc_in", acc_in, f32, (B, H, ld)),
             _kv_arg(me, at, "acc_out", acc_out, f32, (B, H, ld)), ld, _kv_arg(me, at, "out", out, dt, (B, Hq, shape.Dv)),
             _kv_arg(me, at, "lse", lse, f32, (B, Hq)), _ptr(ws), _nbytes(ws, ws_bytes))


def coli_kv_attn_shared_workspace_bytes(shape: KvShape, n_groups: int) -> int:
    cs = shape.c()
    return lib().coli_kv_attn_shared_workspace_bytes(C.byref(cs), n_groups)


def coli_kv_attn_shared(shape: KvShape, q, cache: KvCache, out, scale: float, shared, group_start, lse=None, ws=None, ws_bytes=None,
                        stream=None) -> None:
    """q [B][Hq][Dk], out [B][Hq][Dv], lse fp32 [B][Hq], shared int32 [B], group_start int32 [n_groups + 1]."""
    me = "coli_kv_attn_shared"
    cs, cc, dt, at, torch = _kv_handles(me, shape, cache)
    B, Hq, i32, groups = shape.B, shape.Hq, torch.int32, () if group_start is None else group_start.shape
    if len(groups) != 1 or groups[0] < 1:
        raise ValueError(f"{me}: group_start must have one dimension and at least one entry")
    if ws is not None and ws.get_device() != at:
        raise ValueError(f"{me}: ws is on {ws.device}, the cache on device {at}")
    _kv_call(torch, me, at, stream, cs, _kv_arg(me, at, "q", q, dt, (B, Hq, shape.Dk)), cc, scale,
             _kv_arg(me, at, "shared", shared, i32, (B,)), _kv_arg(me, at, "group_start", group_start, i32, groups), groups[0] - 1,
             _kv_arg(me, at, "out", out, dt, (B, Hq, shape.Dv)), _kv_arg(me, at, "lse", lse, torch.float32, (B, Hq)), _ptr(ws),
             _nbytes(ws, ws_bytes))


def coli_kv_evict(shape: KvShape, cache: KvCache, acc, k: int, new_table, new_lens, kept, tail: int = 0, new_acc=None,
                  stream=None) -> None:
    """acc fp32 [B][Hkv][ld], new_table int32 [B][pages], new_lens int32 [B], kept int32 [B][Hkv][k],
    new_acc fp32 [B][Hkv][new_ld]."""
    me = "coli_kv_evict"
    cs, cc, _, at, torch = _kv_handles(me, shape, cache)
    B, H, f32, i32 = shape.B, shape.Hkv, torch.float32, torch.int32
    ld, cols = acc.shape[-1], new_table.shape[-1]
    new_ld = 0 if new_acc is None else new_acc.shape[-1]
    if new_acc is not None and new_ld == 0:
        raise ValueError("coli_kv_evict: new_acc must not be empty")
    _kv_call(torch, me, at, stream, cs, cc, _kv_arg(me, at, "acc", acc, f32, (B, H, ld)), ld, k, tail,
             _kv_arg(me, at, "new_table", new_table, i32, (B, cols)), cols, _kv_arg(me, at, "new_lens", new_lens, i32, (B,)),
             _kv_arg(me, at, "kept", kept, i32, (B, H, k)), _kv_arg(me, at, "new_acc", new_acc, f32, (B, H, new_ld)), new_ld)


def coli_kv_plan(shape: KvShape, table, lens, want, ring, state, start, slot, pos, shared=None, new_lens=None, new_state=None,
                 stream=None) -> None:
    """All int32 on one GPU: table [B][max_pages], lens, want, shared and new_lens [B], ring [n_pages], state and new_state
    [4], start [B + 1], slot and pos [rows].  new_lens or new_state None: lens or state is written in place.  shared: pages
    that other sequences read too; it stays when a sequence ends, until the last of them passes 0 and gives them back."""
    me = "coli_kv_plan"
    import torch
    if ring is None or slot is None:
        raise ValueError(f"{me}: ring and slot must be given")
    i32, arg, at, B, rows = torch.int32, _kv_arg, ring.get_device(), (shape.B,), slot.shape
    if at < 0:
        raise ValueError(f"{me}: ring must be on a GPU, not on {ring.device}")
    if len(rows) != 1:
        raise ValueError(f"{me}: slot must have one dimension")
    plens, pstate = arg(me, at, "lens", lens, i32, B), arg(me, at, "state", state, i32, (4,))
    _kv_call(torch, me, at, stream, _shape_ref(shape), arg(me, at, "table", table, i32, (shape.B, shape.max_pages)), plens,
             arg(me, at, "want", want, i32, B), arg(me, at, "shared", shared, i32, B), arg(me, at, "ring", ring, i32, (shape.n_pages,)),
             pstate, plens if new_lens is None else arg(me, at, "new_lens", new_lens, i32, B),
             pstate if new_state is None else arg(me, at, "new_state", new_state, i32, (4,)),
             arg(me, at, "start", start, i32, (shape.B + 1,)), rows[0], arg(me, at, "slot", slot, i32, rows),
             arg(me, at, "pos", pos, i32, rows))


ROPE_SCALINGS = ("plain", "linear", "ntk", "yarn")


def coli_rope_freqs(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, length: float = 4096):
    """The angle per position of each pair (float64 tensor [rot / 2] on the CPU) and the factor on cosines and sines.
    "yarn" blends by turns; a checkpoint that was trained with a blend by the pair's index, or with other borders or
    another amplitude, needs a table of its own (Rope takes any)."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"coli_rope_freqs: scaling must be one of {ROPE_SCALINGS}, got {scaling!r}")
    freq, amp = (C.c_double * max(rot // 2, 1))(), C.c_float()
    _check(lib().coli_rope_freqs(rot, base, ROPE_SCALINGS.index(scaling), factor, length, freq, C.byref(amp)), "coli_rope_freqs")
    return torch.tensor(list(freq), dtype=torch.float64), amp.value


@dataclass(frozen=True)
class Rope:
    """Rotation by positions, see coli_rope.  freq: float64 on the GPU, one of each pair; 2 * its length elements of a
    head are rotated, from rot_at on."""
    freq: object
    rot_at: int = 0
    interleaved: bool = False
    amp: float = 1.0

    def c(self, where: str, at: int, f64) -> CRope:
        n = self.freq.shape
        if len(n) != 1:
            raise ValueError(f"{where}: rope.freq must have one dimension")
        return CRope(_kv_arg(where, at, "rope.freq", self.freq, f64, n), 2 * n[0], self.rot_at, 1 if self.interleaved else 0, self.amp)


@dataclass(frozen=True)
class QkNorm:
    """Norm of each head's first elements, see coli_qk_norm; as many as the weights have."""
    q_w: object = None
    k_w: object = None
    eps: float = 1e-6

    def c(self, where: str, at: int, dt) -> CQkNorm:
        n = (self.k_w if self.q_w is None else self.q_w).shape
        if len(n) != 1:
            raise ValueError(f"{where}: the norm's weights must have one dimension")
        return CQkNorm(_kv_arg(where, at, "norm.q_w", self.q_w, dt, n), _kv_arg(where, at, "norm.k_w", self.k_w, dt, n), n[0], self.eps)


def _kv_rows(where: str, at: int, name: str, t, dtype, size):
    """Address of [rows][heads][width] values and the elements from a row to the next; only whole rows may lie apart."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != size:
        raise ValueError(f"{where}: {name} must be {dtype} {list(size)}, got {t.dtype} {list(t.shape)}")
    if t.get_device() != at:
        raise ValueError(f"{where}: {name} is on {t.device}, the other tensors on device {at}")
    _, H, D = size
    ld, across, along = t.stride()
    if (D > 1 and along != 1) or (H > 1 and across != D):
        raise ValueError(f"{where}: the heads of a row of {name} must lie side by side")
    if size[0] < 2:                                  # (of one row the stride says nothing)
        ld = H * D
    return t.data_ptr(), ld


def coli_kv_rope(shape: KvShape, q, k, v, q_out, pos=None, rope: Optional[Rope] = None, norm: Optional[QkNorm] = None, k_out=None,
                 pool_k=None, pool_v=None, slot=None, stream=None) -> None:
    """q [rows][Hq][Dk], k [rows][Hkv][Dk], v [rows][Hkv][Dv] (slices of a wider tensor may be passed), q_out and k_out of
    their sizes, pos and slot int32 [rows], the cache's pools."""
    me = "coli_kv_rope"
    import torch
    some = k if q is None else q
    if some is None:
        raise ValueError(f"{me}: q or k must be given")
    at, rows = some.get_device(), some.shape[0]
    if at < 0:
        raise ValueError(f"{me}: the tensors must be on a GPU, not on {some.device}")
    dt, i32, row, arg = torch.float32 if shape.dtype == COLI_F32 else torch.bfloat16, torch.int32, (rows,), _kv_arg
    Hq, H, Dk, Dv = shape.Hq, shape.Hkv, shape.Dk, shape.Dv
    pq, q_ld = _kv_rows(me, at, "q", q, dt, (rows, Hq, Dk))
    pk, k_ld = _kv_rows(me, at, "k", k, dt, (rows, H, Dk))
    pv, v_ld = _kv_rows(me, at, "v", v, dt, (rows, H, Dv))
    cn = None if norm is None or (norm.q_w is None and norm.k_w is None) else C.byref(norm.c(me, at, dt))
    cr = None if rope is None else C.byref(rope.c(me, at, torch.float64))
    _kv_call(torch, me, at, stream, _shape_ref(shape), rows, pq, q_ld, pk, k_ld, pv, v_ld, cn, cr,
             arg(me, at, "pos", pos, i32, row), arg(me, at, "slot", slot, i32, row),
             arg(me, at, "q_out", q_out, dt, (rows, Hq, Dk)), arg(me, at, "k_out", k_out, dt, (rows, H, Dk)),
             arg(me, at, "pool_k", pool_k, dt, (shape.n_pages, H, shape.page, Dk)),
             arg(me, at, "pool_v", pool_v, dt, (shape.n_pages, H, shape.page, Dv)))


NOALLOC_SCRATCH_BYTES = 32 << 20


def coli_moe_ffn_noalloc(shape: Shape, x, routing: Routing, weights: Weights, y, residual=None,
                         y_bf16=None, stream=None) -> None:
    """coli_moe_ffn with the library's own per-GPU scratch array as workspace."""
    cs, cr, cw = shape.c(), routing.c(), weights.c()
    _check(lib().coli_moe_ffn_noalloc(C.byref(cs), _ptr(x), C.byref(cr), C.byref(cw), _ptr(residual),
                                      _ptr(y), _ptr(y_bf16), _stream(stream)), "coli_moe_ffn_noalloc")
