"""Python binding for libengram, the Engram forward path on MI355X (gfx950).

Argument marshalling only: every step of the path runs in the HIP kernels of
``libengram.so``.  PyTorch provides device memory and the current stream;
the functions below check dtypes, devices and shapes, pass raw device
pointers through the C ABI declared in ``include/engram.h`` and raise
``EngramError`` on a non-zero status.  There is no CPU fallback: if the
library is not built, every call raises.

Functions carry the C names:
    engram_hash, engram_gather, engram_wkv, engram_wkv_gathered, engram_gate_add,
    engram_forward, engram_forward_workspace_size, engram_wkv_gathered_scratch_size,
    engram_gate_partials_supported, engram_wkv_gate_partials, engram_gate_from_partials,
    engram_check_geometry,
    engram_wkv_adapters, engram_wkv_adapters_scratch_size, engram_forward_adapted,
    engram_forward_adapted_workspace_size, engram_norm_quant, engram_beam_select,
    engram_beam_select_scratch_size, engram_beam_reorder
plus ``Geometry`` / ``HashTables`` (the C structs), ``Adapters`` (the low-rank
adapters of a layer's projection) and ``EngramLayer``, a holder for one layer's
device tables, weights and workspace.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

__all__ = [
    "Geometry", "HashTables", "EngramError", "EngramLayer", "load", "library_path",
    "engram_check_geometry", "engram_hash", "engram_hash_layers", "engram_gather", "engram_wkv",
    "engram_wkv_gathered", "engram_wkv_gathered_scratch_size",
    "engram_gate_partials_supported", "engram_wkv_gate_partials", "engram_gate_from_partials",
    "engram_gate_add", "engram_forward", "engram_forward_hashed", "engram_forward_workspace_size",
    "Adapters", "engram_wkv_adapters", "engram_wkv_adapters_scratch_size",
    "engram_forward_adapted", "engram_forward_adapted_workspace_size", "engram_norm_quant",
    "engram_beam_select", "engram_beam_select_scratch_size", "engram_beam_reorder",
    "ERRBIT_TOKEN", "ERRBIT_HASH", "ERRBIT_ROW", "ERRBIT_ADAPTER", "ERRBIT_LOGIT",
    "ERRBIT_PARENT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libengram.so")

ERRBIT_TOKEN, ERRBIT_HASH, ERRBIT_ROW = 0x1, 0x2, 0x4
ERRBIT_ADAPTER, ERRBIT_LOGIT, ERRBIT_PARENT = 0x8, 0x10, 0x20
_SCALE_FORMATS = {"e8m0_32": 0, "f32_128": 1, "f32_row": 2}
_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported geometry",
           3: "workspace missing or too small", 4: "HIP runtime error",
           5: "call needs more than the fixed scratch array holds"}
ERR_TOO_LARGE = 5


class EngramError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s failed: %s (status %d)" % (fn, _STATUS.get(status, "?"), status))
        self.status = status


class Geometry(C.Structure):
    _fields_ = [("dim", C.c_int32), ("hc_mult", C.c_int32), ("max_ngram_size", C.c_int32),
                ("n_heads", C.c_int32), ("head_dim", C.c_int32), ("vocab", C.c_int32),
                ("pad_id", C.c_int32), ("reserved", C.c_int32), ("num_embeddings", C.c_int64),
                ("norm_eps", C.c_float), ("reserved2", C.c_int32)]

    @classmethod
    def make(cls, dim, hc_mult, max_ngram_size, n_heads, head_dim, num_embeddings, vocab,
             pad_id=0, norm_eps=1e-6) -> "Geometry":
        return cls(dim, hc_mult, max_ngram_size, n_heads, head_dim, vocab, pad_id, 0,
                   num_embeddings, norm_eps, 0)

    @property
    def n_hash_cols(self) -> int:
        return (self.max_ngram_size - 1) * self.n_heads

    @property
    def K(self) -> int:
        return self.n_hash_cols * self.head_dim

    @property
    def N(self) -> int:
        return self.dim * (self.hc_mult + 1)


class HashTables(C.Structure):
    _fields_ = [("token_map", C.c_void_p), ("mult", C.c_void_p), ("prime", C.c_void_p),
                ("offset", C.c_void_p)]


class _CAdapters(C.Structure):
    _fields_ = [("down", C.c_void_p), ("up", C.c_void_p), ("scale", C.c_void_p),
                ("n", C.c_int32), ("rank", C.c_int32)]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libengram.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libengram.so is not built; run `python -m gram_memory_layer_amd.build`")
    L = C.CDLL(_LIB_PATH)
    P, G, HT = C.c_void_p, C.POINTER(Geometry), C.POINTER(HashTables)
    i32, i64 = C.c_int32, C.c_int64
    L.engram_status_string.restype = C.c_char_p
    L.engram_status_string.argtypes = [C.c_int]
    L.engram_check_geometry.restype = C.c_int
    L.engram_check_geometry.argtypes = [G]
    L.engram_hash.restype = C.c_int
    L.engram_hash.argtypes = [G, HT, P, P, i32, i32, P, P, P]
    L.engram_hash_layers.restype = C.c_int
    L.engram_hash_layers.argtypes = [G, HT, i32, P, P, i32, i32, P, P, P]
    L.engram_gather.restype = C.c_int
    L.engram_gather.argtypes = [G, P, P, P, i64, P, P, P]
    L.engram_wkv.restype = C.c_int
    L.engram_wkv.argtypes = [G, P, P, i64, P, P]
    L.engram_wkv_gathered_scratch_size.restype = C.c_size_t
    L.engram_wkv_gathered_scratch_size.argtypes = [G, i64]
    L.engram_wkv_gathered.restype = C.c_int
    L.engram_wkv_gathered.argtypes = [G, P, P, P, i64, P, P, P, C.c_size_t, P, P]
    L.engram_gate_partials_supported.restype = C.c_int
    L.engram_gate_partials_supported.argtypes = [G, i64]
    L.engram_wkv_gate_partials.restype = C.c_int
    L.engram_wkv_gate_partials.argtypes = [G, P, P, P, i64, P, P, P, P, P, P, P, C.c_size_t, P, P]
    L.engram_gate_from_partials.restype = C.c_int
    L.engram_gate_from_partials.argtypes = [G, P, P, P, P, i64, P, P, P]
    L.engram_gate_add.restype = C.c_int
    L.engram_gate_add.argtypes = [G, P, P, P, P, P, i64, P, P, P]
    L.engram_forward_hashed.restype = C.c_int
    L.engram_forward_hashed.argtypes = [G, P, P, P, P, P, P, P, P, i64, P, P, P, C.c_size_t, P, P]
    L.engram_forward_workspace_size.restype = C.c_size_t
    L.engram_forward_workspace_size.argtypes = [G, i64]
    L.engram_forward.restype = C.c_int
    L.engram_forward.argtypes = [G, HT, P, P, P, P, P, P, P, P, P, i32, i32, P, P, P, C.c_size_t,
                                 P, P]
    L.engram_fixed_scratch_bytes.restype = C.c_size_t
    L.engram_fixed_scratch_bytes.argtypes = []
    L.engram_forward_noalloc.restype = C.c_int
    L.engram_forward_noalloc.argtypes = [G, HT, P, P, P, P, P, P, P, P, P, i32, i32, P, P, P, P]
    A = C.POINTER(_CAdapters)
    L.engram_wkv_adapters_scratch_size.restype = C.c_size_t
    L.engram_wkv_adapters_scratch_size.argtypes = [G, A, i64]
    L.engram_wkv_adapters.restype = C.c_int
    L.engram_wkv_adapters.argtypes = [G, A, P, P, P, i64, P, P, C.c_size_t, P, P]
    L.engram_forward_adapted_workspace_size.restype = C.c_size_t
    L.engram_forward_adapted_workspace_size.argtypes = [G, A, i64]
    L.engram_forward_adapted.restype = C.c_int
    L.engram_forward_adapted.argtypes = [G, HT, A, P, P, P, P, P, P, P, P, P, P, i32, i32, P, P, P,
                                         C.c_size_t, P, P]
    L.engram_norm_quant.restype = C.c_int
    L.engram_norm_quant.argtypes = [P, P, P, i64, i32, C.c_float, i32, P, P, P, P]
    L.engram_beam_select_scratch_size.restype = C.c_size_t
    L.engram_beam_select_scratch_size.argtypes = [i32, i32, i32]
    L.engram_beam_select.restype = C.c_int
    L.engram_beam_select.argtypes = [P, i32, i64, P, P, i32, i32, i32, i32, i32, P, P, P, P, P,
                                     C.c_size_t, P, P]
    L.engram_beam_reorder.restype = C.c_int
    L.engram_beam_reorder.argtypes = [P, P, i32, P, i32, i32, P, P]
    _lib = L
    return L


# ------------------------------------------------------------------ helpers
def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


_Tensor = torch.Tensor


def _dev(t, name, dtype, shape=None, device=None):
    # what nearly every call passes, in a few comparisons; the rest below says what is wrong
    if (type(t) is _Tensor and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape) and (device is None or t.device == device)):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device.type != "cuda":
        raise ValueError("%s must be a device tensor (got %s)" % (name, t.device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    return t


def _check(fn, status):
    if status != 0:
        raise EngramError(fn, status)


def _tables(tables: dict, g: Geometry, device) -> HashTables:
    nc = g.n_hash_cols
    tm = _dev(tables["token_map"], "token_map", torch.int32, (g.vocab,), device)
    mult = _dev(tables["mult"], "mult", torch.uint64, (nc, g.max_ngram_size), device)
    prime = _dev(tables["prime"], "prime", torch.uint64, (nc,), device)
    offset = _dev(tables["offset"], "offset", torch.uint64, (nc,), device)
    return HashTables(tm.data_ptr(), mult.data_ptr(), prime.data_ptr(), offset.data_ptr())


# ------------------------------------------------------------------ C entry points
def engram_check_geometry(g: Geometry) -> int:
    return load().engram_check_geometry(C.byref(g))


def engram_forward_workspace_size(g: Geometry, n_tok: int) -> int:
    return load().engram_forward_workspace_size(C.byref(g), int(n_tok))


def engram_hash(g: Geometry, tables: dict, ids: torch.Tensor, state=None, hash_ids=None, err=None):
    """ids int32 [B, T] -> hash_ids int32 [B, T, n_hash_cols]; `state` int32
    [B, max_ngram_size-1] is read and updated in place (None = fresh)."""
    L = load()
    dev = ids.device
    _dev(ids, "ids", torch.int32, None, dev)
    if ids.dim() != 2:
        raise ValueError("ids must be [B, T]")
    B, T = ids.shape
    ht = _tables(tables, g, dev)
    if state is not None:
        _dev(state, "state", torch.int32, (B, g.max_ngram_size - 1), dev)
    if hash_ids is None:
        hash_ids = torch.empty((B, T, g.n_hash_cols), dtype=torch.int32, device=dev)
    _dev(hash_ids, "hash_ids", torch.int32, (B, T, g.n_hash_cols), dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_hash", L.engram_hash(C.byref(g), C.byref(ht), _ptr(state), ids.data_ptr(), B, T,
                                        hash_ids.data_ptr(), _ptr(err), _stream(dev)))
    return hash_ids


def engram_hash_layers(geoms, tables, ids: torch.Tensor, states=None, hash_ids=None, err=None):
    """Several layers' hashes in one launch: geoms / tables are lists (one
    per layer; only num_embeddings and the tables may differ), ids int32
    [B, T] -> hash_ids int32 [n_layers, B, T, n_hash_cols]; `states` None or a
    list of per-layer int32 [B, max_ngram_size-1] states, updated in place."""
    L = load()
    dev = ids.device
    _dev(ids, "ids", torch.int32, None, dev)
    if ids.dim() != 2:
        raise ValueError("ids must be [B, T]")
    n = len(geoms)
    if len(tables) != n or (states is not None and len(states) != n):
        raise ValueError("one geometry, table set and state per layer")
    B, T = ids.shape
    g0 = geoms[0]
    garr = (Geometry * n)(*geoms)
    tarr = (HashTables * n)(*[_tables(tables[l], geoms[l], dev) for l in range(n)])
    sarr = None
    if states is not None:
        for st in states:
            _dev(st, "state", torch.int32, (B, g0.max_ngram_size - 1), dev)
        sarr = (C.c_void_p * n)(*[st.data_ptr() for st in states])
    if hash_ids is None:
        hash_ids = torch.empty((n, B, T, g0.n_hash_cols), dtype=torch.int32, device=dev)
    _dev(hash_ids, "hash_ids", torch.int32, (n, B, T, g0.n_hash_cols), dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_hash_layers", L.engram_hash_layers(
        garr, tarr, n, sarr, ids.data_ptr(), B, T, hash_ids.data_ptr(), _ptr(err), _stream(dev)))
    return hash_ids


def engram_gather(g: Geometry, table, scales, hash_ids, rows=None, err=None):
    """table uint8 [num_embeddings, head_dim], scales uint8 [num_embeddings, head_dim/32],
    hash_ids int32 [n_tok, n_hash_cols] -> rows bf16 [n_tok, n_hash_cols*head_dim]."""
    L = load()
    dev = hash_ids.device
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(hash_ids, "hash_ids", torch.int32, None, dev)
    hid = hash_ids.reshape(-1, g.n_hash_cols)
    n_tok = hid.shape[0]
    if rows is None:
        rows = torch.empty((n_tok, g.K), dtype=torch.bfloat16, device=dev)
    _dev(rows, "rows", torch.bfloat16, (n_tok, g.K), dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_gather", L.engram_gather(C.byref(g), table.data_ptr(), scales.data_ptr(),
                                            hid.data_ptr(), n_tok, rows.data_ptr(), _ptr(err),
                                            _stream(dev)))
    return rows


def engram_wkv(g: Geometry, a, w, kv=None):
    """a bf16 [M, K], w bf16 [N, K] -> kv bf16 [M, N]."""
    L = load()
    dev = a.device
    _dev(a, "a", torch.bfloat16, None, dev)
    if a.dim() != 2 or a.shape[1] != g.K:
        raise ValueError("a must be [M, %d]" % g.K)
    M = a.shape[0]
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    if kv is None:
        kv = torch.empty((M, g.N), dtype=torch.bfloat16, device=dev)
    _dev(kv, "kv", torch.bfloat16, (M, g.N), dev)
    _check("engram_wkv", L.engram_wkv(C.byref(g), a.data_ptr(), w.data_ptr(), M, kv.data_ptr(),
                                      _stream(dev)))
    return kv


def engram_wkv_gathered_scratch_size(g: Geometry, M: int) -> int:
    return load().engram_wkv_gathered_scratch_size(C.byref(g), int(M))


def engram_wkv_gathered(g: Geometry, table, scales, hash_ids, w, kv=None, scratch=None, err=None):
    """Gather + projection in one: table/scales/hash_ids as in engram_gather,
    w bf16 [N, K] -> kv bf16 [n_tok, N] (head_dim 64 only)."""
    L = load()
    dev = hash_ids.device
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(hash_ids, "hash_ids", torch.int32, None, dev)
    hid = hash_ids.reshape(-1, g.n_hash_cols)
    M = hid.shape[0]
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    if kv is None:
        kv = torch.empty((M, g.N), dtype=torch.bfloat16, device=dev)
    _dev(kv, "kv", torch.bfloat16, (M, g.N), dev)
    need = engram_wkv_gathered_scratch_size(g, M)
    if scratch is None:
        scratch = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(scratch, "scratch", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_wkv_gathered", L.engram_wkv_gathered(
        C.byref(g), table.data_ptr(), scales.data_ptr(), hid.data_ptr(), M, w.data_ptr(),
        kv.data_ptr(), scratch.data_ptr(), scratch.numel(), _ptr(err), _stream(dev)))
    return kv


def engram_gate_partials_supported(g: Geometry, M: int) -> bool:
    return bool(load().engram_gate_partials_supported(C.byref(g), int(M)))


def engram_wkv_gate_partials(g: Geometry, table, scales, hash_ids, w, x, q, k, v=None, part=None,
                             scratch=None, err=None):
    """Fused gather + projection whose key columns become the gate's partial
    sums: returns (v bf16 [n_tok, dim], part fp32 [n_tok, hc, dim/128, 2])."""
    L = load()
    dev = hash_ids.device
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(hash_ids, "hash_ids", torch.int32, None, dev)
    hid = hash_ids.reshape(-1, g.n_hash_cols)
    M = hid.shape[0]
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    _dev(x, "x", torch.bfloat16, None, dev)
    if x.numel() != M * g.hc_mult * g.dim:
        raise ValueError("x must hold n_tok*hc_mult*dim values")
    _dev(q, "q", torch.bfloat16, (g.hc_mult, g.dim), dev)
    _dev(k, "k", torch.bfloat16, (g.hc_mult, g.dim), dev)
    if v is None:
        v = torch.empty((M, g.dim), dtype=torch.bfloat16, device=dev)
    _dev(v, "v", torch.bfloat16, (M, g.dim), dev)
    if part is None:
        part = torch.empty((M, g.hc_mult, g.dim // 128, 2), dtype=torch.float32, device=dev)
    _dev(part, "part", torch.float32, (M, g.hc_mult, g.dim // 128, 2), dev)
    need = engram_wkv_gathered_scratch_size(g, M)
    if scratch is None:
        scratch = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(scratch, "scratch", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_wkv_gate_partials", L.engram_wkv_gate_partials(
        C.byref(g), table.data_ptr(), scales.data_ptr(), hid.data_ptr(), M, w.data_ptr(),
        x.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), part.data_ptr(),
        scratch.data_ptr(), scratch.numel(), _ptr(err), _stream(dev)))
    return v, part


def engram_gate_from_partials(g: Geometry, x, v, part, mask=None, out=None, gate=None):
    """x bf16 [n_tok, hc, dim] (any leading shape), v bf16 [n_tok, dim], part from
    engram_wkv_gate_partials -> out (like x); `out` may be x."""
    L = load()
    dev = x.device
    _dev(x, "x", torch.bfloat16, None, dev)
    n_tok = x.numel() // (g.hc_mult * g.dim)
    if x.numel() != n_tok * g.hc_mult * g.dim or x.shape[-1] != g.dim:
        raise ValueError("x must be [..., hc_mult, dim]")
    _dev(v, "v", torch.bfloat16, (n_tok, g.dim), dev)
    _dev(part, "part", torch.float32, (n_tok, g.hc_mult, g.dim // 128, 2), dev)
    m = _mask(mask, n_tok, dev)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", torch.bfloat16, tuple(x.shape), dev)
    if gate is not None:
        _dev(gate, "gate", torch.float32, None, dev)
        if gate.numel() != n_tok * g.hc_mult:
            raise ValueError("gate must hold n_tok*hc_mult values")
    _check("engram_gate_from_partials", L.engram_gate_from_partials(
        C.byref(g), x.data_ptr(), v.data_ptr(), part.data_ptr(), _ptr(m), n_tok, out.data_ptr(),
        _ptr(gate), _stream(dev)))
    return out


def engram_gate_add(g: Geometry, x, kv, q, k, mask=None, out=None, gate=None):
    """x bf16 [n_tok, hc, dim] (any leading shape), kv bf16 [n_tok, dim*(hc+1)],
    q/k bf16 [hc, dim], mask bool/uint8 [n_tok] or None -> out (same shape as x);
    `out` may be x (in place); `gate` fp32 [n_tok, hc] is filled if given."""
    L = load()
    dev = x.device
    _dev(x, "x", torch.bfloat16, None, dev)
    n_tok = x.numel() // (g.hc_mult * g.dim)
    if x.numel() != n_tok * g.hc_mult * g.dim or x.shape[-1] != g.dim:
        raise ValueError("x must be [..., hc_mult, dim]")
    _dev(kv, "kv", torch.bfloat16, None, dev)
    if kv.numel() != n_tok * g.N:
        raise ValueError("kv must be [n_tok, dim*(hc_mult+1)]")
    _dev(q, "q", torch.bfloat16, (g.hc_mult, g.dim), dev)
    _dev(k, "k", torch.bfloat16, (g.hc_mult, g.dim), dev)
    m = _mask(mask, n_tok, dev)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", torch.bfloat16, tuple(x.shape), dev)
    if gate is not None:
        _dev(gate, "gate", torch.float32, None, dev)
        if gate.numel() != n_tok * g.hc_mult:
            raise ValueError("gate must hold n_tok*hc_mult values")
    _check("engram_gate_add", L.engram_gate_add(C.byref(g), x.data_ptr(), kv.data_ptr(),
                                                q.data_ptr(), k.data_ptr(), _ptr(m), n_tok,
                                                out.data_ptr(), _ptr(gate), _stream(dev)))
    return out


def _mask(mask, n_tok, dev):
    if mask is None:
        return None
    if mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    _dev(mask, "mask", torch.uint8, None, dev)
    if mask.numel() != n_tok:
        raise ValueError("mask must hold one value per position")
    return mask


def engram_forward(g: Geometry, tables: dict, table, scales, w, q, k, x, ids, mask=None,
                   state=None, out=None, gate=None, workspace=None, err=None):
    """The whole forward: x bf16 [B, T, hc, dim], ids int32 [B, T] -> out (like x)."""
    L = load()
    dev = x.device
    _dev(ids, "ids", torch.int32, None, dev)
    if ids.dim() != 2:
        raise ValueError("ids must be [B, T]")
    B, T = ids.shape
    _dev(x, "x", torch.bfloat16, (B, T, g.hc_mult, g.dim), dev)
    ht = _tables(tables, g, dev)
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    _dev(q, "q", torch.bfloat16, (g.hc_mult, g.dim), dev)
    _dev(k, "k", torch.bfloat16, (g.hc_mult, g.dim), dev)
    if state is not None:
        _dev(state, "state", torch.int32, (B, g.max_ngram_size - 1), dev)
    m = _mask(mask, B * T, dev)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", torch.bfloat16, (B, T, g.hc_mult, g.dim), dev)
    if gate is not None:
        _dev(gate, "gate", torch.float32, (B, T, g.hc_mult), dev)
    need = engram_forward_workspace_size(g, B * T)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_forward", L.engram_forward(
        C.byref(g), C.byref(ht), table.data_ptr(), scales.data_ptr(), w.data_ptr(), q.data_ptr(),
        k.data_ptr(), _ptr(state), x.data_ptr(), ids.data_ptr(), _ptr(m), B, T, out.data_ptr(),
        _ptr(gate), workspace.data_ptr(), workspace.numel(), _ptr(err), _stream(dev)))
    return out


def engram_forward_hashed(g: Geometry, table, scales, w, q, k, x, hash_ids, mask=None, out=None,
                          gate=None, workspace=None, err=None):
    """The forward from given hash ids (the block's forward signature): x bf16
    [..., hc, dim], hash_ids int32 [..., n_hash_cols] (same leading shape),
    mask bool/uint8 over the positions or None -> out (like x)."""
    L = load()
    dev = x.device
    _dev(hash_ids, "hash_ids", torch.int32, None, dev)
    n_tok = hash_ids.numel() // g.n_hash_cols
    if hash_ids.numel() != n_tok * g.n_hash_cols or hash_ids.shape[-1] != g.n_hash_cols:
        raise ValueError("hash_ids must be [..., n_hash_cols]")
    _dev(x, "x", torch.bfloat16, None, dev)
    if x.numel() != n_tok * g.hc_mult * g.dim or x.shape[-1] != g.dim:
        raise ValueError("x must be [..., hc_mult, dim] with one position per hash-id row")
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    _dev(q, "q", torch.bfloat16, (g.hc_mult, g.dim), dev)
    _dev(k, "k", torch.bfloat16, (g.hc_mult, g.dim), dev)
    m = _mask(mask, n_tok, dev)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", torch.bfloat16, tuple(x.shape), dev)
    if gate is not None:
        _dev(gate, "gate", torch.float32, None, dev)
        if gate.numel() != n_tok * g.hc_mult:
            raise ValueError("gate must hold n_tok*hc_mult values")
    need = engram_forward_workspace_size(g, n_tok)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_forward_hashed", L.engram_forward_hashed(
        C.byref(g), table.data_ptr(), scales.data_ptr(), w.data_ptr(), q.data_ptr(), k.data_ptr(),
        x.data_ptr(), hash_ids.data_ptr(), _ptr(m), n_tok, out.data_ptr(), _ptr(gate),
        workspace.data_ptr(), workspace.numel(), _ptr(err), _stream(dev)))
    return out


def engram_fixed_scratch_bytes() -> int:
    """Size of the library's fixed per-GPU scratch array (engram_forward_noalloc)."""
    return int(load().engram_fixed_scratch_bytes())


def engram_forward_noalloc(g: Geometry, tables: dict, table, scales, w, q, k, x, ids, out,
                           mask=None, state=None, gate=None, err=None):
    """engram_forward with the library's fixed scratch array as its workspace:
    nothing is allocated by this call (out, and gate/err if wanted, are the
    caller's).  Raises EngramError (ENGRAM_ERR_TOO_LARGE) when the call's
    workspace would not fit the array."""
    L = load()
    dev = x.device
    _dev(ids, "ids", torch.int32, None, dev)
    if ids.dim() != 2:
        raise ValueError("ids must be [B, T]")
    B, T = ids.shape
    _dev(x, "x", torch.bfloat16, (B, T, g.hc_mult, g.dim), dev)
    ht = _tables(tables, g, dev)
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    _dev(q, "q", torch.bfloat16, (g.hc_mult, g.dim), dev)
    _dev(k, "k", torch.bfloat16, (g.hc_mult, g.dim), dev)
    if state is not None:
        _dev(state, "state", torch.int32, (B, g.max_ngram_size - 1), dev)
    m = _mask(mask, B * T, dev)
    _dev(out, "out", torch.bfloat16, (B, T, g.hc_mult, g.dim), dev)
    if gate is not None:
        _dev(gate, "gate", torch.float32, (B, T, g.hc_mult), dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _check("engram_forward_noalloc", L.engram_forward_noalloc(
        C.byref(g), C.byref(ht), table.data_ptr(), scales.data_ptr(), w.data_ptr(), q.data_ptr(),
        k.data_ptr(), _ptr(state), x.data_ptr(), ids.data_ptr(), _ptr(m), B, T, out.data_ptr(),
        _ptr(gate), _ptr(err), _stream(dev)))
    return out


# ------------------------------------------------------------------ around the layer
# the current stream's handle without a Stream object around it (2 us a call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


# the current device, without the check that torch is initialised (a tensor is there)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(name, fn, dev, *args):
    """Call a C entry on `dev`'s current stream, with `dev` the current device."""
    index = dev.index
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        raise EngramError(name, status)


class Adapters:
    """Low-rank adapters of a layer's wkv projection, on the device: down bf16
    [n, rank, K], up bf16 [n, N, rank], scale fp32 [n] or None (1 for all).
    Position m with adapter j gets scale[j] * up[j] (down[j] a[m]) added."""

    def __init__(self, down, up, scale=None):
        _dev(down, "down", torch.bfloat16)
        if down.dim() != 3:
            raise ValueError("down must be [n, rank, K]")
        n, rank, K = down.shape
        _dev(up, "up", torch.bfloat16, None, down.device)
        if up.dim() != 3 or up.shape[0] != n or up.shape[2] != rank:
            raise ValueError("up must be [n, N, rank]")
        if scale is not None:
            _dev(scale, "scale", torch.float32, (n,), down.device)
        self.down, self.up, self.scale = down, up, scale
        self.n, self.rank, self.K, self.N = n, rank, K, up.shape[1]
        self._c = _CAdapters(down.data_ptr(), up.data_ptr(), _ptr(scale), n, rank)

    def _for(self, g: Geometry, dev):
        if self.K != g.K or self.N != g.N:
            raise ValueError("adapters of a [%d -> %d] projection, the geometry's is [%d -> %d]" % (
                self.K, self.N, g.K, g.N))
        if self.down.device != dev:
            raise ValueError("adapters are on %s, expected %s" % (self.down.device, dev))
        return C.byref(self._c)


def engram_wkv_adapters_scratch_size(g: Geometry, adapters: Adapters, M: int) -> int:
    return load().engram_wkv_adapters_scratch_size(C.byref(g), C.byref(adapters._c), int(M))


def engram_wkv_adapters(g: Geometry, adapters: Adapters, a, w, adapter_ids, kv=None, scratch=None,
                        err=None):
    """The projection with each position's own adapter: a bf16 [M, K], w bf16
    [N, K], adapter_ids int32 [M] (-1: none) -> kv bf16 [M, N]."""
    L = load()
    dev = a.device
    _dev(a, "a", torch.bfloat16, None, dev)
    if a.dim() != 2 or a.shape[1] != g.K:
        raise ValueError("a must be [M, %d]" % g.K)
    M = a.shape[0]
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    ad = adapters._for(g, dev)
    _dev(adapter_ids, "adapter_ids", torch.int32, (M,), dev)
    if kv is None:
        kv = torch.empty((M, g.N), dtype=torch.bfloat16, device=dev)
    _dev(kv, "kv", torch.bfloat16, (M, g.N), dev)
    if scratch is None:
        scratch = torch.empty(max(engram_wkv_adapters_scratch_size(g, adapters, M), 1),
                              dtype=torch.uint8, device=dev)
    _dev(scratch, "scratch", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _launch("engram_wkv_adapters", L.engram_wkv_adapters, dev, C.byref(g), ad, a.data_ptr(),
            w.data_ptr(), adapter_ids.data_ptr(), M, kv.data_ptr(), scratch.data_ptr(),
            scratch.numel(), _ptr(err))
    return kv


def engram_forward_adapted_workspace_size(g: Geometry, adapters: Adapters, n_tok: int) -> int:
    return load().engram_forward_adapted_workspace_size(C.byref(g), C.byref(adapters._c),
                                                        int(n_tok))


def engram_forward_adapted(g: Geometry, tables: dict, adapters: Adapters, table, scales, w, q, k,
                           x, ids, adapter_ids, mask=None, state=None, out=None, gate=None,
                           workspace=None, err=None):
    """The whole forward with adapters: as engram_forward, adapter_ids int32 [B]
    naming each sequence's adapter (-1: none)."""
    L = load()
    dev = x.device
    _dev(ids, "ids", torch.int32, None, dev)
    if ids.dim() != 2:
        raise ValueError("ids must be [B, T]")
    B, T = ids.shape
    _dev(x, "x", torch.bfloat16, (B, T, g.hc_mult, g.dim), dev)
    ht = _tables(tables, g, dev)
    ad = adapters._for(g, dev)
    _dev(adapter_ids, "adapter_ids", torch.int32, (B,), dev)
    _dev(table, "table", torch.uint8, (g.num_embeddings, g.head_dim), dev)
    _dev(scales, "scales", torch.uint8, (g.num_embeddings, g.head_dim // 32), dev)
    _dev(w, "w", torch.bfloat16, (g.N, g.K), dev)
    _dev(q, "q", torch.bfloat16, (g.hc_mult, g.dim), dev)
    _dev(k, "k", torch.bfloat16, (g.hc_mult, g.dim), dev)
    if state is not None:
        _dev(state, "state", torch.int32, (B, g.max_ngram_size - 1), dev)
    m = _mask(mask, B * T, dev)
    if out is None:
        out = torch.empty_like(x)
    _dev(out, "out", torch.bfloat16, (B, T, g.hc_mult, g.dim), dev)
    if gate is not None:
        _dev(gate, "gate", torch.float32, (B, T, g.hc_mult), dev)
    if workspace is None:
        workspace = torch.empty(max(engram_forward_adapted_workspace_size(g, adapters, B * T), 1),
                                dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _launch("engram_forward_adapted", L.engram_forward_adapted, dev, C.byref(g), C.byref(ht), ad,
            table.data_ptr(), scales.data_ptr(), w.data_ptr(), q.data_ptr(), k.data_ptr(),
            _ptr(state), x.data_ptr(), ids.data_ptr(), adapter_ids.data_ptr(), _ptr(m), B, T,
            out.data_ptr(), _ptr(gate), workspace.data_ptr(), workspace.numel(), _ptr(err))
    return out


def engram_norm_quant(x, weight=None, residual=None, eps=1e-6, scale_format="e8m0_32", codes=None,
                      scales=None, total=None):
    """Root-mean-square norm of h = x + residual with an e4m3 output: x bf16
    [..., dim], residual the same or None, weight bf16 [dim] or None ->
    (codes uint8 like x, scales, total).  scale_format "e8m0_32": scales uint8
    [..., ceil(dim/32)]; "f32_128": fp32 [..., ceil(dim/128)]; "f32_row": fp32
    [..., 1].  total = bf16(h) (may be x or residual; None without a residual
    unless given)."""
    L = load()
    if scale_format not in _SCALE_FORMATS:
        raise ValueError("scale_format must be one of %s" % ", ".join(_SCALE_FORMATS))
    _dev(x, "x", torch.bfloat16)
    dev, shape = x.device, x.shape
    if not shape or shape[-1] == 0:
        raise ValueError("x must be [..., dim]")
    dim = shape[-1]
    if weight is not None:
        _dev(weight, "weight", torch.bfloat16, (dim,), dev)
    if residual is not None:
        _dev(residual, "residual", torch.bfloat16, shape, dev)
        if total is None:
            total = torch.empty_like(x)
    if total is not None:
        _dev(total, "total", torch.bfloat16, shape, dev)
    if codes is None:
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
    else:
        _dev(codes, "codes", torch.uint8, shape, dev)
    group = 32 if scale_format == "e8m0_32" else 128 if scale_format == "f32_128" else dim
    kind = torch.uint8 if scale_format == "e8m0_32" else torch.float32
    s_shape = (*shape[:-1], (dim + group - 1) // group)
    if scales is None:
        scales = torch.empty(s_shape, dtype=kind, device=dev)
    else:
        _dev(scales, "scales", kind, s_shape, dev)
    _launch("engram_norm_quant", L.engram_norm_quant, dev, x.data_ptr(), _ptr(residual),
            _ptr(weight), x.numel() // dim, dim, float(eps), _SCALE_FORMATS[scale_format],
            _ptr(total), codes.data_ptr(), scales.data_ptr())
    return codes, scales, total


def engram_beam_select_scratch_size(B: int, W: int, V: int) -> int:
    return load().engram_beam_select_scratch_size(int(B), int(W), int(V))


def engram_beam_select(logits, scores, finished=None, eos_id=-1, pad_id=0, tokens=None,
                       parents=None, new_scores=None, new_finished=None, scratch=None, err=None):
    """Beam search's selection: logits bf16 or fp32 [B*W, V] (or [B, W, V]; rows
    may be strided), scores fp32 [B, W], finished bool/uint8 [B, W] or None ->
    (tokens int32, parents int32, new_scores fp32, new_finished uint8, or bool
    if such a tensor is given), all [B, W], best first.  new_scores may be
    scores, new_finished finished."""
    L = load()
    dev = logits.device
    _dev(scores, "scores", torch.float32, None, dev)
    shape = scores.shape
    if len(shape) != 2:
        raise ValueError("scores must be [B, W]")
    B, W = shape
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor (got %s)" % dev)
    f32 = logits.dtype is torch.float32
    if not f32 and logits.dtype is not torch.bfloat16:
        raise TypeError("logits must be torch.float32 or torch.bfloat16 (got %s)" % logits.dtype)
    V = logits.shape[-1] if logits.dim() else 0
    if logits.shape != (B * W, V) and logits.shape != (B, W, V):
        raise ValueError("logits must be [B*W, V] or [B, W, V]")
    stride = logits.stride()
    ld = stride[-2] if B * W > 1 else V
    if len(stride) == 3 and W == 1 and B > 1:
        ld = stride[0]
    if (V > 1 and stride[-1] != 1) or ld < V or (
            len(stride) == 3 and B > 1 and W > 1 and stride[0] != W * ld):
        raise ValueError("logits must have contiguous rows, evenly apart")
    if finished is not None:
        if finished.dtype is torch.bool:
            finished = finished.view(torch.uint8)
        _dev(finished, "finished", torch.uint8, shape, dev)
    if tokens is None:
        tokens = torch.empty(shape, dtype=torch.int32, device=dev)
    else:
        _dev(tokens, "tokens", torch.int32, shape, dev)
    if parents is None:
        parents = torch.empty(shape, dtype=torch.int32, device=dev)
    else:
        _dev(parents, "parents", torch.int32, shape, dev)
    if new_scores is None:
        new_scores = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _dev(new_scores, "new_scores", torch.float32, shape, dev)
    if new_finished is None:
        new_finished = torch.empty(shape, dtype=torch.uint8, device=dev)
    else:
        kind = torch.bool if getattr(new_finished, "dtype", None) is torch.bool else torch.uint8
        _dev(new_finished, "new_finished", kind, shape, dev)
    if scratch is None:
        scratch = torch.empty(max(engram_beam_select_scratch_size(B, W, V), 1), dtype=torch.uint8,
                              device=dev)
    _dev(scratch, "scratch", torch.uint8, None, dev)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    _launch("engram_beam_select", L.engram_beam_select, dev, logits.data_ptr(),
            1 if f32 else 0, ld, scores.data_ptr(), _ptr(finished), B, W, V,
            int(eos_id), int(pad_id), tokens.data_ptr(), parents.data_ptr(),
            new_scores.data_ptr(), new_finished.data_ptr(), scratch.data_ptr(), scratch.numel(),
            _ptr(err))
    return tokens, parents, new_scores, new_finished


_array_types: dict = {}  # ctypes array types (making one takes longer than filling it)


def _ptr_array(n):
    if n not in _array_types:
        _array_types[n] = (C.c_void_p * n, C.c_int64 * n)
    return _array_types[n][0]


def _size_array(n):
    _ptr_array(n)
    return _array_types[n][1]


def engram_beam_reorder(states, parents, err=None):
    """state[b][w] = state[b][parents[b][w]] in place for every tensor of the
    list `states` (any dtype, [B*W, ...] or [B, W, ...], contiguous, rows of a
    multiple of 4 bytes; for instance each layer's engram_hash state);
    parents int32 [B, W]."""
    L = load()
    dev = parents.device
    _dev(parents, "parents", torch.int32, None, dev)
    if parents.dim() != 2:
        raise ValueError("parents must be [B, W]")
    B, W = parents.shape
    rows, n = B * W, len(states)
    ptr, size = [], []
    for st in states:
        if not (type(st) is torch.Tensor and st.is_cuda and st.is_contiguous() and st.device == dev):
            _dev(st, "state", st.dtype if isinstance(st, torch.Tensor) else None, None, dev)
        shape = st.shape
        if not len(shape) or (shape[0] != rows and tuple(shape[:2]) != (B, W)):
            raise ValueError("a state must be [B*W, ...] or [B, W, ...] (got %s)" % (tuple(shape),))
        ptr.append(st.data_ptr())
        size.append(st.nbytes // rows if rows else 0)
    if err is not None:
        _dev(err, "err", torch.int32, (1,), dev)
    if rows == 0:
        return states
    _launch("engram_beam_reorder", L.engram_beam_reorder, dev, _ptr_array(n)(*ptr),
            _size_array(n)(*size), n, parents.data_ptr(), B, W, _ptr(err))
    return states


class EngramLayer:
    """One Engram layer's device-resident inputs: geometry, hash tables, the
    fp8 table and scales, the wkv weight and q/k weights, plus a reusable
    workspace, which grows as calls need it (one that a graph was captured with
    is kept).  `forward` is engram_forward, or with adapters
    engram_forward_adapted."""

    def __init__(self, g: Geometry, tables: dict, table, scales, w, q, k):
        self.g, self.tables = g, tables
        self.table, self.scales, self.w, self.q, self.k = table, scales, w, q, k
        self._ws = None
        self._ws_captured, self._kept = False, []

    def _room(self, need: int):
        if self._ws is None or self._ws.numel() < need:
            if self._ws_captured:  # the graph's replays write there
                self._kept.append(self._ws)
            self._ws = torch.empty(max(need, 1), dtype=torch.uint8, device=self.w.device)
            self._ws_captured = False
        if not self._ws_captured and self._ws.is_cuda:
            self._ws_captured = torch.cuda.is_current_stream_capturing()
        return self._ws

    def workspace(self, n_tok: int):
        return self._room(engram_forward_workspace_size(self.g, n_tok))

    def forward(self, x, ids, mask=None, state=None, out=None, gate=None, err=None, adapters=None,
                adapter_ids=None):
        if adapters is None and adapter_ids is not None:
            raise ValueError("adapter_ids without adapters")
        if adapters is not None:
            ws = self._room(engram_forward_adapted_workspace_size(self.g, adapters, ids.numel()))
            return engram_forward_adapted(self.g, self.tables, adapters, self.table, self.scales,
                                          self.w, self.q, self.k, x, ids, adapter_ids, mask=mask,
                                          state=state, out=out, gate=gate, workspace=ws, err=err)
        return engram_forward(self.g, self.tables, self.table, self.scales, self.w, self.q, self.k,
                              x, ids, mask=mask, state=state, out=out, gate=gate,
                              workspace=self.workspace(ids.numel()), err=err)
