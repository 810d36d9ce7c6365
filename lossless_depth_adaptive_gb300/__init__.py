"""GB300 (sm_103a) Depth Exploration Decoding: Python binding of the C ABI in include/dex.h.

This module only marshals arguments into ``_build/libdex.so``; every step of a DEX round
runs in the library's CUDA kernels and host scheduler.  Device memory and streams come
from PyTorch tensors / streams (``tensor.data_ptr()``, ``stream.cuda_stream``).

Importing does not need a GPU.  The library itself must exist (``build()`` in
``lossless_depth_adaptive_gb300.build`` or ``__graft_entry__.build()``); a missing library
raises ``DexLibraryMissing`` -- there is no fallback path.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Dict, List, Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libdex.so")

LAYER_TENSORS = ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "wg", "wu", "wd")

DEX_OK, DEX_EINVAL, DEX_ENOMEM, DEX_ECUDA, DEX_ECAPACITY, DEX_ETIMEOUT, DEX_ESTATE, DEX_ENODEV, DEX_ERANGE = \
    0, -1, -2, -3, -4, -5, -6, -7, -8


class DexLibraryMissing(ImportError):
    pass


class DexError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {code} ({strerror(code)})")


class dex_model(C.Structure):
    _fields_ = [("n_layers", C.c_int32), ("d_model", C.c_int32), ("n_heads", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("d_ff", C.c_int32),
                ("vocab", C.c_int32), ("rms_eps", C.c_float), ("rope_theta", C.c_float),
                ("embed", C.c_void_p), ("final_norm", C.c_void_p), ("lm_head", C.c_void_p),
                ("layers", C.POINTER(C.c_void_p)), ("adapters", C.POINTER(C.c_void_p)),
                ("adapter_alpha", C.POINTER(C.c_float))]


class dex_decode_cfg(C.Structure):
    _fields_ = [("batch", C.c_int32), ("max_ctx", C.c_int32), ("max_new", C.c_int32),
                ("sample", C.c_int32), ("tau", C.c_float), ("seed", C.c_uint64),
                ("decs", C.c_int32), ("debug_logits", C.c_int32), ("max_branch", C.c_int32)]


class dex_stats(C.Structure):
    _fields_ = [("rounds", C.c_int64), ("commits", C.c_int64), ("nodes", C.c_int64),
                ("max_round_nodes", C.c_int64), ("layer_passes", C.c_int64),
                ("node_layers", C.c_int64), ("depth_charge", C.c_int64),
                ("kstar_hist", C.c_int64 * 16), ("weight_bytes", C.c_int64), ("kv_bytes", C.c_int64),
                ("h2d_bytes", C.c_int64), ("d2h_bytes", C.c_int64), ("kernel_launches", C.c_int64),
                ("gemm_launches", C.c_int64), ("gemm_bytes", C.c_int64), ("ms_gemm", C.c_double),
                ("ms_expand", C.c_double), ("ms_exit", C.c_double), ("ms_collapse", C.c_double),
                ("ms_host", C.c_double), ("attn_launches", C.c_int64), ("ms_attn", C.c_double)]

    def as_dict(self) -> Dict:
        d = {k: getattr(self, k) for k, _ in self._fields_}
        d["kstar_hist"] = list(self.kstar_hist)
        return d


class dex_exit_node(C.Structure):
    _fields_ = [("seq", C.c_int32), ("target_pos", C.c_int32), ("unmasked", C.c_int32),
                ("prior_off", C.c_int32), ("n_prior", C.c_int32)]


class dex_kv_geom(C.Structure):
    _fields_ = [("batch", C.c_int32), ("n_layers", C.c_int32), ("n_kv_heads", C.c_int32),
                ("head_dim", C.c_int32), ("max_ctx", C.c_int32), ("n_slots", C.c_int32)]


class dex_copy_job(C.Structure):
    _fields_ = [("seq", C.c_int32), ("slot", C.c_int32), ("pos", C.c_int32), ("n_layers", C.c_int32)]


class dex_plan_node(C.Structure):
    _fields_ = [("seq", C.c_int32), ("heap", C.c_int32), ("stage", C.c_int32), ("plen", C.c_int32),
                ("pos", C.c_int32), ("c_end", C.c_int32), ("slot", C.c_int32), ("kv_commit", C.c_int32),
                ("token", C.c_int32), ("target_pos", C.c_int32), ("unmasked", C.c_int32),
                ("n_prior", C.c_int32), ("n_tail", C.c_int32), ("prior", C.c_int32 * 16),
                ("tail", C.c_int32 * 16)]


class dex_paged_kv(C.Structure):
    _fields_ = [("pages", C.c_void_p), ("table", C.c_void_p), ("page_stride", C.c_int64), ("n_pages", C.c_int32),
                ("page_size", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("batch", C.c_int32),
                ("table_width", C.c_int32), ("table_stride", C.c_int32), ("dtype", C.c_int32)]


class dex_append_args(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("q_out", C.c_void_p),
                ("q_stride", C.c_int64), ("k_stride", C.c_int64), ("v_stride", C.c_int64),
                ("q_out_stride", C.c_int64), ("seq", C.c_void_p), ("pos", C.c_void_p), ("rope_pos", C.c_void_p),
                ("n_tokens", C.c_int32), ("n_heads", C.c_int32), ("in_dtype", C.c_int32), ("rope_theta", C.c_float)]


class dex_attention_args(C.Structure):
    _fields_ = [("q", C.c_void_p), ("out", C.c_void_p), ("lse", C.c_void_p), ("q_stride", C.c_int64),
                ("out_stride", C.c_int64), ("q_start", C.c_void_p), ("seq_len", C.c_void_p),
                ("prefix_table", C.c_void_p), ("tree_mask", C.c_void_p), ("n_tokens", C.c_int32),
                ("n_heads", C.c_int32), ("max_q", C.c_int32), ("prefix_len", C.c_int32), ("scale", C.c_float)]


DEX_DT_BF16, DEX_DT_FP16, DEX_DT_FP32 = 0, 1, 2
DEX_ATTN_BAD_PAGE, DEX_ATTN_BAD_RANGE, DEX_ATTN_TIMEOUT = 1, 2, 4

P = C.c_void_p
I32P = C.POINTER(C.c_int32)
# name -> (restype, argtypes): every symbol of include/dex.h
SIGNATURES = {
    "dex_init": (C.c_int, [C.POINTER(dex_model), I32P, C.c_int32, C.POINTER(dex_decode_cfg), P, C.POINTER(P)]),
    "dex_prefill": (C.c_int, [P, C.c_int32, I32P, C.c_int32]),
    "dex_step": (C.c_int, [P, I32P, I32P]),
    "dex_generate": (C.c_int, [P, I32P]),
    "dex_ar_step": (C.c_int, [P, I32P, I32P]),
    "dex_ar_generate": (C.c_int, [P, I32P]),
    "dex_get_stats": (C.c_int, [P, C.POINTER(dex_stats)]),
    "dex_reset_stats": (C.c_int, [P]),
    "dex_set_timing": (C.c_int, [P, C.c_int32]),
    "dex_last_round_nodes": (C.c_int, [P, I32P, C.c_int32, I32P]),
    "dex_debug_logits": (C.c_int, [P, C.POINTER(C.c_float), C.c_int32, I32P]),
    "dex_strerror": (C.c_char_p, [C.c_int]),
    "dex_free": (None, [P]),
    "dex_selftest_stall": (C.c_int, [P, C.c_int32]),
    "dex_exit_head_decs": (C.c_int, [P, C.c_int32, C.c_int32, P, C.c_float, P, C.c_int32, P, P, C.c_int32,
                                     C.c_float, C.c_uint64, P, P, P]),
    "dex_exit_head_decs_noalloc": (C.c_int, [P, C.c_int32, C.c_int32, P, C.c_float, P, C.c_int32, P, P,
                                             C.c_int32, C.c_float, C.c_uint64, P, P, P]),
    "dex_kv_collapse": (C.c_int, [P, P, C.POINTER(dex_kv_geom), P, C.c_int32, P, P]),
    "dex_paged_append": (C.c_int, [C.POINTER(dex_paged_kv), C.POINTER(dex_append_args), P, P]),
    "dex_prefix_attention_workspace": (C.c_int, [C.POINTER(dex_paged_kv), C.POINTER(dex_attention_args),
                                                 C.POINTER(C.c_size_t)]),
    "dex_prefix_attention": (C.c_int, [C.POINTER(dex_paged_kv), C.POINTER(dex_attention_args), P, C.c_size_t, P,
                                       P]),
    "dex_lattice_new": (C.c_int, [I32P, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.POINTER(P)]),
    "dex_lattice_start": (C.c_int, [P, C.c_int32, C.c_int32, C.c_int32]),
    "dex_lattice_plan": (C.c_int, [P, C.POINTER(dex_plan_node), C.c_int32, I32P]),
    "dex_lattice_update": (C.c_int, [P, I32P, I32P, I32P, C.POINTER(dex_copy_job), C.c_int32, I32P]),
    "dex_lattice_state": (C.c_int, [P, C.c_int32, I32P, I32P, I32P]),
    "dex_lattice_free": (None, [P]),
}

_lib: Optional[C.CDLL] = None


def lib() -> C.CDLL:
    """Load libdex.so (once).  Raises DexLibraryMissing when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise DexLibraryMissing(f"{LIB_PATH} is missing: run lossless_depth_adaptive_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(code: int) -> str:
    try:
        return lib().dex_strerror(code).decode()
    except DexLibraryMissing:
        return str(code)


def check(code: int, where: str) -> int:
    if code != DEX_OK:
        raise DexError(code, where)
    return code


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise DexError(DEX_EINVAL, message)


def i32(values: Sequence[int]):
    return (C.c_int32 * len(values))(*values)


# ---- thin wrappers with the C names ---------------------------------------------------------

def dex_init(model: dex_model, X: Sequence[int], cfg: dex_decode_cfg, stream: int = 0) -> C.c_void_p:
    h = C.c_void_p()
    check(lib().dex_init(C.byref(model), i32(X), len(X), C.byref(cfg), C.c_void_p(stream), C.byref(h)),
          "dex_init")
    return h


def dex_prefill(h, seq: int, tokens: Sequence[int]) -> None:
    check(lib().dex_prefill(h, seq, i32(tokens), len(tokens)), "dex_prefill")


def dex_step(h, batch: int, ar: bool = False):
    out, nc = (C.c_int32 * batch)(), (C.c_int32 * batch)()
    fn = lib().dex_ar_step if ar else lib().dex_step
    check(fn(h, out, nc), "dex_ar_step" if ar else "dex_step")
    return list(out), list(nc)


def dex_ar_step(h, batch: int):
    return dex_step(h, batch, ar=True)


def dex_generate(h, batch: int, max_new: int, ar: bool = False, out=None) -> List[List[int]]:
    """Generate into ``out`` (a ctypes int32 array of batch*max_new, reused if given)."""
    if out is None:
        out = (C.c_int32 * (batch * max_new))(*([-1] * (batch * max_new)))
    fn = lib().dex_ar_generate if ar else lib().dex_generate
    check(fn(h, out), "dex_ar_generate" if ar else "dex_generate")
    return [list(out[b * max_new:(b + 1) * max_new]) for b in range(batch)]


def dex_ar_generate(h, batch: int, max_new: int) -> List[List[int]]:
    return dex_generate(h, batch, max_new, ar=True)


def dex_get_stats(h) -> Dict:
    s = dex_stats()
    check(lib().dex_get_stats(h, C.byref(s)), "dex_get_stats")
    return s.as_dict()


def dex_reset_stats(h) -> None:
    check(lib().dex_reset_stats(h), "dex_reset_stats")


def dex_set_timing(h, level: int) -> None:
    check(lib().dex_set_timing(h, level), "dex_set_timing")


def dex_last_round_nodes(h, max_rows: int = 4096) -> List[Dict]:
    buf, n = (C.c_int32 * (8 * max_rows))(), C.c_int32()
    check(lib().dex_last_round_nodes(h, buf, max_rows, C.byref(n)), "dex_last_round_nodes")
    keys = ("seq", "heap", "stage", "plen", "target_pos", "token", "n_prior", "pos")
    return [dict(zip(keys, buf[8 * k:8 * k + 8])) for k in range(n.value)]


def dex_debug_logits(h, vocab: int, max_rows: int = 512):
    import numpy as np
    out = np.zeros((max_rows, vocab), dtype=np.float32)
    n = C.c_int32()
    check(lib().dex_debug_logits(h, out.ctypes.data_as(C.POINTER(C.c_float)), max_rows, C.byref(n)),
          "dex_debug_logits")
    return out[:n.value]


def dex_free(h) -> None:
    if h:
        lib().dex_free(h)


def dex_exit_head_decs(h_ptr: int, n: int, d: int, final_norm_ptr: int, rms_eps: float, lm_head_ptr: int,
                       vocab: int, nodes_ptr: int, priors_ptr: int, sample: bool, tau: float, seed: int,
                       tokens_ptr: int, logits_ptr: int = 0, stream: int = 0) -> None:
    check(lib().dex_exit_head_decs(P(h_ptr), n, d, P(final_norm_ptr), rms_eps, P(lm_head_ptr), vocab,
                                   P(nodes_ptr), P(priors_ptr), int(sample), tau, seed, P(tokens_ptr),
                                   P(logits_ptr or None), P(stream)), "dex_exit_head_decs")


def dex_exit_head_decs_noalloc(h_ptr: int, n: int, d: int, final_norm_ptr: int, rms_eps: float,
                               lm_head_ptr: int, vocab: int, nodes_ptr: int, priors_ptr: int, sample: bool,
                               tau: float, seed: int, tokens_ptr: int, logits_ptr: int = 0, stream: int = 0) -> int:
    """Allocation-free exit head + DECS; returns the status code (raises on other errors)."""
    rc = lib().dex_exit_head_decs_noalloc(P(h_ptr), n, d, P(final_norm_ptr), rms_eps, P(lm_head_ptr), vocab,
                                          P(nodes_ptr), P(priors_ptr), int(sample), tau, seed, P(tokens_ptr),
                                          P(logits_ptr or None), P(stream))
    if rc not in (DEX_OK, DEX_ECAPACITY):
        check(rc, "dex_exit_head_decs_noalloc")
    return rc


def dex_kv_collapse(committed_ptr: int, pool_ptr: int, geom: dex_kv_geom, jobs_ptr: int, n_jobs: int,
                    stream: int = 0, rejected_ptr: int = 0) -> None:
    """rejected_ptr: device int32 that receives the number of out-of-range jobs skipped (or 0)."""
    check(lib().dex_kv_collapse(P(committed_ptr), P(pool_ptr), C.byref(geom), P(jobs_ptr), n_jobs,
                                P(rejected_ptr or None), P(stream)), "dex_kv_collapse")


def dex_paged_append(kv: dex_paged_kv, args: dex_append_args, rejected_ptr: int = 0, stream: int = 0) -> None:
    """rejected_ptr: device int32 that receives the number of out-of-range tokens skipped (or 0)."""
    check(lib().dex_paged_append(C.byref(kv), C.byref(args), P(rejected_ptr or None), P(stream)), "dex_paged_append")


def dex_prefix_attention_workspace(kv: dex_paged_kv, args: dex_attention_args) -> int:
    """Bytes of device scratch dex_prefix_attention needs (reads the integer fields only)."""
    n = C.c_size_t()
    check(lib().dex_prefix_attention_workspace(C.byref(kv), C.byref(args), C.byref(n)),
          "dex_prefix_attention_workspace")
    return n.value


def dex_prefix_attention(kv: dex_paged_kv, args: dex_attention_args, workspace_ptr: int, workspace_bytes: int,
                         status_ptr: int = 0, stream: int = 0) -> None:
    """status_ptr: device int32 into which the call ORs DEX_ATTN_* bits (or 0)."""
    check(lib().dex_prefix_attention(C.byref(kv), C.byref(args), P(workspace_ptr or None), workspace_bytes,
                                     P(status_ptr or None), P(stream)), "dex_prefix_attention")


# ---- model marshalling (PyTorch tensors -> dex_model) -------------------------------------------

class ModelRef:
    """Keeps the ctypes model description and the layer-pointer array alive."""

    def __init__(self, shape, weights: Dict, adapters: Optional[Sequence[Dict]] = None):
        ptrs = []
        for l in range(shape.n_layers):
            for name in LAYER_TENSORS:
                t = weights[f"l{l}.{name}"]
                assert t.is_cuda and t.is_contiguous()
                ptrs.append(t.data_ptr())
        self._layers = (C.c_void_p * len(ptrs))(*ptrs)
        head = weights["embed"] if shape.tied_head else weights["lm_head"]
        self.model = dex_model(shape.n_layers, shape.d_model, shape.n_heads, shape.n_kv_heads, shape.head_dim,
                               shape.d_ff, shape.vocab, shape.rms_eps, shape.rope_theta,
                               weights["embed"].data_ptr(), weights["final_norm"].data_ptr(), head.data_ptr(),
                               C.cast(self._layers, C.POINTER(C.c_void_p)))
        self.weights = weights
        self.adapters = adapters
        if adapters:
            aptrs = []
            for ad in adapters:
                for name in ("g", "w1", "b1", "w2", "b2"):
                    t = ad[name]
                    assert t.is_cuda and t.is_contiguous()
                    aptrs.append(t.data_ptr())
            self._adapters = (C.c_void_p * len(aptrs))(*aptrs)
            self._alpha = (C.c_float * len(adapters))(*[float(ad["alpha"]) for ad in adapters])
            self.model.adapters = C.cast(self._adapters, C.POINTER(C.c_void_p))
            self.model.adapter_alpha = C.cast(self._alpha, C.POINTER(C.c_float))


class Decoder:
    """A handle plus the model it references: init / prefill / step / generate / stats."""

    def __init__(self, shape, weights: Dict, X: Sequence[int], batch: int, max_ctx: int, max_new: int,
                 sample: bool = False, tau: float = 1.0, seed: int = 0, decs: bool = True,
                 debug_logits: bool = False, stream: Optional[int] = None, max_branch: int = 0,
                 adapters: Optional[Sequence[Dict]] = None):
        import torch
        self.shape, self.X, self.batch, self.max_new = shape, list(X), batch, max_new
        self.ref = ModelRef(shape, weights, adapters)
        cfg = dex_decode_cfg(batch, max_ctx, max_new, int(sample), tau, seed, int(decs), int(debug_logits),
                             int(max_branch))
        self.stream = torch.cuda.current_stream().cuda_stream if stream is None else stream
        self.h = dex_init(self.ref.model, self.X, cfg, self.stream)

    def prefill(self, seq: int, tokens: Sequence[int]) -> None:
        dex_prefill(self.h, seq, [int(t) for t in tokens])

    def step(self, ar: bool = False):
        return dex_step(self.h, self.batch, ar)

    def generate(self, ar: bool = False, out=None) -> List[List[int]]:
        return dex_generate(self.h, self.batch, self.max_new, ar, out)

    def stats(self) -> Dict:
        return dex_get_stats(self.h)

    def reset_stats(self) -> None:
        dex_reset_stats(self.h)

    def set_timing(self, level: int) -> None:
        dex_set_timing(self.h, level)

    def last_round_nodes(self) -> List[Dict]:
        return dex_last_round_nodes(self.h)

    def debug_logits(self):
        return dex_debug_logits(self.h, self.shape.vocab)

    def selftest_stall(self, limit_us: int) -> int:
        """Return code of dex_selftest_stall (DEX_ETIMEOUT when the bounded wait gave up)."""
        return lib().dex_selftest_stall(self.h, int(limit_us))

    def close(self) -> None:
        if self.h:
            dex_free(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedCache:
    """One layer of a paged K/V cache: append with rotary positions, shared-prefix attention.

    ``pages``: [n_pages, 2 (K, V), kv_heads, page_size, head_dim] bf16 or fp16, contiguous within a
    page (a slice of a larger allocation is fine, so the layers of a model can share one).
    ``table``: int32 [batch, width] page ids; position p of sequence b is row ``p % page_size`` of page
    ``table[b, p // page_size]``.  Both stay the caller's and may be changed in place between calls.

    Calls run on the pages' device and its current stream, never synchronise and can be captured into
    a CUDA graph.  A bad argument raises DexError before anything is launched; the device-side checks
    of ``dex_paged_append`` and ``dex_prefix_attention`` (include/dex.h) report through ``rejected`` and
    ``status``.
    """

    def __init__(self, pages, table):
        import torch
        self._torch = torch
        self._code = {torch.bfloat16: DEX_DT_BF16, torch.float16: DEX_DT_FP16}
        _need(pages.dim() == 5 and pages.shape[1] == 2, "pages must be [n_pages, 2, kv_heads, page_size, head_dim]")
        n, _, kvh, ps, hd = pages.shape
        _need(pages.dtype in self._code, "pages must be bf16 or fp16")
        _need(n > 0 and pages.stride()[1:] == (kvh * ps * hd, ps * hd, hd, 1), "each page must be contiguous")
        _need(table.dim() == 2 and table.dtype == torch.int32 and table.stride(1) == 1 and table.shape[0] > 0,
              "table must be int32 [batch, width], contiguous rows")
        self.pages, self.table, self.device = pages, table, pages.device
        page_stride = pages.stride(0) if n > 1 else 2 * kvh * ps * hd
        table_stride = table.stride(0) if table.shape[0] > 1 else table.shape[1]
        self.kv = dex_paged_kv(pages.data_ptr(), table.data_ptr(), page_stride, n, ps, kvh, hd, table.shape[0],
                               table.shape[1], table_stride, self._code[pages.dtype])
        self.kv_heads, self.head_dim = kvh, hd
        # the geometry checks of the library, which look at the sizes alone
        dex_prefix_attention_workspace(self.kv, dex_attention_args(n_heads=kvh, max_q=1, scale=1.0))
        self._on_device(table=table)
        # what every call needs: a small one is bound by the time it takes to get to its launch
        self._dev = pages.get_device() if pages.is_cuda else None
        self._kv_ref, self._dtype, self._i32 = C.byref(self.kv), pages.dtype, torch.int32
        self._lib_append, self._lib_attention = lib().dex_paged_append, lib().dex_prefix_attention

    def _on_device(self, **tensors):
        for name, t in tensors.items():
            _need(t is None or (t.is_cuda and t.device == self.device), f"{name} must be on the pages' CUDA device")

    def _rows(self, name, t, heads, n):
        """[n, heads, head_dim] with the rows of a token contiguous: the stride between tokens."""
        hd = self.head_dim
        if t.dim() == 3:
            (rows, h, d), (between, s1, s2) = t.shape, t.stride()
            if rows == n and d == hd and s2 == 1 and (s1 == hd or h == 1) and (h == heads or heads is None):
                return between if n > 1 else h * hd
        raise DexError(DEX_EINVAL, f"{name} must be [tokens = {n}, {heads or 'heads'}, {hd}] with contiguous heads")

    def _vector(self, name, t, n, dtype):
        if not (t.dtype == dtype and t.dim() == 1 and t.shape[0] == n and t.is_contiguous()):
            raise DexError(DEX_EINVAL, f"{name} must be a contiguous {dtype} vector of {n}")
        return t.data_ptr()

    def _run(self, fn, where, *args):
        cuda = self._torch._C
        if cuda._cuda_getDevice() == self._dev:
            rc = fn(*args, cuda._cuda_getCurrentRawStream(self._dev))
        else:
            with self._torch.cuda.device(self._dev):
                rc = fn(*args, cuda._cuda_getCurrentRawStream(self._dev))
        if rc != DEX_OK:
            check(rc, where)

    def append(self, k, v, seq, pos, q=None, q_out=None, theta: float = 10000.0, rope_pos=None, rejected=None):
        """Store k (rotated) and v of token t at position pos[t] of sequence seq[t]; return q rotated.

        k, v: [tokens, kv_heads, head_dim], q: [tokens, heads, head_dim] or None, in the cache's type or
        fp32 (slices of a fused projection are fine).  seq, pos, rope_pos: int32 [tokens]; seq -1 skips a
        token, rope_pos (default: pos) is the rotation position.  theta 0 stores k unrotated.  q_out:
        [tokens, heads, head_dim] in the cache's type, allocated when not given; it may be q itself.
        rejected: int32 [1], receives the number of tokens out of range, which are skipped.
        """
        n, dt, dev = k.shape[0], k.dtype, self._dev
        f32 = dt == self._torch.float32
        if v.dtype != dt or not (f32 or dt == self._dtype):
            raise DexError(DEX_EINVAL, "k and v must have the cache's type or fp32")
        k_stride, v_stride = self._rows("k", k, self.kv_heads, n), self._rows("v", v, self.kv_heads, n)
        here = k.get_device() == dev and v.get_device() == dev and seq.get_device() == dev and pos.get_device() == dev
        q_ptr, out_ptr, q_stride, out_stride, heads = None, None, 0, 0, 0
        if q is not None:
            heads = q.shape[1]
            q_stride = self._rows("q", q, None, n)
            if q.dtype != dt:
                raise DexError(DEX_EINVAL, "q must have the type of k")
            if q_out is None:
                q_out = self._torch.empty(q.shape, dtype=self._dtype, device=q.device)
            elif q_out.dtype != self._dtype:
                raise DexError(DEX_EINVAL, "q_out must have the cache's type")
            out_stride = self._rows("q_out", q_out, heads, n)
            q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
            here = here and q.get_device() == dev and q_out.get_device() == dev
        elif q_out is not None:
            raise DexError(DEX_EINVAL, "q_out needs q")
        rope_ptr = None
        if rope_pos is not None:
            rope_ptr = self._vector("rope_pos", rope_pos, n, self._i32)
            here = here and rope_pos.get_device() == dev
        a = dex_append_args(q_ptr, k.data_ptr(), v.data_ptr(), out_ptr, q_stride, k_stride, v_stride, out_stride,
                            self._vector("seq", seq, n, self._i32), self._vector("pos", pos, n, self._i32), rope_ptr, n,
                            heads, DEX_DT_FP32 if f32 else self.kv.dtype, theta)
        rejected_ptr = None if rejected is None else self._vector("rejected", rejected, 1, self._i32)
        if not here or (rejected is not None and rejected.get_device() != dev):
            self._on_device(k=k, v=v, q=q, q_out=q_out, seq=seq, pos=pos, rope_pos=rope_pos, rejected=rejected)
        self._run(self._lib_append, "dex_paged_append", self._kv_ref, C.byref(a), rejected_ptr)
        return q_out

    def attention_workspace(self, q, max_q: int, prefix_len: int = 0):
        """A scratch tensor for attention() calls of these sizes (any lengths); calls that may overlap
        on the GPU need one each."""
        a = dex_attention_args(n_tokens=q.shape[0], n_heads=q.shape[1], max_q=max_q, prefix_len=prefix_len, scale=1.0)
        return self._torch.empty(max(1, dex_prefix_attention_workspace(self.kv, a)), dtype=self._torch.uint8,
                                 device=self.device)

    def attention(self, q, q_start, seq_len, max_q: int, prefix_len: int = 0, prefix_table=None, tree_mask=None,
                  scale: Optional[float] = None, out=None, lse=None, workspace=None, status=None):
        """Attention of q over the cache; returns out ([tokens, heads, head_dim], the cache's type).

        The queries of sequence b are tokens q_start[b] .. q_start[b+1]-1 (int32 [batch + 1], at most max_q
        each) and stand at its last positions; seq_len (int32 [batch]) counts them.  Query i of n sees
        positions 0 .. seq_len - n + i, or with tree_mask (int64 [tokens]) everything before the last n and
        of those the ones whose bit is set.  prefix_len promises that the positions below it are the same for
        every sequence with queries (and named by its table, usually the same pages); where it pays they are
        read once for the batch, through prefix_table (int32; default: row 0 of the table).  scale defaults to
        head_dim**-0.5.  lse: fp32 [tokens, heads], receives the log of the softmax denominator.  workspace: from
        attention_workspace(), allocated when not given.  status: int32 [1], receives DEX_ATTN_* bits.
        Rows of out and lse that belong to no sequence are left as they were.  out must not overlap q, and what
        the cache holds at positions below seq_len and prefix_len must be finite.
        """
        i32, batch = self._i32, self.kv.batch
        n, heads = q.shape[0], q.shape[1]
        if not (0 <= prefix_len < 2 ** 31 and 0 < max_q < 2 ** 31):
            raise DexError(DEX_EINVAL, "prefix_len or max_q out of range")
        if q.dtype != self._dtype:
            raise DexError(DEX_EINVAL, "q must have the cache's type")
        if out is None:
            out = self._torch.empty((n, heads, self.head_dim), dtype=q.dtype, device=q.device)
        elif out.dtype != q.dtype:
            raise DexError(DEX_EINVAL, "out must have the cache's type")
        a = dex_attention_args(q.data_ptr(), out.data_ptr(), None, self._rows("q", q, None, n),
                               self._rows("out", out, heads, n), self._vector("q_start", q_start, batch + 1, i32),
                               self._vector("seq_len", seq_len, batch, i32), None, None, n, heads, max_q, prefix_len,
                               self.head_dim ** -0.5 if scale is None else scale)
        if prefix_table is not None:
            a.prefix_table = self._vector("prefix_table", prefix_table, prefix_table.numel(), i32)
            _need(prefix_table.numel() * self.kv.page_size >= prefix_len, "prefix_table is shorter than prefix_len")
        if tree_mask is not None:
            a.tree_mask = self._vector("tree_mask", tree_mask, n, self._torch.int64)
        if lse is not None:
            if not (lse.dtype == self._torch.float32 and lse.is_contiguous() and lse.shape == q.shape[:2]):
                raise DexError(DEX_EINVAL, "lse must be contiguous fp32 [tokens, heads]")
            a.lse = lse.data_ptr()
        status_ptr = None if status is None else self._vector("status", status, 1, i32)
        if workspace is None:
            workspace = self.attention_workspace(q, max_q, prefix_len)
        elif not workspace.is_contiguous():
            raise DexError(DEX_EINVAL, "workspace must be contiguous")
        for t in (q, out, q_start, seq_len, workspace, prefix_table, tree_mask, lse, status):
            if t is not None and t.get_device() != self._dev:
                self._on_device(q=q, out=out, q_start=q_start, seq_len=seq_len, prefix_table=prefix_table,
                                tree_mask=tree_mask, lse=lse, workspace=workspace, status=status)
        self._run(self._lib_attention, "dex_prefix_attention", self._kv_ref, C.byref(a), workspace.data_ptr(),
                  workspace.nbytes, status_ptr)
        return out


class Lattice:
    """Host-only lattice scheduler (the library's FSM), usable without a GPU."""

    def __init__(self, X: Sequence[int], batch: int, decs: bool = True, max_branch: int = 0):
        self.h = C.c_void_p()
        self.batch = batch
        check(lib().dex_lattice_new(i32(X), len(X), batch, int(decs), int(max_branch), C.byref(self.h)),
              "dex_lattice_new")
        self.cap = batch << (len(X) - 1)

    def start(self, seq: int, p_c: int, last_token: int) -> None:
        check(lib().dex_lattice_start(self.h, seq, p_c, last_token), "dex_lattice_start")

    def plan(self) -> List[Dict]:
        buf, n = (dex_plan_node * self.cap)(), C.c_int32()
        check(lib().dex_lattice_plan(self.h, buf, self.cap, C.byref(n)), "dex_lattice_plan")
        out = []
        for k in range(n.value):
            p = buf[k]
            d = {f: getattr(p, f) for f, _ in dex_plan_node._fields_ if f not in ("prior", "tail")}
            d["prior"] = list(p.prior[:p.n_prior])
            d["tail"] = list(p.tail[:p.n_tail])
            out.append(d)
        return out

    def update(self, tokens: Sequence[int]):
        committed, kstar = (C.c_int32 * self.batch)(), (C.c_int32 * self.batch)()
        jobs, nj = (dex_copy_job * self.batch)(), C.c_int32()
        check(lib().dex_lattice_update(self.h, i32(tokens) if tokens else None, committed, kstar, jobs,
                                       self.batch, C.byref(nj)), "dex_lattice_update")
        return list(committed), list(kstar), [(j.seq, j.slot, j.pos, j.n_layers) for j in jobs[:nj.value]]

    def state(self, seq: int):
        q, p_c, used = C.c_int32(), C.c_int32(), C.c_int32()
        check(lib().dex_lattice_state(self.h, seq, C.byref(q), C.byref(p_c), C.byref(used)), "dex_lattice_state")
        return q.value, p_c.value, used.value

    def __del__(self):
        try:
            if self.h:
                lib().dex_lattice_free(self.h)
        except Exception:
            pass
