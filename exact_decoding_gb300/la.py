"""ctypes binding of include/la.h (argument marshalling only).

Each `la_*` function here calls the C entry point of the same name; errors
become `LaError`.  `Decoder` is a convenience owner: it uploads a weight dict
(from `synth`) to the device with torch and keeps those tensors alive for the
handle's lifetime.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import List, Optional, Tuple

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libla.so")

LA_F32, LA_BF16 = 0, 1
LA_POOL_FIFO, LA_POOL_LRU, LA_POOL_LFU = 0, 1, 2
_lib = None


class LaError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {msg} (code {code})")
        self.code = code


class la_model_dims(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("rms_eps", ctypes.c_float), ("rope_base", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


_PP = ctypes.POINTER(ctypes.c_void_p)


class la_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("final_norm", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("attn_norm", _PP), ("wq", _PP), ("wk", _PP), ("wv", _PP), ("wo", _PP), ("ffn_norm", _PP),
                ("w_gate", _PP), ("w_up", _PP), ("w_down", _PP)]


class la_opts(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("W", ctypes.c_int32), ("G", ctypes.c_int32), ("max_seq", ctypes.c_int32),
                ("prompt_as_reference", ctypes.c_int32), ("pool_cap", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("seed", ctypes.c_uint64), ("cuda_stream", ctypes.c_void_p),
                ("profile", ctypes.c_int32), ("top_k", ctypes.c_int32), ("top_p", ctypes.c_float),
                ("pool_policy", ctypes.c_int32)]


class la_stats_t(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int64), ("generated", ctypes.c_int64), ("last_accept", ctypes.c_int32),
                ("last_candidates", ctypes.c_int32), ("prefix_len", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("gemm_ms", ctypes.c_double), ("gemm_bytes", ctypes.c_double), ("gemm_launches", ctypes.c_int64),
                ("attn_ms", ctypes.c_double), ("attn_bytes", ctypes.c_double), ("attn_launches", ctypes.c_int64),
                ("kernel_launches", ctypes.c_int64), ("elem_ms", ctypes.c_double), ("spec_ms", ctypes.c_double),
                ("h2d_bytes", ctypes.c_int64), ("d2h_bytes", ctypes.c_int64)]


_I32P = ctypes.POINTER(ctypes.c_int32)
LA_ERR_CAPACITY = -3   # include/la.h


class la_state_t(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("tokens_cap", ctypes.c_int32), ("tokens", _I32P),
                ("window", _I32P), ("n_records", ctypes.c_int32), ("records_cap", ctypes.c_int32),
                ("records", _I32P), ("uses", _I32P)]


class la_kv8_cache(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("n_seqs", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class la_kv8_attn(ctypes.Structure):
    _fields_ = [("layer", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("max_len", ctypes.c_int32), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("row_start", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("vis", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("scale", ctypes.c_float)]


class la_kv8_rows(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int32), ("n_src", ctypes.c_int32), ("max_rows", ctypes.c_int32),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("k_layer_stride", ctypes.c_int64),
                ("v_layer_stride", ctypes.c_int64), ("row_start", ctypes.c_void_p), ("row_idx", ctypes.c_void_p),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("stored", ctypes.c_void_p)]


class la_kv8_qkv(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("type", ctypes.c_int32),
                ("weight_type", ctypes.c_int32), ("eps", ctypes.c_float), ("rope_base", ctypes.c_float),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64), ("v_out_stride", ctypes.c_int64),
                ("row_start", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("depth", ctypes.c_void_p),
                ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p)]


class la_logprobs_args(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("type", ctypes.c_int32),
                ("n_tokens", ctypes.c_int32), ("n_top", ctypes.c_int32), ("stride", ctypes.c_int64),
                ("logits", ctypes.c_void_p), ("tokens", ctypes.c_void_p), ("logprob", ctypes.c_void_p),
                ("entropy", ctypes.c_void_p), ("top_ids", ctypes.c_void_p), ("top_logprob", ctypes.c_void_p)]


_KV8_QKV = struct.Struct("@4i2f6q12P")     # la_kv8_qkv
_LOGPROBS = struct.Struct("@5i4xq6P")      # la_logprobs_args
assert _KV8_QKV.size == ctypes.sizeof(la_kv8_qkv) and _LOGPROBS.size == ctypes.sizeof(la_logprobs_args)
_KV8_ATTN = struct.Struct("@5i4q6Pf4x")    # la_kv8_attn
_KV8_ROWS = struct.Struct("@3i4q5P")       # la_kv8_rows
assert _KV8_ATTN.size == ctypes.sizeof(la_kv8_attn) and _KV8_ROWS.size == ctypes.sizeof(la_kv8_rows)


def load_library():
    """Load libla.so; raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m exact_decoding_gb300.build`")
    lib = ctypes.CDLL(LIB_PATH)
    H = ctypes.c_void_p
    lib.la_create.argtypes = [ctypes.POINTER(la_model_dims), ctypes.POINTER(la_weights), ctypes.POINTER(la_opts),
                              ctypes.POINTER(H)]
    lib.la_create_kv8.argtypes = [ctypes.POINTER(la_model_dims), ctypes.POINTER(la_weights), ctypes.POINTER(la_opts),
                                  ctypes.POINTER(la_kv8_cache), ctypes.c_int32, ctypes.POINTER(H)]
    lib.la_fork.argtypes = [H, H]
    lib.la_prefill.argtypes = [H, _I32P, ctypes.c_int32, _I32P]
    lib.la_step.argtypes = [H, _I32P, _I32P]
    lib.la_ar_step.argtypes = [H, _I32P]
    lib.la_generate.argtypes = [H, _I32P, ctypes.c_int32, ctypes.c_int32, _I32P, _I32P, _I32P]
    lib.la_stats.argtypes = [H, ctypes.POINTER(la_stats_t)]
    lib.la_export_state.argtypes = [H, ctypes.POINTER(la_state_t)]
    lib.la_import_state.argtypes = [H, ctypes.POINTER(la_state_t)]
    lib.la_debug_logits.argtypes = [H, ctypes.c_void_p, _I32P, _I32P]
    lib.la_gemm_bf16.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                 ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
    lib.la_gemm_bf16_noalloc.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                         ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]
    lib.la_gemm_status.argtypes = [ctypes.c_void_p]
    lib.la_selftest_timeout.argtypes = [H, ctypes.c_int64, ctypes.c_void_p]
    lib.la_step_tables.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _I32P,
                                   ctypes.POINTER(ctypes.c_uint32), _I32P, ctypes.c_int32, _I32P, _I32P]
    lib.la_gemm_schedule.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _I32P,
                                     ctypes.c_int32, _I32P, _I32P, _I32P, _I32P]
    KV8 = ctypes.POINTER(la_kv8_cache)
    lib.la_kv8_workspace.argtypes = [KV8, ctypes.POINTER(ctypes.c_int64)]
    lib.la_kv8_attention.argtypes = [KV8, ctypes.POINTER(la_kv8_attn), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
    lib.la_kv8_attention_window.argtypes = [KV8, ctypes.POINTER(la_kv8_attn), ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_void_p]
    lib.la_kv8_append.argtypes = [KV8, ctypes.POINTER(la_kv8_rows), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]
    lib.la_kv8_fork.argtypes = [KV8, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    lib.la_kv8_free.argtypes = [KV8, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]
    lib.la_kv8_compact.argtypes = [KV8, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_int64, ctypes.c_void_p]
    lib.la_kv8_status.argtypes = [KV8, ctypes.POINTER(ctypes.c_uint32), ctypes.c_void_p]
    lib.la_kv8_norm_rope.argtypes = [KV8, ctypes.POINTER(la_kv8_qkv), ctypes.c_void_p]
    lib.la_logprobs.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.la_gemv_w4_workspace.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_int64)]
    lib.la_gemv_w4.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                               ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64,
                               ctypes.c_void_p]
    lib.la_destroy.argtypes = [H]
    lib.la_destroy.restype = None
    lib.la_strerror.argtypes = [ctypes.c_int]
    lib.la_strerror.restype = ctypes.c_char_p
    lib.la_last_error.argtypes = []
    lib.la_last_error.restype = ctypes.c_char_p
    for name in ("la_create", "la_prefill", "la_step", "la_ar_step", "la_generate", "la_stats", "la_export_state",
                 "la_import_state", "la_debug_logits", "la_gemm_bf16", "la_gemm_bf16_noalloc", "la_gemm_status",
                 "la_selftest_timeout", "la_gemm_schedule", "la_step_tables", "la_kv8_workspace", "la_kv8_attention",
                 "la_kv8_append", "la_kv8_fork", "la_kv8_free", "la_kv8_compact", "la_kv8_status", "la_create_kv8",
                 "la_fork", "la_kv8_attention_window", "la_kv8_norm_rope", "la_logprobs", "la_gemv_w4", "la_gemv_w4_workspace"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def la_strerror(code: int) -> str:
    return load_library().la_strerror(code).decode()


def _check(rc: int, where: str):
    if rc != 0:
        lib = load_library()
        raise LaError(rc, where, lib.la_last_error().decode() or lib.la_strerror(rc).decode())


def _i32(a: np.ndarray):
    return a.ctypes.data_as(_I32P)


# ---------------------------------------------------------------------------- entry points
def la_create(dims: la_model_dims, weights: la_weights, opts: la_opts) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load_library().la_create(ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(opts),
                                    ctypes.byref(h)), "la_create")
    return h


def la_create_kv8(dims: la_model_dims, weights: la_weights, opts: la_opts, cache: la_kv8_cache, slot: int) -> ctypes.c_void_p:
    h = ctypes.c_void_p()
    _check(load_library().la_create_kv8(ctypes.byref(dims), ctypes.byref(weights), ctypes.byref(opts), ctypes.byref(cache),
                                        slot, ctypes.byref(h)), "la_create_kv8")
    return h


def la_fork(src, dst) -> None:
    _check(load_library().la_fork(src, dst), "la_fork")


def la_prefill(h, prompt) -> int:
    p = np.ascontiguousarray(prompt, dtype=np.int32)
    first = np.zeros(1, dtype=np.int32)
    _check(load_library().la_prefill(h, _i32(p), len(p), _i32(first)), "la_prefill")
    return int(first[0])


def la_step(h, N: int) -> List[int]:
    out = np.zeros(max(N, 8), dtype=np.int32)
    n = np.zeros(1, dtype=np.int32)
    _check(load_library().la_step(h, _i32(out), _i32(n)), "la_step")
    return out[: int(n[0])].tolist()


def la_ar_step(h) -> int:
    tok = np.zeros(1, dtype=np.int32)
    _check(load_library().la_ar_step(h, _i32(tok)), "la_ar_step")
    return int(tok[0])


def la_generate(h, prompt, max_new: int) -> Tuple[List[int], int]:
    p = np.ascontiguousarray(prompt, dtype=np.int32)
    out = np.zeros(max_new, dtype=np.int32)
    n = np.zeros(1, dtype=np.int32)
    steps = np.zeros(1, dtype=np.int32)
    _check(load_library().la_generate(h, _i32(p), len(p), max_new, _i32(out), _i32(n), _i32(steps)),
           "la_generate")
    return out[: int(n[0])].tolist(), int(steps[0])


def la_stats(h) -> dict:
    s = la_stats_t()
    _check(load_library().la_stats(h, ctypes.byref(s)), "la_stats")
    return {f: getattr(s, f) for f, _ in la_stats_t._fields_}


def la_export_state(h, N: int, W: int, tokens_cap: int = 1 << 16, records_cap: int = 1 << 16) -> dict:
    toks = np.zeros(tokens_cap, dtype=np.int32)
    win = np.zeros((N - 1) * W, dtype=np.int32)
    recs = np.zeros(records_cap * N, dtype=np.int32)
    uses = np.zeros(records_cap, dtype=np.int32)
    st = la_state_t(0, tokens_cap, _i32(toks), _i32(win), 0, records_cap, _i32(recs), _i32(uses))
    _check(load_library().la_export_state(h, ctypes.byref(st)), "la_export_state")
    r = recs[: st.n_records * N].reshape(st.n_records, N)
    return {"tokens": toks[: st.n_tokens].tolist(), "window": win.reshape(N - 1, W).copy(),
            "records": [(int(x[0]), tuple(int(t) for t in x[1:])) for x in r],
            "uses": uses[: st.n_records].tolist()}


def la_import_state(h, N: int, W: int, tokens, window, records, uses=None) -> None:
    toks = np.ascontiguousarray(tokens, dtype=np.int32)
    win = np.ascontiguousarray(np.asarray(window).reshape(-1), dtype=np.int32)
    recs = np.ascontiguousarray(np.array([[k, *s] for k, s in records], dtype=np.int32).reshape(-1, N))
    u = None if uses is None else np.ascontiguousarray(uses, dtype=np.int32)
    st = la_state_t(len(toks), len(toks), _i32(toks), _i32(win), len(recs), len(recs), _i32(recs),
                    _i32(u) if u is not None else None)
    _check(load_library().la_import_state(h, ctypes.byref(st)), "la_import_state")


def la_debug_logits(h) -> np.ndarray:
    rows = np.zeros(1, dtype=np.int32)
    vocab = np.zeros(1, dtype=np.int32)
    lib = load_library()
    _check(lib.la_debug_logits(h, None, _i32(rows), _i32(vocab)), "la_debug_logits")
    out = np.zeros((int(rows[0]), int(vocab[0])), dtype=np.float32)
    _check(lib.la_debug_logits(h, out.ctypes.data, _i32(rows), _i32(vocab)), "la_debug_logits")
    return out


def la_gemm_bf16(x_ptr: int, w_ptr: int, y_ptr: int, rows: int, out: int, k: int, splits: int = 1,
                 workspace_ptr: Optional[int] = None, stream: Optional[int] = None) -> None:
    _check(load_library().la_gemm_bf16(x_ptr, w_ptr, y_ptr, rows, out, k, splits, workspace_ptr, stream),
           "la_gemm_bf16")


def la_gemm_bf16_noalloc(x_ptr: int, w_ptr: int, y_ptr: int, rows: int, out: int, k: int, splits: int = 1,
                         stream: Optional[int] = None) -> None:
    """la_gemm_bf16 without a caller workspace: for callers that cannot allocate
    device memory at call time.  The split-K partials live in a fixed device
    array inside the library (LA_NOALLOC_SCRATCH_FLOATS floats); overlapping
    calls race on it."""
    _check(load_library().la_gemm_bf16_noalloc(x_ptr, w_ptr, y_ptr, rows, out, k, splits, stream),
           "la_gemm_bf16_noalloc")


NOALLOC_SCRATCH_FLOATS = 4 * 1024 * 1024


def la_gemm_status(stream: Optional[int] = None) -> None:
    """Raise LaError(-5) if a bounded wait inside an earlier la_gemm_bf16,
    la_gemm_bf16_noalloc or la_gemv_w4 kernel on this device gave up; clears the status."""
    _check(load_library().la_gemm_status(stream), "la_gemm_status")


def la_selftest_timeout(h, limit_ns: int, stream: Optional[int] = None) -> None:
    """Launch the bounded-wait self-test kernel (its wait gives up after
    limit_ns and sets a timeout bit in h's error word, or with h None in the
    standalone GEMMs' words)."""
    _check(load_library().la_selftest_timeout(h, limit_ns, stream), "la_selftest_timeout")


def la_step_tables(N: int, W: int, G: int):
    """The static tables of a step's rows, from the library's host code:
    (depth [M], visibility words [M][8] as uint32, used rows [U]) as numpy
    arrays.  No GPU is touched."""
    import numpy as np
    lib = load_library()
    depth = np.zeros(256, dtype=np.int32)
    vis = np.zeros((256, 8), dtype=np.uint32)
    used = np.zeros(256, dtype=np.int32)
    m = np.zeros(1, dtype=np.int32)
    u = np.zeros(1, dtype=np.int32)
    rc = lib.la_step_tables(N, W, G, depth.ctypes.data_as(_I32P), vis.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32)),
                            used.ctypes.data_as(_I32P), 256, m.ctypes.data_as(_I32P), u.ctypes.data_as(_I32P))
    _check(rc, "la_step_tables")
    return depth[:m[0]].copy(), vis[:m[0]].copy(), used[:u[0]].copy()


def la_gemm_schedule(tiles: int, n_kb: int, ctas: int, whole_first: bool):
    """The projection GEMMs' work split, from the library's host code: returns
    (segments [n][4] of (tile, kb0, kb1, plane), cta_first [ctas_used + 1],
    planes per tile [tiles]) as int32 numpy arrays.  No GPU is touched."""
    import numpy as np
    lib = load_library()
    cap = tiles + ctas + 16                      # a run adds at most one segment per tile boundary
    while True:
        segs = np.zeros((cap, 4), dtype=np.int32)
        first = np.zeros(ctas + 1, dtype=np.int32)
        used = np.zeros(1, dtype=np.int32)
        nseg = np.zeros(1, dtype=np.int32)
        planes = np.zeros(tiles, dtype=np.int32)
        ptr = lambda a: a.ctypes.data_as(_I32P)
        rc = lib.la_gemm_schedule(tiles, n_kb, ctas, int(bool(whole_first)), ptr(segs), cap, ptr(nseg), ptr(first),
                                  ptr(used), ptr(planes))
        if rc == LA_ERR_CAPACITY:
            cap *= 2
            continue
        _check(rc, "la_gemm_schedule")
        return segs[:nseg[0]].copy(), first[:used[0] + 1].copy(), planes


def la_kv8_workspace(cache: la_kv8_cache) -> int:
    n = ctypes.c_int64()
    _check(load_library().la_kv8_workspace(cache, ctypes.byref(n)), "la_kv8_workspace")
    return n.value


def la_kv8_attention(cache: la_kv8_cache, args: la_kv8_attn, workspace_ptr: int, workspace_bytes: int,
                     stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_attention(cache, args, workspace_ptr, workspace_bytes, stream), "la_kv8_attention")


def la_kv8_attention_window(cache: la_kv8_cache, args: la_kv8_attn, window: int, sinks: int, workspace_ptr: int, workspace_bytes: int,
                            stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_attention_window(cache, args, window, sinks, workspace_ptr, workspace_bytes, stream),
           "la_kv8_attention_window")


def la_kv8_norm_rope(cache: la_kv8_cache, args: la_kv8_qkv, stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_norm_rope(cache, args, stream), "la_kv8_norm_rope")


def la_logprobs(args: la_logprobs_args, stream: Optional[int] = None) -> None:
    _check(load_library().la_logprobs(ctypes.byref(args), stream), "la_logprobs")


def la_gemv_w4_workspace(rows: int, out: int, k: int, group: int) -> int:
    n = ctypes.c_int64()
    _check(load_library().la_gemv_w4_workspace(rows, out, k, group, ctypes.byref(n)), "la_gemv_w4_workspace")
    return n.value


def la_gemv_w4(x_ptr: int, x_stride: int, w_ptr: int, scales_ptr: int, y_ptr: int, y_stride: int, rows: int, out: int, k: int,
               group: int, workspace_ptr: Optional[int] = None, workspace_bytes: int = 0, stream: Optional[int] = None) -> None:
    _check(load_library().la_gemv_w4(x_ptr, x_stride, w_ptr, scales_ptr, y_ptr, y_stride, rows, out, k, group, workspace_ptr, workspace_bytes,
                                     stream), "la_gemv_w4")


def la_kv8_append(cache: la_kv8_cache, rows: la_kv8_rows, workspace_ptr: int, workspace_bytes: int,
                  stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_append(cache, rows, workspace_ptr, workspace_bytes, stream), "la_kv8_append")


def la_kv8_fork(cache: la_kv8_cache, src_ptr: int, dst_ptr: int, n: int, stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_fork(cache, src_ptr, dst_ptr, n, stream), "la_kv8_fork")


def la_kv8_free(cache: la_kv8_cache, slots_ptr: int, keep_ptr: Optional[int], n: int,
                stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_free(cache, slots_ptr, keep_ptr, n, stream), "la_kv8_free")


def la_kv8_compact(cache: la_kv8_cache, table_out_ptr: int, refs_out_ptr: int, n_live_ptr: Optional[int],
                   workspace_ptr: int, workspace_bytes: int, stream: Optional[int] = None) -> None:
    _check(load_library().la_kv8_compact(cache, table_out_ptr, refs_out_ptr, n_live_ptr, workspace_ptr, workspace_bytes,
                                         stream), "la_kv8_compact")


def la_kv8_status(cache: la_kv8_cache, stream: Optional[int] = None) -> None:
    """Raise LaError if a call on this cache met no free page (-3), something
    outside the cache (-6) or a wait that gave up (-5); clears the status."""
    _check(load_library().la_kv8_status(cache, None, stream), "la_kv8_status")


def la_destroy(h) -> None:
    if h:
        load_library().la_destroy(h)


# ---------------------------------------------------------------------------- operators on tensors
_torch_module = None


def _torch():
    """torch, which this module needs for its tensors alone."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _on(index: int, stream, fn, where: str, *args) -> None:
    """fn(*args, stream) with CUDA device `index` current; stream None: torch's current one there."""
    c = _torch()._C
    st = c._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if c._cuda_getDevice() == index:
        rc = fn(*args, st)
    else:
        with _torch().cuda.device(index):
            rc = fn(*args, st)
    if rc:
        _check(rc, where)


def _empty(stream, *shape, dtype, device):
    """A new tensor whose memory belongs to the stream that writes it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _cuda_index(t, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, not on {t.device}")
    return t.get_device()


def logprobs(logits, tokens=None, top: int = 0, out=None, stream=None):
    """Log probabilities of given tokens, the entropy, and the most probable
    tokens of every row of logits [rows, vocab] (float32 or bfloat16, rows at
    any stride); see la_logprobs.  tokens: int32 [rows] or [rows, n], or None;
    top: alternatives of a row, 0 .. 32.  Returns (logprob like tokens or
    None, entropy [rows], ids [rows, top] int32, their log probabilities
    [rows, top]); `out` has tensors of these shapes to write to.  Runs on
    `stream` (default: torch's current one of the logits' device) and does not
    synchronise."""
    torch = _torch()
    f32, sh, st, kind = torch.float32, logits.shape, logits.stride(), logits.dtype
    if len(sh) != 2 or (kind is not f32 and kind is not torch.bfloat16) or (st[1] != 1 and sh[1] > 1):
        raise ValueError(f"logits must be float32 or bfloat16 [rows, vocab] with dense rows, not {kind} {tuple(sh)} strides {st}")
    index = logits.get_device()
    if index < 0:
        _cuda_index(logits, "logits")
    rows, vocab = sh
    n, given = 0, None
    if tokens is not None:
        given = tokens.shape
        if tokens.dtype is not torch.int32 or not 1 <= len(given) <= 2 or given[0] != rows or not tokens.is_contiguous() or tokens.get_device() != index:
            raise ValueError(f"tokens must be a contiguous int32 tensor [{rows}] or [{rows}, n] on {logits.device}, not {tokens.dtype} "
                             f"{tuple(given)} on {tokens.device}")
        n = given[1] if len(given) == 2 else 1
    if out is None:
        f = {"dtype": f32, "device": logits.device}
        lp, entropy = None if tokens is None else _empty(stream, *given, **f), _empty(stream, rows, **f)
        ids, best = _empty(stream, rows, max(top, 0), dtype=torch.int32, device=logits.device), _empty(stream, rows, max(top, 0), **f)
        out = lp, entropy, ids, best
    else:
        lp, entropy, ids, best = out
        if (lp is None) != (given is None):
            raise ValueError(f"out's logprob must be {'None' if given is None else f'a float32 tensor {tuple(given)}'}")
        listed = (rows, top)
        for name, t, shape, dtype in (("logprob", lp, given, f32), ("entropy", entropy, (rows,), f32), ("ids", ids, listed, torch.int32), ("top logprob", best, listed, f32)):
            if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != index) or t is None and name != "logprob":
                raise ValueError(f"out's {name} must be a contiguous {dtype} tensor {tuple(shape)} on {logits.device}")
    args = _LOGPROBS.pack(rows, vocab, LA_F32 if kind is f32 else LA_BF16, n, top, st[0] if rows > 1 else vocab, logits.data_ptr(), tokens.data_ptr() if n else 0,
                          lp.data_ptr() if n else 0, entropy.data_ptr(), ids.data_ptr() if top > 0 else 0, best.data_ptr() if top > 0 else 0)
    _on(index, stream, load_library().la_logprobs, "la_logprobs", args)
    return out


class W4Matrix:
    """A matrix [out, k] of 4-bit weights: w uint8 [out, k / 2] (the even k in a
    byte's low half), scales bfloat16 [out, k / group], group 32, 64 or 128.
    Element (o, k) is (q - 8) * scales[o, k / group]; see la_gemv_w4."""

    def __init__(self, w, scales):
        import torch
        self._torch = torch
        if w.dtype is not torch.uint8 or w.dim() != 2 or not w.is_contiguous() or scales.dtype is not torch.bfloat16 or scales.dim() != 2 \
                or not scales.is_contiguous() or scales.device != w.device or scales.shape[0] != w.shape[0] or scales.shape[1] < 1 \
                or 2 * w.shape[1] % scales.shape[1]:
            raise ValueError(f"W4Matrix needs contiguous uint8 [out, k / 2] and bfloat16 [out, k / group] on one device, not {w.dtype} "
                             f"{tuple(w.shape)} on {w.device} and {scales.dtype} {tuple(scales.shape)} on {scales.device}")
        self._index = _cuda_index(w, "w")
        self.w, self.scales = w, scales
        self.out, self.k, self.group = w.shape[0], 2 * w.shape[1], 2 * w.shape[1] // scales.shape[1]
        self._w_ptr, self._s_ptr, self._fn, self._need = w.data_ptr(), scales.data_ptr(), load_library().la_gemv_w4, {}

    def matvec(self, x, out=None, stream=None):
        """x W^T for the bfloat16 rows x [rows, k] (or [k]), as float32 [rows, out]
        (or [out]).  For a batch of single tokens: the matrix is read once for
        every 16 rows.  Runs on `stream` (default: torch's current one of the
        matrix's device) and does not synchronise."""
        torch, sh, st = self._torch, x.shape, x.stride()
        if x.dtype is not torch.bfloat16 or not 1 <= len(sh) <= 2 or sh[-1] != self.k or st[-1] != 1 or x.get_device() != self._index:
            raise ValueError(f"x must be bfloat16 [rows, {self.k}] with dense rows on {self.w.device}, not {x.dtype} {tuple(sh)} strides {st} on {x.device}")
        rows, shape = (1, (self.out,)) if len(sh) == 1 else (sh[0], (sh[0], self.out))
        if out is None:
            out = _empty(stream, *shape, dtype=torch.float32, device=self.w.device)
        elif out.dtype is not torch.float32 or out.shape != shape or (out.stride(-1) != 1 and self.out > 1) or out.get_device() != self._index:
            raise ValueError(f"out must be float32 {shape} with dense rows on {self.w.device}, not {out.dtype} {tuple(out.shape)} strides "
                             f"{out.stride()} on {out.device}")
        need = self._need.get(rows)
        if need is None:
            with torch.cuda.device(self._index):
                need = self._need[rows] = la_gemv_w4_workspace(rows, self.out, self.k, self.group)
        # the allocator keeps it for the stream that uses it
        ws = _empty(stream, need, dtype=torch.uint8, device=self.w.device) if need else None
        _on(self._index, stream, self._fn, "la_gemv_w4", x.data_ptr(), st[0] if rows > 1 else self.k, self._w_ptr, self._s_ptr, out.data_ptr(),
            out.stride(0) if rows > 1 else self.out, rows, self.out, self.k, self.group, 0 if ws is None else ws.data_ptr(), need)
        return out


# ---------------------------------------------------------------------------- owners
class DeviceWeights:
    """Device copies (torch tensors) of a weight dict in the synth.model_weights
    layout, and the la_weights / la_model_dims structs that point at them."""

    def __init__(self, weights: dict, device="cuda"):
        import torch
        dims = weights["dims"]
        self.dims = dims
        self._keep = []

        def up(a):
            if a.dtype == np.uint16:
                t = torch.from_numpy(a.view(np.int16)).to(device)
            else:
                t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device)
            self._keep.append(t)
            return t.data_ptr()

        def arr(ptrs):
            a = (ctypes.c_void_p * len(ptrs))(*ptrs)
            self._keep.append(a)
            return ctypes.cast(a, _PP)

        names = ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down")
        per = {k: [] for k in names}
        for lw in weights["layers"]:
            for k in names:
                per[k].append(up(lw[k]))
        self.struct = la_weights(up(weights["embed"]), up(weights["final_norm"]), up(weights["lm_head"]),
                                 *[arr(per[k]) for k in names])
        self.dims_struct = la_model_dims(dims.n_layers, dims.d_model, dims.n_heads, dims.n_kv_heads, dims.head_dim,
                                         dims.ffn, dims.vocab, dims.rms_eps, dims.rope_base,
                                         LA_BF16 if dims.dtype == "bf16" else LA_F32)
        self.device = self._keep[0].device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self._keep if hasattr(t, "numel"))


class Kv8Cache:
    """A paged 8-bit KV cache (la_kv8_*): the pool, its scales, the sequences'
    table and lengths, and a workspace, all as torch tensors on one device.

    k, v        uint8 (e4m3) [layers, pages, kv heads, page, dim] and, V
                transposed, [layers, pages, kv heads, dim, page]
    k_scale, v_scale   float32 [layers, pages, kv heads], powers of two
    table, lens, refs  int32 [seqs, max_pages], [seqs], [pages]

    `tensors` adopts existing tensors by those names.  Calls run on `stream`
    (default: torch's current stream of the cache's device) and do not
    synchronise; status() does, and raises what they met.  Calls that overlap
    (streams, captured graphs) need a `workspace` of their own (workspace()).
    On another stream than their own, the cache's tensors and the arguments
    have to live until that stream is through with them."""

    def __init__(self, n_layers: int, n_pages: int, page: int, n_kv_heads: int, head_dim: int, n_seqs: int,
                 max_pages: int, device="cuda", tensors: Optional[dict] = None):
        import torch
        self._torch, self._bf16, self._f32, self._i32 = torch, torch.bfloat16, torch.float32, torch.int32
        tensors = dict(tensors or {})
        given = next(iter(tensors.values()), None)
        dev = torch.device(given.device if given is not None else device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._index = dev.index if dev.type == "cuda" else -1
        pool = (n_layers, n_pages, n_kv_heads)
        shapes = {"k": (*pool, page, head_dim), "v": (*pool, head_dim, page), "k_scale": pool, "v_scale": pool,
                  "table": (n_seqs, max_pages), "lens": (n_seqs,), "refs": (n_pages,), "status": (1,)}
        types = {"k": torch.uint8, "v": torch.uint8, "k_scale": torch.float32, "v_scale": torch.float32}
        for name, shape in shapes.items():
            t = tensors.pop(name, None)
            if t is None:
                t = torch.zeros(shape, dtype=types.get(name, torch.int32), device=dev)
                if name == "table":
                    t.fill_(-1)
                elif name.endswith("scale"):
                    t.fill_(1.0)
            self._checked(t, name, types.get(name, torch.int32), shape)
            setattr(self, "status_word" if name == "status" else name, t)
        if tensors:
            raise ValueError(f"unknown tensors: {sorted(tensors)}")
        self.n_layers, self.n_pages, self.page, self.n_kv_heads = n_layers, n_pages, page, n_kv_heads
        self.head_dim, self.n_seqs, self.max_pages = head_dim, n_seqs, max_pages
        self.struct = la_kv8_cache(n_layers, n_pages, page, n_kv_heads, head_dim, n_seqs, max_pages,
                                   *[getattr(self, "status_word" if n == "status" else n).data_ptr()
                                     for n in shapes])
        self._ref = ctypes.addressof(self.struct)
        lib, P, I = load_library(), ctypes.c_void_p, ctypes.c_int32
        # The arguments as packed bytes: a ctypes structure costs more to fill than a call to launch.
        self._fn = {}
        for name, kinds in (("la_kv8_attention", (P, ctypes.c_int64)), ("la_kv8_append", (P, ctypes.c_int64)),
                            ("la_kv8_fork", (P, I)), ("la_kv8_free", (P, I)),
                            ("la_kv8_compact", (P, P, P, ctypes.c_int64)), ("la_kv8_status", ()), ("la_kv8_norm_rope", ()),
                            ("la_kv8_attention_window", (I, I, P, ctypes.c_int64))):
            f = lib[name]
            f.argtypes, f.restype = [P, P, *kinds, P], ctypes.c_int
            self._fn[name] = f
        self._ws = self.workspace()
        self._ws_ptr, self._ws_bytes = self._ws.data_ptr(), self._ws.numel()
        self._stored = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self._live = torch.zeros(1, dtype=torch.int32, device=dev)

    def workspace(self):
        """A workspace for calls that overlap with others on this cache."""
        with self._torch.cuda.device(self.device):
            return self._torch.empty(la_kv8_workspace(self.struct), dtype=self._torch.uint8, device=self.device)

    # -------------------------------------------------------------- checks
    def _checked(self, t, name, dtype, shape):
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {self.device}, not "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _ints(self, t, name, n):
        """Address of an int32 device vector of n values; 0 for None."""
        return 0 if t is None else self._checked(t, name, self._torch.int32, (n,))

    def _rows(self, t, name, heads, dtype=None):
        """bf16 (or `dtype`) [rows, heads, dim] with dense (heads, dim): rows, row stride."""
        dtype, sh, st = dtype or self._bf16, t.shape, t.stride()
        if len(sh) == 3:
            (n, h, d), (row, head, one) = sh, st
            if d == self.head_dim and one == 1 and (head == d or h == 1) and (h == heads or not heads) and t.dtype is dtype and t.get_device() == self._index:
                return n, row if n > 1 else h * d
        raise ValueError(f"{name} must be a {str(dtype)[6:]} tensor [rows, {heads or 'heads'}, {self.head_dim}] on {self.device} "
                         f"with dense heads, not {t.dtype} {tuple(sh)} strides {st} on {t.device}")

    def _layers(self, t, name, rows):
        """bf16 [layers, rows, kv heads, dim] with dense (heads, dim): row and layer strides."""
        sh, st, h, d = t.shape, t.stride(), self.n_kv_heads, self.head_dim
        if t.dtype is not self._torch.bfloat16 or t.get_device() != self._index or sh != (self.n_layers, rows, h, d) or st[3] != 1 \
                or (st[2] != d and h > 1):
            raise ValueError(f"{name} must be a bfloat16 tensor [{self.n_layers} layers, {rows or 'rows'}, {h}, {d}] on {self.device} "
                             f"with dense heads, not {t.dtype} {tuple(sh)} strides {st} on {t.device}")
        return st[1] if rows > 1 else h * d, st[0]

    def _workspace(self, ws):
        if ws is None:
            return self._ws_ptr, self._ws_bytes
        if ws.get_device() != self._index or not ws.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def _call(self, fn, where, *args, stream=None):
        """fn(cache, *args, stream) with the cache's device current."""
        c = self._torch._C
        st = c._cuda_getCurrentRawStream(self._index) if stream is None else stream.cuda_stream
        if c._cuda_getDevice() == self._index:
            rc = fn(self._ref, *args, st)
        else:
            with self._torch.cuda.device(self._index):
                rc = fn(self._ref, *args, st)
        if rc:
            _check(rc, where)

    # -------------------------------------------------------------- calls
    def attention(self, q, k=None, v=None, row_start=None, layer: int = 0, vis=None, out=None, scale: float = 0.0,
                  max_rows: int = 0, max_len: int = 0, workspace=None, stream=None, window: int = 0, sinks: int = 0):
        """Attention of the rows q [rows, heads, dim] over their sequences'
        cached tokens and the visible new rows k, v [rows, kv heads, dim];
        see la_kv8_attention.  max_rows and max_len are bounds that the host
        knows (0: none); they steer the split of the work only, and a batch
        without max_rows is slow.  window (0: none) and sinks: a row sees the
        last `window` and the first `sinks` of its keys alone; see
        la_kv8_attention_window.  Returns out."""
        rows, qs = self._rows(q, "q", 0)
        heads = q.shape[1]
        if out is None:
            out = _empty(stream, rows, heads, self.head_dim, dtype=q.dtype, device=self.device)
        n, os_ = self._rows(out, "out", heads)
        kp = vp = ks = vs = 0
        if k is not None and v is not None:
            nk, ks = self._rows(k, "k", self.n_kv_heads)
            nv, vs = self._rows(v, "v", self.n_kv_heads)
            if nk != rows or nv != rows:
                raise ValueError(f"k and v must have q's {rows} rows, not {nk} and {nv}")
            kp, vp = k.data_ptr(), v.data_ptr()
        elif k is not None or v is not None:
            raise ValueError("k and v come together")
        if n != rows:
            raise ValueError(f"out must have q's {rows} rows, not {n}")
        ws, wb = self._workspace(workspace)
        args = _KV8_ATTN.pack(layer, heads, rows, max_rows, max_len, qs, ks, vs, os_,
                              self._ints(row_start, "row_start", self.n_seqs + 1), q.data_ptr(), kp, vp,
                              0 if vis is None else self._checked(vis, "vis", self._torch.int32, (rows, 8)), out.data_ptr(), scale)
        if window == 0 and sinks == 0:
            self._call(self._fn["la_kv8_attention"], "la_kv8_attention", args, ws, wb, stream=stream)
        else:
            if abs(window) >> 31 or abs(sinks) >> 31:   # ctypes would cut them
                raise ValueError(f"window must be 1 .. 2^30 and sinks 0 .. 2^30, not {window} and {sinks}")
            self._call(self._fn["la_kv8_attention_window"], "la_kv8_attention_window", args, window, sinks, ws, wb, stream=stream)
        return out

    def norm_rope(self, q, k, v=None, q_weight=None, k_weight=None, eps: float = 1e-5, rope_base: float = 10000.0, inv_freq=None,
                  row_start=None, pos=None, depth=None, out=None, stream=None):
        """Rows of a projection for attention() and append(): the heads of q
        [rows, heads, dim] and k [rows, kv heads, dim] (float32 or bfloat16) are
        normed (with q_weight, k_weight [dim]; None: not), rotated by their
        positions behind the sequences' cached tokens, and rounded to bfloat16,
        with v rounded along; see la_kv8_norm_rope.  pos [rows]: positions that
        have nothing to do with the cache; depth [rows]: places of a tree's
        rows.  Returns (q, k) or (q, k, v), or writes to `out`, which may be
        the bfloat16 inputs themselves."""
        dtype, bf16, f32, heads, kv = q.dtype, self._bf16, self._f32, q.shape[1] if q.dim() == 3 else 0, self.n_kv_heads
        if dtype is not f32 and dtype is not bf16:
            raise ValueError(f"q must be float32 or bfloat16, not {dtype}")
        n, qs = self._rows(q, "q", 0, dtype)
        n_k, ks = self._rows(k, "k", kv, dtype)
        n_v, vs = (n, 0) if v is None else self._rows(v, "v", kv, dtype)
        if n_k != n or n_v != n:
            raise ValueError(f"k and v must have q's {n} rows, not {n_k} and {n_v}")
        if out is None:
            out = tuple([_empty(stream, *t.shape, dtype=bf16, device=self.device) for t in ((q, k) if v is None else (q, k, v))])
        elif len(out) != (2 if v is None else 3):
            raise ValueError(f"out must be {'q and k' if v is None else 'q, k and v'}, not {len(out)} tensors")
        qo, ko, vo = out if v is not None else (*out, None)
        m, qos = self._rows(qo, "out's q", heads)
        m_k, kos = self._rows(ko, "out's k", kv)
        m_v, vos = (n, 0) if vo is None else self._rows(vo, "out's v", kv)
        if m != n or m_k != n or m_v != n:
            raise ValueError(f"out must have q's {n} rows, not {m}, {m_k} and {m_v}")
        weight = k_weight if q_weight is None else q_weight
        kind = bf16 if weight is None else weight.dtype
        if kind is not f32 and kind is not bf16:
            raise ValueError(f"q_weight and k_weight must be float32 or bfloat16, not {kind}")
        dim = (self.head_dim,)
        args = _KV8_QKV.pack(heads, n, LA_F32 if dtype is f32 else LA_BF16, LA_F32 if kind is f32 else LA_BF16, eps, rope_base, qs, ks, vs, qos, kos, vos,
                             0 if row_start is None else self._ints(row_start, "row_start", self.n_seqs + 1), 0 if pos is None else self._ints(pos, "pos", n),
                             0 if depth is None else self._ints(depth, "depth", n), q.data_ptr(), k.data_ptr(), 0 if v is None else v.data_ptr(),
                             0 if q_weight is None else self._checked(q_weight, "q_weight", kind, dim), 0 if k_weight is None else self._checked(k_weight, "k_weight", kind, dim),
                             0 if inv_freq is None else self._checked(inv_freq, "inv_freq", f32, (self.head_dim // 2,)),
                             qo.data_ptr(), ko.data_ptr(), 0 if vo is None else vo.data_ptr())
        self._call(self._fn["la_kv8_norm_rope"], "la_kv8_norm_rope", args, stream=stream)
        return out if type(out) is tuple else tuple(out)

    def append(self, k, v, row_start=None, row_idx=None, stored=None, max_rows: int = 0, workspace=None, stream=None):
        """Append the rows of k, v [layers, rows, kv heads, dim] (or the rows
        row_idx of them) behind the sequences; see la_kv8_append.  max_rows:
        the most rows of one sequence; with many slots the call is slow without.
        Returns stored [seqs], the rows stored for each sequence (without `stored`, a
        tensor that the next append overwrites)."""
        n = k.shape[1] if k.dim() == 4 else 0
        ks, vs = self._layers(k, "k", n), self._layers(v, "v", n)
        stored = self._stored if stored is None else stored
        ws, wb = self._workspace(workspace)
        args = _KV8_ROWS.pack(n if row_idx is None else row_idx.numel(), n, max_rows, ks[0], vs[0], ks[1], vs[1],
                              self._ints(row_start, "row_start", self.n_seqs + 1),
                              0 if row_idx is None else self._ints(row_idx, "row_idx", row_idx.numel()), k.data_ptr(), v.data_ptr(),
                              self._ints(stored, "stored", self.n_seqs))
        self._call(self._fn["la_kv8_append"], "la_kv8_append", args, ws, wb, stream=stream)
        return stored

    def fork(self, src, dst, stream=None) -> None:
        """The empty slots dst continue the sequences src (int32 device vectors); see la_kv8_fork."""
        n = src.numel()
        self._call(self._fn["la_kv8_fork"], "la_kv8_fork", self._ints(src, "src", n), self._ints(dst, "dst", n), n, stream=stream)

    def free(self, slots, keep=None, stream=None) -> None:
        """Shorten the sequences in slots to keep tokens (None: 0); see la_kv8_free."""
        n = slots.numel()
        self._call(self._fn["la_kv8_free"], "la_kv8_free", self._ints(slots, "slots", n), self._ints(keep, "keep", n), n, stream=stream)

    def compact(self, table_out=None, refs_out=None, n_live=None, workspace=None, stream=None):
        """Move the used pages to the pool's front; see la_kv8_compact.  The new
        table and counts go to table_out, refs_out (default: in place).
        Returns n_live, an int32 tensor with the number of used pages."""
        table_out = self.table if table_out is None else table_out
        refs_out = self.refs if refs_out is None else refs_out
        n_live = self._live if n_live is None else n_live
        ws, wb = self._workspace(workspace)
        self._call(self._fn["la_kv8_compact"], "la_kv8_compact",
                   self._checked(table_out, "table_out", self._torch.int32, (self.n_seqs, self.max_pages)),
                   self._ints(refs_out, "refs_out", self.n_pages), self._ints(n_live, "n_live", 1), ws, wb, stream=stream)
        return n_live

    def status(self, stream=None) -> None:
        """Wait for the stream and raise LaError for what earlier calls met; see la_kv8_status."""
        self._call(self._fn["la_kv8_status"], "la_kv8_status", None, stream=stream)


class Decoder:
    """A la_handle over DeviceWeights (or a host weight dict, uploaded here).
    With `kv_cache` (a Kv8Cache) its KV cache is slot `slot` of that cache."""

    def __init__(self, weights, N: int, W: int, G: int, max_seq: int, temperature: float = 0.0,
                 seed: int = 0, prompt_as_reference: bool = False, pool_cap: int = 0, stream=None, device="cuda",
                 profile: bool = False, top_k: int = 0, top_p: float = 1.0, pool_policy: str = "fifo",
                 kv_cache: Optional["Kv8Cache"] = None, slot: int = 0):
        self.weights = weights if isinstance(weights, DeviceWeights) else DeviceWeights(weights, device)
        self.dims, self.N, self.W, self.G = self.weights.dims, N, W, G
        self.stream = stream
        sp = stream.cuda_stream if stream is not None else None
        policies = {"fifo": LA_POOL_FIFO, "lru": LA_POOL_LRU, "lfu": LA_POOL_LFU}
        if pool_policy not in policies:
            raise ValueError(f"pool_policy must be 'fifo', 'lru' or 'lfu', not {pool_policy!r}")
        o = la_opts(N, W, G, max_seq, int(prompt_as_reference), pool_cap, temperature, seed, sp, int(profile),
                    top_k, top_p, policies[pool_policy])
        self.kv_cache, self.slot = kv_cache, slot
        if kv_cache is None:
            self.h = la_create(self.weights.dims_struct, self.weights.struct, o)
        else:
            if kv_cache.device != self.weights.device:
                raise ValueError(f"kv_cache must be on the weights' device {self.weights.device}, not {kv_cache.device}")
            if stream is not None:   # the cache's tensors are written on the current one
                stream.wait_stream(kv_cache._torch.cuda.current_stream(kv_cache.device))
            self.h = la_create_kv8(self.weights.dims_struct, self.weights.struct, o, kv_cache.struct, slot)

    def prefill(self, prompt) -> int:
        return la_prefill(self.h, prompt)

    def step(self) -> List[int]:
        return la_step(self.h, self.N)

    def ar_step(self) -> int:
        return la_ar_step(self.h)

    def generate(self, prompt, max_new: int):
        return la_generate(self.h, prompt, max_new)

    def stats(self) -> dict:
        return la_stats(self.h)

    def export_state(self) -> dict:
        return la_export_state(self.h, self.N, self.W)

    def import_state(self, tokens, window, records, uses=None) -> None:
        la_import_state(self.h, self.N, self.W, tokens, window, records, uses)

    def debug_logits(self) -> np.ndarray:
        return la_debug_logits(self.h)

    def fork_from(self, src: "Decoder") -> None:
        """Continue from src's state in this decoder's slot of the same cache."""
        la_fork(src.h, self.h)

    def close(self):
        if getattr(self, "h", None):
            la_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
