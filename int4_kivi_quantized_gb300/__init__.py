"""Python binding of libs4kv.so, the int4 KIVI-style paged KV cache for GB300.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. Functions carry the C ABI's names (include/s4kv.h); pointer arguments
accept a torch tensor (its data_ptr), an int address or None; `stream` accepts a
torch.cuda.Stream, an int handle or None (the current torch stream).

There is no fallback: if the shared library is missing or fails to load,
importing this package raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libs4kv.so")

S4KV_OK = 0
S4KV_ERR_INVALID_ARG = 1
S4KV_ERR_UNSUPPORTED = 2
S4KV_ERR_CUDA = 3
S4KV_ERR_POOL_TOO_SMALL = 4
S4KV_ERR_DEVICE = 5
S4KV_ERR_DEVICE_TIMEOUT = 6
S4KV_ERR_WORKSPACE_TOO_SMALL = 7

S4KV_F16, S4KV_BF16, S4KV_F32 = 0, 1, 2

S4KV_DEV_BAD_PAGE, S4KV_DEV_BAD_LENGTH, S4KV_DEV_BAD_SLOT = 1, 2, 3
S4KV_DEV_BAD_TABLE, S4KV_DEV_BAD_CU, S4KV_DEV_TIMEOUT = 4, 5, 6
S4KV_DEV_BAD_POSITION = 7

S4KV_BITS_INT8 = 0x108

S4KV_OPT_DECODE_WARPS, S4KV_OPT_DECODE_IMPL, S4KV_OPT_WAIT_NS, S4KV_OPT_TAIL_COST = 1, 2, 3, 4
S4KV_OPT_KEY_SPLIT = 5
S4KV_OPT_MQ_KERNEL = 6
S4KV_OPT_WINDOW_FORM = 7


class S4KVError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {s4kv_strerror(code)} (status {code})")
        self.code = code


class s4kv_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_layers", "num_pages", "page_size", "num_kv_heads", "head_dim", "group_k", "group_v",
        "residual_v", "max_slots", "dtype", "bits")]


class s4kv_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "pool_bytes", "status_offset", "lens_offset", "layer_offset", "layer_stride", "page_stride",
        "record_bytes", "kcode_offset", "kmeta_offset", "vcode_offset", "vmeta_offset",
        "kring_offset", "kring_slot_stride", "kring_head_stride", "kring_row_stride",
        "vring_offset", "vring_slot_stride", "vring_head_stride", "vring_row_stride", "scale_offset")]


class s4kv_rope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("max_positions", ctypes.c_int), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class s4kv_scores(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("window", ctypes.c_int),
                ("num_sinks", ctypes.c_int), ("first", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


class s4kv_kv_bytes_report(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in (
        "fp16_equiv_bytes", "code_bytes", "meta_bytes", "residual_bytes", "paged_bytes")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(or python int4_kivi_quantized_gb300/build.py)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "s4kv_cache_bytes": [ctypes.POINTER(s4kv_config), ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
        "s4kv_cache_create": [ctypes.POINTER(s4kv_config), P, SZ, ctypes.POINTER(P)],
        "s4kv_cache_destroy": [P],
        "s4kv_get_layout": [P, ctypes.POINTER(s4kv_layout)],
        "s4kv_append": [P, I, P, P, I, P, P, P, P, I, I, P],
        "s4kv_decode_workspace_bytes": [P, I, I, I, ctypes.POINTER(SZ)],
        "s4kv_decode_attention": [P, I, P, I, P, I, P, P, I, ctypes.c_float, P, I, P, SZ, I, P],
        "s4kv_decode_attention_noalloc": [P, I, P, I, P, I, P, P, I, ctypes.c_float, P, I, I, P],
        "s4kv_decode_step": [P, I, P, P, P, I, P, I, P, P, I, ctypes.c_float, P, I, P, SZ, I, P],
        "s4kv_multi_query_workspace_bytes": [P, I, I, I, I, ctypes.POINTER(SZ)],
        "s4kv_multi_query_attention": [P, I, P, I, I, P, I, P, P, I, ctypes.c_float, P, I, P, SZ, I, P],
        "s4kv_append_rope": [P, I, ctypes.POINTER(s4kv_rope), P, P, I, P, P, P, P, I, I, P, I, P, P],
        "s4kv_window_workspace_bytes": [P, I, I, I, I, ctypes.POINTER(SZ)],
        "s4kv_window_attention": [P, I, P, I, I, I, I, P, I, P, P, I, ctypes.c_float, P, I, P, SZ, I, P],
        "s4kv_score_attention": [P, I, ctypes.POINTER(s4kv_scores), P, I, I, P, I, P, P, I, ctypes.c_float, P, I, P, SZ, I, P],
        "s4kv_prompt_workspace_bytes": [P, I, I, I, I, ctypes.c_longlong, ctypes.POINTER(SZ)],
        "s4kv_prompt_attention": [P, I, ctypes.POINTER(s4kv_scores), P, I, P, I, P, I, P, P, I, ctypes.c_float, P, I, P,
                                  SZ, I, ctypes.c_longlong, P],
        "s4kv_take_pages": [P, P, P, I, I, P, P, P, I, P, P],
        "s4kv_release_pages": [P, P, P, I, I, P, P, P, I, P],
        "s4kv_fork": [P, P, P, I, I, P, P, P, I, P, P],
        "s4kv_gather": [P, I, P, I, P, P, P, P, I, I, P, P, I, P],
        "s4kv_dequant_debug": [P, I, I, P, I, P, P, P],
        "s4kv_get_status": [P, P, ctypes.POINTER(I)],
        "s4kv_kv_bytes": [ctypes.POINTER(s4kv_config), ctypes.c_double, ctypes.c_double,
                          ctypes.POINTER(s4kv_kv_bytes_report)],
        "s4kv_set_option": [P, I, ctypes.c_longlong],
        "s4kv_capacity_tokens": [ctypes.POINTER(s4kv_config), ctypes.c_double, ctypes.POINTER(ctypes.c_longlong),
                                 ctypes.POINTER(ctypes.c_longlong)],
        "s4kv_set_fp8_scales": [P, I, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_float), P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = I
    L.s4kv_strerror.argtypes = [I]
    L.s4kv_strerror.restype = ctypes.c_char_p
    return L


_lib = _load()


def _ptr(x):
    # an int or None goes to a c_void_p argument as it is
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, what: str):
    if rc != S4KV_OK:
        raise S4KVError(rc, what)


def s4kv_strerror(code: int) -> str:
    return _lib.s4kv_strerror(int(code)).decode()


def make_config(num_layers, num_pages, num_kv_heads, residual_v, max_slots, dtype=S4KV_F16,
                head_dim=128, page_size=16, group_k=32, group_v=32, bits=4) -> s4kv_config:
    return s4kv_config(num_layers, num_pages, page_size, num_kv_heads, head_dim, group_k, group_v,
                       residual_v, max_slots, dtype, bits)


def s4kv_capacity_tokens(cfg: s4kv_config, budget_bytes: float):
    """(tokens, pages) of KV that fit in budget_bytes for this configuration."""
    t, p = ctypes.c_longlong(), ctypes.c_longlong()
    _check(_lib.s4kv_capacity_tokens(ctypes.byref(cfg), float(budget_bytes), ctypes.byref(t), ctypes.byref(p)),
           "s4kv_capacity_tokens")
    return t.value, p.value


def s4kv_cache_bytes(cfg: s4kv_config):
    pool = ctypes.c_size_t()
    per = ctypes.c_size_t()
    _check(_lib.s4kv_cache_bytes(ctypes.byref(cfg), ctypes.byref(pool), ctypes.byref(per)),
           "s4kv_cache_bytes")
    return pool.value, per.value


def s4kv_kv_bytes(cfg: s4kv_config, batch: float, tokens: float) -> dict:
    r = s4kv_kv_bytes_report()
    _check(_lib.s4kv_kv_bytes(ctypes.byref(cfg), float(batch), float(tokens), ctypes.byref(r)),
           "s4kv_kv_bytes")
    return {n: getattr(r, n) for n, _ in r._fields_}


def s4kv_cache_create(cfg: s4kv_config, pool, pool_bytes: int):
    h = ctypes.c_void_p()
    _check(_lib.s4kv_cache_create(ctypes.byref(cfg), _ptr(pool), int(pool_bytes), ctypes.byref(h)),
           "s4kv_cache_create")
    return h


def s4kv_set_fp8_scales(h, layer, k_scale, v_scale, stream=None):
    """FP8 pools: per-kv-head key and value scales of one layer (host sequences)."""
    ks = (ctypes.c_float * len(k_scale))(*[float(x) for x in k_scale])
    vs = (ctypes.c_float * len(v_scale))(*[float(x) for x in v_scale])
    _check(_lib.s4kv_set_fp8_scales(h, int(layer), ks, vs, _stream(stream)), "s4kv_set_fp8_scales")


def s4kv_cache_destroy(h):
    _check(_lib.s4kv_cache_destroy(h), "s4kv_cache_destroy")


def s4kv_get_layout(h) -> s4kv_layout:
    lay = s4kv_layout()
    _check(_lib.s4kv_get_layout(h, ctypes.byref(lay)), "s4kv_get_layout")
    return lay


def s4kv_set_option(h, option: int, value: int):
    _check(_lib.s4kv_set_option(h, int(option), int(value)), "s4kv_set_option")


def s4kv_append(h, layer, k, v, num_new_tokens, cu_new, slot_ids, seq_lens_before, block_table,
                bt_stride, n, stream=None):
    _check(_lib.s4kv_append(h, int(layer), _ptr(k), _ptr(v), int(num_new_tokens), _ptr(cu_new),
                            _ptr(slot_ids), _ptr(seq_lens_before), _ptr(block_table),
                            int(bt_stride), int(n), _stream(stream)), "s4kv_append")


def s4kv_decode_workspace_bytes(h, B, num_q_heads, max_seq_len) -> int:
    out = ctypes.c_size_t()
    _check(_lib.s4kv_decode_workspace_bytes(h, int(B), int(num_q_heads), int(max_seq_len),
                                            ctypes.byref(out)), "s4kv_decode_workspace_bytes")
    return out.value


def s4kv_decode_attention(h, layer, q, num_q_heads, block_table, bt_stride, seq_lens, slot_ids, B,
                          sm_scale, out, out_dtype, workspace, ws_bytes, max_seq_len, stream=None):
    _check(_lib.s4kv_decode_attention(h, int(layer), _ptr(q), int(num_q_heads), _ptr(block_table),
                                      int(bt_stride), _ptr(seq_lens), _ptr(slot_ids), int(B),
                                      float(sm_scale), _ptr(out), int(out_dtype), _ptr(workspace),
                                      int(ws_bytes), int(max_seq_len), _stream(stream)),
           "s4kv_decode_attention")


def s4kv_multi_query_workspace_bytes(h, B, num_q_tokens, num_q_heads, max_seq_len) -> int:
    out = ctypes.c_size_t()
    _check(_lib.s4kv_multi_query_workspace_bytes(h, int(B), int(num_q_tokens), int(num_q_heads),
                                                 int(max_seq_len), ctypes.byref(out)),
           "s4kv_multi_query_workspace_bytes")
    return out.value


def s4kv_multi_query_attention(h, layer, q, num_q_tokens, num_q_heads, block_table, bt_stride, seq_lens,
                               slot_ids, B, sm_scale, out, out_dtype, workspace, ws_bytes, max_seq_len,
                               stream=None):
    _check(_lib.s4kv_multi_query_attention(h, int(layer), _ptr(q), int(num_q_tokens), int(num_q_heads),
                                           _ptr(block_table), int(bt_stride), _ptr(seq_lens), _ptr(slot_ids),
                                           int(B), float(sm_scale), _ptr(out), int(out_dtype), _ptr(workspace),
                                           int(ws_bytes), int(max_seq_len), _stream(stream)),
           "s4kv_multi_query_attention")


def s4kv_append_rope(h, layer, rope: s4kv_rope, k, v, num_new_tokens, cu_new, slot_ids, seq_lens_before, block_table,
                     bt_stride, n, q=None, num_q_heads=0, q_out=None, stream=None):
    """s4kv_append with the keys (and the queries q into q_out) rotated by their positions on the way."""
    _check(_lib.s4kv_append_rope(h, int(layer), ctypes.byref(rope), _ptr(k), _ptr(v), int(num_new_tokens),
                                 _ptr(cu_new), _ptr(slot_ids), _ptr(seq_lens_before), _ptr(block_table),
                                 int(bt_stride), int(n), _ptr(q), int(num_q_heads), _ptr(q_out),
                                 _stream(stream)), "s4kv_append_rope")


def s4kv_window_workspace_bytes(h, B, num_q_tokens, num_q_heads, max_seq_len) -> int:
    out = ctypes.c_size_t()
    _check(_lib.s4kv_window_workspace_bytes(h, int(B), int(num_q_tokens), int(num_q_heads), int(max_seq_len),
                                            ctypes.byref(out)), "s4kv_window_workspace_bytes")
    return out.value


def s4kv_window_attention(h, layer, q, num_q_tokens, num_q_heads, window, num_sinks, block_table, bt_stride,
                          seq_lens, slot_ids, B, sm_scale, out, out_dtype, workspace, ws_bytes, max_seq_len,
                          stream=None):
    """Causal attention of the last tokens within a sliding window, the first tokens kept visible."""
    _check(_lib.s4kv_window_attention(h, int(layer), _ptr(q), int(num_q_tokens), int(num_q_heads), int(window),
                                      int(num_sinks), _ptr(block_table), int(bt_stride), _ptr(seq_lens),
                                      _ptr(slot_ids), int(B), float(sm_scale), _ptr(out), int(out_dtype),
                                      _ptr(workspace), int(ws_bytes), int(max_seq_len), _stream(stream)),
           "s4kv_window_attention")


def s4kv_score_attention(h, layer, scores: s4kv_scores, q, num_q_tokens, num_q_heads, block_table, bt_stride, seq_lens,
                         slot_ids, B, sm_scale, out, out_dtype, workspace, ws_bytes, max_seq_len, stream=None):
    """Causal attention of the last tokens with a score form."""
    _check(_lib.s4kv_score_attention(h, int(layer), ctypes.byref(scores), _ptr(q), int(num_q_tokens), int(num_q_heads),
                                     _ptr(block_table), int(bt_stride), _ptr(seq_lens), _ptr(slot_ids), int(B),
                                     float(sm_scale), _ptr(out), int(out_dtype), _ptr(workspace), int(ws_bytes),
                                     int(max_seq_len), _stream(stream)), "s4kv_score_attention")


def s4kv_prompt_workspace_bytes(h, n, num_q, num_q_heads, max_seq_len, sum_seq_lens) -> int:
    out = ctypes.c_size_t()
    _check(_lib.s4kv_prompt_workspace_bytes(h, int(n), int(num_q), int(num_q_heads), int(max_seq_len), int(sum_seq_lens),
                                            ctypes.byref(out)), "s4kv_prompt_workspace_bytes")
    return out.value


def s4kv_prompt_attention(h, layer, scores, q, num_q, cu_q, num_q_heads, block_table, bt_stride, seq_lens, slot_ids, n,
                          sm_scale, out, out_dtype, workspace, ws_bytes, max_seq_len, sum_seq_lens, stream=None):
    """Causal attention of ragged prompt chunks with a score form (an s4kv_scores, or None)."""
    _check(_lib.s4kv_prompt_attention(h, int(layer), None if scores is None else ctypes.byref(scores), _ptr(q), int(num_q),
                                      _ptr(cu_q), int(num_q_heads), _ptr(block_table), int(bt_stride), _ptr(seq_lens),
                                      _ptr(slot_ids), int(n), float(sm_scale), _ptr(out), int(out_dtype), _ptr(workspace),
                                      int(ws_bytes), int(max_seq_len), int(sum_seq_lens), _stream(stream)),
           "s4kv_prompt_attention")


def s4kv_take_pages(h, refs, block_table, bt_stride, rows, lens, new_lens, slot_ids, n, taken, stream=None):
    """Free pages into the table rows of growing sequences."""
    _check(_lib.s4kv_take_pages(h, _ptr(refs), _ptr(block_table), int(bt_stride), int(rows), _ptr(lens), _ptr(new_lens),
                                _ptr(slot_ids), int(n), _ptr(taken), _stream(stream)), "s4kv_take_pages")


def s4kv_release_pages(h, refs, block_table, bt_stride, rows, first, last, slot_ids, n, stream=None):
    """Table entries given up, their pages' counts down by one."""
    _check(_lib.s4kv_release_pages(h, _ptr(refs), _ptr(block_table), int(bt_stride), int(rows), _ptr(first), _ptr(last),
                                   _ptr(slot_ids), int(n), _stream(stream)), "s4kv_release_pages")


def s4kv_fork(h, refs, block_table, bt_stride, rows, src, dst, seq_lens, n, taken, stream=None):
    """Sequences continued in other slots on shared pages."""
    _check(_lib.s4kv_fork(h, _ptr(refs), _ptr(block_table), int(bt_stride), int(rows), _ptr(src), _ptr(dst), _ptr(seq_lens),
                          int(n), _ptr(taken), _stream(stream)), "s4kv_fork")


def s4kv_gather(h, layer, block_table, bt_stride, seq_lens, slot_ids, first_token, cu_rows, num_rows, n, out_k, out_v,
                out_dtype, stream=None):
    """Restores token ranges of n sequences into dense rows."""
    _check(_lib.s4kv_gather(h, int(layer), _ptr(block_table), int(bt_stride), _ptr(seq_lens), _ptr(slot_ids),
                            _ptr(first_token), _ptr(cu_rows), int(num_rows), int(n), _ptr(out_k), _ptr(out_v),
                            int(out_dtype), _stream(stream)), "s4kv_gather")


def s4kv_decode_step(h, layer, k_new, v_new, q, num_q_heads, block_table, bt_stride, seq_lens, slot_ids, B,
                     sm_scale, out, out_dtype, workspace, ws_bytes, max_seq_len, stream=None):
    """One token appended per sequence and decode attention over the result, in one launch."""
    _check(_lib.s4kv_decode_step(h, int(layer), _ptr(k_new), _ptr(v_new), _ptr(q), int(num_q_heads),
                                 _ptr(block_table), int(bt_stride), _ptr(seq_lens), _ptr(slot_ids), int(B),
                                 float(sm_scale), _ptr(out), int(out_dtype), _ptr(workspace), int(ws_bytes),
                                 int(max_seq_len), _stream(stream)), "s4kv_decode_step")


def s4kv_decode_attention_noalloc(h, layer, q, num_q_heads, block_table, bt_stride, seq_lens, slot_ids,
                                  B, sm_scale, out, out_dtype, max_seq_len, stream=None):
    """Decode attention with the library's built-in device scratch (no workspace)."""
    _check(_lib.s4kv_decode_attention_noalloc(h, int(layer), _ptr(q), int(num_q_heads),
                                              _ptr(block_table), int(bt_stride), _ptr(seq_lens),
                                              _ptr(slot_ids), int(B), float(sm_scale), _ptr(out),
                                              int(out_dtype), int(max_seq_len), _stream(stream)),
           "s4kv_decode_attention_noalloc")


def s4kv_dequant_debug(h, layer, slot, block_table_row, seq_len, out_k, out_v, stream=None):
    _check(_lib.s4kv_dequant_debug(h, int(layer), int(slot), _ptr(block_table_row), int(seq_len),
                                   _ptr(out_k), _ptr(out_v), _stream(stream)), "s4kv_dequant_debug")


def s4kv_get_status(h, stream=None):
    """Returns (status, detail); does not raise on a device-side status."""
    detail = ctypes.c_int(0)
    rc = _lib.s4kv_get_status(h, _stream(stream), ctypes.byref(detail))
    return rc, detail.value


class Rope:
    """A rotation table for append_rope: `table` [max_positions, rotary_dim] in fp32 on the cache's
    device, the cosines of the rotary_dim / 2 angles of each position, then their sines. It is
    used in place and kept alive by this object."""

    def __init__(self, table, interleaved=False):
        import torch
        if table.dim() != 2 or table.dtype != torch.float32 or not table.is_contiguous():
            raise ValueError("the rotation table is a contiguous fp32 tensor [max_positions, rotary_dim]")
        self.table = table
        self.interleaved = bool(interleaved)
        self.c = s4kv_rope(table.data_ptr(), table.shape[0], table.shape[1], int(self.interleaved))
        self.ref = ctypes.byref(self.c)


class Scores:
    """A model's score form for attend and prompt: scores capped at cap tanh(x / cap) (0: as they
    are), less slopes[head] |p - t| (fp32 [H_q] on the cache's device, kept alive by this object),
    within the newest `window` tokens (0: all) and the sequence's first `num_sinks` (which every document
    packed behind them sees, too)."""

    def __init__(self, cap=0.0, slopes=None, window=0, num_sinks=0):
        if slopes is not None:
            import torch
            if slopes.dim() != 1 or slopes.dtype != torch.float32 or not slopes.is_contiguous():
                raise ValueError("the slopes are a contiguous fp32 tensor [H_q]")
        if cap != 0 and not 2.0 ** -60 <= cap <= 2.0 ** 60:
            raise ValueError("a cap is 2^-60 .. 2^60, or 0 for none")
        if window < 0 or num_sinks < 0:
            raise ValueError("window and num_sinks are not negative")
        self.cap, self.slopes = float(cap), slopes
        wide = 0x7fffffff
        self.window, self.num_sinks = min(int(window), wide), min(int(num_sinks), wide)

        self._alone = ctypes.byref(s4kv_scores(self.cap, _address(slopes), self.window, self.num_sinks, None, None))

    def __setattr__(self, name, value):
        if hasattr(self, "_alone"):   # (which holds the slopes' address)
            raise AttributeError("a Scores does not change: make another")
        object.__setattr__(self, name, value)

    def ref(self, first, prefix):
        """The s4kv_scores of a call, by reference."""
        if first is None and prefix is None:
            return self._alone
        return ctypes.byref(s4kv_scores(self.cap, _address(self.slopes), self.window, self.num_sinks, _address(first), _address(prefix)))


def _on_its_device(f):
    """A method that runs with the cache's device as the current one."""
    @functools.wraps(f)
    def call(self, *args, **kwargs):
        if self._current_device() == self._index:
            return f(self, *args, **kwargs)
        with self._torch.cuda.device(self._index):
            return f(self, *args, **kwargs)
    return call


def _address(t):
    return None if t is None else t.data_ptr()


_PLAIN = Scores()


class KVCache:
    """A cache bound to a torch-allocated device pool (torch provides memory only).

    bits: 4 (default), 2, 8 (FP8 E4M3) or "int8" (one scale per 16-token block and head).

    A call with stream= runs on that stream, and results that it makes itself are that stream's
    memory, as under torch.cuda.stream(stream); order other streams behind it before they read them."""

    def __init__(self, num_layers, num_pages, num_kv_heads, residual_v, max_slots, dtype="fp16",
                 device="cuda", bits=4):
        import torch
        self._torch = torch   # (an import statement takes a few hundred nanoseconds of a call)
        self.dtype = dtype
        self.cdtype = S4KV_F16 if dtype == "fp16" else S4KV_BF16
        self.torch_dtype = torch.float16 if dtype == "fp16" else torch.bfloat16
        bits = S4KV_BITS_INT8 if bits == "int8" else bits
        self.bits = bits
        self.cfg = make_config(num_layers, num_pages, num_kv_heads, residual_v, max_slots,
                               self.cdtype, bits=bits)
        self.pool_bytes, self.bytes_per_token_head = s4kv_cache_bytes(self.cfg)
        # 256-byte alignment is guaranteed by the caching allocator
        self.pool = torch.empty(self.pool_bytes, dtype=torch.uint8, device=device)
        self.h = s4kv_cache_create(self.cfg, self.pool, self.pool_bytes)
        self.layout = s4kv_get_layout(self.h)
        self.H = num_kv_heads
        self.R = residual_v
        self._ws = None
        self._index = self.pool.get_device()
        # (torch.cuda.current_stream builds a Stream object for every call)
        self._current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        self._current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        self._sizes = {}

    def close(self):
        if getattr(self, "h", None):
            s4kv_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_option(self, option, value):
        s4kv_set_option(self.h, option, value)

    def set_fp8_scales(self, layer, k_scale, v_scale, stream=None):
        """FP8 pools (bits=8): key and value scale of every kv head of `layer`."""
        if len(k_scale) != self.H or len(v_scale) != self.H:
            raise ValueError("one key and one value scale per kv head")
        s4kv_set_fp8_scales(self.h, layer, k_scale, v_scale, stream)

    def append(self, layer, k, v, cu_new, seq_lens_before, block_table, slot_ids=None, stream=None):
        n = seq_lens_before.numel()
        s4kv_append(self.h, layer, k, v, k.shape[0], cu_new, slot_ids, seq_lens_before,
                    block_table, block_table.shape[1], n, stream)

    def workspace(self, B, num_q_heads, max_seq_len):
        import torch
        nbytes = s4kv_decode_workspace_bytes(self.h, B, num_q_heads, max_seq_len)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.pool.device)
        return self._ws, nbytes

    def decode(self, layer, q, block_table, seq_lens, max_seq_len, out=None, out_dtype=S4KV_F32,
               slot_ids=None, sm_scale=0.0, stream=None):
        import torch
        B, Hq, _ = q.shape
        if out is None:
            dt = torch.float32 if out_dtype == S4KV_F32 else self.torch_dtype
            out = self._made(stream, torch.empty, (B, Hq, 128), dtype=dt, device=q.device)
        if self.bits == S4KV_BITS_INT8:
            nbytes = self._window_bytes(B, 1, Hq, max_seq_len)
            ws, stream = self._scratch(nbytes, stream), self._handle(stream)
        else:
            ws, nbytes = self.workspace(B, Hq, max_seq_len)
        s4kv_decode_attention(self.h, layer, q, Hq, block_table, block_table.shape[1], seq_lens,
                              slot_ids, B, sm_scale, out, out_dtype, ws, nbytes, max_seq_len, stream)
        return out

    def multi_query(self, layer, q, block_table, seq_lens, max_seq_len, out=None, out_dtype=S4KV_F32,
                    slot_ids=None, sm_scale=0.0, stream=None):
        """Causal attention of the last nq tokens: q [B, nq, H_q, 128] -> out [B, nq, H_q, 128]."""
        import torch
        B, nq, Hq, _ = q.shape
        if out is None:
            dt = torch.float32 if out_dtype == S4KV_F32 else self.torch_dtype
            out = self._made(stream, torch.empty, (B, nq, Hq, 128), dtype=dt, device=q.device)
        if self.bits == S4KV_BITS_INT8:
            nbytes = self._window_bytes(B, nq, Hq, max_seq_len)
            s4kv_multi_query_attention(self.h, layer, q, nq, Hq, block_table, block_table.shape[1], seq_lens, slot_ids, B,
                                       sm_scale, out, out_dtype, self._scratch(nbytes, stream), nbytes, max_seq_len,
                                       self._handle(stream))
            return out
        nbytes = s4kv_multi_query_workspace_bytes(self.h, B, nq, Hq, max_seq_len)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.pool.device)
        s4kv_multi_query_attention(self.h, layer, q, nq, Hq, block_table, block_table.shape[1], seq_lens,
                                   slot_ids, B, sm_scale, out, out_dtype, self._ws, nbytes, max_seq_len, stream)
        return out

    # ---- calls that check their tensors and take scratch of their own ----
    def _tensor(self, t, name, dtype, shape):
        """t is a contiguous tensor of this cache's device; shape: sizes, None for any."""
        got = t.shape
        if got == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == self._index:
            return got
        good = t.dtype is dtype and len(got) == len(shape)
        if good:
            for w, g in zip(shape, got):
                good = good and (w is None or w == g)
        if not good:
            raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} is wanted, got {t.dtype} {tuple(got)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} is not contiguous")
        if t.get_device() != self._index:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.pool.device}")
        return got

    def _handle(self, stream):
        """The cudaStream_t of `stream`: of the cache's device's current stream for None."""
        if stream is None:
            return self._current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _made(self, stream, make, *args, **kwargs):
        """make(...), a result of a call on `stream`: of that stream's memory, and kept from it while
        the current stream still uses what it was handed."""
        if stream is None:
            return make(*args, **kwargs)
        torch = self._torch
        st = torch.cuda.ExternalStream(stream, device=self.pool.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(st):
            t = make(*args, **kwargs)
        t.record_stream(torch.cuda.current_stream(self.pool.device))
        return t

    def _scratch(self, nbytes, stream):
        """Scratch of one call, allocated on its stream: calls on other streams and captured graphs share none of it."""
        torch = self._torch
        if stream is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=self.pool.device)
        st = torch.cuda.ExternalStream(stream, device=self.pool.device) if isinstance(stream, int) else stream
        with torch.cuda.stream(st):
            return torch.empty(nbytes, dtype=torch.uint8, device=self.pool.device)

    def _window_bytes(self, B, nq, Hq, max_seq_len):
        """Scratch of a window call (on INT8 pages of any attention call): it goes by these sizes alone."""
        n = self._sizes.get((B, nq, Hq))
        if n is None:
            n = self._sizes[B, nq, Hq] = max(16, s4kv_window_workspace_bytes(self.h, B, nq, Hq, max_seq_len))
        return n

    def _out(self, out, name, shape, out_dtype, stream, like=None):
        """`out`, checked, or a new tensor (like: a checked tensor of this shape, which torch is quicker to copy)."""
        torch = self._torch
        if out_dtype == self.cdtype:
            dt = self.torch_dtype
        elif out_dtype == S4KV_F32:
            dt = torch.float32
        else:
            raise ValueError("out_dtype is S4KV_F32 or the cache's dtype")
        if out is None:
            if like is None:
                return self._made(stream, torch.empty, shape, dtype=dt, device=self.pool.device)
            if stream is None:
                return torch.empty_like(like) if like.dtype is dt else torch.empty_like(like, dtype=dt)
            return self._made(stream, torch.empty_like, like, dtype=dt)
        self._tensor(out, name, dt, shape)
        return out

    @_on_its_device
    def append_rope(self, layer, k, v, cu_new, seq_lens_before, block_table, rope, slot_ids=None, q=None, q_out=None,
                    stream=None):
        """append() with the new keys rotated by their positions on the way (rope: a Rope). With q
        [tokens, H_q, 128], the new tokens' queries are rotated too, into q_out (a new tensor if
        None; q itself is allowed), which is returned."""
        torch = self._torch
        i32, dt, n = torch.int32, self.torch_dtype, seq_lens_before.shape[0]
        tokens = self._tensor(k, "k", dt, (None, self.H, 128))[0]
        self._tensor(v, "v", dt, (tokens, self.H, 128))
        self._tensor(cu_new, "cu_new", i32, (n + 1,))
        self._tensor(seq_lens_before, "seq_lens_before", i32, (n,))
        rows, width = self._tensor(block_table, "block_table", i32, (None, None))
        if rows < n:
            raise ValueError("block_table has fewer rows than there are sequences")
        if rope.table.get_device() != self._index:
            raise ValueError(f"the rotation table is on {rope.table.device}, the cache on {self.pool.device}")
        if slot_ids is not None:
            self._tensor(slot_ids, "slot_ids", i32, (n,))
        heads = 0
        if q is not None:
            heads = self._tensor(q, "q", dt, (tokens, None, 128))[1]
            if q_out is None:
                q_out = torch.empty_like(q) if stream is None else self._made(stream, torch.empty_like, q)
            elif q_out is not q:
                self._tensor(q_out, "q_out", dt, (tokens, heads, 128))
        elif q_out is not None:
            raise ValueError("q_out without q")
        _check(_lib.s4kv_append_rope(self.h, int(layer), rope.ref, k.data_ptr(), v.data_ptr(), tokens, cu_new.data_ptr(),
                                     _address(slot_ids), seq_lens_before.data_ptr(), block_table.data_ptr(), width, n,
                                     _address(q), heads, _address(q_out), self._handle(stream)), "s4kv_append_rope")
        return q_out

    @_on_its_device
    def window(self, layer, q, block_table, seq_lens, max_seq_len, window, num_sinks=0, out=None, out_dtype=S4KV_F32,
               slot_ids=None, sm_scale=0.0, stream=None):
        """Causal attention of the last nq tokens, q [B, nq, H_q, 128], within the newest `window` tokens
        of each query's position and the first `num_sinks` tokens -> out [B, nq, H_q, 128]."""
        torch = self._torch
        B, nq, Hq, _ = self._tensor(q, "q", self.torch_dtype, (None, None, None, 128))
        rows, width = self._tensor(block_table, "block_table", torch.int32, (None, None))
        self._tensor(seq_lens, "seq_lens", torch.int32, (B,))
        if rows < B:
            raise ValueError("block_table has fewer rows than there are sequences")
        if slot_ids is not None:
            self._tensor(slot_ids, "slot_ids", torch.int32, (B,))
        out = self._out(out, "out", (B, nq, Hq, 128), out_dtype, stream, q)
        max_seq_len = int(max_seq_len)
        nbytes = self._window_bytes(B, nq, Hq, max_seq_len)
        ws = self._scratch(nbytes, stream)
        wide = 0x7fffffff   # as wide as any sequence
        _check(_lib.s4kv_window_attention(self.h, int(layer), q.data_ptr(), nq, Hq, min(int(window), wide),
                                          min(int(num_sinks), wide), block_table.data_ptr(),
                                          width, seq_lens.data_ptr(), _address(slot_ids), B, float(sm_scale), out.data_ptr(),
                                          out_dtype, ws.data_ptr(), nbytes, max_seq_len, self._handle(stream)),
               "s4kv_window_attention")
        return out

    def _form(self, scores, first, prefix, queries, n, Hq):
        """The s4kv_scores of a call, by reference: `first` has the shape `queries`, `prefix` one entry a sequence."""
        torch = self._torch
        if scores is None:
            scores = _PLAIN
        if scores.slopes is not None:
            self._tensor(scores.slopes, "slopes", torch.float32, (Hq,))
        if first is not None:
            self._tensor(first, "first", torch.int32, queries)
        if prefix is not None:
            self._tensor(prefix, "prefix", torch.int32, (n,))
        return scores.ref(first, prefix)

    @_on_its_device
    def attend(self, layer, q, block_table, seq_lens, max_seq_len, scores, first=None, prefix=None, out=None,
               out_dtype=S4KV_F32, slot_ids=None, sm_scale=0.0, stream=None):
        """Causal attention of the last nq tokens (1 to 16), q [B, nq, H_q, 128] -> out of the same shape,
        with a score form (scores: a Scores). first [B, nq]: the first token that each query's document
        has; prefix [B]: how many first tokens see one another whole."""
        torch = self._torch
        B, nq, Hq, _ = self._tensor(q, "q", self.torch_dtype, (None, None, None, 128))
        rows, width = self._tensor(block_table, "block_table", torch.int32, (None, None))
        self._tensor(seq_lens, "seq_lens", torch.int32, (B,))
        if rows < B:
            raise ValueError("block_table has fewer rows than there are sequences")
        if slot_ids is not None:
            self._tensor(slot_ids, "slot_ids", torch.int32, (B,))
        form = self._form(scores, first, prefix, (B, nq), B, Hq)
        out = self._out(out, "out", (B, nq, Hq, 128), out_dtype, stream, q)
        max_seq_len = int(max_seq_len)
        nbytes = self._window_bytes(B, nq, Hq, max_seq_len)
        ws = self._scratch(nbytes, stream)
        _check(_lib.s4kv_score_attention(self.h, int(layer), form, q.data_ptr(), nq, Hq, block_table.data_ptr(),
                                         width, seq_lens.data_ptr(), _address(slot_ids), B, float(sm_scale), out.data_ptr(),
                                         out_dtype, ws.data_ptr(), nbytes, max_seq_len, self._handle(stream)),
               "s4kv_score_attention")
        return out

    @_on_its_device
    def prompt(self, layer, q, cu_q, block_table, seq_lens, max_seq_len, sum_seq_lens=None, scores=None, first=None,
               prefix=None, out=None, out_dtype=S4KV_F32, slot_ids=None, sm_scale=0.0, stream=None):
        """Causal attention of prompt chunks, q [tokens, H_q, 128] -> out of the same shape: rows
        cu_q[i] .. cu_q[i + 1] are sequence i's newest tokens, appended before. scores: a Scores;
        first [tokens]: the first token that each query's document has; prefix [n]: how many first
        tokens see one another whole. max_seq_len and sum_seq_lens bound the sequences' lengths and
        their sum (n max_seq_len without it): scratch of 512 bytes a token and kv head is taken."""
        torch = self._torch
        i32, n = torch.int32, seq_lens.shape[0]
        tokens, Hq, _ = self._tensor(q, "q", self.torch_dtype, (None, None, 128))
        self._tensor(cu_q, "cu_q", i32, (n + 1,))
        self._tensor(seq_lens, "seq_lens", i32, (n,))
        rows, width = self._tensor(block_table, "block_table", i32, (None, None))
        if rows < n:
            raise ValueError("block_table has fewer rows than there are sequences")
        if slot_ids is not None:
            self._tensor(slot_ids, "slot_ids", i32, (n,))
        form = self._form(scores, first, prefix, (tokens,), n, Hq)
        out = self._out(out, "out", (tokens, Hq, 128), out_dtype, stream, q)
        max_seq_len = int(max_seq_len)
        total = n * max_seq_len if sum_seq_lens is None else int(sum_seq_lens)
        nbytes = s4kv_prompt_workspace_bytes(self.h, n, tokens, Hq, max_seq_len, total)
        ws = self._scratch(max(16, nbytes), stream)
        _check(_lib.s4kv_prompt_attention(self.h, int(layer), form, q.data_ptr(), tokens, cu_q.data_ptr(), Hq,
                                          block_table.data_ptr(), width, seq_lens.data_ptr(), _address(slot_ids), n,
                                          float(sm_scale), out.data_ptr(), out_dtype, ws.data_ptr(), nbytes, max_seq_len,
                                          total, self._handle(stream)), "s4kv_prompt_attention")
        return out

    @_on_its_device
    def gather(self, layer, block_table, seq_lens, cu_rows, num_rows, first=None, slot_ids=None, out_k=None, out_v=None,
               out_dtype=S4KV_F32, stream=None):
        """Restores tokens first[i] .. of sequence i (0 without first) into rows [cu_rows[i], cu_rows[i+1])
        of two dense tensors [num_rows, H_kv, 128], which are returned as (k, v)."""
        torch = self._torch
        i32, n = torch.int32, seq_lens.shape[0]
        rows, width = self._tensor(block_table, "block_table", i32, (None, None))
        self._tensor(seq_lens, "seq_lens", i32, (n,))
        self._tensor(cu_rows, "cu_rows", i32, (n + 1,))
        if rows < n:
            raise ValueError("block_table has fewer rows than there are sequences")
        if first is not None:
            self._tensor(first, "first", i32, (n,))
        if slot_ids is not None:
            self._tensor(slot_ids, "slot_ids", i32, (n,))
        num_rows = int(num_rows)
        shape = (num_rows, self.H, 128)
        out_k = self._out(out_k, "out_k", shape, out_dtype, stream)
        out_v = self._out(out_v, "out_v", shape, out_dtype, stream, out_k)
        _check(_lib.s4kv_gather(self.h, int(layer), block_table.data_ptr(), width, seq_lens.data_ptr(), _address(slot_ids),
                                _address(first), cu_rows.data_ptr(), num_rows, n, out_k.data_ptr(), out_v.data_ptr(),
                                out_dtype, self._handle(stream)), "s4kv_gather")
        return out_k, out_v

    def _pages(self, refs, block_table, slot_ids, n):
        """Checks what the calls on pages share; the table's (rows, width)."""
        torch = self._torch
        self._tensor(refs, "refs", torch.int32, (self.cfg.num_pages,))
        rows, width = self._tensor(block_table, "block_table", torch.int32, (None, None))
        if slot_ids is not None:
            self._tensor(slot_ids, "slot_ids", torch.int32, (n,))
        elif rows < n:
            raise ValueError("block_table has fewer rows than there are sequences")
        return rows, width

    def _taken(self, taken, like, stream):
        """`taken`, checked, or a new tensor like the checked one."""
        torch = self._torch
        if taken is None:
            return torch.empty_like(like) if stream is None else self._made(stream, torch.empty_like, like)
        self._tensor(taken, "taken", torch.int32, like.shape)
        return taken

    @_on_its_device
    def take_pages(self, refs, block_table, lens, new_lens, slot_ids=None, taken=None, stream=None):
        """Free pages (refs [num_pages]: the table entries that name each; 0: free) for sequences that
        grow from `lens` to `new_lens` tokens, into their rows of block_table [slots, entries], lowest
        page first. Returns `taken` [n]: how many each got, -1 where too few are free or an entry to
        fill names a page already. `taken` lies apart from the other tensors."""
        torch = self._torch
        n = lens.shape[0]
        self._tensor(lens, "lens", torch.int32, (n,))
        self._tensor(new_lens, "new_lens", torch.int32, (n,))
        rows, width = self._pages(refs, block_table, slot_ids, n)
        taken = self._taken(taken, lens, stream)
        _check(_lib.s4kv_take_pages(self.h, refs.data_ptr(), block_table.data_ptr(), width, rows, lens.data_ptr(),
                                    new_lens.data_ptr(), _address(slot_ids), n, taken.data_ptr(), self._handle(stream)),
               "s4kv_take_pages")
        return taken

    @_on_its_device
    def release_pages(self, refs, block_table, first, last, slot_ids=None, stream=None):
        """Gives up the pages of tokens first .. last - 1 of each sequence (whole pages from `first`
        on, the one that holds `last` - 1 included): their entries become -1, their counts go down.
        Of a sequence of T tokens that goes on, on KIVI pages, `last` is T - residual_v at most, rounded
        down to 32 tokens: later values have still to be written."""
        torch = self._torch
        n = first.shape[0]
        self._tensor(first, "first", torch.int32, (n,))
        self._tensor(last, "last", torch.int32, (n,))
        rows, width = self._pages(refs, block_table, slot_ids, n)
        _check(_lib.s4kv_release_pages(self.h, refs.data_ptr(), block_table.data_ptr(), width, rows, first.data_ptr(),
                                       last.data_ptr(), _address(slot_ids), n, self._handle(stream)), "s4kv_release_pages")

    @_on_its_device
    def fork(self, refs, block_table, src, dst, seq_lens, taken=None, stream=None):
        """Continues the sequences of slots src (seq_lens tokens) in slots dst too, in every layer: pages
        that are done with are shared (refs up by one), the others taken and copied, rings and
        lengths copied. block_table has a row for each slot. Returns `taken` [n] as take_pages does."""
        torch = self._torch
        n = src.shape[0]
        self._tensor(src, "src", torch.int32, (n,))
        self._tensor(dst, "dst", torch.int32, (n,))
        self._tensor(seq_lens, "seq_lens", torch.int32, (n,))
        rows, width = self._pages(refs, block_table, src, n)
        taken = self._taken(taken, src, stream)
        _check(_lib.s4kv_fork(self.h, refs.data_ptr(), block_table.data_ptr(), width, rows, src.data_ptr(), dst.data_ptr(),
                              seq_lens.data_ptr(), n, taken.data_ptr(), self._handle(stream)), "s4kv_fork")
        return taken

    def dequant(self, layer, slot, block_table_row, seq_len, stream=None):
        torch = self._torch
        k = self._made(stream, torch.empty, (self.H, seq_len, 128), dtype=torch.float32, device=self.pool.device)
        v = self._made(stream, torch.empty_like, k)
        s4kv_dequant_debug(self.h, layer, slot, block_table_row, seq_len, k, v, stream)
        return k, v

    def status(self, stream=None):
        return s4kv_get_status(self.h, stream)
