"""Python binding for `liblsa.so` (the C-ABI declared in include/lsa.h).

This module only marshals arguments. Every step of the selection path runs in
the library's HIP kernels. Tensors are passed by `data_ptr()`, `*_host` offset
arrays are int64 numpy arrays (or CPU tensors), and the stream defaults to
torch's current stream. If the library has not been built, importing this
module raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblsa.so")

F32, BF16, FP8_E4M3 = 0, 1, 2
DTYPES = {"f32": F32, "bf16": BF16, "fp8": FP8_E4M3}
MAX_LAYERS = 8
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_HIP, ERR_WORKSPACE = 0, -1, -2, -3, -4


class LsaError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build the HIP library first (__graft_entry__.build())")
_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_i32, _i64, _f32, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class ProjLayer(ctypes.Structure):
    _fields_ = [("h", _vp), ("w_dq", _vp), ("w_iuq", _vp), ("w_w", _vp),
                ("c_out", _vp), ("q_out", _vp), ("w_out", _vp)]


class ScoreLayer(ctypes.Structure):
    _fields_ = [("q", _vp), ("w", _vp), ("keys", _vp), ("key_scale", _vp),
                ("mask_out", _vp), ("score_out", _vp)]


class ScoreOptions(ctypes.Structure):
    _fields_ = [("kernel", _i32), ("chunk_words", _i32), ("ring", _i32), ("guard", _i32)]


SCORE_KERNELS = {"auto": 0, "stream": 1, "pairs": 2}


class TopkLayer(ctypes.Structure):
    _fields_ = [("q", _vp), ("w", _vp), ("keys", _vp), ("key_scale", _vp),
                ("topk_idx_out", _vp), ("topk_score_out", _vp)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_table", _vp), ("kv_len", _vp),
                ("table_stride", _i64), ("n_pages", _i32), ("n_kv", _i32), ("page_tokens", _i32), ("d_h", _i32),
                ("dtype", _i32)]


class _AttendForm(ctypes.Structure):
    _fields_ = [("softcap", _f32), ("slopes", _vp), ("doc_start", _vp), ("prefix_end", _vp)]


class _KvPool(ctypes.Structure):
    _fields_ = [("refs", _vp), ("page_table", _vp), ("kv_len", _vp), ("table_stride", _i64), ("B", _i32), ("n_pages", _i32),
                ("page_tokens", _i32)]


ROPE = {None: 0, "none": 0, "halves": 1, "pairs": 2}


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_project = _sig("lsa_project", _i32, [ctypes.POINTER(ProjLayer), _i32, _i32, _i32, _i32, _i32, _i32, _i32, _vp])
_pack_size = _sig("lsa_pack_weights_size", _sz, [_i32, _i32])
_pack = _sig("lsa_pack_weights", _i32, [_vp, _i32, _i32, _vp, _sz, _vp])
_project_packed = _sig("lsa_project_packed", _i32, [ctypes.POINTER(ProjLayer), _i32, _i32, _i32, _i32, _i32, _i32,
                                                     _vp])
_score_select = _sig("lsa_score_select", _i32, [ctypes.POINTER(ScoreLayer), _i32, _i32, _vp, _vp, _vp, _vp,
                                                 _i32, _i32, _i32, _f32, _vp])
_score_select_ex = _sig("lsa_score_select_ex", _i32, [ctypes.POINTER(ScoreLayer), _i32, _i32, _vp, _vp, _vp, _vp,
                                                       _i32, _i32, _i32, _f32, ctypes.POINTER(ScoreOptions), _vp])
_union_compact = _sig("lsa_union_compact", _i32, [ctypes.POINTER(_vp), _i32, _i32, _vp, _vp, _vp, _vp,
                                                   _vp, _vp, _vp, _vp])
_topk_ws = _sig("lsa_topk_workspace_size", _sz, [_i32, _i32, _i64, _i32])
_topk = _sig("lsa_topk", _i32, [ctypes.POINTER(TopkLayer), _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                 _i32, _vp, _vp, _sz, _vp])
_topk_score = _sig("lsa_topk_score", _i32, [ctypes.POINTER(TopkLayer), _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32,
                                             _i32, _vp, _sz, _vp])
_topk_step = _sig("lsa_topk_step", _i32, [ctypes.POINTER(TopkLayer), _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32,
                                           _i32, _i32, _vp, _vp, _sz, _vp])
_topk_step_noalloc = _sig("lsa_topk_step_noalloc", _i32, [ctypes.POINTER(TopkLayer), _i32, _i32, _vp, _vp, _vp, _vp,
                                                           _i32, _i32, _i32, _i32, _vp, _vp])
_topk_select = _sig("lsa_topk_select", _i32, [ctypes.POINTER(TopkLayer), _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp,
                                               _vp, _sz, _vp])
_gather = _sig("lsa_gather", _i32, [_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp])
_fetch_host = _sig("lsa_fetch_host", _i32, [_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp])
_golden_ws = _sig("lsa_golden_workspace_size", _sz, [_i32, _i32, _i64])
_golden = _sig("lsa_golden_labels", _i32, [_vp, _i64, _i32, _i32, _vp, _f32, _i32, _vp, _vp, _vp, _vp, _vp, _sz,
                                           _vp])
_train_ws = _sig("lsa_train_workspace_size", _sz, [_i32, _vp, _i32])
_train = _sig("lsa_train_step", _i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                       _i32, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _sz, _vp])
_kv_append = _sig("lsa_kv_append", _i32, [ctypes.POINTER(_KvCache), _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _vp,
                                          _vp, _i32, _vp, _i32, _vp, _vp])
_attend_ws = _sig("lsa_attend_workspace_size", _sz, [_i32, _i32, _i32, _i32, _vp, _i32, _i32, _i32])
_attend = _sig("lsa_attend", _i32, [ctypes.POINTER(_KvCache), _i32, _vp, _i64, _i32, _vp, _vp, _i32, _f32, _i32, _i32,
                                    _vp, _i64, _vp, _vp, _sz, _vp])
_attend_topk_ws = _sig("lsa_attend_topk_workspace_size", _sz, [_i32] * 8)
_attend_topk = _sig("lsa_attend_topk", _i32, [ctypes.POINTER(_KvCache), _i32, _vp, _i64, _i32, _vp, _vp, _i32, _i32,
                                              _f32, _i32, _i32, _vp, _i64, _vp, _vp, _sz, _vp])
_attend_ex = _sig("lsa_attend_ex", _i32, [ctypes.POINTER(_KvCache), _i32, _vp, _i64, _i32, _vp, _vp, _i32, _f32, _i32, _i32,
                                          ctypes.POINTER(_AttendForm), _vp, _i64, _vp, _vp, _sz, _vp])
_attend_topk_ex = _sig("lsa_attend_topk_ex", _i32, [ctypes.POINTER(_KvCache), _i32, _vp, _i64, _i32, _vp, _vp, _i32, _i32,
                                                    _f32, _i32, _i32, ctypes.POINTER(_AttendForm), _vp, _i64, _vp, _vp, _sz,
                                                    _vp])
_kv_kept = _sig("lsa_kv_kept", _i32, [ctypes.POINTER(_KvCache), _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp])
_kv_compact = _sig("lsa_kv_compact", _i32, [ctypes.POINTER(_KvCache), ctypes.POINTER(_KvCache), _i32, _i32, _vp, _vp, _vp,
                                            _i32, _i32, _i32, _i32, _vp])
_kv_extend = _sig("lsa_kv_extend", _i32, [ctypes.POINTER(_KvPool), _vp, _vp, _vp])
_kv_fork_ws = _sig("lsa_kv_fork_workspace_size", _sz, [_i32])
_kv_fork = _sig("lsa_kv_fork", _i32, [ctypes.POINTER(_KvPool), ctypes.POINTER(_KvCache), _i32, _i32, _vp, _vp, _vp, _vp, _sz,
                                      _vp])
_kv_free = _sig("lsa_kv_free", _i32, [ctypes.POINTER(_KvPool), _i32, _vp, _vp])
_debug_range_errors = _sig("lsa_debug_range_errors", _i32, [_vp, ctypes.POINTER(_i64)])
_last_error = _sig("lsa_last_error", ctypes.c_char_p, [])
_version = _sig("lsa_version", _i32, [])

EXPORTED = ("lsa_project", "lsa_pack_weights_size", "lsa_pack_weights", "lsa_project_packed", "lsa_score_select",
            "lsa_score_select_ex", "lsa_topk_step", "lsa_topk_step_noalloc",
            "lsa_topk_score", "lsa_topk_select", "lsa_union_compact", "lsa_topk_workspace_size", "lsa_topk",
            "lsa_gather", "lsa_fetch_host", "lsa_golden_workspace_size", "lsa_golden_labels", "lsa_train_workspace_size",
            "lsa_train_step", "lsa_kv_append", "lsa_attend_workspace_size", "lsa_attend",
            "lsa_attend_topk_workspace_size", "lsa_attend_topk", "lsa_attend_ex", "lsa_attend_topk_ex", "lsa_kv_kept",
            "lsa_kv_compact", "lsa_kv_extend", "lsa_kv_fork_workspace_size", "lsa_kv_fork", "lsa_kv_free",
            "lsa_debug_range_errors", "lsa_last_error", "lsa_version")


def last_error() -> str:
    return _last_error().decode()


def version() -> int:
    return int(_version())


def debug_range_errors(stream=None) -> int:
    """lsa_debug_range_errors: out-of-range list entries met since the last call (debug builds only;
    waits for the stream)."""
    n = _i64(0)
    _check("lsa_debug_range_errors", _debug_range_errors(_stream(stream), ctypes.byref(n)))
    return int(n.value)


def _p(t):
    """Device pointer of a tensor (or None/int passthrough)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _host64(a):
    """Host int64 array -> (keep-alive object, pointer)."""
    if a is None:
        return None, None
    if hasattr(a, "numpy"):
        a = a.detach().cpu().numpy()
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int64))
    return arr, arr.ctypes.data


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    """Size in bytes of a tensor (0 for None)."""
    return 0 if t is None else t.numel() * t.element_size()


def _check(fn, st):
    if st != OK:
        raise LsaError(fn, st, last_error())


def project(layers, *, B, d, r, n_h, d_h, dtype, stream=None):
    """lsa_project. `layers`: list of dicts with h, w_dq, w_iuq, w_w, c_out, q_out, w_out tensors."""
    arr = (ProjLayer * len(layers))(*[ProjLayer(*[_p(x[k]) for k in ("h", "w_dq", "w_iuq", "w_w", "c_out",
                                                                      "q_out", "w_out")]) for x in layers])
    _check("lsa_project", _project(arr, len(layers), B, d, r, n_h, d_h, DTYPES.get(dtype, dtype), _stream(stream)))


def pack_weights_size(rows, K) -> int:
    """lsa_pack_weights_size: bytes of the packed operand layout of a rows x K bf16 matrix."""
    return int(_pack_size(rows, K))


def pack_weights(w, rows, K, out, out_bytes=None, stream=None):
    """lsa_pack_weights: `w` a [rows, K] bf16 (int16 bits) tensor, `out` a byte tensor of pack_weights_size bytes."""
    if out_bytes is None:
        out_bytes = out.numel() * out.element_size()
    _check("lsa_pack_weights", _pack(_p(w), rows, K, _p(out), int(out_bytes), _stream(stream)))


def project_packed(layers, *, B, d, r, n_h, d_h, stream=None):
    """lsa_project_packed: as project(), with w_dq, w_iuq, w_w packed by pack_weights (bf16)."""
    arr = (ProjLayer * len(layers))(*[ProjLayer(*[_p(x[k]) for k in ("h", "w_dq", "w_iuq", "w_w", "c_out",
                                                                      "q_out", "w_out")]) for x in layers])
    _check("lsa_project_packed", _project_packed(arr, len(layers), B, d, r, n_h, d_h, _stream(stream)))


def score_select(layers, *, B, key_offsets, key_offsets_host, mask_word_offsets, mask_word_offsets_host,
                 n_h, d_h, key_dtype, threshold=0.5, options=None, stream=None):
    """lsa_score_select. `layers`: dicts with q, w, keys, key_scale (fp8), mask_out, score_out (optional).

    With `options` (a dict with any of kernel ("auto", "stream", "pairs"), chunk_words, ring, guard),
    lsa_score_select_ex with those launch options instead."""
    arr = (ScoreLayer * len(layers))(*[ScoreLayer(_p(x["q"]), _p(x["w"]), _p(x["keys"]), _p(x.get("key_scale")),
                                                  _p(x["mask_out"]), _p(x.get("score_out"))) for x in layers])
    ko, kop = _host64(key_offsets_host)
    mo, mop = _host64(mask_word_offsets_host)
    args = (arr, len(layers), B, _p(key_offsets), kop, _p(mask_word_offsets), mop, n_h, d_h,
            DTYPES.get(key_dtype, key_dtype), float(threshold))
    if options is None:
        _check("lsa_score_select", _score_select(*args, _stream(stream)))
        return
    o = ScoreOptions(SCORE_KERNELS.get(options.get("kernel", 0), options.get("kernel", 0)),
                     int(options.get("chunk_words", 0)), int(options.get("ring", 0)), int(options.get("guard", 0)))
    _check("lsa_score_select_ex", _score_select_ex(*args, ctypes.byref(o), _stream(stream)))


def union_compact(masks, *, B, key_offsets, key_offsets_host, mask_word_offsets, mask_word_offsets_host,
                  idx_out, count_out, union_mask_out=None, stream=None):
    """lsa_union_compact over a list of per-layer mask tensors."""
    marr = (_vp * len(masks))(*[_p(m) for m in masks])
    ko, kop = _host64(key_offsets_host)
    mo, mop = _host64(mask_word_offsets_host)
    _check("lsa_union_compact", _union_compact(marr, len(masks), B, _p(key_offsets), kop, _p(mask_word_offsets),
                                               mop, _p(idx_out), _p(count_out), _p(union_mask_out),
                                               _stream(stream)))


def topk_workspace_size(L, B, total_rows, k) -> int:
    return int(_topk_ws(L, B, total_rows, k))


def topk(layers, *, B, key_offsets, key_offsets_host, idx, count, n_h, d_h, key_dtype, k, topk_count_out,
         workspace, stream=None):
    """lsa_topk. `layers`: dicts with q, w, keys, key_scale (fp8), topk_idx_out, topk_score_out (optional)."""
    arr = (TopkLayer * len(layers))(*[TopkLayer(_p(x["q"]), _p(x["w"]), _p(x["keys"]), _p(x.get("key_scale")),
                                                _p(x["topk_idx_out"]), _p(x.get("topk_score_out"))) for x in layers])
    ko, kop = _host64(key_offsets_host)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("lsa_topk", _topk(arr, len(layers), B, _p(key_offsets), kop, _p(idx), _p(count), n_h, d_h,
                             DTYPES.get(key_dtype, key_dtype), k, _p(topk_count_out), _p(workspace), nbytes,
                             _stream(stream)))


def topk_step(layers, *, B, key_offsets, key_offsets_host, idx, count, n_h, d_h, key_dtype, k, topk_count_out,
              workspace, stream=None):
    """lsa_topk_step: as topk, with each layer's `keys` the packed subset keys (one decode step)."""
    arr = (TopkLayer * len(layers))(*[TopkLayer(_p(x["q"]), _p(x["w"]), _p(x["keys"]), _p(x.get("key_scale")),
                                                _p(x["topk_idx_out"]), _p(x.get("topk_score_out"))) for x in layers])
    ko, kop = _host64(key_offsets_host)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("lsa_topk_step", _topk_step(arr, len(layers), B, _p(key_offsets), kop, _p(idx), _p(count), n_h, d_h,
                                       DTYPES.get(key_dtype, key_dtype), k, _p(topk_count_out), _p(workspace),
                                       nbytes, _stream(stream)))


NOALLOC_SCRATCH_BYTES = 32 << 20


def topk_step_noalloc(layers, *, B, key_offsets, key_offsets_host, idx, count, n_h, d_h, key_dtype, k,
                      topk_count_out, stream=None):
    """lsa_topk_step_noalloc: as topk_step, with the library's own fixed scratch instead of a workspace."""
    arr = (TopkLayer * len(layers))(*[TopkLayer(_p(x["q"]), _p(x["w"]), _p(x["keys"]), _p(x.get("key_scale")),
                                                _p(x["topk_idx_out"]), _p(x.get("topk_score_out"))) for x in layers])
    ko, kop = _host64(key_offsets_host)
    _check("lsa_topk_step_noalloc", _topk_step_noalloc(arr, len(layers), B, _p(key_offsets), kop, _p(idx), _p(count),
                                                       n_h, d_h, DTYPES.get(key_dtype, key_dtype), k,
                                                       _p(topk_count_out), _stream(stream)))


def _topk_layers(layers):
    return (TopkLayer * len(layers))(*[TopkLayer(_p(x.get("q")), _p(x.get("w")), _p(x.get("keys")),
                                                 _p(x.get("key_scale")), _p(x.get("topk_idx_out")),
                                                 _p(x.get("topk_score_out"))) for x in layers])


def topk_score(layers, *, B, key_offsets, key_offsets_host, idx, count, n_h, d_h, key_dtype, workspace,
               stream=None):
    """lsa_topk_score: the subset scores into the workspace. `layers`: dicts with q, w, keys, key_scale."""
    ko, kop = _host64(key_offsets_host)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("lsa_topk_score", _topk_score(_topk_layers(layers), len(layers), B, _p(key_offsets), kop, _p(idx),
                                         _p(count), n_h, d_h, DTYPES.get(key_dtype, key_dtype), _p(workspace),
                                         nbytes, _stream(stream)))


def topk_select(layers, *, B, key_offsets, key_offsets_host, idx, count, k, topk_count_out, workspace,
                stream=None):
    """lsa_topk_select: the top-k from the scores in the workspace. `layers`: dicts with topk_idx_out
    and topk_score_out (optional)."""
    ko, kop = _host64(key_offsets_host)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("lsa_topk_select", _topk_select(_topk_layers(layers), len(layers), B, _p(key_offsets), kop, _p(idx),
                                           _p(count), k, _p(topk_count_out), _p(workspace), nbytes,
                                           _stream(stream)))


def gather(pool, *, row_bytes, B, pool_row_offsets, pool_row_offsets_host, idx, idx_offsets, count, out,
           out_row_offsets=None, out_capacity_rows, stream=None):
    """lsa_gather (packed mode when out_row_offsets is None)."""
    po, pop = _host64(pool_row_offsets_host)
    _check("lsa_gather", _gather(_p(pool), int(row_bytes), B, _p(pool_row_offsets), pop, _p(idx), _p(idx_offsets),
                                 _p(count), _p(out), _p(out_row_offsets), int(out_capacity_rows), _stream(stream)))


def fetch_host(pool_host, *, row_bytes, B, pool_row_offsets, pool_row_offsets_host, idx, idx_offsets, count, out,
               out_row_offsets=None, out_capacity_rows, stream=None):
    """lsa_fetch_host: pool_host is a pinned CPU tensor (pin_memory=True); out is on the device."""
    po, pop = _host64(pool_row_offsets_host)
    _check("lsa_fetch_host", _fetch_host(_p(pool_host), int(row_bytes), B, _p(pool_row_offsets), pop, _p(idx),
                                         _p(idx_offsets), _p(count), _p(out), _p(out_row_offsets),
                                         int(out_capacity_rows), _stream(stream)))


def golden_workspace_size(T, L, row_stride) -> int:
    return int(_golden_ws(int(T), int(L), int(row_stride)))


def golden_labels(logits, *, row_stride, T, L, n_valid, top_p, theta, row_mask, golden, workspace,
                  nucleus_size=None, token_golden=None, stream=None):
    """lsa_golden_labels: logits [T, L, row_stride] fp32 and n_valid [T] int32 on the device; the mask
    outputs are int64 tensors of ceil(row_stride / 64) words per row; workspace is a device tensor of at
    least golden_workspace_size(T, L, row_stride) bytes."""
    _check("lsa_golden_labels", _golden(_p(logits), int(row_stride), int(T), int(L), _p(n_valid), float(top_p),
                                        int(theta), _p(row_mask), _p(nucleus_size), _p(token_golden), _p(golden),
                                        _p(workspace), _nbytes(workspace), _stream(stream)))


def train_workspace_size(B, key_offsets_host, r) -> int:
    ko, kop = _host64(key_offsets_host)
    return int(_train_ws(int(B), kop, int(r)))


def train_step(*, h, w_dq, w_iuq, w_w, keys, key_offsets, key_offsets_host, labels, mask_word_offsets,
               mask_word_offsets_host, B, d, r, n_h, d_h, gamma, alpha, loss, g_dq, g_iuq, g_w, workspace,
               stream=None):
    """lsa_train_step: h [B, d], w_dq [r, d], w_iuq [n_h*d_h, r], w_w [n_h, d] and keys [rows, d_h] as bf16
    bits on the device; labels are the selection path's bit masks; loss [1] and the gradients (the
    weights' shapes) are fp32 device tensors; workspace holds train_workspace_size(...) bytes."""
    ko, kop = _host64(key_offsets_host)
    mo, mop = _host64(mask_word_offsets_host)
    _check("lsa_train_step", _train(_p(h), _p(w_dq), _p(w_iuq), _p(w_w), _p(keys), _p(key_offsets), kop, _p(labels),
                                    _p(mask_word_offsets), mop, int(B), int(d), int(r), int(n_h), int(d_h),
                                    float(gamma), float(alpha), _p(loss), _p(g_dq), _p(g_iuq), _p(g_w),
                                    _p(workspace), _nbytes(workspace), _stream(stream)))


# ------------------------------------------------------------------ the paged cache
# These calls take a few microseconds on the device, so their checks are kept to a few comparisons per tensor;
# the text of a refusal is only made when there is one.
def _refuse(fn, msg):
    raise LsaError(fn, ERR_INVALID_ARG, msg)


def _want(fn, name, t, dtype, shape, device):
    """A contiguous tensor of this dtype and shape on the device of this index (-1: host)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(fn, f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on device {device} "
                    f"(got {t.dtype}, {list(t.shape)}, strides {t.stride()}, device {t.get_device()})")


def _rows(fn, name, t, dtype, shape, device):
    """A [rows, heads, d] tensor whose rows are contiguous, at any distance, which is returned."""
    step, head, one = t.stride() if t.dim() == 3 else (0, 0, 0)
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != device or one != 1 or
            (head != shape[2] and shape[1] > 1)):
        _refuse(fn, f"{name} must be a {dtype} tensor of shape {list(shape)} with contiguous rows on device {device} "
                    f"(got {t.dtype}, {list(t.shape)}, strides {t.stride()}, device {t.get_device()})")
    return step if shape[0] > 1 else shape[1] * shape[2]


def check_rows(fn, name, t, shape, device):
    """Refuses, in the name of `fn`, a tensor that lsa_kv_append would refuse as new rows [rows, heads, d_h]."""
    step = _rows(fn, name, t, _torch().bfloat16, shape, device)
    if step % 8 or step < shape[1] * shape[2] or t.data_ptr() % 16:
        _refuse(fn, f"{name} must be 16-byte aligned, with its rows a multiple of 8 elements apart, at least "
                    f"{shape[1] * shape[2]} (got {step})")


def _offsets(fn, name, off, host, B, rows, device):
    """Checks device and host offsets of rows; returns (the host array, its pointer)."""
    if off.dtype is not _torch().int64 or off.shape != (B + 1,) or off.get_device() != device or not off.is_contiguous():
        _want(fn, name, off, _torch().int64, (B + 1,), device)
    if type(host) is not np.ndarray or host.dtype != np.int64 or not host.flags.c_contiguous:
        host = _host64(host)[0]
    if host.shape != (B + 1,) or host[B] > rows:
        _refuse(fn, f"{name}_host must have {B + 1} elements and end within the {rows} rows (got {host.shape[0]}, "
                    f"ending at {host[-1]})")
    if host.flags.writeable:  # half the time of the array interface
        return host, ctypes.addressof(ctypes.c_char.from_buffer(host))
    return host, host.__array_interface__["data"][0]


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_module = None


def _launch(device, fn, call, args, stream):
    """The call on the device of this index, whichever is current, on `stream` or that device's current one."""
    torch = _torch()
    if device < 0:
        _refuse(fn, "the tensors must be on a GPU")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        st = call(*args, stream)
    else:
        with torch.cuda.device(device):
            st = call(*args, stream)
    if st != OK:
        raise LsaError(fn, st, last_error())


class KvCache:
    """The lsa_kv_cache of one layer: k and v [n_pages, n_kv, page_tokens, d_h] in bfloat16, or in
    float8_e4m3fn with k_scale and v_scale [n_pages, n_kv] float32; page_table [B, pages] and kv_len [B] int32.

    Holds the tensors. Their contents may change between calls; the tensors themselves stay."""

    def __init__(self, *, k, v, page_table, kv_len, k_scale=None, v_scale=None):
        fn, torch = "KvCache", _torch()
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or k.dim() != 4:
            _refuse(fn, f"k must be [n_pages, n_kv, page_tokens, d_h] in bfloat16 or float8_e4m3fn (got {k.dtype}, "
                        f"{list(k.shape)})")
        fp8 = k.dtype == torch.float8_e4m3fn
        self.device = dev = k.get_device()
        self.n_pages, self.n_kv, self.page_tokens, self.d_h = k.shape
        _want(fn, "k", k, k.dtype, k.shape, dev)
        _want(fn, "v", v, k.dtype, k.shape, dev)
        if fp8 != (k_scale is not None) or fp8 != (v_scale is not None):
            _refuse(fn, "k_scale and v_scale are needed for float8_e4m3fn, and only for it")
        if fp8:
            _want(fn, "k_scale", k_scale, torch.float32, k.shape[:2], dev)
            _want(fn, "v_scale", v_scale, torch.float32, k.shape[:2], dev)
        if kv_len.dim() != 1 or page_table.dim() != 2:
            _refuse(fn, "kv_len must be [B] and page_table [B, pages]")
        self.B = kv_len.shape[0]
        _want(fn, "kv_len", kv_len, torch.int32, (self.B,), dev)
        _want(fn, "page_table", page_table, torch.int32, (self.B, page_table.shape[1]), dev)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table, self.kv_len = page_table, kv_len
        self._c = _KvCache(_p(k), _p(v), _p(k_scale), _p(v_scale), _p(page_table), _p(kv_len), page_table.shape[1],
                           self.n_pages, self.n_kv, self.page_tokens, self.d_h, FP8_E4M3 if fp8 else BF16)
        self.ref = ctypes.byref(self._c)


def _three(fn, name, t):
    shape = t.shape
    if len(shape) != 3:
        _refuse(fn, f"{name} must be [rows, heads, d_h] (got {list(shape)})")
    return shape


def kv_append(cache, k_new, v_new, *, new_offsets, new_offsets_host, q=None, q_out=None, inv_freq=None, rope="halves",
              positions=None, stream=None):
    """lsa_kv_append: k_new, v_new [rows, n_kv, d_h] and q [rows, n_q, d_h] bfloat16, with contiguous rows at any
    distance; q_out [rows, n_q, d_h] contiguous; new_offsets [B + 1] int64 on the device and on the host; inv_freq
    [rot_dim / 2] float32, None for no rotation; rope "halves" or "pairs"; positions [rows] int32 or None."""
    fn, torch = "lsa_kv_append", _torch()
    dev, B, bf16 = cache.device, cache.B, torch.bfloat16
    shape = _three(fn, "k_new", k_new)
    rows, d = shape[0], cache.d_h
    shape = (rows, cache.n_kv, d)
    ks = _rows(fn, "k_new", k_new, bf16, shape, dev)
    vs = _rows(fn, "v_new", v_new, bf16, shape, dev)
    n_q = qs = rot = 0
    q_at = q_out_at = inv_at = pos_at = None
    if q is not None and q_out is not None:
        n_q = _three(fn, "q", q)[1]
        qs = _rows(fn, "q", q, bf16, (rows, n_q, d), dev)
        _want(fn, "q_out", q_out, bf16, (rows, n_q, d), dev)
        q_at, q_out_at = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        _refuse(fn, "q and q_out must be set together")
    style = ROPE.get(rope, -1)
    if inv_freq is None and style >= 0:
        style = 0
    elif style > 0:
        rot = 2 * inv_freq.shape[0]
        _want(fn, "inv_freq", inv_freq, torch.float32, (rot // 2,), dev)
        inv_at = inv_freq.data_ptr()
    if positions is not None:
        _want(fn, "positions", positions, torch.int32, (rows,), dev)
        pos_at = positions.data_ptr()
    host, host_at = _offsets(fn, "new_offsets", new_offsets, new_offsets_host, B, rows, dev)
    _launch(dev, fn, _kv_append, (cache.ref, B, k_new.data_ptr(), ks, v_new.data_ptr(), vs, q_at, qs, q_out_at, n_q,
                                  new_offsets.data_ptr(), host_at, style, inv_at, rot, pos_at), stream)


def _int32(fn, *values):
    """Refuses numbers that would arrive in the library as others: ctypes takes the lower 32 bits."""
    for x in values:
        if not -0x80000000 <= x <= 0x7FFFFFFF:
            _refuse(fn, f"{x} does not fit 32 bits")


def attend_workspace_size(cache, *, n_q, q_offsets_host, max_kv_len, window=0, sinks=0) -> int:
    """lsa_attend_workspace_size for this cache."""
    _int32("lsa_attend_workspace_size", n_q, max_kv_len, window, sinks)
    off, offp = _host64(q_offsets_host)
    return int(_attend_ws(off.size - 1, n_q, cache.n_kv, cache.d_h, offp, max_kv_len, window, sinks))


def _attend_tensors(fn, cache, q, out, lse, workspace):
    torch, dev = _torch(), cache.device
    shape = _three(fn, "q", q)
    rows, n_q = shape[0], shape[1]
    shape = (rows, n_q, cache.d_h)
    qs = _rows(fn, "q", q, torch.bfloat16, shape, dev)
    os_ = _rows(fn, "out", out, torch.bfloat16, shape, dev)
    lse_at = ws_at = None
    nbytes = 0
    if lse is not None:
        _want(fn, "lse", lse, torch.float32, (rows, n_q), dev)
        lse_at = lse.data_ptr()
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse(fn, f"workspace must be contiguous and on device {dev}")
        ws_at, nbytes = workspace.data_ptr(), workspace.nbytes
    return rows, n_q, qs, os_, lse_at, ws_at, nbytes


def _attend_form(fn, cache, rows, n_q, softcap, slopes, doc_start, prefix_end):
    torch, dev = _torch(), cache.device
    form = _AttendForm(softcap)
    if slopes is not None:
        _want(fn, "slopes", slopes, torch.float32, (n_q,), dev)
        form.slopes = slopes.data_ptr()
    if doc_start is not None:
        _want(fn, "doc_start", doc_start, torch.int32, (rows,), dev)
        form.doc_start = doc_start.data_ptr()
    if prefix_end is not None:
        _want(fn, "prefix_end", prefix_end, torch.int32, (rows,), dev)
        form.prefix_end = prefix_end.data_ptr()
    return form


def attend(cache, q, *, q_offsets, q_offsets_host, max_kv_len, out, scale, window=0, sinks=0, lse=None, workspace=None,
           stream=None, softcap=0.0, slopes=None, doc_start=None, prefix_end=None):
    """lsa_attend: q and out [rows, n_q, d_h] bfloat16 with contiguous rows at any distance, lse [rows, n_q] float32
    or None; q_offsets [B + 1] int64 on the device and on the host; workspace a tensor of at least
    attend_workspace_size(...) bytes for the same arguments.

    With softcap, slopes [n_q] float32, doc_start or prefix_end [rows] int32, lsa_attend_ex with these."""
    fn = "lsa_attend"
    _int32(fn, max_kv_len, window, sinks)
    rows, n_q, qs, os_, lse_at, ws_at, nbytes = _attend_tensors(fn, cache, q, out, lse, workspace)
    host, host_at = _offsets(fn, "q_offsets", q_offsets, q_offsets_host, cache.B, rows, cache.device)
    args = (cache.ref, cache.B, q.data_ptr(), qs, n_q, q_offsets.data_ptr(), host_at, max_kv_len, scale, window, sinks)
    outs = (out.data_ptr(), os_, lse_at, ws_at, nbytes)
    if softcap == 0.0 and slopes is None and doc_start is None and prefix_end is None:
        _launch(cache.device, fn, _attend, args + outs, stream)
    else:
        form = _attend_form("lsa_attend_ex", cache, rows, n_q, softcap, slopes, doc_start, prefix_end)
        _launch(cache.device, "lsa_attend_ex", _attend_ex, (*args, form, *outs), stream)


def attend_topk_workspace_size(cache, *, n_q, k, entry_tokens=1, window=0, sinks=0) -> int:
    """lsa_attend_topk_workspace_size for this cache."""
    _int32("lsa_attend_topk_workspace_size", n_q, k, entry_tokens, window, sinks)
    return int(_attend_topk_ws(cache.B, n_q, cache.n_kv, cache.d_h, k, entry_tokens, window, sinks))


def attend_topk(cache, q, *, idx, count, out, scale, entry_tokens=1, window=0, sinks=0, lse=None, workspace=None,
                stream=None, softcap=0.0, slopes=None):
    """lsa_attend_topk: q and out [B, n_q, d_h] bfloat16, idx [B, k] and count [B] int32 as topk and topk_step
    write them, lse [B, n_q] float32 or None; workspace of at least attend_topk_workspace_size(...) bytes.

    With softcap or slopes [n_q] float32, lsa_attend_topk_ex with these."""
    fn, torch, B = "lsa_attend_topk", _torch(), cache.B
    _int32(fn, entry_tokens, window, sinks)
    rows, n_q, qs, os_, lse_at, ws_at, nbytes = _attend_tensors(fn, cache, q, out, lse, workspace)
    if rows != B or idx.dim() != 2:
        _refuse(fn, f"q must have one row per sequence and idx must be [B, k] (got {rows} rows for {B}, {list(idx.shape)})")
    k = idx.shape[1]
    _want(fn, "idx", idx, torch.int32, (B, k), cache.device)
    _want(fn, "count", count, torch.int32, (B,), cache.device)
    args = (cache.ref, B, q.data_ptr(), qs, n_q, idx.data_ptr(), count.data_ptr(), k, entry_tokens, scale, window, sinks)
    outs = (out.data_ptr(), os_, lse_at, ws_at, nbytes)
    if softcap == 0.0 and slopes is None:
        _launch(cache.device, fn, _attend_topk, args + outs, stream)
    else:
        form = _attend_form("lsa_attend_topk_ex", cache, rows, n_q, softcap, slopes, None, None)
        _launch(cache.device, "lsa_attend_topk_ex", _attend_topk_ex, (*args, form, *outs), stream)


# ------------------------------------------------------------------ kept tokens and pages
def _vector(fn, name, t, dtype, n, device):
    """As _want for a [n] tensor (n None: of any length), and its address."""
    if t.dtype is not dtype or t.dim() != 1 or (n is not None and len(t) != n) or t.get_device() != device or not t.is_contiguous():
        _want(fn, name, t, dtype, (t.numel() if n is None else n,), device)
    return t.data_ptr()


def _lists(fn, cache, idx, idx_offsets, count):
    torch, B, dev = _torch(), cache.B, cache.device
    n = len(idx_offsets)
    if n != B and n != B + 1:
        _refuse(fn, f"idx_offsets must have {B} elements, or one more (got {n})")
    return (_vector(fn, "idx", idx, torch.int32, None, dev), _vector(fn, "idx_offsets", idx_offsets, torch.int64, n, dev),
            _vector(fn, "count", count, torch.int32, B, dev))


def _layers(fn, name, caches, device):
    """The lsa_kv_cache array of these layers."""
    if not caches or any(c.device != device for c in caches):
        _refuse(fn, f"{name} must be caches on device {device}, one at least")
    return (_KvCache * len(caches))(*[c._c for c in caches])


def kv_kept(cache, *, idx, idx_offsets, count, out, entry_tokens=1, window=0, sinks=0, stream=None):
    """lsa_kv_kept: idx [rows] int32, idx_offsets [B] (or [B + 1]) int64 and count [B] int32 as union_compact takes and writes
    them; out [B] int32."""
    fn = "lsa_kv_kept"
    _int32(fn, entry_tokens, window, sinks)
    lists = _lists(fn, cache, idx, idx_offsets, count)
    out_at = _vector(fn, "out", out, _torch().int32, cache.B, cache.device)
    _launch(cache.device, fn, _kv_kept, (cache.ref, cache.B, *lists, entry_tokens, window, sinks, out_at), stream)


def kv_compact(caches, to, *, idx, idx_offsets, count, max_kept, entry_tokens=1, window=0, sinks=0, stream=None):
    """lsa_kv_compact: `caches` and `to` lists of KvCache, one a layer; the lists as for kv_kept."""
    fn = "lsa_kv_compact"
    _int32(fn, entry_tokens, window, sinks, max_kept)
    if len(caches) != len(to) or not caches:
        _refuse(fn, f"as many caches from as to, and one at least (got {len(caches)} and {len(to)})")
    dev, B = caches[0].device, caches[0].B
    if any(c.B != B for c in (*caches, *to)):
        _refuse(fn, f"all caches must have {B} sequences")
    lists = _lists(fn, caches[0], idx, idx_offsets, count)
    _launch(dev, fn, _kv_compact, (_layers(fn, "caches", caches, dev), _layers(fn, "to", to, dev), len(caches), B, *lists,
                                   entry_tokens, window, sinks, max_kept), stream)


class KvPool:
    """The lsa_kv_pool that the caches of one or several layers share: refs [n_pages], page_table [B, pages] and kv_len [B],
    all int32. Holds the tensors; the calls on the pool change their contents."""

    def __init__(self, *, refs, page_table, kv_len, page_tokens):
        fn, i32 = "KvPool", _torch().int32
        if refs.dim() != 1 or kv_len.dim() != 1 or page_table.dim() != 2:
            _refuse(fn, "refs must be [n_pages], kv_len [B] and page_table [B, pages]")
        self.device = dev = refs.get_device()
        self.n_pages, self.B, self.page_tokens = refs.shape[0], kv_len.shape[0], page_tokens
        _int32(fn, page_tokens)
        _want(fn, "refs", refs, i32, (self.n_pages,), dev)
        _want(fn, "kv_len", kv_len, i32, (self.B,), dev)
        _want(fn, "page_table", page_table, i32, (self.B, page_table.shape[1]), dev)
        self.refs, self.page_table, self.kv_len = refs, page_table, kv_len
        self._c = _KvPool(_p(refs), _p(page_table), _p(kv_len), page_table.shape[1], self.B, self.n_pages, page_tokens)
        self.ref = ctypes.byref(self._c)


def kv_extend(pool, n_new, *, missing=None, stream=None):
    """lsa_kv_extend: n_new [B] int32, missing [B] int32 or None."""
    fn, i32 = "lsa_kv_extend", _torch().int32
    at = _vector(fn, "n_new", n_new, i32, pool.B, pool.device)
    missing_at = None if missing is None else _vector(fn, "missing", missing, i32, pool.B, pool.device)
    _launch(pool.device, fn, _kv_extend, (pool.ref, at, missing_at), stream)


def kv_fork_workspace_size(n) -> int:
    return int(_kv_fork_ws(n))


def kv_fork(pool, caches, src, dst, *, status, workspace, stream=None):
    """lsa_kv_fork: `caches` a list of KvCache, one a layer; src, dst and status [n] int32; workspace a tensor of at least
    kv_fork_workspace_size(n) bytes."""
    fn, i32, dev = "lsa_kv_fork", _torch().int32, pool.device
    n = src.numel()
    at = [_vector(fn, name, t, i32, n, dev) for name, t in (("src", src), ("dst", dst), ("status", status))]
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(fn, f"workspace must be contiguous and on device {dev}")
    _launch(dev, fn, _kv_fork, (pool.ref, _layers(fn, "caches", caches, dev), len(caches), n, *at, workspace.data_ptr(),
                                workspace.nbytes), stream)


def kv_free(pool, seqs, *, stream=None):
    """lsa_kv_free: seqs [n] int32."""
    fn = "lsa_kv_free"
    n = seqs.numel()
    _launch(pool.device, fn, _kv_free, (pool.ref, n, _vector(fn, "seqs", seqs, _torch().int32, n, pool.device)), stream)
