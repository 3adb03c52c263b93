"""Device-resident buffers for one workload, and one pass of the whole path.

`Pipeline(inputs)` copies a seeded input set (from `synth.make`) into HBM and
allocates every output and the top-k workspace once. `run()` then enqueues the
five library calls, with no allocation and no host synchronisation, on the
current stream (the load step on a second stream that forks after the union
and joins at the end):

  lsa_project        memory-indexer and native query/gates for every layer (one call, 2L layers);
                     with bf16 weights, lsa_project_packed on weights packed once at set-up
  lsa_score_select   masks for every (layer, sequence) (score_with_sigmoid: a pass that also
                     writes the sigmoid scores)
  lsa_union_compact  OR over the layers -> ascending index list + count per sequence
  lsa_topk           native top-k inside the union, per (layer, sequence)
                     (run() calls its two stages, lsa_topk_score and lsa_topk_select)
  lsa_gather         the union rows of the compressed-KV pool -> packed compact buffer
                     (with host_pool=True, lsa_fetch_host reads them from a copy of the
                     pool in pinned host memory instead: the cold pool)

After a trigger, alloc_steps() / pack_subset_keys() / step() run the decode steps: each
layer's union rows of keys are packed once (lsa_gather), and every step projects its own
native query and calls lsa_topk_step over them.

With alloc_attention(), the steps go on to the core attention of every layer over what was selected:
append_prompt() stores the prompt's keys and values in a paged cache, and attend_step() stores a step's
own (lsa_kv_append) and attends over the step's top-k entries, the sliding window and the first tokens
(lsa_attend_topk).

This module only wires buffers. All arithmetic happens in the HIP kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import sys

import numpy as np
import torch

from . import lsa


class DeviceEvent:
    """A HIP event for ordering or timing work on the streams of one device, with no
    system-scope fence when it is recorded or waited on. The fork and join of run() need only
    device-scope ordering (host visibility comes from the caller's own synchronisation), and a
    default event's system-scope fence left the GPU idle for several microseconds at each fork
    and join. As a timing event (timing=True) it adds less to the interval it brackets than a
    default event, for the same reason. The runtime is the one the library is linked against,
    already loaded."""

    _DISABLE_TIMING = 0x2
    _DISABLE_SYSTEM_FENCE = 0x20000000
    _hip = None

    def __init__(self, timing: bool = False):
        if DeviceEvent._hip is None:
            hip = ctypes.CDLL("libamdhip64.so.7", mode=os.RTLD_NOLOAD)
            hip.hipEventCreateWithFlags.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_uint]
            hip.hipEventRecord.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
            hip.hipStreamWaitEvent.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint]
            hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
            hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
            DeviceEvent._hip = hip
        self._h = ctypes.c_void_p()
        flags = self._DISABLE_SYSTEM_FENCE | (0 if timing else self._DISABLE_TIMING)
        self._check(self._hip.hipEventCreateWithFlags(ctypes.byref(self._h), flags), "hipEventCreateWithFlags")

    @staticmethod
    def _check(rc, what):
        if rc != 0:
            raise RuntimeError(f"{what} failed with HIP error {rc}")

    def record(self, stream):
        self._check(self._hip.hipEventRecord(self._h, ctypes.c_void_p(stream.cuda_stream)), "hipEventRecord")

    def wait(self, stream):
        """Make `stream` wait for the work before this event's last record."""
        self._check(self._hip.hipStreamWaitEvent(ctypes.c_void_p(stream.cuda_stream), self._h, 0),
                    "hipStreamWaitEvent")

    def elapsed_time(self, end: "DeviceEvent") -> float:
        """Milliseconds from this event to `end` (both recorded with timing=True and complete)."""
        ms = ctypes.c_float()
        self._check(self._hip.hipEventElapsedTime(ctypes.byref(ms), self._h, end._h), "hipEventElapsedTime")
        return ms.value

    def __del__(self):
        # at interpreter exit the runtime may already be torn down; the process frees the event
        if self._hip is not None and self._h and not sys.is_finalizing():
            self._hip.hipEventDestroy(self._h)


def _dev(a: np.ndarray, device) -> torch.Tensor:
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    elif a.dtype == np.uint64:
        a = a.view(np.int64)
    return torch.from_numpy(a).to(device)


GUARD_BYTES = 4096
CANARY = 0x5A


class Pipeline:
    def __init__(self, inp, device="cuda", *, with_scores=False, with_topk_scores=True, gather_capacity=None,
                 guard=False, packed=True, overlap=True, host_pool=False, early_fork=True):
        w = inp.workload
        self.w = w
        self.inp = inp
        dev = torch.device(device)
        self.device = dev
        self._guarded = []
        self.guard = guard
        self.overlap = overlap
        self.early_fork = early_fork  # fork the load step before the top-k scoring (else after it)
        self._side = torch.cuda.Stream(device=dev)  # default priority
        self._fork = DeviceEvent()
        self._join = DeviceEvent()
        B, L = w.B, w.L
        self.rows = int(inp.key_offsets[-1])
        self.words = int(inp.mask_word_offsets[-1])
        self.key_off_h = inp.key_offsets.astype(np.int64)
        self.mwo_h = inp.mask_word_offsets.astype(np.int64)
        self.key_off = _dev(self.key_off_h, dev)
        self.mwo = _dev(self.mwo_h, dev)

        self.h = [_dev(inp.h[l], dev) for l in range(L)]
        self.mem = [tuple(_dev(x, dev) for x in (lw.w_dq, lw.w_iuq, lw.w_w)) for lw in inp.mem_w]
        self.nat = [tuple(_dev(x, dev) for x in (lw.w_dq, lw.w_iuq, lw.w_w)) for lw in inp.nat_w]
        # bf16 projection weights are packed once into the matrix-core operand layout
        self.packed = packed and w.act_dtype == "bf16" and B <= 32 and w.r % 64 == 0 and (w.n_h * w.d_h) % 64 == 0
        if self.packed:
            shapes = ((w.r, w.d), (w.n_h * w.d_h, w.r), (w.n_h, w.d))

            def pack(mats):
                out = []
                for m, (rows, K) in zip(mats, shapes):
                    buf = torch.empty(lsa.pack_weights_size(rows, K), dtype=torch.uint8, device=dev)
                    lsa.pack_weights(m, rows, K, buf)
                    out.append(buf)
                return tuple(out)

            self.mem = [pack(m) for m in self.mem]
            self.nat = [pack(m) for m in self.nat]
            torch.cuda.synchronize()
        self.keys = [_dev(inp.keys[l], dev) for l in range(L)]
        self.scale = [None if inp.key_scale[l] is None else _dev(inp.key_scale[l], dev) for l in range(L)]
        self.pool = None if inp.pool is None else _dev(inp.pool, dev)
        # the cold pool: the same rows in pinned host memory, read by lsa_fetch_host
        self.pool_host = None
        if host_pool and inp.pool is not None:
            a = np.ascontiguousarray(inp.pool)
            self.pool_host = torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).pin_memory()

        f32, i32, i64, i16 = torch.float32, torch.int32, torch.int64, torch.int16
        out = self._out
        # 2L projection outputs: first L for the memory indexer, next L for the native indexer
        self.c = [out((B, w.r), f32) for _ in range(2 * L)]
        self.q = [out((B, w.n_h, w.d_h), f32) for _ in range(2 * L)]
        self.g = [out((B, w.n_h), f32) for _ in range(2 * L)]
        self.masks = [out((max(self.words, 1),), i64) for _ in range(L)]
        # with_scores: buffers for a separate score pass that also writes the sigmoid scores
        # (score_with_sigmoid); run() itself writes masks only
        self.scores = [out((max(self.rows, 1),), f32) for _ in range(L)] if with_scores else None
        self.masks_scored = [out((max(self.words, 1),), i64) for _ in range(L)] if with_scores else None
        self.score_options = None  # launch options of run()'s score pass (lsa_score_select_ex), None = defaults
        self.idx = out((max(self.rows, 1),), i32)
        self.count = out((B,), i32)
        self.union_mask = out((max(self.words, 1),), i64)
        self.topk_idx = [out((B, w.k), i32) for _ in range(L)]
        self.topk_score = [out((B, w.k), f32) for _ in range(L)] if with_topk_scores else None
        self.topk_count = out((L, B), i32)
        ws = lsa.topk_workspace_size(L, B, self.rows, w.k)
        self.workspace = out((max(ws, 4),), torch.uint8)
        self.gather_capacity = self.rows if gather_capacity is None else int(gather_capacity)
        if self.pool is not None:
            self.gathered = out((max(self.gather_capacity, 1), w.pool_dim), i16)
        # decode steps (allocated by alloc_steps): each layer's union rows of keys packed once per
        # trigger, the step's native query and gates, and the step's top-k outputs
        self.keys_sub = None

    def alloc_steps(self):
        """Buffers of the per-step top-k over the resident subset (lsa_topk_step)."""
        w, L, B = self.w, self.w.L, self.w.B
        f32, i32 = torch.float32, torch.int32
        kdt = {"f32": torch.float32, "bf16": torch.int16, "fp8": torch.uint8}[w.key_dtype]
        self.key_row_bytes = w.d_h * {"f32": 4, "bf16": 2, "fp8": 1}[w.key_dtype]
        self.keys_sub = [self._out((max(self.rows, 1), w.d_h), kdt) for _ in range(L)]
        self.h_step = [self._out((B, w.d), torch.int16 if w.act_dtype == "bf16" else f32) for _ in range(L)]
        self.c_step = [self._out((B, w.r), f32) for _ in range(L)]
        self.q_step = [self._out((B, w.n_h, w.d_h), f32) for _ in range(L)]
        self.g_step = [self._out((B, w.n_h), f32) for _ in range(L)]
        self.step_idx = [self._out((B, w.k), i32) for _ in range(L)]
        self.step_score = [self._out((B, w.k), f32) for _ in range(L)]
        self.step_count = self._out((L, B), i32)

    def _out(self, shape, dtype):
        """An output buffer. With guard=True it sits between two GUARD_BYTES canary bands."""
        n = 1
        for s_ in shape:
            n *= int(s_)
        if not self.guard:
            return torch.empty(shape, dtype=dtype, device=self.device)
        esz = torch.empty(0, dtype=dtype).element_size()
        nbytes = n * esz
        raw = torch.full((GUARD_BYTES + nbytes + GUARD_BYTES,), CANARY, dtype=torch.uint8, device=self.device)
        self._guarded.append((raw, nbytes))
        return raw[GUARD_BYTES:GUARD_BYTES + nbytes].view(dtype).view(shape)

    def check_guards(self):
        """Return the indices of output buffers whose canary bands were written."""
        bad = []
        for i, (raw, nbytes) in enumerate(self._guarded):
            head = raw[:GUARD_BYTES]
            tail = raw[GUARD_BYTES + nbytes:]
            if not (bool((head == CANARY).all()) and bool((tail == CANARY).all())):
                bad.append(i)
        return bad

    # ------------------------------------------------------------- stages
    def project(self, stream=None):
        w, L = self.w, self.w.L
        layers = []
        for j in range(2 * L):
            wdq, wiuq, ww = (self.mem if j < L else self.nat)[j % L]
            layers.append(dict(h=self.h[j % L], w_dq=wdq, w_iuq=wiuq, w_w=ww, c_out=self.c[j], q_out=self.q[j],
                               w_out=self.g[j]))
        if self.packed:
            lsa.project_packed(layers, B=w.B, d=w.d, r=w.r, n_h=w.n_h, d_h=w.d_h, stream=stream)
        else:
            lsa.project(layers, B=w.B, d=w.d, r=w.r, n_h=w.n_h, d_h=w.d_h, dtype=w.act_dtype, stream=stream)

    def score_select(self, stream=None):
        """The step's score pass: masks only, with score_options if set."""
        self._score_call(self.masks, None, self.score_options, stream)

    def score_with_sigmoid(self, stream=None, options=None):
        """A score pass that also writes the sigmoid scores (into scores and masks_scored)."""
        self._score_call(self.masks_scored, self.scores, options, stream)

    def _score_call(self, masks, scores, options, stream):
        w = self.w
        layers = [dict(q=self.q[l], w=self.g[l], keys=self.keys[l], key_scale=self.scale[l], mask_out=masks[l],
                       score_out=None if scores is None else scores[l]) for l in range(w.L)]
        lsa.score_select(layers, B=w.B, key_offsets=self.key_off, key_offsets_host=self.key_off_h,
                         mask_word_offsets=self.mwo, mask_word_offsets_host=self.mwo_h, n_h=w.n_h, d_h=w.d_h,
                         key_dtype=w.key_dtype, threshold=w.threshold, options=options, stream=stream)

    def union_compact(self, stream=None):
        w = self.w
        lsa.union_compact(self.masks, B=w.B, key_offsets=self.key_off, key_offsets_host=self.key_off_h,
                          mask_word_offsets=self.mwo, mask_word_offsets_host=self.mwo_h, idx_out=self.idx,
                          count_out=self.count, union_mask_out=self.union_mask, stream=stream)

    def _topk_layers(self):
        w, L = self.w, self.w.L
        return [dict(q=self.q[L + l], w=self.g[L + l], keys=self.keys[l], key_scale=self.scale[l],
                     topk_idx_out=self.topk_idx[l],
                     topk_score_out=None if self.topk_score is None else self.topk_score[l]) for l in range(L)]

    def topk(self, stream=None):
        w = self.w
        lsa.topk(self._topk_layers(), B=w.B, key_offsets=self.key_off, key_offsets_host=self.key_off_h,
                 idx=self.idx, count=self.count, n_h=w.n_h, d_h=w.d_h, key_dtype=w.key_dtype, k=w.k,
                 topk_count_out=self.topk_count, workspace=self.workspace, stream=stream)

    def topk_score_stage(self, stream=None):
        w = self.w
        lsa.topk_score(self._topk_layers(), B=w.B, key_offsets=self.key_off, key_offsets_host=self.key_off_h,
                       idx=self.idx, count=self.count, n_h=w.n_h, d_h=w.d_h, key_dtype=w.key_dtype,
                       workspace=self.workspace, stream=stream)

    def topk_select_stage(self, stream=None):
        w = self.w
        lsa.topk_select(self._topk_layers(), B=w.B, key_offsets=self.key_off, key_offsets_host=self.key_off_h,
                        idx=self.idx, count=self.count, k=w.k, topk_count_out=self.topk_count,
                        workspace=self.workspace, stream=stream)

    def gather(self, stream=None):
        if self.pool is None:
            return
        w = self.w
        lsa.gather(self.pool, row_bytes=w.pool_dim * 2, B=w.B, pool_row_offsets=self.key_off,
                   pool_row_offsets_host=self.key_off_h, idx=self.idx, idx_offsets=self.key_off, count=self.count,
                   out=self.gathered, out_capacity_rows=self.gather_capacity, stream=stream)

    def fetch_host(self, stream=None):
        """The gather's rows, read from the pinned host copy of the pool (lsa_fetch_host)."""
        if self.pool_host is None:
            return
        w = self.w
        lsa.fetch_host(self.pool_host, row_bytes=w.pool_dim * 2, B=w.B, pool_row_offsets=self.key_off,
                       pool_row_offsets_host=self.key_off_h, idx=self.idx, idx_offsets=self.key_off, count=self.count,
                       out=self.gathered, out_capacity_rows=self.gather_capacity, stream=stream)

    # ------------------------------------------------------------- decode steps
    def pack_subset_keys(self, stream=None):
        """Once per trigger: each layer's keys of the union rows, packed in list order (lsa_gather)."""
        w = self.w
        for l in range(w.L):
            lsa.gather(self.keys[l], row_bytes=self.key_row_bytes, B=w.B, pool_row_offsets=self.key_off,
                       pool_row_offsets_host=self.key_off_h, idx=self.idx, idx_offsets=self.key_off, count=self.count,
                       out=self.keys_sub[l], out_capacity_rows=self.rows, stream=stream)

    def set_step_hidden(self, h_step):
        """Copy one decode step's hidden states ([layer] -> [B, d] stored values) into HBM."""
        for l, hl in enumerate(h_step):
            a = np.ascontiguousarray(hl)
            self.h_step[l].copy_(torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a))

    def step(self, stream=None):
        """One decode step: the native query and gates of the step's h (lsa_project with the native
        weights), then lsa_topk_step over the packed subset keys."""
        w, L = self.w, self.w.L
        layers = [dict(h=self.h_step[l], w_dq=self.nat[l][0], w_iuq=self.nat[l][1], w_w=self.nat[l][2],
                       c_out=self.c_step[l], q_out=self.q_step[l], w_out=self.g_step[l]) for l in range(L)]
        if self.packed:
            lsa.project_packed(layers, B=w.B, d=w.d, r=w.r, n_h=w.n_h, d_h=w.d_h, stream=stream)
        else:
            lsa.project(layers, B=w.B, d=w.d, r=w.r, n_h=w.n_h, d_h=w.d_h, dtype=w.act_dtype, stream=stream)
        self.step_topk(stream)

    def step_topk(self, stream=None):
        """lsa_topk_step with the step's native query (q_step, g_step) over the packed subset keys."""
        w, L = self.w, self.w.L
        tl = [dict(q=self.q_step[l], w=self.g_step[l], keys=self.keys_sub[l], key_scale=self.scale[l],
                   topk_idx_out=self.step_idx[l], topk_score_out=self.step_score[l]) for l in range(L)]
        lsa.topk_step(tl, B=w.B, key_offsets=self.key_off, key_offsets_host=self.key_off_h, idx=self.idx,
                      count=self.count, n_h=w.n_h, d_h=w.d_h, key_dtype=w.key_dtype, k=w.k,
                      topk_count_out=self.step_count, workspace=self.workspace, stream=stream)

    # ------------------------------------------------------------- core attention of the decode steps
    def alloc_attention(self, *, n_q, n_kv, d_h=128, dtype="bf16", page_tokens=64, entry_tokens=4, window=128, sinks=4,
                        max_steps=64, rot_dim=None, theta=10000.0, softcap=0.0, slopes=None):
        """A paged cache per layer for every sequence's N_b * entry_tokens prompt tokens and max_steps more, and the
        buffers of attend_step. The lists that step() makes hold entries of the prompt, so the steps' own tokens are seen
        through the window alone: it must cover max_steps. softcap and slopes ([n_q] float32 on the device) are the backbone's
        cap of its scores and its biases by distance (lsa_attend_topk_ex)."""
        if window < max_steps:
            raise ValueError(f"a window of {window} tokens would lose steps' tokens within max_steps = {max_steps}")
        if softcap != 0 and not 2.0 ** -10 <= softcap <= 1024:
            raise ValueError(f"softcap must be 0 or in [2^-10, 1024] (got {softcap})")
        if slopes is not None:
            device = torch.empty(0, device=self.device).get_device()
            lsa._want("alloc_attention", "slopes", slopes, torch.float32, (n_q,), device)
        self.softcap, self.slopes = softcap, slopes
        w, L, B = self.w, self.w.L, self.w.B
        bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
        self.entry_tokens, self.window, self.sinks, self.n_q, self.n_kv = entry_tokens, window, sinks, n_q, n_kv
        self.prompt_len = np.diff(self.key_off_h) * entry_tokens
        pages = -(-(self.prompt_len + max_steps) // page_tokens)
        self.capacity = self.prompt_len + max_steps
        first = np.concatenate([[0], np.cumsum(pages)])
        table = np.full((B, int(pages.max())), -1, np.int32)
        for b in range(B):
            table[b, :pages[b]] = np.arange(first[b], first[b + 1])
        self.page_table = _dev(table, self.device)
        self.len_h = np.zeros(B, np.int64)  # kv_len as far as the host has counted it
        self.prompt_len_dev = _dev(self.prompt_len.astype(np.int32), self.device)
        self.kv_len = torch.zeros(B, dtype=i32, device=self.device)
        shape = (int(first[-1]), n_kv, page_tokens, d_h)
        self.caches = []
        for _ in range(L):
            if dtype == "fp8":
                kv = [self._out(shape, torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)]
                scale = [self._out(shape[:2], f32) for _ in range(2)]
            else:
                kv, scale = [self._out(shape, bf16) for _ in range(2)], (None, None)
            self.caches.append(lsa.KvCache(k=kv[0], v=kv[1], k_scale=scale[0], v_scale=scale[1],
                                           page_table=self.page_table, kv_len=self.kv_len))
        rot = d_h if rot_dim is None else rot_dim
        self.inv_freq = _dev((theta ** (-np.arange(rot // 2) * 2.0 / rot)).astype(np.float32), self.device)
        self.prompt_off_h = np.concatenate([[0], np.cumsum(self.prompt_len)]).astype(np.int64)
        self.prompt_off = _dev(self.prompt_off_h, self.device)
        self.one_off_h = np.arange(B + 1, dtype=np.int64)
        self.one_off = _dev(self.one_off_h, self.device)
        self.q_rot = [self._out((B, n_q, d_h), bf16) for _ in range(L)]
        self.attn_out = [self._out((B, n_q, d_h), bf16) for _ in range(L)]
        self.attn_lse = [self._out((B, n_q), f32) for _ in range(L)]
        size = lsa.attend_topk_workspace_size(self.caches[0], n_q=n_q, k=w.k, entry_tokens=entry_tokens, window=window,
                                              sinks=sinks)
        self.attn_workspace = self._out((max(size, 16),), torch.uint8)

    @contextlib.contextmanager
    def _grow(self, by, by_dev, stream):
        """Within, every sequence has `by` tokens more, in the order of `stream`; an exception takes them back, so that what
        a failed call stored lies behind the lengths and is stored again by the next one. Nothing waits for the device."""
        if (self.len_h + by > self.capacity).any():
            raise ValueError("the cache is full: alloc_attention(max_steps=...) bounds the steps")
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.device)
        with torch.cuda.stream(stream):  # None: the current one
            self.kv_len.add_(by_dev)
            captured = self.device.type == "cuda" and torch.cuda.is_current_stream_capturing()
        try:
            yield
        except BaseException:
            with torch.cuda.stream(stream):
                self.kv_len.sub_(by_dev)
            raise
        if not captured:
            self.len_h = self.len_h + by

    def _check_layers(self, fn, name, given, heads, rows):
        """Refuses new rows that are not as the appends take them, for all layers before anything is enqueued: a refused call
        stores nothing in any layer."""
        if len(given) < self.w.L:
            lsa._refuse(fn, f"{name} must hold a tensor for each of the {self.w.L} layers (got {len(given)})")
        for l in range(self.w.L):
            lsa.check_rows(fn, f"{name}[{l}]", given[l], (rows[l], heads, self.q_rot[0].shape[2]), self.kv_len.get_device())

    def append_prompt(self, k, v, stream=None):
        """Once, before the steps: the prompt's keys and values, [layer] -> [sum of N_b * entry_tokens, n_kv, d_h] bfloat16,
        before the rotation, sequence after sequence."""
        if self.len_h.any():
            raise ValueError("the prompt comes once, before the steps: its tokens are the cache's first")
        rows = [max(int(self.prompt_off_h[-1]), t.shape[0]) for t in k]
        self._check_layers("append_prompt", "k", k, self.n_kv, rows)
        self._check_layers("append_prompt", "v", v, self.n_kv, rows)
        with self._grow(self.prompt_len, self.prompt_len_dev, stream):
            for l in range(self.w.L):
                lsa.kv_append(self.caches[l], k[l], v[l], new_offsets=self.prompt_off, new_offsets_host=self.prompt_off_h,
                              inv_freq=self.inv_freq, stream=stream)

    def attend_step(self, qkv, stream=None):
        """The step's core attention, after step(): qkv [layer] -> [B, n_q + 2 n_kv, d_h] bfloat16, the step's queries, keys
        and values before the rotation. Writes attn_out and attn_lse.

        May be captured, with step() before it: every replay is one more step. The host does not count replays (len_h), so
        keeping them within max_steps is the caller's part; a token beyond the cache's pages is not stored."""
        if self.keys_sub is None:
            raise ValueError("attend_step() attends over what step() lists: alloc_steps() first")
        n_q, n_kv, rows = self.n_q, self.n_kv, [self.w.B] * self.w.L
        q, k, v = [x[:, :n_q] for x in qkv], [x[:, n_q:n_q + n_kv] for x in qkv], [x[:, n_q + n_kv:] for x in qkv]
        for name, part, heads in (("queries of qkv", q, n_q), ("keys of qkv", k, n_kv), ("values of qkv", v, n_kv)):
            self._check_layers("attend_step", name, part, heads, rows)
        with self._grow(1, 1, stream):
            for l in range(self.w.L):
                lsa.kv_append(self.caches[l], k[l], v[l], new_offsets=self.one_off, new_offsets_host=self.one_off_h, q=q[l],
                              q_out=self.q_rot[l], inv_freq=self.inv_freq, stream=stream)
                lsa.attend_topk(self.caches[l], self.q_rot[l], idx=self.step_idx[l], count=self.step_count[l],
                                entry_tokens=self.entry_tokens, scale=self.q_rot[l].shape[2] ** -0.5, window=self.window,
                                sinks=self.sinks, out=self.attn_out[l], lse=self.attn_lse[l], workspace=self.attn_workspace,
                                softcap=self.softcap, slopes=self.slopes, stream=stream)

    def load(self, stream=None):
        """The load step: from the host pool when there is one, else from HBM."""
        if self.pool_host is not None:
            self.fetch_host(stream)
        else:
            self.gather(stream)

    def run(self, stream=None):
        """One pass of the path. The load step (gather, or the cold-pool fetch) needs only the
        union list, so it runs on a second stream forked right after the union and compaction,
        overlapping both top-k stages, and joins at the end. (Forking it after the top-k
        scoring instead, so that it overlaps only the selection, is 14 us slower per step on
        the three-layer workload: the scoring and the gather share HBM better than they
        queue. Projecting the native indexer on the second stream while the memory indexer
        scores is 6 us slower per step: score_select is the HBM-bound stage and loses more
        than the projection gains. Projecting it after the union instead, on this stream while
        the load runs on the other, is 24 us slower on the three-layer workload: that phase is
        already bound by HBM, and the split adds a second pair of projection launches.)"""
        main = torch.cuda.current_stream() if stream is None else stream
        self.project(main)
        self.score_select(main)
        self.union_compact(main)
        if self.pool is None or not self.overlap:
            self.topk(main)
            self.load(main)
            return
        if self.early_fork:
            self._fork.record(main)
            self._fork.wait(self._side)
            self.load(self._side)
            self.topk_score_stage(main)
        else:
            self.topk_score_stage(main)
            self._fork.record(main)
            self._fork.wait(self._side)
            self.load(self._side)
        self.topk_select_stage(main)
        self._join.record(self._side)
        self._join.wait(main)

    def capture(self):
        """Record one run() into a HIP graph and return it (replay with .replay()).

        run() allocates nothing and clears nothing with memset, so the graph holds
        exactly the kernel launches of the five calls, with these buffers baked in.
        """
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        torch.cuda.synchronize()
        return g

    def outputs(self):
        """Every output buffer of run(), for comparisons between runs."""
        out = self.c + self.q + self.g + self.masks + [self.idx, self.count, self.union_mask, self.topk_count]
        out += self.topk_idx
        if self.topk_score is not None:
            out += self.topk_score
        if self.pool is not None:
            out.append(self.gathered)
        return out

    # ------------------------------------------------------------- readback
    def masks_bool(self, l, scored=False):
        """Unpack layer l's mask words (of run(), or of score_with_sigmoid) into one bool array per sequence."""
        words = (self.masks_scored if scored else self.masks)[l][: self.words].cpu().numpy().view(np.uint64)
        return self._unpack(words)

    def union_bool(self):
        return self._unpack(self.union_mask[: self.words].cpu().numpy().view(np.uint64))

    def _unpack(self, words):
        out = []
        bits = np.unpackbits(words.view(np.uint8), bitorder="little")
        for b in range(self.w.B):
            w0, w1 = int(self.mwo_h[b]), int(self.mwo_h[b + 1])
            n = int(self.key_off_h[b + 1] - self.key_off_h[b])
            seg = bits[w0 * 64: w1 * 64]
            out.append((seg[:n].astype(bool), seg[n:].astype(bool)))
        return out
