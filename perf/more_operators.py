"""Measured cases of what the paged KV cache is served with beyond appending and plain attention.

Operators (`op` of a case):

  attend   lsa_attend_ex: attention of a ragged batch whose scores are capped by a tanh (`softcap`) or lose
           a slope per head times the distance (`slopes`), and whose rows see their document only (`docs`) or a
           whole prefix (`prefix`)
  topk     lsa_attend_topk_ex: the same scores for one token per sequence over listed entries, the window and
           the first tokens
  compact  lsa_kv_kept and lsa_kv_compact: listed entries, window and first tokens of every layer's cache, dense
           in other pages
  pages    lsa_kv_free, lsa_kv_extend and lsa_kv_fork: finished sequences give their pages back, admitted ones
           take pages, and each is forked into several samples

`run` computes them from elementary torch operations in 32 bits where `own` is false, and calls
the library where it is true. `exact` computes them in 64 bits, sequence by sequence.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases
def _case(name, op, *, B, ctx, new=(1, 1), n_q=64, n_kv=8, d=128, pt=64, dtype="fp8", window=0, sinks=0, lens_seed=1, **more):
    c = dict(op=op, B=B, ctx_lo=ctx[0], ctx_hi=ctx[1], n_kv=n_kv, d=d, pt=pt, dtype=dtype, lens_seed=lens_seed)
    if op in ("attend", "topk"):
        c.update(new_lo=new[0], new_hi=new[1], n_q=n_q, window=window, sinks=sinks, softcap=0.0, slopes=False)
        c.update(dict(docs=0, prefix=0) if op == "attend" else dict(k=0, r=1))
    elif op == "compact":
        c.update(window=window, sinks=sinks, keep=0.135, r=4, L=3)
    else:
        c.update(admit=1, ways=4, L=3, spare=64)
    c.update(more)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one request alone with distance biases: the shortest decode call, where latency is all
        _case("biased_token_bf16", "attend", B=1, ctx=(4095, 4095), dtype="bf16", slopes=True),
        # a decode step of 32 requests with capped scores, lengths spread as the ragged workload's entries
        _case("capped_decode_fp8", "attend", B=32, ctx=(4096, 131071), softcap=50.0, lens_seed=4),
        # whole prompts through layers with capped scores
        _case("capped_prompt_bf16", "attend", B=2, ctx=(0, 0), new=(2900, 5600), dtype="bf16", softcap=50.0, lens_seed=6),
        # a prompt's chunk on top of a long cached part, with distance biases
        _case("biased_chunk_fp8", "attend", B=1, ctx=(30_720, 30_720), new=(2048, 2048), slopes=True),
        # documents packed into one row of 8192 tokens, each seen by itself only
        _case("documents_bf16", "attend", B=1, ctx=(0, 0), new=(8192, 8192), dtype="bf16", docs=700, lens_seed=8),
        # prompts whose first part (an instruction with its context) sees itself in both directions, page size 16
        _case("prefix_fp8", "attend", B=3, ctx=(0, 0), new=(1800, 4500), prefix=1500, pt=16, lens_seed=9),
        # a decode step with capped scores over the native top-k of the main workload
        _case("capped_topk_fp8", "topk", B=8, ctx=(125_000, 125_000), k=2048, window=128, sinks=4, softcap=30.0),
        # one key head for all queries, distance biases, entries of four tokens, ragged
        _case("biased_topk_mqa_bf16", "topk", B=32, ctx=(4096, 131071), k=512, r=4, n_kv=1, window=512, dtype="bf16",
              slopes=True, lens_seed=4),
        # a short request thinned to what the indexer kept: latency
        _case("compact_one_bf16", "compact", B=1, ctx=(4096, 4096), dtype="bf16", window=128, sinks=4, L=1),
        # the main workload's eight requests, three layers, thinned to the share that the indexer keeps
        _case("compact_b8_fp8", "compact", B=8, ctx=(125_000, 125_000), window=128, sinks=4),
        # one request admitted and sampled four ways beside seven running ones
        _case("pages_one_bf16", "pages", B=8, ctx=(1, 4096), dtype="bf16", L=1),
        # sixteen of sixty-four long requests replaced and sampled eight ways
        _case("pages_many_fp8", "pages", B=64, ctx=(4096, 65_536), admit=16, ways=8, spare=2000, n_kv=2, lens_seed=5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1))))))))


def draw(rng):
    n_kv = rng.choice((1, 2, 4, 8))
    n_q = n_kv * rng.choice((1, 3, 4, 7, 8)) if n_kv > 1 else rng.choice((8, 16, 40, 64))
    c = dict(n_kv=n_kv, d=rng.choice((64, 128)), pt=rng.choice((16, 32, 64, 128)), dtype=rng.choice(("bf16", "fp8")),
             lens_seed=rng.randrange(1 << 20))
    form = rng.choice((dict(softcap=rng.choice((10.0, 30.0, 50.0, 120.0))), dict(slopes=True), dict(softcap=30.0, slopes=True)))
    kind = rng.choice(("decode", "chunk", "prompt", "window", "documents", "prefix", "topk", "compact", "pages"))
    window, sinks = _log_int(rng, 1, 4096), rng.choice((0, 1, 4, 5, 64))
    if kind in ("decode", "window"):
        top = _log_int(rng, 64, 40_000)
        more = dict(window=window, sinks=sinks) if kind == "window" else {}
        return _case(None, "attend", B=_log_int(rng, 1, 32), ctx=(top // 16, top), new=(1, rng.choice((1, 1, 2, 4))), n_q=n_q,
                     **c, **form, **more)
    if kind == "chunk":
        return _case(None, "attend", B=_log_int(rng, 1, 4), ctx=(0, _log_int(rng, 100, 12_000)), new=(1, _log_int(rng, 17, 700)),
                     n_q=n_q, **c, **form)
    if kind in ("prompt", "documents", "prefix"):
        if kind != "prompt":
            form = rng.choice(({}, {}, form))
            form = dict(form, **{"docs" if kind == "documents" else "prefix": _log_int(rng, 5, 1500)})
        return _case(None, "attend", B=_log_int(rng, 1, 4), ctx=(0, 0), new=(1, _log_int(rng, 100, 4000)), n_q=n_q, **c, **form)
    if kind == "topk":
        top = _log_int(rng, 64, 100_000)
        return _case(None, "topk", B=_log_int(rng, 1, 32), ctx=(top // 8, top), k=_log_int(rng, 1, 2048), n_q=n_q,
                     r=rng.choice((1, 1, 2, 4)), window=rng.choice((0, 1, window)), sinks=sinks, **c, **form)
    if kind == "compact":
        top = _log_int(rng, 100, 30_000)
        return _case(None, "compact", B=_log_int(rng, 1, 8), ctx=(top // 8, top), keep=rng.choice((0.01, 0.135, 0.3)),
                     r=rng.choice((1, 2, 4, 7)), L=rng.choice((1, 2, 3)), window=rng.choice((0, 1, window)), sinks=sinks, **c)
    c["n_kv"] = min(n_kv, 2)
    top = _log_int(rng, 64, 20_000)
    return _case(None, "pages", B=_log_int(rng, 2, 64), ctx=(top // 16, top), admit=_log_int(rng, 1, 8), ways=rng.choice((1, 2, 5, 8)),
                 spare=_log_int(rng, 1, 3000), L=rng.choice((1, 2, 3)), **c)


def _lens(case):
    """(new tokens, cached tokens with the new ones) of every sequence."""
    r = random.Random(case["lens_seed"])

    def some(lo, hi):
        return _log_int(r, lo, hi) if lo else r.randint(lo, hi)

    new = [some(case["new_lo"], case["new_hi"]) if "new_lo" in case else 0 for _ in range(case["B"])]
    return new, [n + some(case["ctx_lo"], case["ctx_hi"]) for n in new]


def _seen(case):
    """doc_start and prefix_end of every query row, as lists of positions, or None."""
    new, total = _lens(case)
    r = random.Random(case["lens_seed"] + 1)
    first, end = ([] if case["docs"] else None), ([] if case["prefix"] else None)
    for n, t in zip(new, total):
        if case["docs"]:
            starts, at = [], 0
            while at < t:
                m = _log_int(r, max(case["docs"] // 8, 1), 3 * case["docs"])
                starts += [at] * min(m, t - at)
                at += m
            first += starts[t - n:]
        if case["prefix"]:
            end += [min(t, _log_int(r, 1, case["prefix"]))] * n
    return first, end


def _pairs(case):
    """Visible (query, key) pairs of one head, and cached tokens that some query sees, over the batch."""
    new, total = _lens(case)
    W, S = case["window"], case["sinks"]
    pairs = rows = at = 0
    first, end = _seen(case) if case["op"] == "attend" else (None, None)
    for n, t in zip(new, total):
        if case["op"] == "topk":
            listed_tokens = min(case["k"], -(-t // case["r"])) * case["r"]
            v = min(t, listed_tokens + (min(W, t) + S if W else S))  # overlaps make it less
            pairs, rows = pairs + v, rows + v
            continue
        p = np.arange(t - n, t, dtype=np.int64)
        lo = np.maximum(p - W + 1, 0) if W else np.zeros_like(p)
        hi = p if end is None else np.maximum(p, np.asarray(end[at:at + n]) - 1)
        if first is not None:
            lo = np.maximum(lo, np.asarray(first[at:at + n]))
        pairs += int((hi - lo + 1 + (np.minimum(lo, S) if W else 0)).sum())
        rows += int(hi.max() - lo[0] + 1 + (min(int(lo[0]), S) if W else 0))
        at += n
    return pairs, rows


def _entries(case):
    """Listed entries of every sequence of a compaction."""
    _, total = _lens(case)
    return [max(1, int(round(-(-t // case["r"]) * case["keep"]))) for t in total]


def _most_kept(case):
    _, total = _lens(case)
    return max(min(t, n * case["r"] + case["window"] + case["sinks"]) for t, n in zip(total, _entries(case)))


def _admitted(case):
    r = random.Random(case["lens_seed"] + 2)
    return [_log_int(r, max(case["ctx_lo"], 1), case["ctx_hi"]) for _ in range(min(case["admit"], case["B"]))]


def work(case):
    d, n_kv, pt = case["d"], case["n_kv"], case["pt"]
    size = 2 if case["dtype"] == "bf16" else 1
    if case["op"] == "compact":
        _, total = _lens(case)
        kept = sum(min(t, n * case["r"] + case["window"] + case["sinks"]) for t, n in zip(total, _entries(case)))
        return {"bytes": 4 * kept * n_kv * d * size * case["L"] + 4 * sum(_entries(case)), "flops": 4 * kept * n_kv * d * case["L"]}
    if case["op"] == "pages":
        pages = sum(-(-t // pt) for t in _admitted(case))
        tails = sum(t % pt for t in _admitted(case)) * (case["ways"] - 1) * case["L"]
        # entries given back, taken and shared, their counts, and the copied part of the last pages
        return {"bytes": 4 * tails * n_kv * d * size + 12 * pages * (case["ways"] + 1), "flops": pages * (case["ways"] + 1)}
    new, _ = _lens(case)
    T, n_q = sum(new), case["n_q"]
    pairs, rows = _pairs(case)
    return {"bytes": 2 * rows * n_kv * d * size + T * n_q * (d * 4 + 4), "flops": 4 * pairs * n_q * d}


# ------------------------------------------------------------------ inputs
def _cache(g, dev, shape, fp8):
    """k, k_scale, v, v_scale with `shape` [n_pages, n_kv, pt, d]."""
    parts = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
        if fp8:  # the largest value of a page lies in the top binade of the format
            parts.append(x.mul_(80).clamp_(-448, 448).to(torch.float8_e4m3fn))
            e = torch.randint(-7, -5, shape[:2], generator=g, device=dev)
            parts.append(torch.ldexp(torch.ones_like(e, dtype=torch.float32), e))
        else:
            parts += [x, None]
    return parts


def _table(order, per, width, dev):
    """Rows of `per` pages each, in the order given; a row's end that no token uses holds -1."""
    table = torch.full((len(per), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _lists(g, dev, total, r, counts):
    """Ascending entry numbers of every sequence, one tensor each."""
    return [torch.randperm(-(-t // r), generator=g, device=dev)[:n].sort().values.to(torch.int32) for t, n in zip(total, counts)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case=case, library=None)
    if own:
        from sparse_kv_retrieval_amd import lsa
        s["library"] = lsa
    return {"compact": _prepare_compact, "pages": _prepare_pages}.get(case["op"], _prepare_attention)(s, case, g, dev)


def _prepare_attention(s, case, g, dev):
    new, total = _lens(case)
    B, T, pt, d, n_q, n_kv = case["B"], sum(new), case["pt"], case["d"], case["n_q"], case["n_kv"]
    per = [-(-t // pt) for t in total]
    # the pages of a serving process come in no order
    order = torch.randperm(sum(per), generator=g, device=dev).to(torch.int32)
    s["table"] = _table(order, per, max(per), dev)
    s["k"], s["k_scale"], s["v"], s["v_scale"] = _cache(g, dev, (sum(per) + 1, n_kv, pt, d), case["dtype"] == "fp8")
    off = np.zeros(B + 1, np.int64)
    off[1:] = np.cumsum(new)
    # scores with a spread of some units, so that a cap bends the largest
    s["q"] = torch.randn((T, n_q, d), generator=g, device=dev).mul_(4).to(torch.bfloat16)
    s.update(T=T, kv_len=torch.tensor(total, dtype=torch.int32, device=dev), off_host=off, off=torch.from_numpy(off).to(dev),
             max_new=max(new), max_len=max(total), scale=1.0 / math.sqrt(d),
             out=torch.empty((T, n_q, d), dtype=torch.bfloat16, device=dev), lse=torch.empty((T, n_q), dtype=torch.float32, device=dev))
    # the usual geometric sequence of slopes
    s["slopes"] = torch.exp2(-8.0 * (torch.arange(n_q, device=dev) + 1) / n_q).float() if case["slopes"] else None
    if case["op"] == "topk":
        count = [min(case["k"], -(-t // case["r"])) for t in total]
        s["idx"] = torch.full((B, case["k"]), -1, dtype=torch.int32, device=dev)
        for b, some in enumerate(_lists(g, dev, total, case["r"], count)):
            s["idx"][b, :count[b]] = some
        s["count"] = torch.tensor(count, dtype=torch.int32, device=dev)
    else:
        for name, x in zip(("doc_start", "prefix_end"), _seen(case)):
            s[name] = None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)
    if own:
        lsa = s["library"]
        s["cache"] = lsa.KvCache(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], page_table=s["table"],
                                 kv_len=s["kv_len"])
        if case["op"] == "attend":
            size = lsa.attend_workspace_size(s["cache"], n_q=n_q, q_offsets_host=off, max_kv_len=s["max_len"],
                                             window=case["window"], sinks=case["sinks"])
        else:
            size = lsa.attend_topk_workspace_size(s["cache"], n_q=n_q, k=case["k"], entry_tokens=case["r"],
                                                  window=case["window"], sinks=case["sinks"])
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    return s


def _prepare_compact(s, case, g, dev):
    _, total = _lens(case)
    B, pt, d, n_kv, fp8 = case["B"], case["pt"], case["d"], case["n_kv"], case["dtype"] == "fp8"
    most = _most_kept(case)
    per, per_to = [-(-t // pt) for t in total], [-(-most // pt)] * B
    s["table"] = _table(torch.randperm(sum(per), generator=g, device=dev).to(torch.int32), per, max(per), dev)
    s["table_to"] = _table(torch.randperm(sum(per_to), generator=g, device=dev).to(torch.int32), per_to, per_to[0], dev)
    s["layers"] = [_cache(g, dev, (sum(per), n_kv, pt, d), fp8) for _ in range(case["L"])]
    s["to"] = []
    for _ in range(case["L"]):
        x = [torch.zeros((sum(per_to), n_kv, pt, d), dtype=torch.bfloat16, device=dev) for _ in range(2)]
        scale = [torch.ones((sum(per_to), n_kv), device=dev) if fp8 else None for _ in range(2)]
        s["to"].append([y for a, b in zip(x, scale) for y in (a.to(torch.float8_e4m3fn) if fp8 else a, b)])
    count = _entries(case)
    s["idx"] = torch.cat(_lists(g, dev, total, case["r"], count))
    at = np.zeros(B + 1, np.int64)
    at[1:] = np.cumsum(count)
    s.update(most=most, kv_len=torch.tensor(total, dtype=torch.int32, device=dev), idx_offsets=torch.from_numpy(at).to(dev),
             count=torch.tensor(count, dtype=torch.int32, device=dev), kept=torch.zeros(B, dtype=torch.int32, device=dev))
    if own:
        s["caches"] = [[s["library"].KvCache(k=x[0], k_scale=x[1], v=x[2], v_scale=x[3], page_table=table, kv_len=length)
                        for x in layers] for layers, table, length in ((s["layers"], s["table"], s["kv_len"]),
                                                                       (s["to"], s["table_to"], s["kept"]))]
    return s


def _prepare_pages(s, case, g, dev):
    """Rows 0 .. B - 1 run, the first of them have finished; behind them come the rows of the samples."""
    _, total = _lens(case)
    B, pt, fp8 = case["B"], case["pt"], case["dtype"] == "fp8"
    admitted, ways = _admitted(case), case["ways"]
    A = len(admitted)
    more = [-(-t // pt) for t in admitted]
    per = [-(-t // pt) for t in total] + [0] * (A * (ways - 1))
    n_pages = sum(per) + sum(more) + A * (ways - 1) + case["spare"]
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    s["table"] = _table(order, per, max(per + more), dev)
    s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    s["refs"][order[:sum(per)].long()] = 1
    s["kv_len"] = torch.tensor(total + [0] * (A * (ways - 1)), dtype=torch.int32, device=dev)
    s["layers"] = [_cache(g, dev, (n_pages, case["n_kv"], pt, case["d"]), fp8) for _ in range(case["L"])]
    rows = list(range(A)) + list(range(B, B + A * (ways - 1)))
    i32 = dict(dtype=torch.int32, device=dev)
    s.update(gone=torch.tensor(rows, **i32), grow=torch.tensor(admitted + [0] * (len(per) - A), **i32),
             src=torch.tensor([i // (ways - 1) for i in range(A * (ways - 1))] if ways > 1 else [], **i32),
             dst=torch.tensor(rows[A:], **i32), missing=torch.empty(len(per), **i32), status=torch.empty(len(rows) - A, **i32))
    if own:
        lsa = s["library"]
        s["pool"] = lsa.KvPool(refs=s["refs"], page_table=s["table"], kv_len=s["kv_len"], page_tokens=pt)
        s["caches"] = [lsa.KvCache(k=x[0], k_scale=x[1], v=x[2], v_scale=x[3], page_table=s["table"], kv_len=s["kv_len"])
                       for x in s["layers"]]
        s["workspace"] = torch.empty(max(lsa.kv_fork_workspace_size(len(rows) - A), 1), dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c, lsa = s["case"], s["library"]
    if c["op"] == "compact":
        if own:
            want = dict(idx=s["idx"], idx_offsets=s["idx_offsets"], count=s["count"], entry_tokens=c["r"], window=c["window"],
                        sinks=c["sinks"])
            lsa.kv_kept(s["caches"][0][0], out=s["kept"], **want)
            lsa.kv_compact(s["caches"][0], s["caches"][1], max_kept=s["most"], **want)
        else:
            _plain_compact(s)
        return {"kept": s["kept"], "to": [[x for x in layer if x is not None] for layer in s["to"]]}
    if c["op"] == "pages":
        if own:
            lsa.kv_free(s["pool"], s["gone"])
            lsa.kv_extend(s["pool"], s["grow"], missing=s["missing"])
            if len(s["dst"]):
                lsa.kv_fork(s["pool"], s["caches"], s["src"], s["dst"], status=s["status"], workspace=s["workspace"])
        else:
            _plain_free(s)
            _plain_extend(s)
            if len(s["dst"]):
                _plain_fork(s)
        return {"refs": s["refs"], "table": s["table"], "kv_len": s["kv_len"], "missing": s["missing"], "status": s["status"],
                "layers": [[x for x in layer if x is not None] for layer in s["layers"]]}
    if own and c["op"] == "attend":
        lsa.attend(s["cache"], s["q"], q_offsets=s["off"], q_offsets_host=s["off_host"], max_kv_len=s["max_len"],
                   scale=s["scale"], window=c["window"], sinks=c["sinks"], softcap=c["softcap"], slopes=s["slopes"],
                   doc_start=s["doc_start"], prefix_end=s["prefix_end"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    elif own:
        lsa.attend_topk(s["cache"], s["q"], idx=s["idx"], count=s["count"], entry_tokens=c["r"], scale=s["scale"],
                        window=c["window"], sinks=c["sinks"], softcap=c["softcap"], slopes=s["slopes"], out=s["out"], lse=s["lse"],
                        workspace=s["workspace"])
    else:
        return _plain_topk(s) if c["op"] == "topk" else _plain_attend(s)
    return {"out": s["out"], "lse": s["lse"]}


def _rows(s, name, seq, pos):
    """The cached rows of positions `pos` [n, K] of sequences `seq` [n], as fp32 [n, n_kv, K, d]."""
    pt = s["case"]["pt"]
    page = s["table"][seq[:, None], pos // pt].long()
    x = s[name][page, :, pos % pt].float()
    if s[name + "_scale"] is not None:
        x *= s[name + "_scale"][page][..., None]
    return x.transpose(1, 2)


def _softmax_rows(s, q, K, V, seen, distance):
    """q [n, C, n_q, d], K and V [n, n_kv, keys, d], seen and distance [n, C, keys] -> out [n, C, n_q, d], lse [n, C, n_q]."""
    n, C, n_q, d = q.shape
    n_kv, cap = K.shape[1], s["case"]["softcap"]
    x = q.float().view(n, C, n_kv, n_q // n_kv, d).permute(0, 2, 3, 1, 4).reshape(n, n_kv, -1, d)
    x = torch.matmul(x * s["scale"], K.transpose(2, 3).contiguous()).view(n, n_kv, n_q // n_kv, C, -1)
    if cap:
        x.div_(cap).tanh_().mul_(cap)
    if s["slopes"] is not None:
        x.addcmul_(s["slopes"].view(1, n_kv, -1, 1, 1), distance[:, None, None], value=-1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    most = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    x.sub_(most).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(n, n_kv, -1, x.shape[-1]), V.contiguous()).view(n, n_kv, n_q // n_kv, C, d) / total.clamp_min(1e-37)
    lse = (total.log() + most).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(n, C, n_q, d), lse.permute(0, 3, 1, 2).reshape(n, C, n_q)


def _plain_attend(s):
    c, dev, W, S, C = s["case"], s["q"].device, s["case"]["window"], s["case"]["sinks"], s["max_new"]
    seq = torch.arange(c["B"], device=dev)
    at = torch.arange(C, device=dev).expand(c["B"], C)  # query of its sequence
    n_new, length = s["off"].diff(), s["kv_len"].long()
    real = at < n_new[:, None]
    row = s["off"][:-1, None] + torch.minimum(at, n_new[:, None] - 1)
    p = length[:, None] - n_new[:, None] + at
    key = torch.arange(s["max_len"], device=dev).expand(c["B"], -1)
    last = p if s["prefix_end"] is None else torch.maximum(p, s["prefix_end"][row] - 1)
    seen = (key < length[:, None])[:, None] & (key[:, None] <= last[..., None])
    if s["doc_start"] is not None:
        seen &= key[:, None] >= s["doc_start"][row][..., None]
    if W:
        seen &= (key[:, None] > p[..., None] - W) | (key[:, None] < S)
    at_key = torch.where(key < length[:, None], key, 0)
    out, lse = _softmax_rows(s, s["q"][row], _rows(s, "k", seq, at_key), _rows(s, "v", seq, at_key), seen,
                             (p[..., None] - key[:, None]).abs().float() if c["slopes"] else None)
    s["out"][row[real]] = out[real].to(s["out"].dtype)
    s["lse"][row[real]] = lse[real]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_topk(s):
    c, dev, W, S, r, B = s["case"], s["q"].device, s["case"]["window"], s["case"]["sinks"], s["case"]["r"], s["case"]["B"]
    length = s["kv_len"].long()[:, None]
    near = torch.cat([torch.arange(S, device=dev).expand(B, S), length - W + torch.arange(W, device=dev)], 1)
    ok = torch.cat([near[:, :S] < length, near[:, S:] >= S], 1)
    idx = torch.where(torch.arange(c["k"], device=dev) < s["count"][:, None], s["idx"].long(), -1)
    far = (idx[..., None] * r + torch.arange(r, device=dev)).flatten(1)
    ok = torch.cat([ok, (far >= S) & (far < length - W)], 1)
    key = torch.where(ok, torch.cat([near, far], 1), 0)
    seq = torch.arange(B, device=dev)
    out, lse = _softmax_rows(s, s["q"][:, None], _rows(s, "k", seq, key), _rows(s, "v", seq, key), ok[:, None],
                             (length - 1 - key)[:, None].float())
    return {"out": out[:, 0].to(s["out"].dtype), "lse": lse[:, 0]}


def _least_scale(a):
    """The least power of two s with a <= 448 s, for a > 0, and 2^-118 at least."""
    m, e = torch.frexp(a)  # a = m 2^e, 0.5 <= m < 1, and 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-118)
    return torch.ldexp(torch.ones_like(a), torch.where(a > 0, e, torch.full_like(e, -118)))


def _plain_compact(s):
    c, dev, B, pt, r = s["case"], s["idx"].device, s["case"]["B"], s["case"]["pt"], s["case"]["r"]
    length, n = s["kv_len"].long()[:, None], s["table"].shape[1] * pt
    width = s["table_to"].shape[1]
    token = torch.arange(n, device=dev)
    in_list = torch.zeros((B, -(-n // r)), dtype=torch.bool, device=dev)
    seq = torch.searchsorted(s["idx_offsets"], torch.arange(len(s["idx"]), device=dev), right=True) - 1
    in_list[seq, s["idx"].long()] = True
    keep = in_list.repeat_interleave(r, 1)[:, :n] | (token < c["sinks"]) | (token >= length - c["window"])
    upto = (keep & (token < length)).int().cumsum(1)
    s["kept"].copy_(upto[:, -1])
    # the token that place i takes is the first one with i + 1 kept ones up to it
    place = torch.arange(width * pt, device=dev).expand(B, -1)
    source = torch.searchsorted(upto, (place + 1).to(upto.dtype).contiguous()).clamp_max(n - 1)
    real = (place < s["kept"][:, None]).view(B, width, pt)
    page, slot = s["table"].gather(1, source // pt).long(), source % pt
    page = torch.where(real.flatten(1), page, 0)
    to = s["table_to"].long()
    used = real.any(-1)
    for layer, dest in zip(s["layers"], s["to"]):
        for x, scale, y, y_scale in (layer[:2] + dest[:2], layer[2:] + dest[2:]):
            rows = x[page, :, slot].view(B, width, pt, *x.shape[1::2])  # [B, pages, pt, n_kv, d]
            if scale is not None:
                rows = rows.float() * scale[page].view(B, width, pt, -1, 1)
                after = _least_scale(torch.where(real[..., None, None], rows.abs(), 0).amax((2, 4)))
                rows = (rows / after[:, :, None, :, None]).to(y.dtype)
                y_scale[to] = torch.where(used[..., None], after, y_scale[to])
            old = y[to].transpose(2, 3)
            y[to] = torch.where(real[..., None, None], rows.view(torch.uint8), old.view(torch.uint8)).view(y.dtype).transpose(2, 3) \
                if scale is not None else torch.where(real[..., None, None], rows, old).transpose(2, 3)


def _held(s, rows):
    """Which entries of these rows of the table hold pages."""
    n = -(-s["kv_len"][rows].long() // s["case"]["pt"])
    return torch.arange(s["table"].shape[1], device=n.device) < n[:, None]


def _plain_free(s):
    rows = s["gone"].long()
    held = _held(s, rows)
    s["refs"].index_add_(0, s["table"][rows].clamp_min(0).flatten(), -held.int().flatten())
    s["table"][rows] = torch.where(held, -1, s["table"][rows])
    s["kv_len"][rows] = 0


def _lowest_free(s):
    """Pages with the free ones first, in ascending order, and how many are free."""
    free = s["refs"] <= 0
    return torch.argsort((~free).int(), stable=True).int(), free.sum()


def _plain_extend(s):
    pt = s["case"]["pt"]
    order, free = _lowest_free(s)
    length = s["kv_len"].long()
    have, want = -(-length // pt), -(-(length + s["grow"]) // pt)
    upto = (want - have).cumsum(0)
    granted = (upto <= free) | (want == have)
    s["missing"].copy_(torch.where(granted, 0, want - have))
    j = torch.arange(s["table"].shape[1], device=length.device)
    new = (j >= have[:, None]) & (j < want[:, None]) & granted[:, None]
    page = order[((upto - want)[:, None] + j).clamp(0, len(order) - 1)]
    s["table"].copy_(torch.where(new, page, s["table"]))
    s["refs"].index_add_(0, page.flatten(), new.int().flatten())
    s["kv_len"].add_(torch.where(granted, s["grow"], 0))


def _plain_fork(s):
    """The samples' rows are empty: they were freed."""
    pt, src, dst = s["case"]["pt"], s["src"].long(), s["dst"].long()
    length = s["kv_len"][src].long()
    full, tail = length // pt, length % pt
    j = torch.arange(s["table"].shape[1], device=src.device)
    shared = j < full[:, None]
    s["refs"].index_add_(0, s["table"][src].clamp_min(0).flatten(), shared.int().flatten())
    order, free = _lowest_free(s)
    upto = (tail > 0).cumsum(0)
    granted = upto <= free
    copied = (tail > 0) & granted
    page = order[(upto - 1).clamp(0, len(order) - 1)]
    last = (j == full[:, None]) & copied[:, None]
    s["refs"].index_add_(0, page, copied.int())
    s["table"][dst] = torch.where(shared, s["table"][src], torch.where(last, page[:, None], s["table"][dst]))
    s["kv_len"][dst] = torch.where(copied, length, full * pt).int()
    s["status"].copy_((tail > 0) & ~granted)
    used = (torch.arange(pt, device=src.device) < tail[:, None]) & copied[:, None]
    start = s["table"][src, full.clamp_max(s["table"].shape[1] - 1)].clamp_min(0).long()
    to = page.long()
    for layer in s["layers"]:
        for x, scale in (layer[:2], layer[2:]):
            bits = x.view(torch.uint8 if scale is not None else torch.int16)
            bits[to] = torch.where(used[:, None, :, None], bits[start], bits[to])
            if scale is not None:
                scale[to] = torch.where(copied[:, None], scale[start], scale[to])


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """In 64 bits and without the last rounding; what is held in 8 bits in units of its scale."""
    s = prepare(case, seed)
    if case["op"] == "compact":
        return _exact_compact(s)
    return None if case["op"] == "pages" else _exact_attention(s)


def _exact_attention(s):
    c = s["case"]
    new, total = _lens(c)
    W, S, pt, G, d = c["window"], c["sinks"], c["pt"], c["n_q"] // c["n_kv"], c["d"]
    dev = s["q"].device
    out = torch.zeros((s["T"], c["n_q"], d), dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], c["n_q"]), -math.inf, dtype=torch.float64, device=dev)
    begin = 0
    for b, (n, t) in enumerate(zip(new, total)):
        pages = s["table"][b, :-(-t // pt)].long()
        position = torch.arange(t, device=dev)
        in_list = torch.zeros(t, dtype=torch.bool, device=dev)
        if c["op"] == "topk":
            some = s["idx"][b, :int(s["count"][b])].long()
            far = (some[:, None] * c["r"] + torch.arange(c["r"], device=dev)).flatten()
            in_list[far[far < t]] = True
        elif not W:
            in_list[:] = True
        for h in range(c["n_kv"]):
            def cached(name):
                x = s[name][pages, h].double()
                return (x if s[name + "_scale"] is None else x * s[name + "_scale"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]

            K, V, heads = cached("k"), cached("v"), slice(h * G, (h + 1) * G)
            for i in range(0, n, 512):
                m = min(512, n - i)
                rows = slice(begin + i, begin + i + m)
                at = (t - n + i + torch.arange(m, device=dev))[:, None]
                last, first = at, torch.zeros_like(at)
                if c["op"] == "attend" and s["prefix_end"] is not None:
                    last = torch.maximum(at, s["prefix_end"][rows, None].long() - 1)
                if c["op"] == "attend" and s["doc_start"] is not None:
                    first = s["doc_start"][rows, None].long()
                see = (position <= last) & (position >= first) & (in_list | (position < S) | (position > at - W))
                x = torch.matmul(s["q"][rows, heads].double().reshape(m * G, d), K.t().contiguous()) * s["scale"]
                x = x.view(m, G, t)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                if s["slopes"] is not None:
                    x = x - s["slopes"][heads].double()[:, None] * (at - position).abs().double()[:, None]
                x = x.masked_fill(~see[:, None], -math.inf)
                some = see.any(-1)
                l = torch.logsumexp(x, -1)
                y = torch.matmul(torch.exp(x - torch.where(some[:, None], l, 0.0)[..., None]).view(m * G, t), V).view(m, G, d)
                out[rows, heads], lse[rows, heads] = y, l
        begin += n
    return {"out": out, "lse": lse}


def _exact_compact(s):
    c = s["case"]
    _, total = _lens(c)
    pt, at = c["pt"], s["idx_offsets"].tolist()
    to = [[None if x is None else x.double() for x in layer] for layer in s["to"]]
    kept = []
    for b, t in enumerate(total):
        entries = set(s["idx"][at[b]:at[b + 1]].tolist())
        some = [p for p in range(t) if p // c["r"] in entries or p < c["sinks"] or p >= t - c["window"]]
        kept.append(len(some))
        p = torch.tensor(some, dtype=torch.long, device=s["table"].device)
        page = s["table"][b, p // pt].long()
        for layer, dest in zip(s["layers"], to):
            for x, scale, y, y_scale in (layer[:2] + dest[:2], layer[2:] + dest[2:]):
                rows = x[page, :, p % pt].double()  # [kept, n_kv, d]
                if scale is not None:
                    rows = rows * scale[page].double()[..., None]
                for i in range(0, len(some), pt):
                    page_to, part = int(s["table_to"][b, i // pt]), rows[i:i + pt].transpose(0, 1)
                    if scale is not None:
                        y_scale[page_to] = torch.exp2(torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448)).clamp_min(-118))
                        part = part / y_scale[page_to][:, None, None]
                    y[page_to, :, :part.shape[1]] = part
    return {"kept": None, "to": [[x for x in layer if x is not None] for layer in to]}
