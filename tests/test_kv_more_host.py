"""Refusals of lsa_attend_ex, lsa_attend_topk_ex, lsa_kv_kept, lsa_kv_compact, lsa_kv_extend, lsa_kv_fork and lsa_kv_free (CPU):
every call here is rejected by argument checks before anything touches the device, and leaves a text that says why."""
import ctypes

import numpy as np
import pytest

from tests.test_kv_host import BAD_CACHES, FAKE, SHARED, cache, lsa, off, refused  # noqa: F401  (lsa is a fixture)


def form(lsa, **kw):
    return lsa._AttendForm(*[kw.get(f, 0) for f, _ in lsa._AttendForm._fields_])


def attend(lsa, c=None, **kw):
    host = kw.pop("host", off(1, 2))
    a = dict(B=2, q=FAKE, qs=256, n_q=4, off=FAKE, host=host.ctypes.data, max_len=100, scale=1.0, window=0, sinks=0,
             form=form(lsa, softcap=5.0), out=FAKE + 4096, os=256, lse=None, ws=FAKE, nb=1 << 30)
    a.update(kw)
    return lsa._attend_ex(ctypes.byref(c or cache(lsa)), *[a[x] for x in ("B", "q", "qs", "n_q", "off", "host", "max_len", "scale", "window",
                                                                        "sinks", "form", "out", "os", "lse", "ws", "nb")], 0)


def topk(lsa, c=None, **kw):
    a = dict(B=2, q=FAKE, qs=256, n_q=4, idx=FAKE, count=FAKE, k=64, r=1, scale=1.0, window=0, sinks=0, form=form(lsa, slopes=FAKE),
             out=FAKE + 4096, os=256, lse=None, ws=FAKE, nb=1 << 30)
    a.update(kw)
    return lsa._attend_topk_ex(ctypes.byref(c or cache(lsa)), *[a[x] for x in ("B", "q", "qs", "n_q", "idx", "count", "k", "r", "scale",
                                                                             "window", "sinks", "form", "out", "os", "lse", "ws", "nb")], 0)


def kept(lsa, c=None, **kw):
    a = dict(B=2, idx=FAKE, off=FAKE, count=FAKE, r=4, window=0, sinks=0, out=FAKE)
    a.update(kw)
    return lsa._kv_kept(ctypes.byref(c or cache(lsa)), *[a[x] for x in ("B", "idx", "off", "count", "r", "window", "sinks", "out")], 0)


def compact(lsa, c=None, **kw):
    a = dict(frm=[c or cache(lsa)] * 2, to=[cache(lsa)] * 2, L=2, B=2, idx=FAKE, off=FAKE, count=FAKE, r=4, window=0, sinks=0, most=100)
    a.update(kw)
    a["frm"], a["to"] = [x if x is None else (lsa._KvCache * len(x))(*x) for x in (a["frm"], a["to"])]
    return lsa._kv_compact(*[a[x] for x in ("frm", "to", "L", "B", "idx", "off", "count", "r", "window", "sinks", "most")], 0)


def pool(lsa, **kw):
    d = dict(refs=FAKE, page_table=FAKE, kv_len=FAKE, table_stride=8, B=2, n_pages=4, page_tokens=16)
    d.update(kw)
    return lsa._KvPool(*[d[f] for f, _ in lsa._KvPool._fields_])


def extend(lsa, p=None, **kw):
    return lsa._kv_extend(ctypes.byref(p or pool(lsa)), kw.get("n_new", FAKE), None, 0)


def fork(lsa, p=None, **kw):
    a = dict(layers=[cache(lsa)] * 2, L=2, n=3, src=FAKE, dst=FAKE, status=FAKE, ws=FAKE, nb=1 << 20)
    a.update(kw)
    a["layers"] = a["layers"] and (lsa._KvCache * len(a["layers"]))(*a["layers"])
    return lsa._kv_fork(ctypes.byref(p or pool(lsa)), *[a[x] for x in ("layers", "L", "n", "src", "dst", "status", "ws", "nb")], 0)


def free(lsa, p=None, **kw):
    return lsa._kv_free(ctypes.byref(p or pool(lsa)), kw.get("n", 3), kw.get("seqs", FAKE), 0)


@pytest.mark.parametrize("call", [attend, topk, kept, compact], ids=["attend_ex", "topk_ex", "kept", "compact"])
@pytest.mark.parametrize("bad", BAD_CACHES, ids=[f"{list(b[2].items())[-1]}" for b in BAD_CACHES])
def test_cache(lsa, call, bad):
    refused(lsa, getattr(lsa, "ERR_" + bad[0]), bad[1], call(lsa, cache(lsa, **bad[2])))


FORMS = [("UNSUPPORTED", "softcap", dict(softcap=-1.0)), ("UNSUPPORTED", "softcap", dict(softcap=float("nan"))),
         ("UNSUPPORTED", "softcap", dict(softcap=float("inf"))), ("UNSUPPORTED", "softcap", dict(softcap=1025.0)),
         ("UNSUPPORTED", "softcap", dict(softcap=1e-4)), ("INVALID_ARG", "4-byte", dict(slopes=FAKE + 2)),
         ("INVALID_ARG", "4-byte", dict(doc_start=FAKE + 1)), ("INVALID_ARG", "4-byte", dict(prefix_end=FAKE + 3))]


@pytest.mark.parametrize("call", [attend, topk], ids=["attend_ex", "topk_ex"])
@pytest.mark.parametrize("status,match,kw", FORMS)
def test_form(lsa, call, status, match, kw):
    refused(lsa, getattr(lsa, "ERR_" + status), match, call(lsa, form=form(lsa, **kw)))


def test_form_combinations(lsa):
    refused(lsa, lsa.ERR_UNSUPPORTED, "window", attend(lsa, window=10, form=form(lsa, prefix_end=FAKE)))
    refused(lsa, lsa.ERR_UNSUPPORTED, "listed", topk(lsa, form=form(lsa, prefix_end=FAKE)))
    refused(lsa, lsa.ERR_UNSUPPORTED, "listed", topk(lsa, form=form(lsa, doc_start=FAKE)))


@pytest.mark.parametrize("call,more", [(attend, {}), (topk, dict(k=512))], ids=["attend_ex", "topk_ex"])
@pytest.mark.parametrize("status,match,kw", SHARED)
def test_shared_with_the_plain_calls(lsa, call, more, status, match, kw):
    if call is attend:
        more = {"max_len": 1000}
    refused(lsa, getattr(lsa, "ERR_" + status), match, call(lsa, cache(lsa, table_stride=64), **{**more, **kw}))


LISTS = [("UNSUPPORTED", "B must", dict(B=0)), ("UNSUPPORTED", "B must", dict(B=4097)), ("INVALID_ARG", "idx", dict(idx=None)),
         ("INVALID_ARG", "idx_offsets", dict(off=None)), ("INVALID_ARG", "count", dict(count=None)),
         ("UNSUPPORTED", "entry_tokens", dict(r=0)), ("UNSUPPORTED", "entry_tokens", dict(r=129)),
         ("INVALID_ARG", "negative", dict(window=-1)), ("INVALID_ARG", "negative", dict(sinks=-1))]


@pytest.mark.parametrize("call", [kept, compact], ids=["kept", "compact"])
@pytest.mark.parametrize("status,match,kw", LISTS)
def test_lists(lsa, call, status, match, kw):
    refused(lsa, getattr(lsa, "ERR_" + status), match, call(lsa, **kw))


def test_kept(lsa):
    refused(lsa, lsa.ERR_INVALID_ARG, "kept_out", kept(lsa, out=None))


def test_compact(lsa):
    c = cache(lsa)
    bad = lambda **kw: cache(lsa, **kw)
    for status, match, kw in [
            ("INVALID_ARG", "from is NULL", dict(frm=None)), ("INVALID_ARG", "to is NULL", dict(to=None)),
            ("UNSUPPORTED", "L must", dict(L=0)), ("UNSUPPORTED", "L must", dict(L=1025)),
            ("INVALID_ARG", "from\\[1\\] must have the dtype", dict(frm=[c, bad(n_kv=4)])),
            ("INVALID_ARG", "to\\[1\\] must have the dtype", dict(to=[c, bad(n_pages=5)])),
            ("INVALID_ARG", "to\\[1\\] must have the dtype", dict(to=[c, bad(page_tokens=32)])),
            ("INVALID_ARG", "to\\[1\\] must have the dtype", dict(to=[c, bad(d_h=128)])),
            ("INVALID_ARG", "from\\[1\\] must have the page_table", dict(frm=[c, bad(page_table=FAKE + 64)])),
            ("INVALID_ARG", "to\\[1\\] must have the page_table", dict(to=[c, bad(kv_len=FAKE + 64)])),
            ("INVALID_ARG", "to\\[1\\] must have the page_table", dict(to=[c, bad(table_stride=9)])),
            ("INVALID_ARG", "equal dtype", dict(to=[bad(n_kv=1)] * 2)), ("INVALID_ARG", "equal dtype", dict(to=[bad(d_h=128)] * 2)),
            ("INVALID_ARG", "equal dtype", dict(to=[bad(dtype=2, k_scale=FAKE, v_scale=FAKE)] * 2)),
            ("INVALID_ARG", "max_kept", dict(most=-1)), ("INVALID_ARG", "max_kept", dict(most=129)),
            ("UNSUPPORTED", "too many", dict(B=4096, to=[bad(table_stride=1 << 20)] * 2, most=1 << 24))]:
        refused(lsa, getattr(lsa, "ERR_" + status), match, compact(lsa, **kw))
    assert compact(lsa, most=0) == lsa.OK


@pytest.mark.parametrize("call", [extend, fork, free], ids=["extend", "fork", "free"])
@pytest.mark.parametrize("status,match,kw", [
    ("INVALID_ARG", "must be set", dict(refs=None)), ("INVALID_ARG", "must be set", dict(page_table=None)),
    ("INVALID_ARG", "must be set", dict(kv_len=None)), ("INVALID_ARG", "16-byte", dict(refs=FAKE + 4)), ("UNSUPPORTED", "B must", dict(B=0)),
    ("UNSUPPORTED", "B must", dict(B=4097)), ("INVALID_ARG", "n_pages", dict(n_pages=0)), ("UNSUPPORTED", "page_tokens", dict(page_tokens=24)),
    ("INVALID_ARG", "table_stride", dict(table_stride=0)), ("INVALID_ARG", "table_stride", dict(table_stride=1 << 28))])
def test_pool(lsa, call, status, match, kw):
    refused(lsa, getattr(lsa, "ERR_" + status), match, call(lsa, pool(lsa, **kw)))


def test_pool_calls(lsa):
    refused(lsa, lsa.ERR_INVALID_ARG, "pool is NULL", lsa._kv_extend(None, FAKE, None, 0))
    refused(lsa, lsa.ERR_INVALID_ARG, "n_new", extend(lsa, n_new=None))
    refused(lsa, lsa.ERR_INVALID_ARG, "seqs", free(lsa, seqs=None))
    for call in (free, fork):
        refused(lsa, lsa.ERR_UNSUPPORTED, "n must", call(lsa, n=-1))
        refused(lsa, lsa.ERR_UNSUPPORTED, "n must", call(lsa, n=4097))
        assert call(lsa, n=0) == lsa.OK
    for status, match, kw in [
            ("INVALID_ARG", "layers is NULL", dict(layers=None)), ("UNSUPPORTED", "L must", dict(L=0)),
            ("INVALID_ARG", "pool's n_pages", dict(layers=[cache(lsa, n_pages=5)] * 2)),
            ("INVALID_ARG", "pool's n_pages", dict(layers=[cache(lsa, page_tokens=32)] * 2)),
            ("INVALID_ARG", "layers\\[1\\]", dict(layers=[cache(lsa), cache(lsa, n_kv=1)])),
            ("INVALID_ARG", "src, dst", dict(src=None)), ("INVALID_ARG", "src, dst", dict(dst=None)), ("INVALID_ARG", "src, dst", dict(status=None)),
            ("WORKSPACE", "workspace needs", dict(ws=None)), ("WORKSPACE", "workspace needs", dict(nb=47)),
            ("INVALID_ARG", "16-byte", dict(ws=FAKE + 8)),
            ("UNSUPPORTED", "too many", dict(n=4096, L=16, layers=[cache(lsa, n_kv=1024)] * 16))]:
        refused(lsa, getattr(lsa, "ERR_" + status), match, fork(lsa, **kw))
    assert lsa.kv_fork_workspace_size(3) == 48 and lsa.kv_fork_workspace_size(-1) == 0 and lsa.kv_fork_workspace_size(4097) == 0


# ------------------------------------------------------------------ the binding's own checks, with CPU tensors
def make(lsa, torch, **kw):
    d = dict(k=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), page_table=torch.zeros(2, 3, dtype=torch.int32), kv_len=torch.zeros(2, dtype=torch.int32))
    d.update(kw)
    return lsa.KvCache(v=d["k"].clone(), **d)


def says(lsa, match, call, *a, **kw):
    with pytest.raises(lsa.LsaError, match=match):
        call(*a, **kw)


def test_binding_attend(lsa):
    torch = pytest.importorskip("torch")
    c, q = make(lsa, torch), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    kw = dict(q_offsets=torch.tensor([0, 1, 3]), q_offsets_host=np.array([0, 1, 3]), max_kv_len=40, out=q.clone(), scale=1.0)
    says(lsa, "slopes", lsa.attend, c, q, slopes=torch.zeros(3), **kw)
    says(lsa, "slopes", lsa.attend, c, q, slopes=torch.zeros(4, dtype=torch.float64), **kw)
    says(lsa, "doc_start", lsa.attend, c, q, doc_start=torch.zeros(3, dtype=torch.int64), **kw)
    says(lsa, "prefix_end", lsa.attend, c, q, prefix_end=torch.zeros(2, dtype=torch.int32), **kw)
    says(lsa, "on a GPU", lsa.attend, c, q, softcap=3.0, **kw)
    kw = dict(idx=torch.zeros(2, 5, dtype=torch.int32), count=torch.zeros(2, dtype=torch.int32), out=q[:2].clone(), scale=1.0)
    says(lsa, "slopes", lsa.attend_topk, c, q[:2], slopes=torch.zeros(4, 1), **kw)


def test_binding_compact(lsa):
    torch = pytest.importorskip("torch")
    c = make(lsa, torch)
    i32 = dict(dtype=torch.int32)
    kw = dict(idx=torch.zeros(9, **i32), idx_offsets=torch.zeros(3, dtype=torch.int64), count=torch.zeros(2, **i32))
    out = torch.zeros(2, **i32)
    says(lsa, "out", lsa.kv_kept, c, out=torch.zeros(3, **i32), **kw)
    says(lsa, "idx_offsets", lsa.kv_kept, c, out=out, **{**kw, "idx_offsets": torch.zeros(4, dtype=torch.int64)})
    says(lsa, "count", lsa.kv_kept, c, out=out, **{**kw, "count": torch.zeros(2)})
    says(lsa, "32 bits", lsa.kv_kept, c, out=out, window=1 << 40, **kw)
    says(lsa, "as many", lsa.kv_compact, [c], [c, c], max_kept=4, **kw)
    says(lsa, "as many", lsa.kv_compact, [], [], max_kept=4, **kw)
    says(lsa, "sequences", lsa.kv_compact, [c], [make(lsa, torch, kv_len=torch.zeros(1, **i32), page_table=torch.zeros(1, 3, **i32))], max_kept=4, **kw)
    says(lsa, "32 bits", lsa.kv_compact, [c], [c], max_kept=1 << 31, **kw)
    says(lsa, "on a GPU", lsa.kv_compact, [c], [c], max_kept=4, **kw)


def test_binding_pool(lsa):
    torch = pytest.importorskip("torch")
    i32 = dict(dtype=torch.int32)
    kw = dict(refs=torch.zeros(4, **i32), page_table=torch.zeros(2, 3, **i32), kv_len=torch.zeros(2, **i32), page_tokens=16)
    says(lsa, "refs", lsa.KvPool, **{**kw, "refs": torch.zeros(4, 1, **i32)})
    says(lsa, "refs", lsa.KvPool, **{**kw, "refs": torch.zeros(4)})
    says(lsa, "page_table", lsa.KvPool, **{**kw, "page_table": torch.zeros(3, 3, **i32)})
    p, c, x, ws = lsa.KvPool(**kw), make(lsa, torch), torch.zeros(2, **i32), torch.zeros(64, dtype=torch.uint8)
    says(lsa, "n_new", lsa.kv_extend, p, torch.zeros(3, **i32))
    says(lsa, "missing", lsa.kv_extend, p, x, missing=torch.zeros(2))
    says(lsa, "seqs", lsa.kv_free, p, torch.zeros(2))
    says(lsa, "dst", lsa.kv_fork, p, [c], x, x[:1], status=x, workspace=ws)
    says(lsa, "status", lsa.kv_fork, p, [c], x, x, status=x[:1], workspace=ws)
    says(lsa, "caches", lsa.kv_fork, p, [], x, x, status=x, workspace=ws)
    for call, a in ((lsa.kv_extend, (p, x)), (lsa.kv_free, (p, x))):
        says(lsa, "on a GPU", call, *a)
    says(lsa, "on a GPU", lsa.kv_fork, p, [c], x, x, status=x, workspace=ws)
