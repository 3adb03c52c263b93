"""Refusals of lsa_kv_append, lsa_attend and lsa_attend_topk (CPU): every call here is rejected by argument
checks before anything touches the device, and leaves a text that says why."""
import ctypes
import re

import numpy as np
import pytest

FAKE = 1 << 20  # non-null, 16-byte aligned stand-in address (never dereferenced: validation fails first)


@pytest.fixture(scope="module")
def lsa():
    from sparse_kv_retrieval_amd import lsa as mod
    return mod


def off(*n):
    o = np.zeros(len(n) + 1, np.int64)
    o[1:] = np.cumsum(n)
    return o


def cache(lsa, **kw):
    d = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_table=FAKE, kv_len=FAKE, table_stride=8, n_pages=4, n_kv=2,
             page_tokens=16, d_h=64, dtype=lsa.BF16)
    d.update(kw)
    return lsa._KvCache(*[d[f] for f, _ in lsa._KvCache._fields_])


def refused(lsa, status, match, st):
    assert st == status, (st, lsa.last_error())
    assert re.search(match, lsa.last_error()), lsa.last_error()


def append(lsa, c=None, **kw):
    host = kw.pop("host", off(1, 2))
    a = dict(B=2, k=FAKE, ks=128, v=FAKE, vs=128, q=FAKE, qs=256, qo=FAKE + 4096, n_q=4, off=FAKE, host=host.ctypes.data, rope=1,
             inv=FAKE, rot=64, pos=None)
    a.update(kw)
    return lsa._kv_append(ctypes.byref(c or cache(lsa)), *[a[x] for x in ("B", "k", "ks", "v", "vs", "q", "qs", "qo", "n_q",
                                                                        "off", "host", "rope", "inv", "rot", "pos")], 0)


def attend(lsa, c=None, **kw):
    host = kw.pop("host", off(1, 2))
    a = dict(B=2, q=FAKE, qs=256, n_q=4, off=FAKE, host=host.ctypes.data, max_len=100, scale=1.0, window=0, sinks=0,
             out=FAKE + 4096, os=256, lse=None, ws=FAKE, nb=1 << 30)
    a.update(kw)
    return lsa._attend(ctypes.byref(c or cache(lsa)), *[a[x] for x in ("B", "q", "qs", "n_q", "off", "host", "max_len", "scale",
                                                                     "window", "sinks", "out", "os", "lse", "ws", "nb")], 0)


def topk(lsa, c=None, **kw):
    a = dict(B=2, q=FAKE, qs=256, n_q=4, idx=FAKE, count=FAKE, k=64, r=1, scale=1.0, window=0, sinks=0, out=FAKE + 4096,
             os=256, lse=None, ws=FAKE, nb=1 << 30)
    a.update(kw)
    return lsa._attend_topk(ctypes.byref(c or cache(lsa)), *[a[x] for x in ("B", "q", "qs", "n_q", "idx", "count", "k", "r",
                                                                          "scale", "window", "sinks", "out", "os", "lse", "ws",
                                                                          "nb")], 0)


BAD_CACHES = [
    ("INVALID_ARG", "must be set", dict(k=None)), ("INVALID_ARG", "must be set", dict(v=None)),
    ("INVALID_ARG", "must be set", dict(page_table=None)), ("INVALID_ARG", "must be set", dict(kv_len=None)),
    ("UNSUPPORTED", "bf16 or fp8", dict(dtype=0)), ("UNSUPPORTED", "bf16 or fp8", dict(dtype=7)),
    ("UNSUPPORTED", "bf16 or fp8", dict(dtype=-1)),
    ("INVALID_ARG", "needs k_scale", dict(dtype=2)), ("INVALID_ARG", "needs k_scale", dict(dtype=2, k_scale=FAKE)),
    ("INVALID_ARG", "only for an fp8", dict(v_scale=FAKE)),
    ("UNSUPPORTED", "page_tokens", dict(page_tokens=8)), ("UNSUPPORTED", "page_tokens", dict(page_tokens=48)),
    ("UNSUPPORTED", "page_tokens", dict(page_tokens=256)), ("UNSUPPORTED", "d_h", dict(d_h=96)),
    ("UNSUPPORTED", "n_kv", dict(n_kv=0)), ("UNSUPPORTED", "n_kv", dict(n_kv=1025)),
    ("INVALID_ARG", "n_pages", dict(n_pages=0)), ("INVALID_ARG", "table_stride", dict(table_stride=0)),
    ("INVALID_ARG", "table_stride", dict(table_stride=1 << 40)), ("INVALID_ARG", "aligned", dict(k=FAKE + 8)),
    ("INVALID_ARG", "aligned", dict(v=FAKE + 4)),
]


@pytest.mark.parametrize("call", [append, attend, topk], ids=["append", "attend", "topk"])
@pytest.mark.parametrize("bad", BAD_CACHES, ids=[f"{list(b[2].items())[-1]}" for b in BAD_CACHES])
def test_cache(lsa, call, bad):
    refused(lsa, getattr(lsa, "ERR_" + bad[0]), bad[1], call(lsa, cache(lsa, **bad[2])))


@pytest.mark.parametrize("status,match,kw", [
    ("UNSUPPORTED", "B must", dict(B=0)), ("UNSUPPORTED", "B must", dict(B=4097)), ("INVALID_ARG", "new_offsets", dict(off=None)),
    ("INVALID_ARG", "new_offsets_host", dict(host=np.array([-1, 2, 3], np.int64))),
    ("INVALID_ARG", "decreasing", dict(host=np.array([0, 2, 1], np.int64))),
    ("INVALID_ARG", "k_new", dict(k=None)), ("INVALID_ARG", "k_new", dict(v=None)), ("INVALID_ARG", "together", dict(q=None)),
    ("INVALID_ARG", "together", dict(qo=None)), ("INVALID_ARG", "aligned", dict(k=FAKE + 2)), ("INVALID_ARG", "aligned", dict(qo=FAKE + 8)),
    ("INVALID_ARG", "k_stride", dict(ks=120)), ("INVALID_ARG", "k_stride", dict(vs=132)), ("INVALID_ARG", "q_stride", dict(qs=248)),
    ("INVALID_ARG", "contiguous", dict(qo=FAKE, qs=264)), ("UNSUPPORTED", "n_q", dict(n_q=3)), ("UNSUPPORTED", "n_q", dict(n_q=0)),
    ("INVALID_ARG", "rope", dict(rope=3)), ("INVALID_ARG", "rope", dict(rope=-1)), ("INVALID_ARG", "inv_freq", dict(inv=None)),
    ("UNSUPPORTED", "rot_dim", dict(rot=0)), ("UNSUPPORTED", "rot_dim", dict(rot=24)), ("UNSUPPORTED", "rot_dim", dict(rot=80)),
    ("UNSUPPORTED", "2\\^31", dict(host=off(1, 1 << 30))), ("UNSUPPORTED", "too many", dict(host=off(1, 1 << 28))),
])
def test_append(lsa, status, match, kw):
    refused(lsa, getattr(lsa, "ERR_" + status), match, append(lsa, **kw))


SHARED = [
    ("INVALID_ARG", "must be set", dict(q=None)), ("INVALID_ARG", "must be set", dict(out=None)),
    ("INVALID_ARG", "aligned", dict(q=FAKE + 8)), ("INVALID_ARG", "aligned", dict(out=FAKE + 8)),
    ("INVALID_ARG", "overlap", dict(out=FAKE)), ("INVALID_ARG", "q_stride", dict(qs=255)), ("INVALID_ARG", "q_stride", dict(os=248)),
    ("INVALID_ARG", "softmax_scale", dict(scale=float("nan"))), ("INVALID_ARG", "softmax_scale", dict(scale=float("inf"))),
    ("INVALID_ARG", "softmax_scale", dict(scale=3e38)),
    ("INVALID_ARG", "lse", dict(lse=FAKE + 2)), ("UNSUPPORTED", "n_q", dict(n_q=5)), ("UNSUPPORTED", "n_q", dict(n_q=4098)),
    ("INVALID_ARG", "negative", dict(window=-1)), ("INVALID_ARG", "negative", dict(sinks=-1)), ("UNSUPPORTED", "B must", dict(B=0)),
    ("WORKSPACE", "workspace needs", dict(ws=None)), ("WORKSPACE", "workspace needs", dict(nb=100)),
    ("INVALID_ARG", "16-byte", dict(ws=FAKE + 8)),
]


@pytest.mark.parametrize("status,match,kw", SHARED + [
    ("INVALID_ARG", "max_kv_len", dict(max_len=-1)), ("INVALID_ARG", "max_kv_len", dict(max_len=1025)),
    ("INVALID_ARG", "q_offsets", dict(off=None)), ("INVALID_ARG", "decreasing", dict(host=np.array([0, 2, 1], np.int64))),
])
def test_attend(lsa, status, match, kw):
    kw = {"max_len": 1000, **kw}
    c = cache(lsa, table_stride=64)
    refused(lsa, getattr(lsa, "ERR_" + status), match, attend(lsa, c, **kw))


@pytest.mark.parametrize("status,match,kw", SHARED + [
    ("INVALID_ARG", "idx", dict(idx=None)), ("INVALID_ARG", "idx", dict(count=None)), ("UNSUPPORTED", "k must", dict(k=0)),
    ("UNSUPPORTED", "k must", dict(k=65537)), ("UNSUPPORTED", "entry_tokens", dict(r=0)), ("UNSUPPORTED", "entry_tokens", dict(r=129)),
])
def test_topk(lsa, status, match, kw):
    refused(lsa, getattr(lsa, "ERR_" + status), match, topk(lsa, **{"k": 2048, **kw}))


def test_max_kv_len_beyond_the_table(lsa):
    refused(lsa, lsa.ERR_INVALID_ARG, "max_kv_len", attend(lsa, max_len=8 * 16 + 1))


def test_no_rows_is_fine(lsa):
    empty = np.zeros(3, np.int64)
    assert append(lsa, host=empty, k=None, v=None, q=None, qo=None) == lsa.OK
    assert attend(lsa, host=empty, q=None, out=None) == lsa.OK


def test_workspace_sizes(lsa):
    # decode: one fp32 row block, its maxima and sums per worker and sequence (2 * 32 tiles of 32 keys make 16
    # workers of four), and a pair of integers per sequence and key head; none where the rows of a prompt fill the device
    size = lsa._attend_ws(2, 8, 2, 64, off(1, 1).ctypes.data, 1000, 0, 0)
    assert size == (16 + 2) * 2 * 16 * 66 * 4 + 2 * 2 * 8
    assert lsa._attend_ws(2, 8, 2, 64, off(1, 1).ctypes.data, 128, 0, 0) == 0  # four tiles: nothing to share
    assert lsa._attend_ws(1, 64, 8, 128, off(20000).ctypes.data, 20000, 0, 0) == 0
    assert lsa._attend_ws(2, 8, 2, 64, off(1, 1).ctypes.data, 1000, 16, 4) <= size
    assert lsa._attend_ws(2, 7, 2, 64, off(1, 1).ctypes.data, 1000, 0, 0) == 0
    assert lsa._attend_topk_ws(2, 8, 2, 64, 2048, 1, 0, 0) > 0
    # never beyond about 256 MiB, but for two splits
    for n in (1, 60, 500):
        assert lsa._attend_ws(4, 64, 8, 128, off(n, n, n, n).ctypes.data, 1 << 20, 0, 0) <= max(1 << 28, 2 * 4 * n * 64 * 130 * 4)


def test_binding_checks_tensors(lsa):
    import torch
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    table, length = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    good = dict(k=k, v=k.clone(), page_table=table, kv_len=length)
    c = lsa.KvCache(**good)
    for bad in (dict(k=k.half()), dict(v=k[:3]), dict(v=k.transpose(0, 1)), dict(k=k[0]), dict(page_table=table.long()),
                dict(page_table=table[:1]), dict(kv_len=length.long()), dict(k_scale=torch.zeros(4, 2)),
                dict(k=k.to(torch.float8_e4m3fn), v=k.to(torch.float8_e4m3fn)),
                dict(k=k.to(torch.float8_e4m3fn), v=k.to(torch.float8_e4m3fn), k_scale=torch.zeros(4, 2), v_scale=torch.zeros(4, 3))):
        with pytest.raises(lsa.LsaError):
            lsa.KvCache(**{**good, **bad})
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    o, oh = torch.tensor([0, 1, 2]), off(1, 1)  # on the host: the last check refuses it
    base = dict(q_offsets=o, q_offsets_host=oh, max_kv_len=40, out=q.clone(), scale=1.0)
    for bad in (dict(out=q[:1]), dict(out=q.float()), dict(lse=torch.zeros(2, 3)), dict(q_offsets=o[:2]), dict(q_offsets=o.int()),
                dict(q_offsets_host=off(1, 2)), dict(q_offsets_host=off(1)), dict(lse=torch.zeros(2, 4).t().contiguous().t())):
        with pytest.raises(lsa.LsaError):
            lsa.attend(c, q, **{**base, **bad})
    fixed = oh.copy()
    fixed.setflags(write=False)  # read-only offsets and plain lists serve as well
    for host in (fixed, oh.tolist(), torch.from_numpy(oh)):
        with pytest.raises(lsa.LsaError, match="on a GPU"):
            lsa.attend(c, q, **{**base, "q_offsets_host": host})
    for bad_q in (q.float(), q[..., ::2], q.transpose(1, 2), q[:, :, :32]):
        with pytest.raises((lsa.LsaError)):
            lsa.attend(c, bad_q, **base)
    with pytest.raises(lsa.LsaError):
        lsa.attend_topk(c, q[:1], idx=torch.zeros((2, 5), dtype=torch.int32), count=length, out=q[:1].clone(), scale=1.0)
    with pytest.raises(lsa.LsaError):
        lsa.attend_topk(c, q, idx=torch.zeros((2, 5), dtype=torch.int64), count=length, out=q.clone(), scale=1.0)
    kn = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    base = dict(new_offsets=o, new_offsets_host=oh)
    for bad in (dict(q=q), dict(q=q, q_out=q.float()), dict(rope="other"), dict(inv_freq=torch.zeros(32, dtype=torch.float64)),
                dict(positions=torch.zeros(2)), dict(new_offsets_host=off(2, 1))):
        with pytest.raises(lsa.LsaError):
            lsa.kv_append(c, kn, kn, **{**base, **bad})
    with pytest.raises(lsa.LsaError):
        lsa.kv_append(c, kn, kn[:1], **base)
