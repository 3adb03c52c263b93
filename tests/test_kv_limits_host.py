"""The largest calls of lsa_attend, lsa_attend_topk and lsa_kv_append that the header promises (CPU): the host layer takes them,
and refuses what is one step larger. Nothing runs: without a device an accepted call ends in the launch's own error."""
import os

import numpy as np
import pytest

from tests.test_kv_host import FAKE, append, attend, cache, off, refused, topk

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="an accepted call would run on the device, on addresses that are none")


@pytest.fixture(scope="module")
def lsa():
    from sparse_kv_retrieval_amd import lsa as mod
    return mod


def taken(lsa, st):
    assert st == lsa.ERR_HIP, (st, lsa.last_error())


def rows_call(lsa, n_q, n_kv, d, news, *, max_len=None, **kw):
    host = off(*news)
    c = cache(lsa, n_kv=n_kv, d_h=d, page_tokens=128, table_stride=1 << 16)
    return attend(lsa, c, B=len(news), host=host, n_q=n_q, qs=n_q * d, os=n_q * d, out=FAKE + 4096, nb=1 << 40,
                  max_len=max(news) if max_len is None else max_len, **kw)


@pytest.mark.parametrize("n_q,n_kv,d,news,max_len", [
    (128, 8, 128, [1 << 19], None), (64, 8, 128, [1 << 20], None),  # prompts whose rows fill the device: nothing is joined
    (1024, 1024, 64, [17] * 4096, 4096),                            # 17 rows each, and their parts are joined
    (1024, 1024, 64, [17] * 4096, 100),                             # too short to share
    (8, 8, 64, [(1 << 23) + 600] + [1] * 40, 1 << 20),              # prompt and decode rows
    (2, 1, 64, [(1 << 30) - 200], 1 << 20),                         # 2^31 - 400 rows times heads
])
def test_attend_takes_what_it_promises(lsa, n_q, n_kv, d, news, max_len):
    taken(lsa, rows_call(lsa, n_q, n_kv, d, news, max_len=max_len))


def test_attend_refuses_the_rest(lsa):
    refused(lsa, lsa.ERR_UNSUPPORTED, "2\\^31", rows_call(lsa, 2, 1, 64, [1 << 30], max_len=1 << 20))
    # row blocks of a long prompt: (rows / 256 + B) n_kv below 2^23
    taken(lsa, rows_call(lsa, 1024, 1024, 64, [8190 * 256], max_len=1 << 20))
    refused(lsa, lsa.ERR_UNSUPPORTED, "too many", rows_call(lsa, 1024, 1024, 64, [8191 * 256], max_len=1 << 20))
    # 2^11 sequences of 2^20 tiles
    def long(B):
        c = cache(lsa, n_kv=1, page_tokens=128, table_stride=1 << 18)
        return attend(lsa, c, B=B, host=off(*[1] * B), n_q=2, qs=128, os=128, nb=1 << 40, max_len=1 << 25)

    refused(lsa, lsa.ERR_UNSUPPORTED, "too many", long(2048))
    taken(lsa, long(2047))


def test_topk_takes_what_it_promises(lsa):
    def call(B, n_q, n_kv, **kw):
        return topk(lsa, cache(lsa, n_kv=n_kv), B=B, n_q=n_q, qs=n_q * 64, os=n_q * 64, nb=1 << 40, **kw)

    taken(lsa, call(4096, 32768, 512, k=2048))  # 2^27 rows times heads
    taken(lsa, call(4096, 16384, 1024, k=64))
    taken(lsa, call(4095, 128 * 1024, 1024, k=64))  # two row blocks of 64 heads each: 2^23 - 2048 of them
    refused(lsa, lsa.ERR_UNSUPPORTED, "too many", call(4096, 256 * 1024, 1024, k=64))  # 2^24
    refused(lsa, lsa.ERR_UNSUPPORTED, "2\\^31", call(4096, 1 << 19, 1024, k=64))


def test_append_limit(lsa):
    # (T / page_tokens + 2 B) 2 n_kv + T n_q / 32 + 1 blocks, below 2^24
    c = cache(lsa, n_kv=4)
    T = 22369552  # (T / 16 + 4) 8 + T 8 / 32 + 1 = 16777197; 64 tokens more are 48 blocks more
    for n, ok in ((T, True), (T + 64, False)):
        args = dict(B=2, host=np.array([0, 1, n], np.int64), ks=256, vs=256, qs=512, n_q=8)
        st = append(lsa, c, **args)
        if ok:
            taken(lsa, st)
        else:
            refused(lsa, lsa.ERR_UNSUPPORTED, "too many", st)


@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), ((1 << 31) - 1, 0), (5, (1 << 31) - 1), ((1 << 31) - 1, (1 << 31) - 1)])
@pytest.mark.parametrize("B", [32, 128, 4096])
def test_topk_takes_any_window(lsa, B, window, sinks):
    # 8 pages of 16 tokens: four tiles by position at most, whatever the window
    taken(lsa, topk(lsa, cache(lsa), B=B, window=window, sinks=sinks, nb=1 << 40))


def test_topk_counts_the_tiles_of_the_table(lsa):
    # 2^19 tiles by position and 2 of the list: 4095 sequences of them pass, 4096 do not
    c = cache(lsa, page_tokens=128, table_stride=1 << 17)
    for B, ok in ((4095, True), (4096, False)):
        st = topk(lsa, c, B=B, window=(1 << 31) - 1, nb=1 << 40)
        if ok:
            taken(lsa, st)
        else:
            refused(lsa, lsa.ERR_UNSUPPORTED, "too many", st)


@pytest.mark.parametrize("n_q,n_kv", [(128, 128), (64, 8), (64, 1), (1024, 1024), (256, 2), (8, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_workspaces_do_not_grow_with_the_batch(lsa, n_q, n_kv, d):
    # parts are as many as two per block that shares the keys, and a pair of integers per row block says where they are
    for news in ([1], [2], [8] + [1]):
        def size(B):
            host = off(*((news + [1] * B)[:B]))
            return lsa._attend_ws(B, n_q, n_kv, d, host.ctypes.data, 1 << 17, 0, 0)

        most = news[0] * (n_q // n_kv)
        rows = 16 if most <= 16 else 32 if most <= 32 else 64
        if most > 64:
            continue
        for B in (64, 256, 4096):
            assert 0 < size(B) <= 2 * max(512, n_kv) * rows * (d + 2) * 4 + B * n_kv * 8 <= 1 << 28, (B, news)
    per = -(-(n_q // n_kv) // 64)
    for B in (64, 256, 4096):
        assert 0 < lsa._attend_topk_ws(B, n_q, n_kv, d, 2048, 4, 128, 4) <= 2 * max(512, n_kv) * 64 * (d + 2) * 4 + B * per * n_kv * 8
