"""The other forms of attention, the compaction and the fork where memory and order are the point: pages beyond 2^32 bytes, rows with
gaps between them, captured calls whose lists change, two streams at once (marked gpu). Every comparison is exact."""
import numpy as np
import pytest

from oracle import kv_more_oracle as M
from tests.test_gpu_kv import Setup, bf16, lsa, offsets, torch  # noqa: F401  (fixtures)
from tests.test_gpu_kv_forms import geometric, run
from tests.test_gpu_kv_pool import Pool, To, ascending, bits, dev, expected

pytestmark = pytest.mark.gpu


def test_far_pages(torch, lsa):
    """Pages whose bytes lie beyond 2^32 and whose elements lie beyond 2^31: read by attention, copied from and to, forked to."""
    n_pages, pt, d = 140_000, 128, 128
    k, v = (torch.empty((n_pages, 1, pt, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = [139_999, 131_500, 70_000, 139_000]
    g = np.random.default_rng(1)
    table = dev(torch, [pages])
    near = dev(torch, [[2, 0, 3, 1]])
    kn, vn = (torch.empty((4, 1, pt, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, page in enumerate(pages):
        for far, close in ((k, kn), (v, vn)):
            far[page] = bf16(torch, g, (1, pt, d))
            close[int(near[0, i])] = far[page]
    kv_len = dev(torch, [500])
    far, close = lsa.KvCache(k=k, v=v, page_table=table, kv_len=kv_len), lsa.KvCache(k=kn, v=vn, page_table=near, kv_len=kv_len)

    class One:
        totals = [500]

    One.d = d
    for n in (1, 200):
        q = bf16(torch, g, (n, 8, d), 3.0)
        got = []
        for cache in (far, close):
            One.cache = cache
            got.append(run(torch, lsa, One, q, offsets([n]), softcap=20.0, slopes=geometric(8), doc=np.full(n, 3, np.int32)))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])

    # thinned from far pages to far pages
    entries = ascending(g, 500, 140)
    to_table = dev(torch, [[139_998, 139_997]])
    kept = torch.zeros(1, dtype=torch.int32, device="cuda")
    to = lsa.KvCache(k=k, v=v, page_table=to_table, kv_len=kept)
    lists = dict(idx=dev(torch, entries), idx_offsets=dev(torch, [0, 140], np.int64), count=dev(torch, [140]), window=30, sinks=2)
    lsa.kv_kept(far, out=kept, **lists)
    lsa.kv_compact([far], [to], max_kept=256, **lists)
    positions = torch.as_tensor(M.kept_positions(500, entries, 1, 30, 2), device="cuda")
    assert kept.tolist() == [len(positions)]
    for x in (k, v):
        want = x[table[0].long()[positions // pt], 0, positions % pt]
        assert torch.equal(torch.cat([x[139_998, 0], x[139_997, 0]])[:len(positions)], want)

    # the only free page is a far one
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[139_996] = 0
    rows = dev(torch, [pages, [-1] * 4])
    lens = dev(torch, [500, 0])
    pool = lsa.KvPool(refs=refs, page_table=rows, kv_len=lens, page_tokens=pt)
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    lsa.kv_fork(pool, [lsa.KvCache(k=k, v=v, page_table=rows, kv_len=lens)], dev(torch, [0]), dev(torch, [1]), status=status,
                workspace=torch.empty(lsa.kv_fork_workspace_size(1), dtype=torch.uint8, device="cuda"))
    assert status.tolist() == [0] and rows[1].tolist() == pages[:3] + [139_996] and lens.tolist() == [500, 500]
    for x in (k, v):
        assert torch.equal(x[139_996, 0, :500 - 384], x[139_000, 0, :500 - 384])


@pytest.mark.parametrize("news", [[1, 2], [70, 200]])
@pytest.mark.parametrize("G", [3, 8])
def test_rows_with_gaps(torch, lsa, news, G):
    """Rows of q and out that lie apart, and rows that belong to no sequence: the gaps stay as they were."""
    s = Setup(torch, lsa, [300, 260], dtype="fp8", n_kv=2, d=64, pt=32, seed=5)
    n_q, T = 2 * G, sum(news)
    form = dict(softcap=15.0, slopes=torch.from_numpy(geometric(n_q)).cuda())
    wide = bf16(torch, s.g, (T + 5, n_q + 3, 64), 2.0)
    out_wide = torch.full((T + 5, n_q + 1, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 5, n_q), -7.0, device="cuda")
    off = offsets(news, 2)
    doc = dev(torch, np.arange(T + 5) % 40)
    size = lsa.attend_workspace_size(s.cache, n_q=n_q, q_offsets_host=off, max_kv_len=300)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")

    def call(q, off, out, lse, doc):
        lsa.attend(s.cache, q, q_offsets=dev(torch, off, np.int64), q_offsets_host=off, max_kv_len=300, out=out, lse=lse, scale=0.125,
                   workspace=ws, doc_start=doc, **form)

    call(wide[:, :n_q], off, out_wide[:, :n_q], lse, doc)
    q = wide[2:T + 2, :n_q].contiguous()
    out, lse1 = torch.empty_like(q), torch.empty(T, n_q, device="cuda")
    call(q, offsets(news), out, lse1, doc[2:T + 2].contiguous())
    assert torch.equal(out_wide[2:T + 2, :n_q], out) and torch.equal(lse[2:T + 2], lse1)
    out_wide[2:T + 2, :n_q] = -7.0
    lse[2:T + 2] = -7.0
    assert (out_wide == -7.0).all() and (lse == -7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_compact_captured(torch, lsa, dtype):
    """A captured count and copy follow list, lengths and tables of each replay, on a stream of its own."""
    totals, r, window, sinks = [400, 90], 4, 20, 3
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=2, d=64, pt=32, seed=8)
    to = To(torch, lsa, 2, 14, dtype=dtype, n_kv=2, d=64, pt=32, layers=1, seed=2)
    idx = torch.zeros(150, dtype=torch.int32, device="cuda")
    off, count = dev(torch, [0, 110], np.int64), dev(torch, [0, 0])

    def call():
        kw = dict(idx=idx, idx_offsets=off, count=count, entry_tokens=r, window=window, sinks=sinks)
        lsa.kv_kept(s.cache, out=to.kept, **kw)
        lsa.kv_compact([s.cache], to.caches, max_kept=14 * 32, **kw)

    call()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for step in range(3):
        lens = [400 - 90 * step, 90 - 45 * step]
        lists = [ascending(s.g, -(-t // r), -(-t // r) // (2 + step)) for t in lens]
        for i, x in enumerate(lists):
            idx[110 * i:110 * i + len(x)] = dev(torch, x)
        count.copy_(dev(torch, [len(x) for x in lists]))
        s.kv_len.copy_(dev(torch, lens))
        to.table = np.roll(to.table, step, 1)
        to.table_dev.copy_(torch.from_numpy(to.table))
        positions = [M.kept_positions(t, x, r, window, sinks) for t, x in zip(lens, lists)]
        want = expected(torch, s, to, 0, positions, dtype, 32, 14 * 32)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert to.kept.tolist() == [len(p) for p in positions]
        for name in ("k", "v"):
            assert (bits(torch, to.parts[0][name]) == want[name]).all()
            if dtype == "fp8":
                assert (to.parts[0][name + "_scale"].cpu().numpy() == want[name + "_scale"]).all()


def test_two_streams(torch, lsa):
    """Calls on two streams at once, each with its own workspace, give what each gives alone; so does a pool beside them."""
    sides = []
    for i in range(2):
        s = Setup(torch, lsa, [2000, 900], dtype=("bf16", "fp8")[i], n_kv=2, d=128, pt=64, seed=i)
        q = bf16(torch, s.g, (101, 16, 128), 2.0)
        off = offsets([100, 1])
        size = lsa.attend_workspace_size(s.cache, n_q=16, q_offsets_host=off, max_kv_len=2000)
        pool = Pool(torch, lsa, 8, 4, 40, 16)
        sides.append(dict(s=s, q=q, off=off, off_dev=dev(torch, off, np.int64), ws=torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"),
                          out=torch.empty_like(q), lse=torch.empty(101, 16, device="cuda"), stream=torch.cuda.Stream(), pool=pool,
                          slopes=torch.from_numpy(geometric(16)).cuda(), n_new=dev(torch, [20] * 8)))

    def call(x, stream=None):
        lsa.attend(x["s"].cache, x["q"], q_offsets=x["off_dev"], q_offsets_host=x["off"], max_kv_len=2000, out=x["out"], lse=x["lse"],
                   scale=0.088, workspace=x["ws"], softcap=30.0, slopes=x["slopes"], stream=stream)
        lsa.kv_extend(x["pool"].pool, x["n_new"], stream=stream)

    alone = []
    for x in sides:
        call(x)
        torch.cuda.synchronize()
        alone.append((x["out"].clone(), x["lse"].clone()))
        x["pool"].want.extend([20] * 8)
        x["pool"].same()
    for _ in range(3):
        for x in sides:
            x["out"].fill_(-7)
        torch.cuda.synchronize()
        for x in sides:
            call(x, x["stream"].cuda_stream)
        torch.cuda.synchronize()
        for x, (out, lse) in zip(sides, alone):
            assert torch.equal(x["out"], out) and torch.equal(x["lse"], lse)
            x["pool"].want.extend([20] * 8)
            x["pool"].same()
