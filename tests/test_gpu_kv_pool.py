"""lsa_kv_kept, lsa_kv_compact, lsa_kv_extend, lsa_kv_fork and lsa_kv_free against the oracle (marked gpu). Everything here is
copied, counted or rounded once, so every comparison is exact."""
import numpy as np
import pytest

from oracle import kv_more_oracle as M
from oracle import kv_oracle as K
from tests.test_gpu_kv import Setup, bf16, lsa, offsets, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def dev(torch, x, t=np.int32):
    return torch.from_numpy(np.asarray(x, t)).cuda()


class To:
    """Destination caches of some layers, the same value in every slot."""

    def __init__(self, torch, lsa, B, width, *, dtype, n_kv, d, pt, layers, seed=0):
        g = np.random.default_rng(seed)
        n_pages = B * width + 1
        self.table = g.permutation(n_pages)[:B * width].reshape(B, width).astype(np.int32)
        self.table_dev, self.kept = dev(torch, self.table), torch.full((B,), -5, dtype=torch.int32, device="cuda")
        self.parts, self.caches = [], []
        for _ in range(layers):
            x = {}
            for name in ("k", "v"):
                if dtype == "fp8":
                    x[name] = torch.full((n_pages, n_kv, pt, d), 0x31, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                    x[name + "_scale"] = torch.full((n_pages, n_kv), 3.0, device="cuda")
                else:
                    x[name] = torch.full((n_pages, n_kv, pt, d), 9.0, dtype=torch.bfloat16, device="cuda")
            self.parts.append(x)
            self.caches.append(lsa.KvCache(page_table=self.table_dev, kv_len=self.kept, **x))


def bits(torch, t):
    return t.view(torch.uint8 if t.dtype == torch.float8_e4m3fn else torch.int16).cpu().numpy()


def expected(torch, src, to, layer, positions, dtype, pt, max_kept):
    """What `to` should hold after the call, from what it holds now: (k, k_scale, v, v_scale) as bits and scales."""
    want = {}
    for name in ("k", "v"):
        y, x = bits(torch, to.parts[layer][name]), bits(torch, src.parts[name])
        ys = to.parts[layer][name + "_scale"].cpu().numpy().copy() if dtype == "fp8" else None
        xs = src.parts[name + "_scale"].cpu().numpy() if dtype == "fp8" else None
        y = y.copy()
        for b, kept in enumerate(positions):
            kept = kept[:max_kept]
            for p0 in range(0, len(kept), pt):
                page = int(to.table[b, p0 // pt])
                if not 0 <= page < len(y):
                    continue
                rows = [(i, int(src.table[b, s // src.pt]), s % src.pt) for i, s in enumerate(kept[p0:p0 + pt])]
                rows = [r for r in rows if 0 <= r[1] < len(x)]
                if not rows:
                    continue
                for h in range(x.shape[1]):
                    if dtype != "fp8":
                        for i, pg, slot in rows:
                            y[page, h, i] = x[pg, h, slot]
                        continue
                    vals = np.stack([K.e4m3_values()[x[pg, h, slot]].astype(np.float32) * xs[pg, h] for _, pg, slot in rows])
                    codes, ys[page, h] = M.compact_page(vals.astype(np.float64))
                    for (i, _, _), c in zip(rows, codes):
                        y[page, h, i] = c
        want[name], want[name + "_scale"] = y, ys
    return want


def same_codes(a, b):
    return ((a == b) | (((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F))).all()


def run_compact(torch, lsa, srcs, to, lists, r, window, sinks, max_kept, *, base=3, stream=None):
    idx = np.concatenate([np.full(base, -9)] + [np.asarray(x, np.int64) for x in lists] + [[7]]).astype(np.int32)
    off = offsets([len(x) for x in lists], base)
    kw = dict(idx=dev(torch, idx), idx_offsets=dev(torch, off, np.int64), count=dev(torch, [len(x) for x in lists]), entry_tokens=r,
              window=window, sinks=sinks)
    lsa.kv_kept(srcs[0].cache, out=to.kept, **kw)
    lsa.kv_compact([s.cache for s in srcs], to.caches, max_kept=max_kept, **kw)
    torch.cuda.synchronize()


def ascending(g, entries, n):
    return np.sort(g.permutation(entries)[:n])


@pytest.mark.parametrize("dtype,d,n_kv,pt,pt_to", [("bf16", 128, 2, 64, 64), ("bf16", 64, 1, 16, 128), ("bf16", 128, 3, 128, 128),
                                                   ("fp8", 128, 2, 64, 64), ("fp8", 64, 3, 32, 16), ("fp8", 128, 1, 16, 128),
                                                   ("fp8", 64, 2, 128, 32), ("bf16", 64, 2, 32, 32), ("fp8", 64, 1, 16, 64),
                                                   ("fp8", 128, 2, 32, 16), ("fp8", 128, 2, 64, 32), ("fp8", 64, 2, 64, 128),
                                                   ("bf16", 128, 1, 32, 16), ("bf16", 64, 1, 64, 16)])
@pytest.mark.parametrize("r,window,sinks", [(1, 0, 0), (4, 40, 3), (7, 1, 10), (128, 300, 130)])
def test_compact(torch, lsa, dtype, d, n_kv, pt, pt_to, r, window, sinks):
    totals = [0, 1, 63, 500, 700, 129]
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=r)
    lists = [ascending(s.g, -(-t // r), int(s.g.integers(0, -(-t // r) + 1))) for t in totals]
    positions = [M.kept_positions(t, x, r, window, sinks) for t, x in zip(totals, lists)]
    most = max(len(p) for p in positions)
    to = To(torch, lsa, len(totals), -(-most // pt_to) + 1, dtype=dtype, n_kv=n_kv, d=d, pt=pt_to, layers=1, seed=r)
    want = expected(torch, s, to, 0, positions, dtype, pt_to, most)
    run_compact(torch, lsa, [s], to, lists, r, window, sinks, most)
    assert to.kept.tolist() == [len(p) for p in positions]
    for name in ("k", "v"):
        got = bits(torch, to.parts[0][name])
        assert same_codes(got, want[name]) if dtype == "fp8" else (got == want[name]).all()
        if dtype == "fp8":
            assert (to.parts[0][name + "_scale"].cpu().numpy() == want[name + "_scale"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_compact_odd(torch, lsa, dtype):
    """Scales that are no powers of two, NaN codes, pages that are not there on either side, a bound below what is kept, lists whose
    last entries lie beyond the sequence, and more layers than one launch takes."""
    totals, layers = [400, 90, 333], 18
    srcs = []
    for l in range(layers):
        s = Setup(torch, lsa, totals, dtype=dtype, n_kv=2, d=64, pt=16, seed=3)  # one table for all
        for name in ("k", "v"):
            x = s.parts[name]
            if dtype == "fp8":
                s.parts[name + "_scale"].mul_(1.0 + 0.01 * l)
                x.view(torch.uint8)[s.table[0, 2], :, 3, l] = 0xFF
            else:
                x.mul_(1.0 + l)
        if srcs:
            s.cache = lsa.KvCache(page_table=srcs[0].table_dev, kv_len=srcs[0].kv_len, **s.parts)
        srcs.append(s)
    table = srcs[0].table
    table[0, 5], table[2, 0], table[2, 1] = -1, 10 ** 8, -(2 ** 31)
    srcs[0].table_dev.copy_(torch.from_numpy(table))
    lists = [ascending(srcs[0].g, 100, 60), [0, 5, 22, 23, 40], [0, 1, 2, 3, 4, 5, 6, 7, 80, 83, 84, 2 ** 31 - 1]]
    positions = [M.kept_positions(t, x, 4, 5, 2) for t, x in zip(totals, lists)]
    to = To(torch, lsa, 3, 20, dtype=dtype, n_kv=2, d=64, pt=16, layers=layers)
    to.table[0, 1], to.table[1, 0] = -1, 10 ** 6
    to.table_dev.copy_(torch.from_numpy(to.table))
    most = 200
    want = []
    for l in range(layers):
        srcs[l].table = table
        want.append(expected(torch, srcs[l], to, l, positions, dtype, 16, most))
    run_compact(torch, lsa, srcs, to, lists, 4, 5, 2, most)
    assert to.kept.tolist() == [len(p) for p in positions] and max(to.kept.tolist()) > most
    for l in range(layers):
        for name in ("k", "v"):
            got = bits(torch, to.parts[l][name])
            assert same_codes(got, want[l][name]) if dtype == "fp8" else (got == want[l][name]).all(), (l, name)
            if dtype == "fp8":
                assert (to.parts[l][name + "_scale"].cpu().numpy() == want[l][name + "_scale"]).all(), (l, name)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_compacted_is_what_topk_sees(torch, lsa, dtype):
    """Attention over the compacted cache against attention over the listed entries of the whole one: the same keys."""
    totals, r = [900, 350], 4
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=2, d=128, pt=64, seed=4)
    lists = [ascending(s.g, -(-t // r), 40) for t in totals]
    to = To(torch, lsa, 2, 6, dtype=dtype, n_kv=2, d=128, pt=64, layers=1)
    run_compact(torch, lsa, [s], to, lists, r, 50, 3, 384)
    q = bf16(torch, s.g, (2, 16, 128))
    a, b = torch.empty_like(q), torch.empty_like(q)
    la, lb = torch.empty(2, 16, device="cuda"), torch.empty(2, 16, device="cuda")
    idx = dev(torch, np.stack(lists))
    size = lsa.attend_topk_workspace_size(s.cache, n_q=16, k=40, entry_tokens=r, window=50, sinks=3)
    lsa.attend_topk(s.cache, q, idx=idx, count=dev(torch, [40, 40]), entry_tokens=r, scale=0.1, window=50, sinks=3, out=a, lse=la,
                    workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    off = offsets([1, 1])
    size = lsa.attend_workspace_size(to.caches[0], n_q=16, q_offsets_host=off, max_kv_len=384)
    lsa.attend(to.caches[0], q, q_offsets=dev(torch, off, np.int64), q_offsets_host=off, max_kv_len=384, scale=0.1, out=b, lse=lb,
               workspace=torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"))
    # Values are N(0, 1) in bf16 and of size 1 in e4m3: at most some 5. Each side rounds probabilities and output once (2^-8);
    # new e4m3 scales change no value but subnormal ones, by half of the smallest step (2^-10) of a scale below 2^-5.
    assert (a.float() - b.float()).abs().max() <= 4 * 2.0 ** -8 * 5 + 2.0 ** -15
    assert (la - lb).abs().max() <= 2.0 ** -11


# ------------------------------------------------------------------ the pool
class Pool:
    def __init__(self, torch, lsa, B, width, n_pages, pt):
        self.torch, self.lsa = torch, lsa
        z = dict(dtype=torch.int32, device="cuda")
        self.refs, self.table, self.kv_len = torch.zeros(n_pages, **z), torch.full((B, width), -1, **z), torch.zeros(B, **z)
        self.pool = lsa.KvPool(refs=self.refs, page_table=self.table, kv_len=self.kv_len, page_tokens=pt)
        self.want = M.Pool([0] * n_pages, [[-1] * width for _ in range(B)], [0] * B, pt)

    def same(self):
        assert self.refs.tolist() == self.want.refs
        assert self.kv_len.tolist() == self.want.kv_len
        assert self.table.tolist() == self.want.table

    def extend(self, n_new):
        missing = self.torch.full((len(n_new),), 77, dtype=self.torch.int32, device="cuda")
        self.lsa.kv_extend(self.pool, dev(self.torch, n_new), missing=missing)
        assert missing.tolist() == self.want.extend(n_new)
        self.same()

    def free(self, seqs):
        self.lsa.kv_free(self.pool, dev(self.torch, seqs))
        self.want.free(seqs)
        self.same()

    def fork(self, caches, src, dst):
        status = self.torch.full((len(src),), 77, dtype=self.torch.int32, device="cuda")
        ws = self.torch.full((max(self.lsa.kv_fork_workspace_size(len(src)), 16),), 0xFF, dtype=self.torch.uint8, device="cuda")
        self.lsa.kv_fork(self.pool, caches, dev(self.torch, src), dev(self.torch, dst), status=status, workspace=ws)
        want, copies = self.want.fork(src, dst)
        assert status.tolist() == want
        self.same()
        return copies


def layers_of(torch, lsa, pool, layers, dtype, n_kv, d, pt, seed=0):
    g = np.random.default_rng(seed)
    out = []
    for _ in range(layers):
        x = {}
        for name in ("k", "v"):
            shape = (pool.refs.numel(), n_kv, pt, d)
            if dtype == "fp8":
                x[name] = torch.from_numpy(g.integers(0, 256, shape).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
                x[name + "_scale"] = torch.from_numpy(g.random(shape[:2]).astype(np.float32)).cuda()
            else:
                x[name] = torch.from_numpy(g.integers(-2 ** 15, 2 ** 15, shape).astype(np.int16)).cuda().view(torch.bfloat16)
        out.append((x, lsa.KvCache(page_table=pool.table, kv_len=pool.kv_len, **x)))
    return out


@pytest.mark.parametrize("dtype,d,n_kv,pt,layers", [("bf16", 64, 1, 16, 1), ("fp8", 128, 3, 64, 2), ("bf16", 128, 2, 128, 3), ("fp8", 64, 1, 32, 18)])
def test_pool_steps(torch, lsa, dtype, d, n_kv, pt, layers):
    """Admissions, growth by a token, forks of forks and retirements."""
    g = np.random.default_rng(pt)
    B, width, n_pages = 12, 6, 40
    p = Pool(torch, lsa, B, width, n_pages, pt)
    caches = layers_of(torch, lsa, p, layers, dtype, n_kv, d, pt)
    for step in range(12):
        p.extend([int(x) for x in g.choice([0, 0, 1, pt, 3 * pt + 5, -4, 7 * pt], B)])
        n = int(g.integers(1, 7))
        src, dst = g.integers(-1, B + 1, n).tolist(), g.integers(-1, B + 1, n).tolist()
        if step % 3 == 0:  # pairs that are all in order
            perm = g.permutation(B).tolist()
            src, dst = [perm[0]] * 3 + [perm[1]] * 3, perm[2:8]
        before = [{k: (bits(torch, v) if "scale" not in k else v.cpu().numpy()).copy() for k, v in x.items()} for x, _ in caches]
        copies = p.fork([c for _, c in caches], src, dst)
        for want, (x, _) in zip(before, caches):
            for a, b, m in copies:
                for name in ("k", "v"):
                    want[name][b, :, :m] = want[name][a, :, :m]
                    if dtype == "fp8":
                        want[name + "_scale"][b] = want[name + "_scale"][a]
            for k, v in x.items():
                assert ((bits(torch, v) if "scale" not in k else v.cpu().numpy()) == want[k]).all(), (step, k)
        p.free(g.integers(-2, B + 2, int(g.integers(1, 5))).tolist())
    p.free(list(range(B)))
    assert p.want.refs == [0] * n_pages


def test_pool_runs_out(torch, lsa):
    """Seven pages: growth and forks that get none, in their order, and what they leave as it was."""
    p = Pool(torch, lsa, 6, 6, 7, 16)
    caches = [c for _, c in layers_of(torch, lsa, p, 1, "fp8", 1, 64, 16)]
    p.extend([40, 20, 0, 0, 0, 0])                               # five pages
    assert len(p.fork(caches, [0, 0, 1], [2, 3, 4])) == 2        # two tails: the third pair keeps its full page only
    assert p.want.kv_len == [40, 20, 40, 40, 16, 0]
    p.extend([1, 12, 8, 9, 0, 1])                                # nobody who needs a page gets one
    assert p.want.kv_len == [41, 32, 48, 40, 16, 0]
    assert p.fork(caches, [0], [1]) and p.want.refs[3] == 1      # dst's own pages come back first
    p.free([4, 3])
    p.extend([0, 0, 0, 0, 33, 16])                               # three for the first: none is left for the second
    p.extend([0, 0, 0, 0, 0, 16])


def test_pool_sizes(torch, lsa):
    """Many sequences and pages: the search goes over several chunks, and over more pages than are held at once."""
    B, pt, n_pages = 4096, 16, 40_003
    p = Pool(torch, lsa, B, 40, n_pages, pt)
    taken = np.random.default_rng(1).random(n_pages) < 0.4  # pages that others hold
    p.refs.copy_(dev(torch, taken))
    p.want.refs = [int(x) for x in taken]
    free = int((~taken).sum())

    def extend(n_new):
        """As Pool.extend; the oracle's search is too slow here, and its rule is short for an empty pool."""
        missing = torch.full((B,), 77, dtype=torch.int32, device="cuda")
        lsa.kv_extend(p.pool, dev(torch, n_new), missing=missing)
        need = -(-np.asarray(n_new) // pt)
        ok = (np.cumsum(need) <= free) | (need == 0)
        pages = np.flatnonzero(~taken)[: need[ok].sum()]
        want, refs = np.full((B, 40), -1), taken.astype(int)
        want[np.arange(40) < np.where(ok, need, 0)[:, None]] = pages
        refs[pages] = 1
        assert (missing.cpu().numpy() == np.where(ok, 0, need)).all()
        assert (p.refs.cpu().numpy() == refs).all() and (p.table.cpu().numpy() == want).all()
        assert (p.kv_len.cpu().numpy() == np.where(ok, n_new, 0)).all()
        lsa.kv_free(p.pool, torch.arange(B, dtype=torch.int32, device="cuda"))
        assert (p.refs.cpu().numpy() == taken).all() and (p.table == -1).all() and (p.kv_len == 0).all()

    g = np.random.default_rng(2)
    extend(g.integers(0, 3 * pt, B))          # some 8000 pages
    extend(g.integers(0, 10 * pt, B))         # some 20,000: nearly all
    extend(g.integers(0, 16 * pt, B))         # more than there are
    extend(np.where(np.arange(B) == 4095, 640, 0))
    extend(np.full(B, 1))
    extend(np.zeros(B, int))


def test_pool_odd(torch, lsa):
    """Lengths out of range, refs below zero, entries that hold no page."""
    p = Pool(torch, lsa, 5, 4, 20, 16)
    p.kv_len.copy_(dev(torch, [-7, 1000, 2 ** 31 - 1, 30, 0]))
    p.want.kv_len = [-7, 1000, 2 ** 31 - 1, 30, 0]
    p.refs[3] = -5
    p.want.refs[3] = -5
    p.table[3, :2] = dev(torch, [99, 7])
    p.want.table[3][:2] = [99, 7]
    p.refs[7] = p.want.refs[7] = 1
    p.extend([5, 1, 1, 40, 0])
    caches = [c for _, c in layers_of(torch, lsa, p, 1, "bf16", 1, 64, 16)]
    # sequence 3 has no page for more than 64 tokens; its first entry is no page and stays none; sequence 1 fills its row
    assert p.fork(caches, [3, 1], [4, 0]) == [(7, p.want.table[4][1], 14)]
    p.free([2, 1, 0, 3, 4])


def test_steps_in_one(torch, lsa):
    """A prompt is admitted, stored, sampled three ways, and every sample goes its own way for some steps; each sample's attention is
    that of its own tokens."""
    from tests.test_gpu_kv_forms import check, geometric
    n_kv, n_q, d, pt, B = 1, 8, 64, 16, 4
    p = Pool(torch, lsa, B, 8, 40, pt)
    (parts, cache), = layers_of(torch, lsa, p, 1, "bf16", n_kv, d, pt)
    for x in parts.values():
        x.fill_(float("nan"))
    g = np.random.default_rng(5)
    prompt = 37
    p.extend([prompt, 0, 0, 0])
    history = [[torch.empty(0, n_kv, d, device="cuda") for _ in range(2)] for _ in range(B)]

    def append(n_new):
        new = [bf16(torch, g, (sum(n_new), n_kv, d)) for _ in range(2)]
        off = offsets(n_new)
        lsa.kv_append(cache, *new, new_offsets=dev(torch, off, np.int64), new_offsets_host=off)
        for b in range(B):
            for i in range(2):
                history[b][i] = torch.cat([history[b][i], new[i][off[b]:off[b + 1]].float()])

    append([prompt, 0, 0, 0])
    p.fork([cache], [0, 0, 0], [1, 2, 3])
    for b in (1, 2, 3):
        history[b] = list(history[0])
    for step in range(14):
        n = [1, 1, 1, 1] if step != 5 else [0, 3, 1, 0]
        p.extend(n)
        append(n)
    off = offsets([1] * B)
    q = bf16(torch, g, (B, n_q, d))
    out, lse, slopes = torch.empty_like(q), torch.empty(B, n_q, device="cuda"), torch.from_numpy(geometric(n_q)).cuda()
    lens = p.kv_len.tolist()
    size = lsa.attend_workspace_size(cache, n_q=n_q, q_offsets_host=off, max_kv_len=max(lens))
    lsa.attend(cache, q, q_offsets=dev(torch, off, np.int64), q_offsets_host=off, max_kv_len=max(lens), out=out, lse=lse, scale=0.125,
               workspace=torch.empty(max(size, 16), dtype=torch.uint8, device="cuda"), slopes=slopes, softcap=9.0)

    class S:  # what check() wants, from the history
        pass

    s = S()
    s.n_kv, s.d, s.totals, s.table = n_kv, d, lens, np.arange(B)[:, None]
    s.decoded = {}
    for i, name in enumerate(("k", "v")):
        one = np.zeros((B, n_kv, max(lens), d))
        for b in range(B):
            assert len(history[b][i]) == lens[b]
            one[b, :, :lens[b]] = history[b][i].cpu().double().numpy().transpose(1, 0, 2)
        s.decoded[name] = one
    check(s, q, out, lse, [(b, b, lens[b] - 1) for b in range(B)], scale=0.125, softcap=9.0, slopes=geometric(n_q))


def test_pool_captured(torch, lsa):
    """Free, extend and fork as one graph: every replay starts from what the one before left, and does what the eager calls do."""
    p, e = Pool(torch, lsa, 6, 5, 30, 16), Pool(torch, lsa, 6, 5, 30, 16)
    cp, ce = [[c for _, c in layers_of(torch, lsa, x, 2, "fp8", 1, 64, 16)] for x in (p, e)]
    grow, gone = dev(torch, [20, 0, 0, 0, 0, 3]), dev(torch, [0, 1, 2])
    src, dst = dev(torch, [0, 0, 5]), dev(torch, [1, 2, 3])
    st, ws = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")

    def step(x, caches):
        lsa.kv_free(x.pool, gone)
        lsa.kv_extend(x.pool, grow)
        lsa.kv_fork(x.pool, caches, src, dst, status=st, workspace=ws)

    step(p, cp)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(p, cp)
    step(e, ce)
    for i in range(4):
        grow.add_(i)
        graph.replay()
        torch.cuda.synchronize()
        step(e, ce)
        torch.cuda.synchronize()
        for a, b in ((p.refs, e.refs), (p.table, e.table), (p.kv_len, e.kv_len)):
            assert torch.equal(a, b), i
        for a, b in zip(cp, ce):
            assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.v_scale, b.v_scale)
