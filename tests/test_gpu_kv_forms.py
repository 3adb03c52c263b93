"""lsa_attend_ex and lsa_attend_topk_ex against the float64 oracle (marked gpu). Inputs and tolerances as in test_gpu_kv.py,
with what the scores' forms add, in natural units:
  * cap: 1 - 2 / (1 + e^(2z)) is formed from an exponential and a reciprocal of one unit in the last place each (2^-23), the
    roundings of 1 + e, of the argument (|z| e^(2z) / (1 + e^(2z))^2 <= 0.23) and of the product: less than 9 * 2^-24 of 2 softcap,
    so 2^-20 softcap bounds it; the score's own error is not enlarged, as tanh is nowhere steeper than 1;
  * bias: slope log2(e), its product with a distance below 2^24 and the sum are rounded: 2^-22 (|bias| + softcap or |score|).
"""
import numpy as np
import pytest

from oracle import kv_more_oracle as M
from oracle import kv_oracle as K
from tests.parity import say
from tests.test_gpu_kv import Setup, U, bf16, lsa, offsets, torch  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def check(s, q, out, lse, rows, *, scale, softcap=0.0, slopes=None, window=0, sinks=0, doc=None, prefix=None, listed=None, r=1, tag=""):
    """rows: (row, sequence, position)."""
    n_q = q.shape[1]
    G = n_q // s.n_kv
    got, got_l, qq = out.cpu().double().numpy(), lse.cpu().double().numpy(), q.cpu().double().numpy()
    cached = {}
    for row, b, p in rows:
        t = max(s.totals[b], 0)
        see = M.sees(p, t, window, sinks, None if doc is None else max(int(doc[row]), 0), None if prefix is None else int(prefix[row]),
                     None if listed is None else listed[b], r)
        for h in range(s.n_kv):
            if (b, h) not in cached:
                cached[b, h] = [K.rows_of(s.decoded[x], s.table[b], t, h) for x in ("k", "v")]
            (Kc, there), (Vc, _) = cached[b, h]
            seen = see & there
            for head in range(h * G, h * G + G):
                slope = 0.0 if slopes is None else float(slopes[head])
                o, l, A, big, bias = M.attend_row(qq[row, head], Kc, Vc, seen, p, scale, softcap, slope)
                dx = 2 * (s.d + 4) * 2.0 ** -24 * big + 2.0 ** -22 * (big if np.isfinite(l) else 0) + 2.0 ** -20 * softcap
                dx += 2.0 ** -22 * (bias + (softcap or big)) if slope else 0.0
                n = int(seen.sum())
                tol = (U + 4 * dx + n * 2.0 ** -24 + 2.0 ** -16) * A + U * np.abs(o) + 1e-30
                where = f"{tag} row {row} seq {b} pos {p} head {head}"
                with np.errstate(invalid="ignore"):
                    g = got[row, head]
                    same = (np.isnan(o) & np.isnan(g)) | (o == g) | (np.abs(g - o) <= tol)
                assert same.all(), (where, np.abs(g - o).max(), o[:4], g[:4])
                if np.isinf(l):
                    assert got_l[row, head] == l, (where, got_l[row, head])
                elif np.isfinite(l):
                    assert abs(got_l[row, head] - l) <= 2 * dx + n * 2.0 ** -24 + 2.0 ** -20 * (1 + abs(l)), (where, got_l[row, head], l)


def run(torch, lsa, s, q, off, *, scale=None, window=0, sinks=0, softcap=0.0, slopes=None, doc=None, prefix=None, max_len=None, ws=None):
    scale = s.d ** -0.5 if scale is None else scale
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], -7.0, device="cuda")
    max_len = max(max(s.totals), 0) if max_len is None else max_len
    if ws is None:
        size = lsa.attend_workspace_size(s.cache, n_q=q.shape[1], q_offsets_host=off, max_kv_len=max_len, window=window, sinks=sinks)
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")

    def dev(x, t):
        return None if x is None else torch.from_numpy(np.asarray(x, t)).cuda()

    lsa.attend(s.cache, q, q_offsets=torch.from_numpy(off).cuda(), q_offsets_host=off, max_kv_len=max_len, out=out, lse=lse, scale=scale,
               window=window, sinks=sinks, workspace=ws, softcap=softcap, slopes=dev(slopes, np.float32), doc_start=dev(doc, np.int32),
               prefix_end=dev(prefix, np.int32))
    return out, lse


def some_rows(news, totals, most=24):
    """(row, sequence, position) of up to `most` rows of each sequence, first and last among them."""
    out, at = [], 0
    for b, (n, t) in enumerate(zip(news, totals)):
        for i in sorted(set(np.linspace(0, n - 1, min(n, most)).astype(int))) if n else []:
            out.append((at + i, b, t - n + i))
        at += n
    return out


def geometric(n_q):
    return (2.0 ** (-8.0 * (np.arange(n_q) + 1) / n_q)).astype(np.float32)


FORMS = {"cap": dict(softcap=5.0), "cap_wide": dict(softcap=1024.0), "bias": dict(slopes=True), "both": dict(softcap=30.0, slopes=True),
         "neg": dict(slopes=-0.01)}


def form_of(name, n_q):
    f = dict(FORMS[name])
    if f.get("slopes") is True:
        f["slopes"] = geometric(n_q)
    elif "slopes" in f:
        f["slopes"] = np.full(n_q, f["slopes"], np.float32)
    return f


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,d,G,pt", [("bf16", 128, 8, 64), ("fp8", 128, 1, 16), ("bf16", 64, 3, 32), ("fp8", 64, 20, 128),
                                          ("fp8", 128, 33, 64), ("bf16", 128, 40, 64)])
def test_tokens(torch, lsa, form, dtype, d, G, pt):
    """One to three new tokens of short and long sequences: the split kernel, shared and not."""
    n_kv = 2
    for totals, news in (([1, 17, 64, 65, 700, 0], [1, 1, 1, 1, 1, 0]), ([9, 2100, 40], [3, 1, 2])):
        s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=G)
        q = bf16(torch, s.g, (sum(news), n_kv * G, d), 3.0)
        f = form_of(form, n_kv * G)
        out, lse = run(torch, lsa, s, q, offsets(news), **f)
        check(s, q, out, lse, some_rows(news, totals), scale=d ** -0.5, tag=f"{form} {totals}", **f)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,d,G,pt", [("bf16", 128, 8, 64), ("fp8", 128, 4, 16), ("bf16", 64, 8, 32), ("fp8", 64, 16, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_prompts(torch, lsa, form, dtype, d, G, pt, window, sinks):
    """Prompts and chunks: the tile kernel, whole and split, and a mixed batch."""
    n_kv = 2
    for totals, news in (([300, 97, 70], [300, 66, 1]), ([5000], [70])):
        s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=3)
        q = bf16(torch, s.g, (sum(news), n_kv * G, d), 3.0)
        f = form_of(form, n_kv * G)
        out, lse = run(torch, lsa, s, q, offsets(news), window=window, sinks=sinks, **f)
        check(s, q, out, lse, some_rows(news, totals, 8), scale=d ** -0.5, window=window, sinks=sinks, tag=f"{form} {totals}", **f)


def documents(g, news, totals, least, most):
    """doc_start of every row: documents of random lengths over each sequence's positions."""
    rows = []
    for n, t in zip(news, totals):
        start = []
        while len(start) < t:
            start += [len(start)] * int(g.integers(least, most + 1))
        rows += start[t - n:t]
    return np.array(rows, np.int32)


@pytest.mark.parametrize("form", [None, "cap", "bias"])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 8), ("fp8", 64, 4), ("fp8", 128, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 4), (500, 100)])
@pytest.mark.parametrize("least,most", [(1, 9), (50, 200)])
def test_documents(torch, lsa, form, dtype, d, G, window, sinks, least, most):
    n_kv = 2
    for totals, news in (([400, 500, 33], [400, 90, 3]), ([3000, 40], [140, 5])):
        s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=16, seed=5)
        doc = documents(s.g, news, totals, least, most)
        q = bf16(torch, s.g, (sum(news), n_kv * G, d), 2.0)
        f = form_of(form, n_kv * G) if form else {}
        out, lse = run(torch, lsa, s, q, offsets(news), window=window, sinks=sinks, doc=doc, **f)
        check(s, q, out, lse, some_rows(news, totals, 12), scale=d ** -0.5, window=window, sinks=sinks, doc=doc, tag=f"{form} {totals}", **f)


@pytest.mark.parametrize("form", [None, "cap", "bias", "both"])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 8), ("fp8", 64, 4)])
def test_prefix(torch, lsa, form, dtype, d, G):
    """A prefix that every row sees, per sequence and with documents, and one that reaches beyond the cache."""
    n_kv = 2
    for totals, news, ends in (([400, 500, 33], [400, 90, 3], [150, 480, 20]), ([3000, 40, 200], [140, 5, 200], [2900, 10 ** 9, 0])):
        s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=32, seed=6)
        prefix = np.repeat(np.array(ends, np.int32), news)
        q = bf16(torch, s.g, (sum(news), n_kv * G, d), 2.0)
        f = form_of(form, n_kv * G) if form else {}
        for doc in (None, documents(s.g, news, totals, 20, 150)):
            out, lse = run(torch, lsa, s, q, offsets(news), doc=doc, prefix=prefix, **f)
            check(s, q, out, lse, some_rows(news, totals, 12), scale=d ** -0.5, doc=doc, prefix=prefix, tag=f"{form} {totals}", **f)


@pytest.mark.parametrize("rows", [5, 90])
def test_odd_masks(torch, lsa, rows):
    """Rows that see nothing, bounds at the ends of int32, positions before the cache, pages that are not there."""
    totals, news = [rows + 200, rows - 3, rows], [rows, rows, rows]  # the second one's first three tokens are not cached
    s = Setup(torch, lsa, totals, dtype="bf16", n_kv=1, d=64, pt=16, seed=7)
    s.table[0, 3] = -1
    s.table[2, 0] = 10 ** 9
    s.table_dev.copy_(torch.from_numpy(s.table))
    q = bf16(torch, s.g, (3 * rows, 8, 64))
    g = np.random.default_rng(8)
    doc = g.choice(np.array([-2 ** 31, -1, 0, 1, 40, rows, rows + 199, rows + 200, 2 ** 31 - 1]), 3 * rows).astype(np.int32)
    prefix = g.choice(np.array([-2 ** 31, -1, 0, 1, 47, rows, rows + 200, 2 ** 31 - 1]), 3 * rows).astype(np.int32)
    for d, p in ((doc, None), (None, prefix), (doc, prefix)):
        for f in ({}, form_of("cap", 8), form_of("bias", 8)):
            out, lse = run(torch, lsa, s, q, offsets(news), doc=d, prefix=p, **f)
            check(s, q, out, lse, some_rows(news, totals, 40), scale=0.125, doc=d, prefix=p, **f)
    assert torch.isinf(lse).any() and (out[torch.isinf(lse)] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("rows", [6, 100])
def test_not_finite(torch, lsa, dtype, rows):
    """What another document holds has no effect on a row, infinities and NaN too; the own document's show."""
    totals, news = [rows + 30], [rows]
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=1, d=64, pt=16, seed=9)
    half = 30 + rows // 2
    doc = np.where(np.arange(30, 30 + rows) < half, 20, half).astype(np.int32)
    q = bf16(torch, s.g, (rows, 8, 64))
    for pos in (3, 25, half + 1):  # seen by nobody, by the first document, by the second
        page, slot = s.table[0, pos // 16], pos % 16
        for name in ("k", "v"):
            if dtype == "fp8":
                s.parts[name].view(torch.uint8)[page, 0, slot, pos % 64] = 0x7F
            else:
                s.parts[name][page, 0, slot, pos % 64] = float("inf") if name == "v" else float("nan")
    s.decode()
    for f in ({}, form_of("cap", 8), form_of("bias", 8), form_of("both", 8)):
        out, lse = run(torch, lsa, s, q, offsets(news), doc=doc, **f)
        bad = ~torch.isfinite(out.float()).all(-1).all(-1).cpu().numpy()
        want = np.array([any(d <= x <= 30 + i for x in (3, 25, half + 1)) for i, d in enumerate(doc)])
        assert (bad == want).all(), (f, np.flatnonzero(bad != want))


def test_values_not_finite_in_some_rows(torch, lsa):
    """An infinite value, with finite keys: exact rows against the oracle on both sides of it."""
    for rows in (6, 100):
        s = Setup(torch, lsa, [rows + 30], dtype="bf16", n_kv=1, d=64, pt=16, seed=10)
        doc = np.where(np.arange(rows) < rows // 2, 0, 31).astype(np.int32)
        s.parts["v"][s.table[0, 1], 0, 14, 5] = float("-inf")  # position 30
        s.decode()
        q = bf16(torch, s.g, (rows, 8, 64))
        for f in ({}, form_of("cap", 8), form_of("bias", 8)):
            out, lse = run(torch, lsa, s, q, offsets([rows]), doc=doc, **f)
            check(s, q, out, lse, some_rows([rows], [rows + 30]), scale=0.125, doc=doc, **f)
            assert torch.isinf(out[: rows // 2, :, 5]).all() and torch.isfinite(out[rows // 2:].float()).all()


@pytest.mark.parametrize("rows", [4, 80])
def test_scales(torch, lsa, rows):
    """Negative and zero softmax scales, scores far beyond the cap and beyond fp32, page scales that are no powers of two."""
    s = Setup(torch, lsa, [rows + 100], dtype="fp8", n_kv=1, d=64, pt=16, seed=11)
    for name in ("k", "v"):
        s.parts[name + "_scale"].mul_(1.37)
    s.decode()
    q = bf16(torch, s.g, (rows, 8, 64))
    for scale in (-0.125, 0.0, 3.0):
        for f in (form_of("cap", 8), form_of("bias", 8), form_of("both", 8)):
            out, lse = run(torch, lsa, s, q, offsets([rows]), scale=scale, **f)
            check(s, q, out, lse, some_rows([rows], [rows + 100], 8), scale=scale, tag=f"scale {scale}", **f)
    # Every score is far beyond the cap: each key has one of two weights, e^(2 softcap) apart. Where the products themselves are beyond
    # fp32 (1e48, of both signs in every row), their sum is infinity less infinity: that shows as NaN.
    s = Setup(torch, lsa, [rows + 100], dtype="bf16", n_kv=1, d=64, pt=16, seed=12)
    q = bf16(torch, s.g, (rows, 8, 64), 1e30)
    s.parts["k"].mul_(1e18)
    s.decode()
    for amp in (1.0, 1e-30):
        q.mul_(amp)
        out, lse = run(torch, lsa, s, q, offsets([rows]), softcap=2.0)
        if amp == 1.0:
            assert torch.isnan(out).all() and torch.isnan(lse).all()
            continue
        qq, got, got_l = q.cpu().double().numpy(), out.cpu().double().numpy(), lse.cpu().double().numpy()
        (Kc, _), (Vc, _) = [K.rows_of(s.decoded[x], s.table[0], rows + 100, 0) for x in ("k", "v")]
        for row in range(rows):
            see = M.sees(101 + row - 1, rows + 100)
            for head in range(8):
                o, l, A, _, _ = M.attend_row(qq[row, head], Kc, Vc, see, 100 + row, 0.125, 2.0)
                tol = (U + 4 * 2.0 ** -19 + 2.0 ** -15) * A + U * np.abs(o)
                assert (np.abs(got[row, head] - o) <= tol).all() and abs(got_l[row, head] - l) <= 2.0 ** -17


def test_zero_form_is_plain(torch, lsa):
    """A form without anything in it gives lsa_attend's results bit for bit."""
    import ctypes
    totals, news = [300, 900], [100, 1]
    s = Setup(torch, lsa, totals, dtype="bf16", n_kv=2, d=128, pt=64, seed=13)
    q, off = bf16(torch, s.g, (101, 16, 128)), offsets(news)
    want = run(torch, lsa, s, q, off)
    size = lsa.attend_workspace_size(s.cache, n_q=16, q_offsets_host=off, max_kv_len=900)
    ws, off_dev = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.from_numpy(off).cuda()
    for form in (None, ctypes.byref(lsa._AttendForm())):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        st = lsa._attend_ex(s.cache.ref, 2, q.data_ptr(), 16 * 128, 16, off_dev.data_ptr(), off.ctypes.data, 900, 128 ** -0.5, 0, 0, form,
                            out.data_ptr(), 16 * 128, lse.data_ptr(), ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,d,n_kv,G,r", [("fp8", 128, 2, 8, 1), ("bf16", 64, 1, 40, 4), ("fp8", 64, 1, 70, 3), ("bf16", 128, 2, 3, 1)])
def test_listed(torch, lsa, form, dtype, d, n_kv, G, r):
    totals, k = [1, 50, 900, 333, 0], 60
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=32, seed=14)
    idx, count = np.full((5, k), -1, np.int32), np.zeros(5, np.int32)
    for b, t in enumerate(totals):
        e = -(-t // r)
        some = np.sort(s.g.permutation(e)[: min(k, e)])
        idx[b, :len(some)], count[b] = some, len(some)
    q = bf16(torch, s.g, (5, n_kv * G, d), 3.0)
    f = form_of(form, n_kv * G)
    for window, sinks in ((0, 0), (40, 3)):
        out, lse = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], -7.0, device="cuda")
        size = lsa.attend_topk_workspace_size(s.cache, n_q=n_kv * G, k=k, entry_tokens=r, window=window, sinks=sinks)
        lsa.attend_topk(s.cache, q, idx=torch.from_numpy(idx).cuda(), count=torch.from_numpy(count).cuda(), entry_tokens=r, scale=d ** -0.5,
                        window=window, sinks=sinks, out=out, lse=lse, workspace=torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda"),
                        softcap=f.get("softcap", 0.0), slopes=None if "slopes" not in f else torch.from_numpy(f["slopes"]).cuda())
        listed = [idx[b, :count[b]].tolist() for b in range(5)]
        check(s, q, out, lse, [(b, b, t - 1) for b, t in enumerate(totals)], scale=d ** -0.5, window=window, sinks=sinks, listed=listed, r=r, **f)


def test_packed_documents_are_single_ones(torch, lsa):
    """Two prompts packed into one sequence, each its own document with a bidirectional prefix, and the same tokens as two sequences:
    their scores and masks are the same. Sums come in another order."""
    a, b = 150, 90
    s = Setup(torch, lsa, [a + b], dtype="bf16", n_kv=2, d=64, pt=16, seed=15)
    t = Setup(torch, lsa, [a, b], dtype="bf16", n_kv=2, d=64, pt=16, seed=16)
    for name in ("k", "v"):
        for p in range(a + b):
            row = s.parts[name][s.table[0, p // 16], :, p % 16]
            seq, at = (0, p) if p < a else (1, p - a)
            t.parts[name][t.table[seq, at // 16], :, at % 16] = row
    q = bf16(torch, s.g, (a + b, 16, 64), 2.0)
    doc = np.repeat(np.array([0, a], np.int32), [a, b])
    prefix = np.repeat(np.array([40, a + 30], np.int32), [a, b])
    f = form_of("both", 16)
    one = run(torch, lsa, s, q, offsets([a + b]), doc=doc, prefix=prefix, **f)
    two = run(torch, lsa, t, q, offsets([a, b]), prefix=np.repeat(np.array([40, 30], np.int32), [a, b]), **f)
    # each is within its own tolerance of the oracle; together twice the roundings of probabilities and output
    assert (one[0].float() - two[0].float()).abs().max() <= 4 * U * 4  # values are N(0, 1): at most some 4
    # scores: 2 (d + 4) 2^-24 of scale * sum |q K| (at most some 40), the cap's error and the sum's
    assert (one[1] - two[1]).abs().max() <= 4 * (2 * 68 * 2.0 ** -24 * 40 + 2.0 ** -20 * 30 + 2.0 ** -16)


def test_captured(torch, lsa):
    """A captured call follows kv_len, doc_start and the slopes of each replay, on a stream of its own."""
    s = Setup(torch, lsa, [700, 60], dtype="bf16", n_kv=1, d=64, pt=16, seed=17)
    q, off = bf16(torch, s.g, (62, 8, 64)), offsets([2, 60])
    doc = torch.zeros(62, dtype=torch.int32, device="cuda")
    slopes = torch.from_numpy(geometric(8)).cuda()
    size = lsa.attend_workspace_size(s.cache, n_q=8, q_offsets_host=off, max_kv_len=700)
    ws, out, lse = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(q), torch.empty(62, 8, device="cuda")
    off_dev = torch.from_numpy(off).cuda()

    def call():
        lsa.attend(s.cache, q, q_offsets=off_dev, q_offsets_host=off, max_kv_len=700, out=out, lse=lse, scale=0.125, workspace=ws,
                   softcap=20.0, slopes=slopes, doc_start=doc)

    call()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for step in range(3):
        s.kv_len.copy_(torch.tensor([700 - 100 * step, 60], dtype=torch.int32))
        doc.fill_(7 * step)
        slopes.mul_(0.5)
        out.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        s.totals = [700 - 100 * step, 60]
        check(s, q, out, lse, some_rows([2, 60], s.totals, 4), scale=0.125, softcap=20.0, slopes=slopes.cpu().numpy(), doc=doc.cpu().numpy())
    say("three replays")
