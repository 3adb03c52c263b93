"""Biases by distance whose size, sign or masks are far from the usual ones, with and without a cap, against the float64 oracle
(marked gpu). Tolerances are those of test_gpu_kv_forms.py, whose check() compares."""
import numpy as np
import pytest

from tests.test_gpu_kv import Setup, bf16, lsa, offsets, torch  # noqa: F401  (fixtures)
from tests.test_gpu_kv_forms import check, documents, run, some_rows

pytestmark = pytest.mark.gpu

# a row's own keys may lie hundreds of units of the bias away from keys that it does not see
CAPPED = {"half": (5.0, -0.5), "one": (30.0, -1.0), "tenth": (30.0, -0.1), "positive": (30.0, 1.0), "both signs": (30.0, None)}


def slopes_of(slope, n_q):
    if slope is None:
        return np.linspace(-1, 1, n_q).astype(np.float32)
    return np.full(n_q, slope, np.float32)


def compare(torch, lsa, s, news, form, G, *, most=14, **kw):
    q = bf16(torch, s.g, (sum(news), s.n_kv * G, s.d), 2.0)
    f = dict(softcap=form[0], slopes=slopes_of(form[1], s.n_kv * G))
    out, lse = run(torch, lsa, s, q, offsets(news), **f, **kw)
    check(s, q, out, lse, some_rows(news, s.totals, most), scale=s.d ** -0.5, tag=f"{form} G {G}", **f, **kw)


@pytest.mark.parametrize("form", CAPPED)
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 1), ("fp8", 64, 1), ("bf16", 64, 3), ("fp8", 128, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_capped_prompts(torch, lsa, form, dtype, d, G, window, sinks):
    """Rows of one block whose positions lie up to 255 apart, and none of whose keys some other rows see."""
    totals, news = [300, 97, 1500], [300, 97, 260]
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=2, d=d, pt=32, seed=21)
    compare(torch, lsa, s, news, CAPPED[form], G, window=window, sinks=sinks)


@pytest.mark.parametrize("form", CAPPED)
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 1), ("fp8", 64, 8)])
@pytest.mark.parametrize("ends", [False, True])
def test_capped_documents(torch, lsa, form, dtype, d, G, ends):
    """Packed documents, short ones beside one of 2000 tokens, each seen from its start, or as a whole from every row."""
    lengths = [[16, 2000, 40, 3, 500], [400, 300]]
    totals = [sum(x) for x in lengths]
    start = np.concatenate([np.repeat(np.cumsum([0] + x[:-1]), x) for x in lengths]).astype(np.int32)
    end = np.concatenate([np.repeat(np.cumsum(x), x) for x in lengths]).astype(np.int32)
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=1, d=d, pt=64, seed=22)
    form = CAPPED[form]
    q = bf16(torch, s.g, (sum(totals), G, d), 2.0)
    f = dict(softcap=form[0], slopes=slopes_of(form[1], G))
    out, lse = run(torch, lsa, s, q, offsets(totals), doc=start, prefix=end if ends else None, **f)
    rows, at = [], 0
    for b, x in enumerate(lengths):  # each document's first, second, middle and last row
        p = 0
        for n in x:
            rows += [(at + p + i, b, p + i) for i in sorted({0, 1, n // 2, n - 1} & set(range(n)))]
            p += n
        at += p
    check(s, q, out, lse, rows, scale=d ** -0.5, doc=start, prefix=end if ends else None, tag=f"{form}", **f)


@pytest.mark.parametrize("form", CAPPED)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_capped_far_keys_only(torch, lsa, form, dtype):
    """The pages around and before the rows are not there, or their documents begin behind them: only far keys are seen."""
    totals, news = [900, 900], [90, 120]
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=1, d=64, pt=16, seed=23)
    s.table[0, 20:] = -1  # positions from 320 on; the rows are 810 .. 899
    s.table_dev.copy_(torch.from_numpy(s.table))
    doc = np.concatenate([np.zeros(90), np.full(120, 880)]).astype(np.int32)
    prefix = np.full(210, 900, np.int32)
    compare(torch, lsa, s, news, CAPPED[form], 1)
    compare(torch, lsa, s, news, CAPPED[form], 3, doc=doc, prefix=prefix)


@pytest.mark.parametrize("form", CAPPED)
@pytest.mark.parametrize("rows", [5, 90])
def test_capped_odd_masks(torch, lsa, form, rows):
    """Rows that see nothing, bounds at the ends of int32, positions before the cache, pages that are not there."""
    totals, news = [rows + 200, rows - 3, rows], [rows, rows, rows]  # the second one's first three tokens are not cached
    s = Setup(torch, lsa, totals, dtype="bf16", n_kv=1, d=64, pt=16, seed=24)
    s.table[0, 3], s.table[2, 0] = -1, 10 ** 9
    s.table_dev.copy_(torch.from_numpy(s.table))
    g = np.random.default_rng(25)
    doc = g.choice(np.array([-2 ** 31, -1, 0, 1, 40, rows, rows + 199, rows + 200, 2 ** 31 - 1]), 3 * rows).astype(np.int32)
    prefix = g.choice(np.array([-2 ** 31, -1, 0, 1, 47, rows, rows + 200, 2 ** 31 - 1]), 3 * rows).astype(np.int32)
    for d, p in ((doc, None), (None, prefix), (doc, prefix)):
        compare(torch, lsa, s, news, CAPPED[form], 8, most=40, doc=d, prefix=p)


@pytest.mark.parametrize("form", CAPPED)
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 8), ("fp8", 64, 1)])
def test_capped_prefixes(torch, lsa, form, dtype, d, G):
    """A prefix that every row sees, per sequence and with documents, and one that reaches beyond the cache."""
    for totals, news, ends in (([400, 500, 33], [400, 90, 3], [150, 480, 20]), ([3000, 40, 200], [140, 5, 200], [2900, 10 ** 9, 0])):
        s = Setup(torch, lsa, totals, dtype=dtype, n_kv=1, d=d, pt=32, seed=26)
        prefix = np.repeat(np.array(ends, np.int32), news)
        for doc in (None, documents(s.g, news, totals, 20, 150)):
            compare(torch, lsa, s, news, CAPPED[form], G, most=10, doc=doc, prefix=prefix)


def test_capped_scores_of_minus_infinity_count(torch, lsa):
    """A visible score of minus infinity is -softcap: rows that see nothing else are the mean of their values, whatever the bias."""
    s = Setup(torch, lsa, [200], dtype="bf16", n_kv=1, d=64, pt=16, seed=27)
    s.parts["k"].fill_(float("-inf"))
    q = torch.ones((200, 2, 64), dtype=torch.bfloat16, device="cuda")
    for slope in (0.0, -0.0):
        out, lse = run(torch, lsa, s, q, offsets([200]), softcap=3.0, slopes=np.full(2, slope, np.float32))
        n = torch.arange(1, 201, device="cuda").double()
        # lse: as in check(), with dx the cap's 2^-20 of 3 and the bias's 2^-22 of it
        assert ((lse.double() + 3.0 - n.log()[:, None]).abs() <= 2 * 3.0 * (2.0 ** -20 + 2.0 ** -22) + 200 * 2.0 ** -24 + 2.0 ** -20 * 9).all()
        v = torch.stack([s.parts["v"][int(s.table[0, p // 16]), 0, p % 16].double() for p in range(200)])
        want = v.cumsum(0) / n[:, None]
        tol = (2.0 ** -8 + 200 * 2.0 ** -24 + 2.0 ** -16) * (v.abs().cumsum(0) / n[:, None]) + 2.0 ** -8 * want.abs()
        assert ((out.double() - want[:, None]).abs() <= tol[:, None]).all()


# ------------------------------------------------------------------ steep ones
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("slope", [3.0, -3.0])
@pytest.mark.parametrize("dtype,d,G", [("bf16", 128, 1), ("fp8", 64, 3), ("fp8", 128, 8)])
def test_steep(torch, lsa, softcap, slope, dtype, d, G):
    """Beyond a slope of 1: prompts, windows, prefixes and documents, and pages that are not there."""
    totals, news = [300, 97, 900], [300, 97, 140]
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=1, d=d, pt=32, seed=31)
    for name in ("k", "v"):
        if dtype == "fp8":
            s.parts[name + "_scale"].mul_(1.37)
    s.decode()
    s.table[2, 5] = -1
    s.table_dev.copy_(torch.from_numpy(s.table))
    form = (softcap, slope)
    compare(torch, lsa, s, news, form, G)
    compare(torch, lsa, s, news, form, G, window=60, sinks=5)
    doc, prefix = documents(s.g, news, totals, 5, 150), np.repeat(np.array([200, 97, 850], np.int32), news)
    compare(torch, lsa, s, news, form, G, doc=doc)
    compare(torch, lsa, s, news, form, G, prefix=prefix)
    compare(torch, lsa, s, news, form, G, doc=doc, prefix=prefix)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("slope", [300.0, 1e6, 1e9, 1e36, 3.4e38])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("rows", [3, 90])
def test_steep_rows_see_themselves(torch, lsa, softcap, slope, dtype, rows):
    """So steep a bias leaves a row its own key, which loses nothing: out is that key's value, lse that key's score."""
    s = Setup(torch, lsa, [rows + 400], dtype=dtype, n_kv=1, d=64, pt=16, seed=32)
    q = bf16(torch, s.g, (rows, 4, 64), 2.0)
    out, lse = run(torch, lsa, s, q, offsets([rows]), softcap=softcap, slopes=np.full(4, slope, np.float32))
    where = [(int(s.table[0, p // 16]), 0, p % 16) for p in range(400, 400 + rows)]
    k, v = (np.stack([s.decoded[x][i] for i in where]) for x in ("k", "v"))
    y = np.einsum("rhd,rd->rh", q.cpu().double().numpy(), k) * 0.125
    big = np.einsum("rhd,rd->rh", np.abs(q.cpu().double().numpy()), np.abs(k)) * 0.125
    want = softcap * np.tanh(y / softcap) if softcap else y
    assert (out.cpu().double().numpy() == v[:, None]).all()  # cached values are bf16 numbers, and the weight is 1
    # as in check(), for one key and a bias of 0
    dx = 2 * (64 + 4) * 2.0 ** -24 * big + 2.0 ** -22 * big + 2.0 ** -20 * softcap
    assert (np.abs(lse.cpu().double().numpy() - want) <= 2 * dx + 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(want))).all()


@pytest.mark.parametrize("rows", [3, 90])
def test_steep_listed(torch, lsa, rows):
    """The same for listed entries and the window."""
    s = Setup(torch, lsa, [100 + rows, 40], dtype="bf16", n_kv=1, d=64, pt=16, seed=33)
    q = bf16(torch, s.g, (2, 4, 64), 2.0)
    idx = torch.tensor([[3, 9], [2, 5]], dtype=torch.int32, device="cuda")
    count = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    size = lsa.attend_topk_workspace_size(s.cache, n_q=4, k=2, window=20)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    for slope in (300.0, 1e9, 3.4e38):
        out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
        lsa.attend_topk(s.cache, q, idx=idx, count=count, out=out, lse=lse, scale=0.125, window=20, workspace=ws,
                        slopes=torch.full((4,), slope, device="cuda"))
        for b, t in enumerate(s.totals):
            v = s.parts["v"][int(s.table[b, (t - 1) // 16]), 0, (t - 1) % 16]
            assert (out[b] == v).all() and torch.isfinite(lse[b]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("scale", [1e-39, 1e-30, -1e-30, 0.0])
def test_biases_alone(torch, lsa, dtype, scale):
    """Scales that leave nothing of the scores: what counts is the bias, on both sides of a row."""
    s = Setup(torch, lsa, [200, 90], dtype=dtype, n_kv=1, d=64, pt=16, seed=34)
    q = bf16(torch, s.g, (290, 2, 64), 2.0)
    prefix = np.repeat(np.array([150, 0], np.int32), [200, 90])
    for slope in (0.3, -0.2, 2.5):
        f = dict(slopes=np.full(2, slope, np.float32))
        out, lse = run(torch, lsa, s, q, offsets([200, 90]), scale=scale, prefix=prefix, **f)
        check(s, q, out, lse, some_rows([200, 90], s.totals, 20), scale=scale, prefix=prefix, tag=f"{scale} {slope}", **f)
