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
