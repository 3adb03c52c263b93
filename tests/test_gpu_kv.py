"""lsa_kv_append, lsa_attend and lsa_attend_topk against the float64 oracle, through the C-ABI (marked gpu).

The inputs are what the kernels get, bit for bit. Slots behind a sequence's length, pages that no sequence
has and their scales hold NaN, so anything read there shows.

Tolerances of one output row, from the arithmetic (u = 2^-8 is half a bf16 step of the value):
  * a score is a sum of d products, exact in fp32 before the sum: off by at most dx = 2 (d + 4) 2^-24 times the
    largest scale * sum_i |q_i K_si|, and the exponential's argument by 2^-22 of its size (|x| <= lse + that);
  * each probability is rounded to bf16 once (u), and out once more: |error| <= (u + 4 dx + n 2^-24 + 2^-16) A + u |out|
    with A = sum_s P_s |V_s|, n the seen keys (fp32 sums);
  * lse: 2 dx + n 2^-24 + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

from oracle import kv_oracle as K
from tests.parity import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


@pytest.fixture(scope="module")
def lsa():
    from sparse_kv_retrieval_amd import lsa as mod
    return mod


class Setup:
    """A cache with `totals` cached tokens a sequence; `torch` tensors on the GPU and decoded float64 copies."""

    def __init__(self, torch, lsa, totals, *, dtype, n_kv, d, pt, seed=0, extra_pages=2, amp=1.0):
        g = np.random.default_rng(seed)
        self.g, self.torch, self.pt, self.d, self.n_kv, self.dtype = g, torch, pt, d, n_kv, dtype
        per = [-(-max(t, 0) // pt) for t in totals]
        n_pages, width = sum(per) + extra_pages, max(max(per), 1) + 1
        order = g.permutation(n_pages)
        self.table = np.full((len(totals), width), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.totals = list(totals)
        used = np.zeros((n_pages, pt), bool)
        for b, t in enumerate(totals):
            for s in range(t):
                used[self.table[b, s // pt], s % pt] = True
        self.used = used
        parts, self.decoded, self.scales = {}, {}, {}
        for name in ("k", "v"):
            if dtype == "fp8":
                codes = g.integers(0, 256, (n_pages, n_kv, pt, d)).astype(np.uint8)
                x = np.clip(g.normal(size=codes.shape) * 80, -448, 448)
                codes = K.to_e4m3(x)
                codes[~np.broadcast_to(used[:, None, :], codes.shape[:3])] = 0x7F
                scale = (2.0 ** g.integers(-8, -5, (n_pages, n_kv)) * amp).astype(np.float32)
                scale[~used.any(1)] = np.nan
                self.decoded[name] = K.e4m3_values()[codes] * scale[:, :, None, None].astype(np.float64)
                parts[name] = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
                parts[name + "_scale"] = torch.from_numpy(scale).cuda()
                self.scales[name] = scale
            else:
                x = torch.from_numpy(g.normal(size=(n_pages, n_kv, pt, d)) * amp).to(torch.bfloat16)
                x[~torch.from_numpy(used)[:, None, :].expand(x.shape[:3])] = float("nan")
                self.decoded[name] = x.double().numpy()
                parts[name] = x.cuda()
        self.kv_len = torch.tensor(totals, dtype=torch.int32, device="cuda")
        self.parts = parts
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.cache = lsa.KvCache(page_table=self.table_dev, kv_len=self.kv_len, **parts)

    def decode(self):
        """The cache as it is now, as float64 values, NaN where a slot is unused."""
        for name in ("k", "v"):
            if self.dtype == "fp8":
                codes = self.parts[name].view(self.torch.uint8).cpu().numpy()
                self.decoded[name] = K.e4m3_values()[codes] * self.parts[name + "_scale"].cpu().numpy().astype(np.float64)[:, :, None, None]
            else:
                self.decoded[name] = self.parts[name].cpu().double().numpy()


def bf16(torch, g, shape, amp=1.0):
    return torch.from_numpy(g.normal(size=shape) * amp).to(torch.bfloat16).cuda()


def offsets(news, base=0):
    off = np.zeros(len(news) + 1, np.int64)
    off[1:] = np.cumsum(news)
    return off + base


def check_rows(s, q, out, lse, rows, scale, window=0, sinks=0, listed=None, entry_tokens=1, n_q=None, tag=""):
    """rows: (row, sequence, position) triples to compare with the oracle."""
    G = n_q // s.n_kv
    got, got_l, qq = out.cpu().double().numpy(), lse.cpu().double().numpy(), q.cpu().double().numpy()
    cached = {}
    for r, b, p in rows:
        n = max(p + 1, 0)
        for h in range(s.n_kv):
            if (b, h) not in cached:
                t = max(s.totals[b], 0)
                cached[b, h] = [K.rows_of(s.decoded[x], s.table[b], t, h) for x in ("k", "v")]
            (Kc, there), (Vc, _) = cached[b, h]
            see = K.visible(p, len(Kc), window, sinks, None if listed is None else listed[b], entry_tokens) & there
            for i in range(G):
                head = h * G + i
                o, l, A, big = K.attend_row(qq[r, head], Kc, Vc, see, scale)
                dx = 2 * (s.d + 4) * 2.0 ** -24 * big + 2.0 ** -22 * (big if np.isfinite(l) else 0)
                n = int(see.sum())
                tol = (U + 4 * dx + n * 2.0 ** -24 + 2.0 ** -16) * A + U * np.abs(o) + 1e-30
                where = f"{tag} row {r} seq {b} pos {p} head {head}"
                with np.errstate(invalid="ignore"):
                    same = (np.isnan(o) & np.isnan(got[r, head])) | (o == got[r, head]) | (np.abs(got[r, head] - o) <= tol)
                assert same.all(), (where, np.abs(got[r, head] - o).max(), o[:4], got[r, head][:4])
                if np.isinf(l):
                    assert got_l[r, head] == l, (where, got_l[r, head])
                elif np.isfinite(l):
                    assert abs(got_l[r, head] - l) <= 2 * dx + n * 2.0 ** -24 + 2.0 ** -20 * (1 + abs(l)), (where, got_l[r, head], l)


def run_attend(torch, lsa, s, q, off, *, window=0, sinks=0, scale=None, out=None, ws=None, max_len=None):
    n_q = q.shape[1]
    scale = scale if scale is not None else s.d ** -0.5
    out = torch.full(q.shape, -7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((q.shape[0], n_q), -7.0, device="cuda")
    max_len = max(max(s.totals), 0) if max_len is None else max_len
    if ws is None:
        size = lsa.attend_workspace_size(s.cache, n_q=n_q, q_offsets_host=off, max_kv_len=max_len, window=window, sinks=sinks)
        ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    lsa.attend(s.cache, q, q_offsets=torch.from_numpy(off).cuda(), q_offsets_host=off, max_kv_len=max_len, out=out, lse=lse,
               scale=scale, window=window, sinks=sinks, workspace=ws)
    return out, lse


# (name, dtype, n_q, n_kv, d, page, [(new, total)], window, sinks)
ATTEND = [
    ("one_token", "bf16", 4, 2, 64, 16, [(1, 1)], 0, 0),
    ("one_token_fp8", "fp8", 8, 1, 128, 64, [(1, 1)], 0, 0),
    ("decode", "bf16", 8, 2, 128, 64, [(1, 33), (1, 32), (1, 31), (1, 700), (1, 64), (1, 65)], 0, 0),
    ("decode_fp8", "fp8", 64, 8, 128, 64, [(1, 257), (1, 1000), (1, 16)], 0, 0),
    ("decode_fp8_d64", "fp8", 16, 4, 64, 128, [(1, 129), (1, 511), (1, 5)], 0, 0),
    ("decode_mqa", "bf16", 40, 1, 64, 32, [(1, 300), (1, 47)], 0, 0),
    ("decode_mqa_fp8", "fp8", 64, 1, 128, 16, [(1, 300), (1, 47)], 0, 0),
    ("decode_mha", "fp8", 5, 5, 64, 16, [(1, 100), (1, 3)], 0, 0),
    ("empty_ones", "bf16", 6, 2, 64, 16, [(0, 40), (1, 0), (2, 1), (3, 3), (0, 0), (1, 50)], 0, 0),
    ("empty_ones_fp8", "fp8", 6, 2, 128, 16, [(0, 40), (1, 0), (2, 1), (3, 3), (0, 0), (1, 50)], 0, 0),
    ("few_tokens", "fp8", 12, 4, 128, 32, [(4, 200), (2, 2), (5, 77)], 0, 0),
    ("chunk", "fp8", 8, 2, 128, 64, [(70, 300), (33, 33), (1, 500)], 0, 0),
    ("chunk_bf16", "bf16", 8, 2, 128, 64, [(70, 300), (33, 33), (1, 500)], 0, 0),
    ("prompt", "bf16", 4, 2, 64, 16, [(200, 200), (131, 131)], 0, 0),
    ("prompt_fp8", "fp8", 7, 1, 64, 128, [(150, 150), (97, 120)], 0, 0),
    ("prompt_long", "bf16", 8, 1, 128, 32, [(600, 600)], 0, 0),
    ("window_decode", "bf16", 8, 2, 128, 16, [(1, 300), (1, 20), (1, 129), (1, 128)], 100, 4),
    ("window_decode_fp8", "fp8", 8, 2, 64, 64, [(1, 300), (1, 20), (1, 129), (1, 128)], 64, 40),
    ("window_one", "fp8", 4, 1, 128, 16, [(1, 90), (3, 64)], 1, 0),
    ("window_prompt", "bf16", 4, 2, 128, 32, [(190, 190), (65, 300)], 50, 3),
    ("window_prompt_fp8", "fp8", 4, 2, 128, 16, [(190, 190), (65, 300)], 33, 33),
    ("many_chunks", "bf16", 8, 1, 64, 16, [(9 + i % 3 if i % 4 else 0, 20 + i % 60) for i in range(70)], 0, 0),
    ("group_beyond_a_block", "fp8", 300, 1, 64, 16, [(2, 70), (1, 33)], 0, 0),
    ("one_token_many_heads", "bf16", 100, 1, 128, 64, [(1, 500), (1, 1)], 0, 0),
    ("many_sequences", "fp8", 4, 2, 64, 16, [(i % 3 != 1, 1 + (i * 197) % 900) for i in range(150)], 0, 0),
    ("many_equal", "bf16", 4, 4, 64, 16, [(1, 400)] * 70, 0, 0),
    ("one_long_of_many", "fp8", 2, 1, 64, 64, [(1, 3)] * 66 + [(2, 9000), (1, 40)], 0, 0),
    ("window_many", "bf16", 2, 1, 64, 16, [(1, 300)] * 65, 200, 7),
    ("window_longer", "bf16", 4, 2, 64, 16, [(20, 60), (1, 9)], 500, 5),
    ("more_queries_than_keys", "bf16", 4, 2, 64, 16, [(100, 60), (90, 0), (80, 1)], 0, 0),
    ("more_queries_than_keys_fp8", "fp8", 8, 1, 128, 64, [(400, 190), (20, 3), (6, 1)], 30, 2),
]


@pytest.mark.parametrize("case", ATTEND, ids=[c[0] for c in ATTEND])
def test_attend(torch, lsa, case):
    name, dtype, n_q, n_kv, d, pt, seqs, window, sinks = case
    say(f"[attend] {name}")
    s = Setup(torch, lsa, [t for _, t in seqs], dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=len(name))
    off = offsets([n for n, _ in seqs], base=3)
    rows = int(off[-1]) + 2
    # rows of a wider projection, and rows before and behind the sequences
    wide = bf16(torch, s.g, (rows, n_q + 2, d))
    q = wide[:, 1:1 + n_q]
    out_wide = torch.full((rows, n_q + 1, d), -7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = run_attend(torch, lsa, s, q, off, window=window, sinks=sinks, out=out_wide[:, :n_q])
    torch.cuda.synchronize()
    assert bool((out_wide[:, n_q] == -7).all()) and bool((out_wide[:3] == -7).all()) and bool((out_wide[rows - 2:] == -7).all())
    assert bool((lse[:3] == -7).all()) and bool((lse[rows - 2:] == -7).all())
    triples = [(int(off[b]) + i, b, t - n + i) for b, (n, t) in enumerate(seqs) for i in range(n)]
    if len(triples) > 60:
        triples = triples[:20] + [triples[i] for i in s.g.choice(len(triples), 30, replace=False)] + triples[-10:]
    check_rows(s, q, out, lse, triples, d ** -0.5, window, sinks, n_q=n_q, tag=name)
    again, lse2 = run_attend(torch, lsa, s, q, off, window=window, sinks=sinks)
    a, b = int(off[0]), int(off[-1])
    assert torch.equal(out[a:b], again[a:b]) and torch.equal(lse[a:b], lse2[a:b]), "two calls differ"


@pytest.mark.parametrize("dtype,window", [("bf16", 0), ("fp8", 0), ("bf16", 40), ("fp8", 40)])
@pytest.mark.parametrize("news", [(3,), (70,), (400,)], ids=["few", "some", "many"])
def test_attend_values_that_are_not_finite(torch, lsa, dtype, window, news):
    # a token's NaN or infinite value reaches the rows that see it, and no other
    say(f"[attend] not finite {dtype} window {window} new {news}")
    n = news[0]
    total = n + 37
    s = Setup(torch, lsa, [total], dtype=dtype, n_kv=1, d=64, pt=16, seed=n)
    for pos, bad in ((total - 2, float("nan")), (total // 2, float("inf")), (total - n, float("-inf"))):
        page, slot = int(s.table[0, pos // 16]), pos % 16
        for name in ("k", "v"):
            x = s.parts[name][page, 0, slot]
            if dtype == "fp8":
                x.view(torch.uint8)[5] = 0x7F if bad > 0 else 0xFF
            elif name == "v":
                x[5] = bad
            else:
                x[5] = float("nan")
    s.decode()
    off = offsets([n])
    q = bf16(torch, s.g, (n, 4, 64))
    out, lse = run_attend(torch, lsa, s, q, off, window=window, sinks=2 if window else 0)
    torch.cuda.synchronize()
    rows = sorted(set([0, 1, n // 2, n - 3, n - 2, n - 1] + list(range(0, n, 13))))
    # keys are NaN at those positions too: rows that see one are NaN in both
    for r in rows:
        p = total - n + r
        see = K.visible(p, total, window, 2 if window else 0)
        bad = any(see[x] for x in (total - 2, total // 2, total - n))
        assert bool(torch.isnan(out[r]).all()) == bad, (r, p)
    check_rows(s, q, out, lse, [(r, 0, total - n + r) for r in rows if not np.isnan(out[r].cpu().double().numpy()).any()],
               64 ** -0.5, window, 2 if window else 0, n_q=4)
    # values alone: infinities keep their sign in the dimension they stand in
    for pos in (total - 2, total // 2, total - n):
        page, slot = int(s.table[0, pos // 16]), pos % 16
        x = s.parts["k"][page, 0, slot]
        (x.view(torch.uint8) if dtype == "fp8" else x)[5] = 0
    s.decode()
    out, lse = run_attend(torch, lsa, s, q, off, window=window, sinks=2 if window else 0)
    torch.cuda.synchronize()
    got = out.cpu().double().numpy()
    for r in rows:
        p = total - n + r
        see = K.visible(p, total, window, 2 if window else 0)
        hit = [x for x in (total - 2, total // 2, total - n) if see[x]]
        assert np.isfinite(np.delete(got[r], 5, axis=-1)).all(), (r, p)
        assert np.isfinite(got[r][:, 5]).all() == (not hit), (r, p, hit)
        if dtype == "bf16" and hit == [total // 2]:
            assert (got[r][:, 5] == np.inf).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,total", [(1, 3000), (100, 3000), (1, 460)])
def test_attend_infinite_values_in_split_rows(torch, lsa, n, total, d):
    # an infinite value in the first and in the last part of rows that are worked on in parts
    s = Setup(torch, lsa, [total], dtype="bf16", n_kv=1, d=d, pt=16, seed=d + n)
    for pos, dim, bad in ((0, 3, float("inf")), (total - n, 9, float("-inf"))):
        s.parts["v"][int(s.table[0, pos // 16]), 0, pos % 16, dim] = bad
    s.decode()
    off = offsets([n])
    q = bf16(torch, s.g, (n, 2, d), 0.1)  # close scores: no probability is 0
    assert lsa.attend_workspace_size(s.cache, n_q=2, q_offsets_host=off, max_kv_len=total) > 0
    out, lse = run_attend(torch, lsa, s, q, off)
    torch.cuda.synchronize()
    assert bool((out[..., 3] == float("inf")).all()) and bool((out[..., 9] == float("-inf")).all())
    check_rows(s, q, out, lse, [(r, 0, total - n + r) for r in sorted({0, n // 2, n - 1})], d ** -0.5, n_q=2)


def test_attend_pages_that_are_not_there(torch, lsa):
    for dtype in ("bf16", "fp8"):
        say(f"[attend] bad pages {dtype}")
        s = Setup(torch, lsa, [200, 90, 64], dtype=dtype, n_kv=2, d=64, pt=16, seed=3)
        s.table[0, 2], s.table[0, 7], s.table[1, 5], s.table[2, :4] = -1, 10 ** 6, -5, 2 ** 31 - 1
        s.table_dev.copy_(torch.from_numpy(s.table))
        off = offsets([3, 1, 2])
        q = bf16(torch, s.g, (6, 4, 64))
        out, lse = run_attend(torch, lsa, s, q, off)
        torch.cuda.synchronize()
        rows = [(0, 0, 197), (1, 0, 198), (2, 0, 199), (3, 1, 89), (4, 2, 62), (5, 2, 63)]
        check_rows(s, q, out, lse, rows, 64 ** -0.5, n_q=4)
        assert bool((out[4:] == 0).all()) and bool(torch.isneginf(lse[4:]).all())


def test_attend_length_beyond_the_bound(torch, lsa):
    # a kv_len beyond max_kv_len counts as it, and a negative one as 0
    s = Setup(torch, lsa, [100, 60], dtype="bf16", n_kv=1, d=64, pt=16, seed=4)
    q = bf16(torch, s.g, (2, 2, 64))
    s.kv_len.copy_(torch.tensor([2 ** 30, -9], dtype=torch.int32))
    out, lse = run_attend(torch, lsa, s, q, offsets([1, 1]), max_len=70)
    torch.cuda.synchronize()
    check_rows(s, q, out, lse, [(0, 0, 69)], 64 ** -0.5, n_q=2)
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())


@pytest.mark.parametrize("n", [40, 300])
def test_attend_largest_window(torch, lsa, n):
    # rows far before the first cached token, and a window whose start before them passes 32 bits
    s = Setup(torch, lsa, [30], dtype="bf16", n_kv=1, d=64, pt=128, seed=n)
    pages = (2 ** 31 - 128) // 128
    s.table_dev = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    s.table_dev[:, :s.table.shape[1]] = torch.from_numpy(s.table).cuda()
    s.cache = lsa.KvCache(page_table=s.table_dev, kv_len=s.kv_len, **s.parts)
    q = bf16(torch, s.g, (n, 1, 64))
    out, lse = run_attend(torch, lsa, s, q, offsets([n]), window=2 ** 31 - 129, max_len=2 ** 31 - 128)
    torch.cuda.synchronize()
    check_rows(s, q, out, lse, [(i, 0, 30 - n + i) for i in range(n - 33, n)], 64 ** -0.5, n_q=1)
    assert bool((out[:n - 30] == 0).all()) and bool(torch.isneginf(lse[:n - 30]).all())


@pytest.mark.parametrize("n", [2, 200])
@pytest.mark.parametrize("scale", [0.0, 30.0, -1.0])
def test_attend_scores_far_apart(torch, lsa, scale, n):
    # scores that grow along the keys by far more than the lazy maximum's slack, and the reverse
    say(f"[attend] far scores {scale}")
    s = Setup(torch, lsa, [333], dtype="bf16", n_kv=1, d=64, pt=32, seed=5)
    ramp = torch.linspace(-1, 1, 333 + 19, device="cuda")
    for p in range(333):
        s.parts["k"][int(s.table[0, p // 32]), 0, p % 32] = ramp[p].to(torch.bfloat16)
    s.decode()
    q = torch.ones((n, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[:, 1] = -1
    out, lse = run_attend(torch, lsa, s, q, offsets([n]), scale=scale)
    torch.cuda.synchronize()
    check_rows(s, q, out, lse, [(r, 0, 333 - n + r) for r in sorted({0, 1, n // 2, n - 1})], scale, n_q=2)


@pytest.mark.parametrize("amp", [1.37, 2.0 ** -110, 3 * 2.0 ** 90])
@pytest.mark.parametrize("n", [1, 90])
def test_attend_scales_of_any_size(torch, lsa, amp, n):
    # page scales that are no power of two, and far from 1 (values only: scores have to stay finite)
    say(f"[attend] scales {amp} rows {n}")
    s = Setup(torch, lsa, [200, 130], dtype="fp8", n_kv=2, d=64, pt=16, seed=6)
    rest = torch.from_numpy(s.g.uniform(0.6, 1.9, s.scales["k"].shape).astype(np.float32)).cuda()
    s.parts["k_scale"] *= rest
    s.parts["v_scale"] *= rest.flip(0) * amp
    s.decode()
    off = offsets([n, n])
    q = bf16(torch, s.g, (2 * n, 4, 64))
    out, lse = run_attend(torch, lsa, s, q, off)
    torch.cuda.synchronize()
    rows = [(b * n + i, b, s.totals[b] - n + i) for b in range(2) for i in sorted({0, n // 2, n - 1})]
    check_rows(s, q, out, lse, rows, 64 ** -0.5, n_q=4)


def test_cache_beyond_32_bit_offsets(torch, lsa):
    """The same contents in a small cache and in the last pages of one of 4.7 GB a side give the same bits."""
    say("[kv] long cache")
    n_kv, d, pt, totals = 2, 128, 64, [300, 90]
    inv = torch.from_numpy((10000.0 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32)).cuda()
    for news in ([1, 1], [70, 40]):
        s = Setup(torch, lsa, totals, dtype="bf16", n_kv=n_kv, d=d, pt=pt, seed=15)
        n = s.parts["k"].shape[0]
        big = {x: torch.empty((145_000, n_kv, pt, d), dtype=torch.bfloat16, device="cuda") for x in ("k", "v")}
        assert big["k"].nbytes > 1 << 32
        shift = 145_000 - n
        for x in big:
            big[x][shift:] = s.parts[x]
        table = s.table_dev.clone()
        table[table >= 0] += shift
        far = lsa.KvCache(k=big["k"], v=big["v"], page_table=table, kv_len=s.kv_len)
        off = offsets(news)
        off_dev = torch.from_numpy(off).cuda()
        T = int(off[-1])
        qkv = bf16(torch, s.g, (T, 8 + 2 * n_kv, d))
        idx = torch.arange(0, 80, 2, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
        count = torch.tensor([40, 20], dtype=torch.int32, device="cuda")
        got = []
        for cache in (s.cache, far):
            q = torch.empty((T, 8, d), dtype=torch.bfloat16, device="cuda")
            lsa.kv_append(cache, qkv[:, 8:8 + n_kv], qkv[:, 8 + n_kv:], new_offsets=off_dev, new_offsets_host=off,
                          q=qkv[:, :8], q_out=q, inv_freq=inv)
            size = max(lsa.attend_workspace_size(cache, n_q=8, q_offsets_host=off, max_kv_len=300),
                       lsa.attend_topk_workspace_size(cache, n_q=8, k=40, entry_tokens=2, window=5))
            ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
            out, top = torch.empty_like(q), torch.empty_like(q[:2])
            lsa.attend(cache, q, q_offsets=off_dev, q_offsets_host=off, max_kv_len=300, out=out, scale=0.1, workspace=ws)
            lsa.attend_topk(cache, q[:2], idx=idx, count=count, out=top, scale=0.1, entry_tokens=2, window=5, workspace=ws)
            torch.cuda.synchronize()
            got.append((q, out, top))
        for a, b in zip(*got):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())
        for x in big:
            assert torch.equal(big[x][shift:].view(torch.int16), s.parts[x].view(torch.int16))
        del big, far
        torch.cuda.empty_cache()


def test_attend_without_lse_and_on_a_given_stream(torch, lsa):
    say("[attend] no lse, own stream")
    s = Setup(torch, lsa, [500, 700], dtype="fp8", n_kv=2, d=64, pt=16, seed=16)
    off = offsets([1, 80])
    q = bf16(torch, s.g, (81, 4, 64))
    want, _ = run_attend(torch, lsa, s, q, off)
    out = torch.zeros_like(q)
    ws = torch.empty(lsa.attend_workspace_size(s.cache, n_q=4, q_offsets_host=off, max_kv_len=700), dtype=torch.uint8, device="cuda")
    off_dev = torch.from_numpy(off).cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    lsa.attend(s.cache, q, q_offsets=off_dev, q_offsets_host=off.tolist(), max_kv_len=700, out=out, scale=0.125, workspace=ws,
               stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# (name, dtype, n_q, n_kv, d, page, lens, k, entry, window, sinks)
TOPK = [
    ("small", "bf16", 4, 2, 64, 16, [1, 5, 100], 8, 1, 0, 0),
    ("all_listed", "fp8", 8, 1, 128, 64, [60, 30], 64, 1, 0, 0),
    ("entries", "fp8", 8, 2, 128, 16, [400, 333, 3], 40, 4, 17, 5),
    ("entries_odd", "bf16", 12, 4, 64, 32, [400, 333, 3], 30, 3, 0, 33),
    ("mqa", "bf16", 64, 1, 128, 64, [1000, 700], 200, 2, 128, 4),
    ("mqa_fp8", "fp8", 40, 1, 64, 128, [1000, 700], 300, 1, 1, 0),
    ("many", "fp8", 16, 2, 128, 64, [3001, 2000, 64, 0], 700, 1, 100, 4),
    ("many_sequences", "fp8", 16, 8, 64, 16, [1 + (i * 131) % 500 for i in range(90)], 150, 1, 20, 2),
    ("heads_beyond_a_block", "bf16", 100, 1, 64, 16, [300, 77, 0], 120, 1, 20, 2),
    ("window_over_all", "bf16", 4, 1, 64, 16, [50], 20, 1, 1000, 1000),
]


@pytest.mark.parametrize("case", TOPK, ids=[c[0] for c in TOPK])
def test_attend_topk(torch, lsa, case):
    name, dtype, n_q, n_kv, d, pt, lens, k, r, window, sinks = case
    say(f"[attend_topk] {name}")
    s = Setup(torch, lsa, lens, dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=len(name) + 7)
    B = len(lens)
    idx, count, listed = np.full((B, k), -1, np.int32), np.zeros(B, np.int32), []
    for b, t in enumerate(lens):
        entries = -(-t // r)
        some = np.sort(s.g.choice(entries, min(k - 2, entries), replace=False)).astype(np.int32) if entries else np.zeros(0, np.int32)
        if b == 0 and some.size > 2:
            some = np.sort(np.concatenate([some, some[1:2]]))  # one entry twice
        if b == 1:
            some = np.concatenate([some, np.array([entries + 3], np.int32)])  # behind the sequence
        idx[b, :some.size], count[b] = some, some.size
        listed.append(some.tolist())
    if name == "small":
        idx[2, 0], listed[2] = -1, listed[2][1:]
    q = bf16(torch, s.g, (B, n_q, d))
    out = torch.full((B, n_q, d), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, n_q), -7.0, device="cuda")
    size = lsa.attend_topk_workspace_size(s.cache, n_q=n_q, k=k, entry_tokens=r, window=window, sinks=sinks)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    args = dict(idx=torch.from_numpy(idx).cuda(), count=torch.from_numpy(count).cuda(), scale=d ** -0.5, entry_tokens=r,
                window=window, sinks=sinks, workspace=ws)
    lsa.attend_topk(s.cache, q, out=out, lse=lse, **args)
    torch.cuda.synchronize()
    check_rows(s, q, out, lse, [(b, b, t - 1) for b, t in enumerate(lens)], d ** -0.5, window, sinks, listed, r, n_q, name)
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    lsa.attend_topk(s.cache, q, out=out2, lse=lse2, **args)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


# (name, dtype, n_q, n_kv, d, page, [(new, total)], rope, rot)
APPEND = [
    ("token", "bf16", 8, 2, 64, 16, [(1, 1), (1, 17), (1, 16), (1, 900)], "halves", 64),
    ("token_fp8", "fp8", 8, 2, 128, 64, [(1, 1), (1, 65), (1, 64), (1, 900)], "halves", 128),
    ("pairs", "bf16", 4, 4, 128, 32, [(1, 10), (40, 73), (0, 5)], "pairs", 64),
    ("pairs_fp8", "fp8", 5, 1, 64, 32, [(1, 10), (40, 73), (0, 5)], "pairs", 48),
    ("prompt", "bf16", 16, 2, 128, 128, [(300, 300), (129, 200)], "halves", 96),
    ("prompt_fp8", "fp8", 16, 2, 128, 128, [(300, 300), (129, 200)], "halves", 96),
    ("prompt_fp8_d64", "fp8", 3, 3, 64, 128, [(300, 333), (1, 128)], "halves", 16),
    ("plain_fp8", "fp8", 0, 2, 64, 16, [(30, 47), (5, 5)], None, 0),
    ("many_sequences", "fp8", 3, 1, 64, 16, [(i % 4, 5 + (i * 37) % 200) for i in range(140)], "pairs", 32),
    ("more_new_than_cached", "fp8", 2, 1, 64, 16, [(20, 13), (3, 0), (2, 1)], "halves", 64),
    ("long", "bf16", 18, 6, 64, 16, [(1500, 1600), (700, 700), (3, 60)], "halves", 64),
    ("long_fp8", "fp8", 10, 10, 128, 16, [(900, 933), (0, 20), (801, 801)], "pairs", 112),
    ("many_of_one", "bf16", 1, 1, 64, 16, [(i % 2, 1 + i % 40) for i in range(1200)], "halves", 32),
]


@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_append(torch, lsa, case):
    """bf16: half a step of the exact value, and 2^-20 of the pair's length for angle, sine and products in fp32.
    e4m3: half a step (2^-4 relative, 2^-10 absolute in units of the scale) and the same 2^-20."""
    name, dtype, n_q, n_kv, d, pt, seqs, rope, rot = case
    say(f"[append] {name}")
    s = Setup(torch, lsa, [t for _, t in seqs], dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=len(name) + 20)
    off = offsets([n for n, _ in seqs], base=2)
    rows = int(off[-1]) + 1
    qkv = bf16(torch, s.g, (rows, n_q + 2 * n_kv, d))
    qkv[2:] *= torch.logspace(-3, 3, rows - 2, device="cuda").to(torch.bfloat16)[:, None, None]  # scales that grow
    q, k_new, v_new = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    q_out = torch.full((rows, max(n_q, 1), d), -7.0, dtype=torch.bfloat16, device="cuda") if n_q else None
    inv = (10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))).astype(np.float32)
    before = {n: x.clone() for n, x in s.parts.items()}
    lsa.kv_append(s.cache, k_new, v_new, new_offsets=torch.from_numpy(off).cuda(), new_offsets_host=off,
                  q=q if n_q else None, q_out=q_out, inv_freq=torch.from_numpy(inv).cuda() if rope else None,
                  rope=rope)
    torch.cuda.synchronize()
    pos = np.zeros(rows)
    for b, (n, t) in enumerate(seqs):
        pos[off[b]:off[b] + n] = np.arange(t - n, t)
    x = {"q": q.cpu().double().numpy(), "k": k_new.cpu().double().numpy(), "v": v_new.cpu().double().numpy()}
    want = {n: (K.rotate(x[n], pos, inv, rope) if rope and n != "v" else x[n]) for n in x}
    if n_q:
        got = q_out.cpu().double().numpy()
        assert (got[:2] == -7).all() and (got[rows - 1:] == -7).all()
        mid = slice(2, rows - 1)
        size = np.abs(x["q"][mid]).max(-1, keepdims=True) * 1.5
        assert (np.abs(got[mid] - want["q"][mid]) <= U * np.abs(want["q"][mid]) + 2.0 ** -20 * size).all()
    for c in ("k", "v"):
        now, was = s.parts[c], before[c]
        values = (K.e4m3_values()[was.view(torch.uint8).cpu().numpy()] if dtype == "fp8" else was.cpu().double().numpy())
        got = (K.e4m3_values()[now.view(torch.uint8).cpu().numpy()] if dtype == "fp8" else now.cpu().double().numpy())
        touched = np.zeros(values.shape[:1] + values.shape[2:3], bool)
        scale = before[c + "_scale"].cpu().numpy().astype(np.float64) if dtype == "fp8" else None
        size = np.zeros(values.shape[:3])
        for b, (n, t) in enumerate(seqs):
            new = want[c][off[b]:off[b] + n]
            if dtype == "fp8":
                values, scale = K.append_fp8(values, scale, s.table[b], t - n, new)
            for i in range(n):
                p = t - n + i
                if p < 0:
                    continue
                page = s.table[b, p // pt]
                touched[page, p % pt] = True
                if dtype == "bf16":
                    values[page, :, p % pt] = new[i]
                size[page, :, p % pt] = np.abs(x[c][off[b] + i]).max(-1) * 1.5
        if dtype == "fp8":
            have = s.parts[c + "_scale"].cpu().numpy().astype(np.float64)
            assert np.array_equal(have, scale, equal_nan=True), (name, c, have.ravel()[:8], scale.ravel()[:8])
            step = np.maximum(np.abs(values) * 2.0 ** -4, 2.0 ** -10) + 2.0 ** -20 * size[..., None] / scale[:, :, None, None]
        else:
            step = np.abs(values) * U + 2.0 ** -20 * size[..., None]
        with np.errstate(invalid="ignore"):
            ok = (np.isnan(values) & np.isnan(got)) | (np.abs(got - values) <= step)
        assert ok.all(), (name, c, np.argwhere(~ok)[:4], got[~ok][:4], values[~ok][:4])
        # slots that no new token took keep their bits, but for earlier tokens of a page whose scale grew
        same = (now.view(torch.uint8) == was.view(torch.uint8)).view(*now.shape[:3], -1).all(-1).cpu().numpy()
        grown = np.zeros(same.shape[:2], bool) if dtype == "bf16" else ~(have <= before[c + "_scale"].cpu().numpy())
        free = ~touched[:, None, :] & (~grown[:, :, None] | ~s.used[:, None, :])
        assert same[np.broadcast_to(free, same.shape)].all(), (name, c)


def test_append_far_positions_and_given_ones(torch, lsa):
    # positions near 2^31 turn as exactly as near ones, and `positions` only replaces the angle's
    say("[append] far positions")
    s = Setup(torch, lsa, [40], dtype="bf16", n_kv=1, d=64, pt=16, seed=9)
    pos = np.array([0, 1, 12345, 999_999, 2 ** 24 + 1, 2 ** 31 - 1], np.int32)
    off = offsets([6])
    k, v = bf16(torch, s.g, (6, 1, 64)), bf16(torch, s.g, (6, 1, 64))
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    q_out = torch.empty_like(k)
    lsa.kv_append(s.cache, k, v, new_offsets=torch.from_numpy(off).cuda(), new_offsets_host=off, q=k, q_out=q_out,
                  inv_freq=torch.from_numpy(inv).cuda(), positions=torch.from_numpy(pos).cuda())
    torch.cuda.synchronize()
    x = k.cpu().double().numpy()
    want = K.rotate(x, pos.astype(np.float64), inv, "halves")
    got = q_out.cpu().double().numpy()
    assert (np.abs(got - want) <= U * np.abs(want) + 2.0 ** -20 * 5).all()
    for i in range(6):
        p = 34 + i
        assert torch.equal(s.parts["k"][int(s.table[0, p // 16]), :, p % 16], q_out[i])
        assert torch.equal(s.parts["v"][int(s.table[0, p // 16]), :, p % 16], v[i])


def test_append_in_place_query_and_bad_pages(torch, lsa):
    say("[append] bad pages")
    s = Setup(torch, lsa, [40, 70], dtype="fp8", n_kv=2, d=64, pt=16, seed=10)
    before = {n: x.clone() for n, x in s.parts.items()}
    s.table[0, 2], s.table[1, 4] = -1, s.parts["k"].shape[0]
    s.table_dev.copy_(torch.from_numpy(s.table))
    s.kv_len.copy_(torch.tensor([40, 10 ** 6], dtype=torch.int32))  # the second lies behind its table
    off = offsets([8, 3])
    q = bf16(torch, s.g, (11, 4, 64))
    k, v = bf16(torch, s.g, (11, 2, 64)), bf16(torch, s.g, (11, 2, 64))
    inv = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    pos = np.array(list(range(32, 40)) + list(range(10 ** 6 - 3, 10 ** 6)))
    want = K.rotate(q.cpu().double().numpy(), pos.astype(np.float64), inv, "halves")
    lsa.kv_append(s.cache, k, v, new_offsets=torch.from_numpy(off).cuda(), new_offsets_host=off, q=q, q_out=q,
                  inv_freq=torch.from_numpy(inv).cuda())
    torch.cuda.synchronize()
    assert (np.abs(q.cpu().double().numpy() - want) <= U * np.abs(want) + 2.0 ** -20 * 8).all()
    for n, x in s.parts.items():
        assert torch.equal(x.view(torch.uint8), before[n].view(torch.uint8)), n


def test_append_not_finite(torch, lsa):
    # NaN and infinities are stored as they are in bf16 and as NaN in e4m3, and do not set a scale
    say("[append] not finite")
    for dtype in ("bf16", "fp8"):
        s = Setup(torch, lsa, [3], dtype=dtype, n_kv=1, d=64, pt=16, seed=11)
        k = torch.ones((3, 1, 64), dtype=torch.bfloat16, device="cuda")
        k[1, 0, 3], k[2, 0, 7], k[2, 0, 8] = float("inf"), float("nan"), float("-inf")
        off = offsets([3])
        lsa.kv_append(s.cache, k, k, new_offsets=torch.from_numpy(off).cuda(), new_offsets_host=off)
        torch.cuda.synchronize()
        page = int(s.table[0, 0])
        for n in ("k", "v"):
            x = s.parts[n][page, 0, :3].float().cpu()
            if dtype == "bf16":
                assert torch.equal(x[~x.isnan()], k[:, 0].float().cpu()[~x.isnan()]) and int(x.isnan().sum()) == 1
            else:
                assert float(s.parts[n + "_scale"][page, 0]) == 2.0 ** -8
                bad = ~torch.isfinite(k[:, 0].float().cpu())
                assert torch.equal(x.isnan(), bad) and bool((x[~bad] == 256).all())


def test_append_then_attend_as_a_model_would(torch, lsa):
    """A prompt and decode steps through append and attend agree with one attention over everything: the run of
    the operators together, against the oracle over the cache as stored."""
    for dtype in ("bf16", "fp8"):
        say(f"[kv] prompt and steps {dtype}")
        n_q, n_kv, d, pt, prompt, steps = 8, 2, 64, 16, [37, 50, 1], 20
        s = Setup(torch, lsa, [p + steps for p in prompt], dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=12)
        inv = torch.from_numpy((10000.0 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32)).cuda()
        now = list(prompt)
        for step in range(steps + 1):
            news = prompt if step == 0 else [1] * 3
            if step:
                now = [n + 1 for n in now]
            s.kv_len.copy_(torch.tensor(now, dtype=torch.int32))
            s.totals = list(now)  # the bound of the lengths that run_attend passes
            off = offsets(news)
            qkv = bf16(torch, s.g, (int(off[-1]), n_q + 2 * n_kv, d))
            q = torch.empty((int(off[-1]), n_q, d), dtype=torch.bfloat16, device="cuda")
            lsa.kv_append(s.cache, qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:], new_offsets=torch.from_numpy(off).cuda(),
                          new_offsets_host=off, q=qkv[:, :n_q], q_out=q, inv_freq=inv)
            window, sinks = (24, 2) if step % 3 == 2 else (0, 0)
            out, lse = run_attend(torch, lsa, s, q, off, window=window, sinks=sinks)
            torch.cuda.synchronize()
            s.decode()
            rows = [(int(off[b]) + i, b, now[b] - n + i) for b, n in enumerate(news) for i in range(n)]
            check_rows(s, q, out, lse, rows, d ** -0.5, window, sinks, n_q=n_q, tag=f"{dtype} step {step}")


def test_captured_step_follows_lengths(torch, lsa):
    """One captured append + attend + attend_topk, replayed while kv_len grows, with eager work between."""
    say("[kv] captured step")
    n_q, n_kv, d, pt = 8, 1, 128, 16
    s = Setup(torch, lsa, [90, 300], dtype="fp8", n_kv=n_kv, d=d, pt=pt, seed=13)
    off = offsets([1, 1])
    off_dev = torch.from_numpy(off).cuda()
    qkv = bf16(torch, s.g, (2, n_q + 2 * n_kv, d))
    inv = torch.from_numpy((10000.0 ** (-np.arange(d // 2) * 2.0 / d)).astype(np.float32)).cuda()
    k = 32
    idx = torch.arange(0, 64, 2, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    count = torch.tensor([20, 32], dtype=torch.int32, device="cuda")
    q = torch.empty((2, n_q, d), dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    size = max(lsa.attend_workspace_size(s.cache, n_q=n_q, q_offsets_host=off, max_kv_len=300),
               lsa.attend_topk_workspace_size(s.cache, n_q=n_q, k=k, entry_tokens=2, window=9, sinks=1))
    assert size > 0  # both calls split their keys here

    def step(outs, ws):
        lsa.kv_append(s.cache, qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:], new_offsets=off_dev, new_offsets_host=off,
                      q=qkv[:, :n_q], q_out=q, inv_freq=inv)
        lsa.attend(s.cache, q, q_offsets=off_dev, q_offsets_host=off, max_kv_len=300, out=outs[0], scale=d ** -0.5, workspace=ws)
        lsa.attend_topk(s.cache, q, idx=idx, count=count, out=outs[1], scale=d ** -0.5, entry_tokens=2, window=9, sinks=1,
                        workspace=ws)

    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    s.kv_len.copy_(torch.tensor([70, 280], dtype=torch.int32))
    step(outs, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs, ws)
    for t in range(6):
        s.kv_len.copy_(torch.tensor([71 + t, 281 + 3 * t], dtype=torch.int32))
        qkv.copy_(bf16(torch, s.g, qkv.shape))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        ws.fill_(0xFF)
        step(outs, ws)  # the same values again, eagerly
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b), f"replay {t}"


def test_two_streams(torch, lsa):
    # calls on two streams at once, each with its own workspace, give what they give alone
    say("[kv] two streams")
    s = Setup(torch, lsa, [700, 900], dtype="fp8", n_kv=2, d=128, pt=64, seed=14)
    off = offsets([1, 1])
    off_dev = torch.from_numpy(off).cuda()
    qs = [bf16(torch, s.g, (2, 8, 128)) for _ in range(2)]
    size = lsa.attend_workspace_size(s.cache, n_q=8, q_offsets_host=off, max_kv_len=900)
    wss = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(qs[0]) for _ in range(2)]

    def call(i, stream=None):
        lsa.attend(s.cache, qs[i], q_offsets=off_dev, q_offsets_host=off, max_kv_len=900, out=outs[i], scale=0.1,
                   workspace=wss[i], stream=stream)

    for i in range(2):
        call(i)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)
