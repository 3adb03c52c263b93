"""Large calls of the paged cache's attention (marked gpu), against the float64 oracle of test_gpu_kv.py, whose tolerances are
used as they are."""
import numpy as np
import pytest

from tests.parity import say
from tests.test_gpu_kv import Setup, bf16, check_rows, lsa, offsets, run_attend, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


class Shared:
    """A bf16 cache of one sequence's pages that several sequences read, as check_rows takes it."""

    def __init__(self, torch, lsa, totals, *, n_kv, d, pt, width, seed):
        g = self.g = np.random.default_rng(seed)
        self.n_kv, self.d, self.totals = n_kv, d, list(totals)
        pages = 40
        x = {n: torch.from_numpy(g.normal(size=(pages, n_kv, pt, d))).to(torch.bfloat16) for n in ("k", "v")}
        self.decoded = {n: y.double().numpy() for n, y in x.items()}
        self.table = np.tile(np.arange(width, dtype=np.int32) % pages, (len(totals), 1))
        self.kv_len = torch.tensor(totals, dtype=torch.int32, device="cuda")
        self.cache = lsa.KvCache(k=x["k"].cuda(), v=x["v"].cuda(), page_table=torch.from_numpy(self.table).cuda(),
                                 kv_len=self.kv_len)


def test_attend_more_rows_than_one_joining_launch(torch, lsa):
    """A prompt of 8,389,208 tokens and 40 decode rows behind it, 8 heads: 67,113,984 rows times heads. The decode
    rows are worked on in parts, and the launch that joins them takes 4 * (2^24 - 1) at a time: they are beyond."""
    say("[attend] many rows")
    n_kv, d, pt, window, tail = 8, 64, 128, 2048, 40
    prompt = (1 << 23) + 600
    decode = [3000 + 17 * i for i in range(tail)]
    s = Shared(torch, lsa, [prompt] + decode, n_kv=n_kv, d=d, pt=pt, width=-(-prompt // pt), seed=2)
    off = offsets([prompt] + [1] * tail)
    rows = int(off[-1])
    assert (prompt * n_kv) > 4 * (2 ** 24 - 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q = torch.empty((rows, n_kv, d), dtype=torch.bfloat16, device="cuda")
    for x in q.split(1 << 20):
        x.normal_(generator=g)
    out = torch.full_like(q, -7.0)
    lse = torch.full((rows, n_kv), -7.0, device="cuda")
    size = lsa.attend_workspace_size(s.cache, n_q=n_kv, q_offsets_host=off, max_kv_len=prompt, window=window)
    assert size > 0
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    lsa.attend(s.cache, q, q_offsets=torch.from_numpy(off).cuda(), q_offsets_host=off, max_kv_len=prompt, out=out, lse=lse,
               scale=d ** -0.5, window=window, workspace=ws)
    torch.cuda.synchronize()
    assert bool((lse != -7).all())
    # the decode rows, as a call of their own would number them
    at = prompt
    s.totals = decode
    s.table = s.table[1:, :-(-max(decode) // pt)]
    check_rows(s, q[at:], out[at:], lse[at:], [(i, i, decode[i] - 1) for i in (0, 1, 19, 38, 39)], d ** -0.5, window, n_q=n_kv)
    # and the prompt's first ones
    s.totals, s.table = [3000], s.table[:1]
    check_rows(s, q[:3000], out[:3000], lse[:3000], [(i, 0, i) for i in (0, 1, 2047, 2048, 2999)], d ** -0.5, window, n_q=n_kv)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (9, 2 ** 31 - 1)])
def test_topk_of_any_window(torch, lsa, window, sinks):
    # more sequences than windows of 2^31 - 1 could have tiles, and a table that ends after 300 tokens or so
    say(f"[attend_topk] window {window} sinks {sinks}")
    B, n_q, n_kv, d, pt, k = 70, 4, 2, 64, 16, 12
    lens = [(7 * b) % 300 for b in range(B)]
    s = Shared(torch, lsa, lens, n_kv=n_kv, d=d, pt=pt, width=19, seed=4)
    idx = np.sort(s.g.integers(0, 150, (B, k)).astype(np.int32), 1)
    listed = [sorted(set(x.tolist())) for x in idx]
    q = bf16(torch, s.g, (B, n_q, d))
    out, lse = torch.full_like(q, -7.0), torch.full((B, n_q), -7.0, device="cuda")
    size = lsa.attend_topk_workspace_size(s.cache, n_q=n_q, k=k, entry_tokens=2, window=window, sinks=sinks)
    ws = torch.full((max(size, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    lsa.attend_topk(s.cache, q, idx=torch.from_numpy(idx).cuda(), count=torch.full((B,), k, dtype=torch.int32, device="cuda"), out=out,
                    lse=lse, scale=d ** -0.5, entry_tokens=2, window=window, sinks=sinks, workspace=ws)
    torch.cuda.synchronize()
    check_rows(s, q, out, lse, [(b, b, lens[b] - 1) for b in range(B)], d ** -0.5, window, sinks, listed, 2, n_q)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("B", [64, 65, 200])
def test_parts_of_more_sequences_than_workers(torch, lsa, dtype, B):
    """8 key heads leave 64 workers a head (32 where rows fill a CU), so their shares end within sequences. The workspace has
    the size asked for, between bytes that have to stay."""
    say(f"[attend] {B} sequences {dtype}")
    n_q, n_kv, d, pt, k = 16, 8, 64, 16, 40
    totals = [1 + (i * 211) % 700 for i in range(B)]
    s = Setup(torch, lsa, totals, dtype=dtype, n_kv=n_kv, d=d, pt=pt, seed=B)
    guard = 4096

    def workspace(size):
        assert size > 0
        raw = torch.full((size + 2 * guard,), 0xFF, dtype=torch.uint8, device="cuda")
        return raw, raw[guard:guard + size]

    def untouched(raw):
        return bool((raw[:guard] == 0xFF).all()) and bool((raw[-guard:] == 0xFF).all())

    news = [1 + i % 2 * (i % 9) for i in range(B)]  # up to nine tokens of two heads each
    for new in ([1] * B, news):
        off = offsets(new)
        q = bf16(torch, s.g, (int(off[-1]), n_q, d))
        raw, ws = workspace(lsa.attend_workspace_size(s.cache, n_q=n_q, q_offsets_host=off, max_kv_len=max(totals)))
        out, lse = run_attend(torch, lsa, s, q, off, ws=ws)
        torch.cuda.synchronize()
        assert untouched(raw)
        check_rows(s, q, out, lse, [(int(off[b]) + i, b, totals[b] - new[b] + i) for b in range(B) for i in range(new[b])],
                   d ** -0.5, n_q=n_q, tag=f"{new[:3]}")
    idx = np.sort(s.g.integers(0, 100, (B, k)).astype(np.int32), 1)
    q = bf16(torch, s.g, (B, n_q, d))
    out, lse = torch.full_like(q, -7.0), torch.full((B, n_q), -7.0, device="cuda")
    raw, ws = workspace(lsa.attend_topk_workspace_size(s.cache, n_q=n_q, k=k, entry_tokens=4, window=100, sinks=3))
    lsa.attend_topk(s.cache, q, idx=torch.from_numpy(idx).cuda(), count=torch.full((B,), k, dtype=torch.int32, device="cuda"), out=out,
                    lse=lse, scale=d ** -0.5, entry_tokens=4, window=100, sinks=3, workspace=ws)
    torch.cuda.synchronize()
    assert untouched(raw)
    check_rows(s, q, out, lse, [(b, b, totals[b] - 1) for b in range(B)], d ** -0.5, 100, 3, [sorted(set(x.tolist())) for x in idx], 4,
               n_q)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [2, 4, 8], ids=lambda n: f"{8 * n}rows")
def test_blocks_that_share_the_keys(torch, lsa, dtype, d, new):
    """As many as the device holds at once, one or two a compute unit: with 8 key heads one long sequence has 32 or 64 parts a
    head. The workspace ends with the pairs (first block, number of parts) that say so."""
    n_q, n_kv = 64, 8
    s = Setup(torch, lsa, [9000], dtype=dtype, n_kv=n_kv, d=d, pt=128, seed=new)
    off = offsets([new])
    q = bf16(torch, s.g, (new, n_q, d))
    size = lsa.attend_workspace_size(s.cache, n_q=n_q, q_offsets_host=off, max_kv_len=9000)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = run_attend(torch, lsa, s, q, off, ws=ws)
    torch.cuda.synchronize()
    pairs = ws[size - 8 * n_kv:].view(torch.int32).view(n_kv, 2).tolist()
    most = 32 if 8 * new * d >= 32 * 128 else 64
    assert all(first == 0 and most * 0.8 < parts <= most for first, parts in pairs), pairs
    check_rows(s, q, out, lse, [(new - 1, 0, 8999)], d ** -0.5, n_q=n_q)
