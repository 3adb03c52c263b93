"""lsa_kv_compact on an e4m3 cache, code by code (marked gpu): what a page's new scale leaves as it was, bit for bit. Exact."""
import numpy as np
import pytest

from tests.test_gpu_kv import Setup, lsa, torch  # noqa: F401  (fixtures)
from tests.test_gpu_kv_pool import To, bits, run_compact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,pt,exponent", [(128, 64, 0), (64, 16, -118), (64, 128, 119), (128, 32, 5)])
def test_codes_of_an_equal_scale_stay(torch, lsa, d, pt, exponent):
    """Every one of the 256 codes, NaN of either sign and negative zero among them, in pages whose scale is the new one's."""
    totals = [4 * pt, 2 * pt + 3]
    s = Setup(torch, lsa, totals, dtype="fp8", n_kv=2, d=d, pt=pt, seed=1)
    g = np.random.default_rng(2)
    for name in ("k", "v"):
        codes = g.integers(0, 256, tuple(s.parts[name].shape)).astype(np.uint8)
        codes[..., 0, 0] = 0x7E  # 448: no lesser power of two holds the page
        s.parts[name].view(torch.uint8).copy_(torch.from_numpy(codes))
        s.parts[name + "_scale"].fill_(2.0 ** exponent)
    to = To(torch, lsa, 2, 4, dtype="fp8", n_kv=2, d=d, pt=pt, layers=1)
    run_compact(torch, lsa, [s], to, [[], []], 1, 4 * pt, 0, 4 * pt)
    assert to.kept.tolist() == totals
    for name in ("k", "v"):
        got, was = bits(torch, to.parts[0][name]), bits(torch, s.parts[name])
        for b, t in enumerate(totals):
            for p in range(t):
                assert (got[to.table[b, p // pt], :, p % pt] == was[s.table[b, p // pt], :, p % pt]).all(), (name, b, p)
        for b, t in enumerate(totals):
            used = to.table[b, :-(-t // pt)]
            assert (to.parts[0][name + "_scale"].cpu().numpy()[used] == 2.0 ** exponent).all()


def test_codes_beside_a_greater_scale(torch, lsa):
    """Tokens of two pages in one: the page whose scale is the new one's keeps its codes, the other's are rounded anew and its NaN is NaN."""
    s = Setup(torch, lsa, [32], dtype="fp8", n_kv=1, d=64, pt=16, seed=3)
    codes = np.tile(np.arange(256, dtype=np.uint8), 8).reshape(2, 1, 16, 64)
    pages = s.table[0, :2]
    for name in ("k", "v"):
        s.parts[name].view(torch.uint8)[torch.from_numpy(pages.astype(np.int64)).cuda()] = torch.from_numpy(codes).cuda()
        s.parts[name + "_scale"][int(pages[0])] = 4.0
        s.parts[name + "_scale"][int(pages[1])] = 1.0
    to = To(torch, lsa, 1, 1, dtype="fp8", n_kv=1, d=64, pt=32, layers=1)
    run_compact(torch, lsa, [s], to, [[]], 1, 32, 0, 32)
    for name in ("k", "v"):
        got = bits(torch, to.parts[0][name])[to.table[0, 0], 0]
        assert (got[:16] == codes[0, 0]).all() and to.parts[0][name + "_scale"][int(to.table[0, 0])].item() == 4.0
        old = codes[1, 0]
        nan = (old & 0x7F) == 0x7F
        assert ((got[16:][nan] & 0x7F) == 0x7F).all()
        big = ~nan & ((old & 0x78) >= 0x18)  # normal codes that stay normal: the exponent falls by two
        assert (got[16:][big] == old[big] - 0x10).all()
