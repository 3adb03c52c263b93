"""The decode steps' core attention over what the native top-k selected, through the pipeline (marked gpu).

One trigger, the prompt's keys and values into the paged caches, then decode steps: every step's top-k
(compared with the oracle elsewhere) feeds lsa_attend_topk, whose outputs are compared with the float64
oracle over the cache as it is stored and the lists as they are.
"""
import numpy as np
import pytest

from oracle import kv_oracle as K
from sparse_kv_retrieval_amd import synth
from tests import parity as P
from tests.test_gpu_kv import check_rows

W = synth.WORKLOADS


class Stored:
    """What check_rows reads: one layer's cache as it is now, in float64."""

    def __init__(self, torch, cache, lens):
        self.n_kv, self.d, self.totals, self.decoded = cache.n_kv, cache.d_h, list(lens), {}
        self.table = cache.page_table.cpu().numpy()
        for name, x, scale in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
            if scale is None:
                self.decoded[name] = x.cpu().double().numpy()
            else:
                codes = x.view(torch.uint8).cpu().numpy()
                self.decoded[name] = K.e4m3_values()[codes] * scale.cpu().numpy().astype(np.float64)[:, :, None, None]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_steps_with_attention(dtype):
    import torch
    from sparse_kv_retrieval_amd.pipeline import Pipeline
    w = synth.scaled(W["three_layer_b8"], N=(700, 64, 1, 333), k=64)
    P.say(f"[steps] core attention {dtype}")
    inp = synth.make(w)
    p = Pipeline(inp, "cuda", guard=True)
    p.alloc_steps()
    p.run()
    p.pack_subset_keys()
    n_q, n_kv, d, steps = 8, 2, 128, 4
    p.alloc_attention(n_q=n_q, n_kv=n_kv, d_h=d, dtype=dtype, page_tokens=32, entry_tokens=4, window=70, sinks=4, max_steps=steps)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def some(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    T = int(p.prompt_len.sum())
    p.append_prompt([some(T, n_kv, d) for _ in range(w.L)], [some(T, n_kv, d) for _ in range(w.L)])
    hs = synth.step_hidden(inp, steps)
    for t in range(steps):
        p.set_step_hidden(hs[t])
        p.step()
        p.attend_step([some(w.B, n_q + 2 * n_kv, d) for _ in range(w.L)])
        torch.cuda.synchronize()
        for l in range(w.L):
            idx, count = p.step_idx[l].cpu().numpy(), p.step_count[l].cpu().numpy()
            listed = [idx[b, :count[b]].tolist() for b in range(w.B)]
            assert count.max() == w.k  # some lists are full
            s = Stored(torch, p.caches[l], p.len_h)
            check_rows(s, p.q_rot[l], p.attn_out[l], p.attn_lse[l], [(b, b, int(p.len_h[b]) - 1) for b in range(w.B)],
                       d ** -0.5, 70, 4, listed, 4, n_q, f"step {t} layer {l}")
    assert p.check_guards() == [], f"writes outside an output buffer: {p.check_guards()}"
    with pytest.raises(ValueError, match="full"):
        p.attend_step([some(w.B, n_q + 2 * n_kv, d) for _ in range(w.L)])
