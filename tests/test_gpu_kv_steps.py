"""Decode steps with core attention through the pipeline where something is unusual (marked gpu): what is expected is
the same steps, bit for bit, of a second pipeline where nothing was."""
import pytest

from sparse_kv_retrieval_amd import synth
from tests import parity as P

pytestmark = pytest.mark.gpu
N_Q, N_KV, D = 8, 2, 128


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def setup(torch, dtype, n=2, steps=4, window=70):
    """n pipelines over the same inputs with the prompt appended, the decode steps' hidden states and a source of qkv."""
    from sparse_kv_retrieval_amd.pipeline import Pipeline
    w = synth.scaled(synth.WORKLOADS["three_layer_b8"], N=(300, 1, 90), k=32)
    inp = synth.make(w)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def some(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    ps = []
    for i in range(n):
        p = Pipeline(inp, "cuda", guard=True)
        p.alloc_steps()
        p.run()
        p.pack_subset_keys()
        p.alloc_attention(n_q=N_Q, n_kv=N_KV, d_h=D, dtype=dtype, page_tokens=32, entry_tokens=4, window=window, sinks=4,
                          max_steps=steps)
        if i == 0:
            T = int(p.prompt_len.sum())
            kv = [[some(T, N_KV, D) for _ in range(w.L)] for _ in range(2)]
        p.append_prompt(*kv)
        ps.append(p)
    return w, ps, synth.step_hidden(inp, steps), lambda: [some(w.B, N_Q + 2 * N_KV, D) for _ in range(w.L)]


def result(torch, p):
    torch.cuda.synchronize()
    assert p.check_guards() == []
    cached = [x.view(torch.uint8).clone() for c in p.caches for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None]
    return [x.clone() for x in p.attn_out + p.attn_lse + p.q_rot + [p.kv_len]] + cached


def same(torch, a, b, what):
    # as stored, NaN of unused slots and scales included
    for i, (x, y) in enumerate(zip(result(torch, a), result(torch, b))):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), f"{what}: buffer {i}"


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_steps_after_refused_ones(torch, dtype):
    P.say(f"[steps] refused {dtype}")
    w, (p, clean), hs, qkv = setup(torch, dtype)
    for t in range(4):
        x = qkv()
        for q in (p, clean):
            q.set_step_hidden(hs[t])
            q.step()
        for l in range(w.L):
            bad = list(x)
            bad[l] = bad[l].float() * 1000  # would raise a page's scale
            with pytest.raises(RuntimeError):
                p.attend_step(bad)
        p.attend_step(x)
        clean.attend_step(x)
        same(torch, p, clean, f"step {t}")
        assert p.len_h.tolist() == clean.len_h.tolist() == p.kv_len.tolist()
