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


def test_captured_step(torch):
    """step() and attend_step() in one graph, replayed with eager work and waits between, against eager steps."""
    P.say("[steps] captured")
    w, (p, clean), hs, qkv = setup(torch, "fp8", steps=6)
    x = qkv()
    for q in (p, clean):  # first step eagerly: everything is loaded
        q.set_step_hidden(hs[0])
        q.step()
        q.attend_step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.step()
        p.attend_step(x)
    same(torch, p, clean, "after the capture")  # which ran nothing
    assert p.len_h.tolist() == clean.len_h.tolist()
    for t in range(1, 6):
        for a, b in zip(x, qkv()):
            a.copy_(b)
        for q in (p, clean):
            q.set_step_hidden(hs[t])
        graph.replay()
        torch.cuda.synchronize()
        clean.step()
        clean.attend_step(x)
        same(torch, p, clean, f"replay {t}")
    assert p.kv_len.tolist() == clean.len_h.tolist()


def test_step_on_a_given_stream_waits_for_nothing(torch):
    """Steps on a stream of their own, given as a stream and as its address; the host enqueues them while it is still
    busy."""
    P.say("[steps] own stream")
    w, (p, clean), hs, qkv = setup(torch, "bf16")
    stream = torch.cuda.Stream()
    xs = [qkv() for _ in range(4)]
    torch.cuda.synchronize()
    busy = torch.zeros((8192, 8192), device="cuda")
    with torch.cuda.stream(stream):
        for _ in range(24):  # some tenths of a second; four steps take the host about a millisecond
            busy = (busy @ busy) * 0
        done = torch.cuda.Event()
        done.record()
    for t in range(4):
        given = stream if t % 2 else stream.cuda_stream
        p.attend_step(xs[t], stream=given)
    assert not done.query(), "the host waited for the stream"
    for t in range(4):
        clean.attend_step(xs[t])
    same(torch, p, clean, "four steps")
