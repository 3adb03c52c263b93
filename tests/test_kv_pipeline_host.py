"""The pipeline's core-attention steps on the host (CPU): what a refused call leaves behind.

The buffers are on the CPU and the binding's checks are real; only the launch behind them is replaced by a
record of what would have been enqueued.
"""
import types

import numpy as np
import pytest
import torch

from sparse_kv_retrieval_amd import lsa
from sparse_kv_retrieval_amd import pipeline as PL

N_Q, N_KV, D = 4, 2, 64
ENTRIES, R, K = (5, 4), 4, 8


@pytest.fixture
def launches(monkeypatch):
    """What was enqueued; .fail_at makes that launch fail (from 0)."""
    log = types.SimpleNamespace(names=[], fail_at=None)

    def launch(device, fn, call, args, stream):
        if log.fail_at == len(log.names):
            raise lsa.LsaError(fn, lsa.ERR_HIP, "as the test asks")
        log.names.append(fn)

    monkeypatch.setattr(lsa, "_launch", launch)
    return log


def pipeline(**kw):
    p = PL.Pipeline.__new__(PL.Pipeline)
    p.w = types.SimpleNamespace(L=2, B=2, k=K)
    p.device, p.guard, p._guarded = torch.device("cpu"), False, []
    p.key_off_h = np.concatenate([[0], np.cumsum(ENTRIES)]).astype(np.int64)
    p.keys_sub = []  # as after alloc_steps()
    p.step_idx = [torch.zeros((2, K), dtype=torch.int32) for _ in range(2)]
    p.step_count = torch.zeros((2, 2), dtype=torch.int32)
    p.alloc_attention(**{**dict(n_q=N_Q, n_kv=N_KV, d_h=D, page_tokens=16, entry_tokens=R, window=16, max_steps=3), **kw})
    return p


def rows(n, heads, dtype=torch.bfloat16):
    return torch.zeros((n, heads, D), dtype=dtype)


def state(p):
    return p.len_h.tolist(), p.kv_len.tolist()


def step_input():
    return [rows(2, N_Q + 2 * N_KV) for _ in range(2)]


T = sum(ENTRIES) * R
BAD = {"float32": lambda x: x.float(), "too few rows": lambda x: x[:1], "heads": lambda x: x[:, :-1], "d_h": lambda x: x[..., :32],
       "stride of a row": lambda x: torch.as_strided(torch.zeros(x.numel() + 4 * x.shape[0], dtype=x.dtype), x.shape,
                                                     (x.shape[1] * D + 4, D, 1)),
       "alignment": lambda x: torch.zeros(x.numel() + 1, dtype=x.dtype)[1:].view(x.shape),
       "heads apart": lambda x: torch.zeros((x.shape[0], x.shape[1], 2 * D), dtype=x.dtype)[..., :D]}


@pytest.mark.parametrize("layer", [0, 1])
@pytest.mark.parametrize("bad", BAD, ids=list(BAD))
def test_refused_step_changes_nothing(launches, bad, layer):
    p = pipeline()
    p.append_prompt([rows(T, N_KV)] * 2, [rows(T, N_KV)] * 2)
    before, n = state(p), len(launches.names)
    assert before == ([20, 16], [20, 16])
    x = step_input()
    x[layer] = BAD[bad](x[layer])
    with pytest.raises(lsa.LsaError):
        p.attend_step(x)
    assert state(p) == before and len(launches.names) == n  # no layer holds the token
    p.attend_step(step_input())
    assert state(p) == ([21, 17], [21, 17]) and len(launches.names) == n + 4


@pytest.mark.parametrize("layer", [0, 1])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("bad", BAD, ids=list(BAD))
def test_refused_prompt_changes_nothing(launches, bad, side, layer):
    p = pipeline()
    kv = {"k": [rows(T, N_KV)] * 2, "v": [rows(T, N_KV)] * 2}
    good = {s: list(x) for s, x in kv.items()}
    kv[side] = list(kv[side])
    kv[side][layer] = BAD[bad](kv[side][layer])
    with pytest.raises(lsa.LsaError):
        p.append_prompt(**kv)
    assert state(p) == ([0, 0], [0, 0]) and launches.names == []
    p.append_prompt(**good)
    assert state(p) == ([20, 16], [20, 16])


def test_missing_layer_changes_nothing(launches):
    p = pipeline()
    with pytest.raises(lsa.LsaError):
        p.append_prompt([rows(T, N_KV)], [rows(T, N_KV)] * 2)
    p.append_prompt([rows(T, N_KV)] * 2, [rows(T, N_KV)] * 2)
    n = len(launches.names)
    with pytest.raises(lsa.LsaError):
        p.attend_step(step_input()[:1])
    assert state(p) == ([20, 16], [20, 16]) and len(launches.names) == n


def test_step_before_alloc_steps_changes_nothing(launches):
    p = pipeline()
    p.append_prompt([rows(T, N_KV)] * 2, [rows(T, N_KV)] * 2)
    n, p.keys_sub = len(launches.names), None
    with pytest.raises(ValueError, match="alloc_steps"):
        p.attend_step(step_input())
    assert state(p) == ([20, 16], [20, 16]) and len(launches.names) == n


@pytest.mark.parametrize("at", range(4))
def test_failed_launch_takes_the_lengths_back(launches, at):
    # whatever a failing launch left in a slot lies behind the length, and the next step writes it again
    p = pipeline()
    launches.fail_at = at % 2
    with pytest.raises(lsa.LsaError):
        p.append_prompt([rows(T, N_KV)] * 2, [rows(T, N_KV)] * 2)
    assert state(p) == ([0, 0], [0, 0])
    launches.fail_at = None
    p.append_prompt([rows(T, N_KV)] * 2, [rows(T, N_KV)] * 2)
    launches.fail_at = len(launches.names) + at
    with pytest.raises(lsa.LsaError):
        p.attend_step(step_input())
    assert state(p) == ([20, 16], [20, 16])
    launches.fail_at = None
    for t in range(1, 4):
        p.attend_step(step_input())
        assert state(p) == ([20 + t, 16 + t], [20 + t, 16 + t])
    with pytest.raises(ValueError, match="full"):
        p.attend_step(step_input())
    assert state(p) == ([23, 19], [23, 19])


def test_window_covers_the_steps(launches):
    # a step sees its own token and the window - 1 before it; the lists hold prompt entries alone
    for window, max_steps in ((16, 17), (0, 1), (1, 64)):
        with pytest.raises(ValueError, match="window"):
            pipeline(window=window, max_steps=max_steps)
    for window, max_steps in ((16, 16), (1, 1), (0, 0), (200, 20)):
        p = pipeline(window=window, max_steps=max_steps)
        p.append_prompt([rows(T, N_KV)] * 2, [rows(T, N_KV)] * 2)
        for _ in range(max_steps):
            p.attend_step(step_input())
        assert (p.kv_len - p.window <= torch.from_numpy(p.prompt_len)).all()  # the last step's window begins in the prompt


def test_prompt_comes_once_and_first(launches):
    p = pipeline(window=64, max_steps=64)  # room for the prompt twice
    prompt = [rows(T, N_KV)] * 2
    p.append_prompt(prompt, prompt)
    n = len(launches.names)
    for _ in range(2):
        with pytest.raises(ValueError, match="prompt"):
            p.append_prompt(prompt, prompt)
        assert state(p)[0] == state(p)[1] and p.len_h[0] in (20, 21) and len(launches.names) == n
        p.attend_step(step_input())
        n = len(launches.names)
    p = pipeline(window=64, max_steps=64)
    p.attend_step(step_input())
    with pytest.raises(ValueError, match="prompt"):
        p.append_prompt(prompt, prompt)
    assert state(p) == ([1, 1], [1, 1])
