"""The example of speculative decoding over a linear-attention block: the states that
the replay leaves are those of exactly the emitted tokens.

Bound on a state: the prefill's of tests/test_gpu_linear.py and the recurrent
path's over the replayed tokens, both relative to the sums of absolute values
(at most 4 (T / 32 + 1) + 80 and 5 T + 4 units of 2^-24 for T tokens).
"""

import importlib.util
import os

import pytest
import torch

from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "speculative_round.py")
spec = importlib.util.spec_from_file_location("speculative_round", PATH)
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_states_follow_the_emitted_tokens(dtype):
    model = ex.Model(V=501, dtype=dtype)
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, model.V, (n,), generator=gen, dtype=torch.int32) for n in (37, 1, 300)]
    rounds, K = 6, 4
    emitted, states = ex.generate(model, prompts, rounds, K)
    again, states2 = ex.generate(model, prompts, rounds, K)
    assert emitted == again and torch.equal(states, states2)
    for b, (p, e) in enumerate(zip(prompts, emitted)):
        assert 1 + rounds <= len(e) <= 1 + rounds * (K + 1) and all(0 <= t < model.V for t in e)
        tokens = torch.cat([p, torch.tensor(e[:-1], dtype=torch.int32)])   # the last one is not in the state yet
        t = tokens.long().to(model.device)
        args = (model.q[t].cpu(), model.k[t].cpu(), model.v[t].cpu(), model.g.cpu(), 1.0, model.Hq, model.Hv, torch.tensor([0, len(tokens)]))
        ref = oo.linear(*args)["final"][0]
        mag = oo.linear(*args, magnitudes=True)["final"][0]
        n = 4 * (len(tokens) // 32 + 1) + 80 + 5 * len(e) + 4
        off = abs(states[b].cpu().double().numpy() - ref)
        assert (off <= n * 2.0 ** -24 * mag + 1e-37).all(), (off / mag).max()


def test_main_runs(capsys):
    ex.main()
    assert capsys.readouterr().out.count("tokens in") == 3
