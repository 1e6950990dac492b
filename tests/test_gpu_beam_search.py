"""The example of a beam search, against a plain search that runs every hypothesis from its first token in 64 bits.

fp32 model: a score is a sum of at most 12 log probabilities of a few hundred fp32 operations each; 1e-3 is three orders
above their rounding, and two orders below the distance of neighbouring hypotheses, which the test asks for."""

import importlib.util
import os

import pytest
import torch

from gpu_common import say

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("beam_search_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm(x, eps=1e-6):
    return x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()


def log_probs(m, tokens):
    """The model in 64 bits over one sequence, token by token: log probabilities of the next token."""
    x = m.embedding.double()[tokens]
    unit = torch.nn.functional.normalize
    T = len(tokens)
    q = unit((x @ m.wq.double()).view(T, m.Hq, m.dk), dim=-1).repeat_interleave(m.Hv // m.Hq, 1)
    k = unit((x @ m.wk.double()).view(T, m.Hq, m.dk), dim=-1).repeat_interleave(m.Hv // m.Hq, 1)
    v = (x @ m.wv.double()).view(T, m.Hv, m.dv)
    alpha = torch.exp(-torch.nn.functional.softplus(x @ m.wg.double()))
    beta = torch.sigmoid(x @ m.wb.double())
    S = torch.zeros(m.Hv, m.dk, m.dv, dtype=torch.float64, device=x.device)
    rows = []
    for t in range(T):
        S = alpha[t][:, None, None] * S
        delta = beta[t][:, None] * (v[t] - (S * k[t][:, :, None]).sum(1))
        S = S + k[t][:, :, None] * delta[:, None]
        rows.append(m.dk ** -0.5 * (S * q[t][:, :, None]).sum(1))
    z = x @ m.wz.double()
    y = norm(torch.stack(rows)).reshape(T, m.D) * z * torch.sigmoid(z)
    h = x + norm(y @ m.wo.double())
    a, b, d = m.heads, m.kv_heads, m.d
    qkv = (norm(h) @ m.wqkv.double()).view(T, a + 2 * b, d)
    turn = torch.arange(T, device=x.device)[:, None].double() * m.inv_freq.double()
    cos, sin = torch.cos(turn)[:, None], torch.sin(turn)[:, None]

    def rotated(u):
        return torch.cat([u[..., :d // 2] * cos - u[..., d // 2:] * sin, u[..., :d // 2] * sin + u[..., d // 2:] * cos], -1)
    q, k, v = rotated(qkv[:, :a]), rotated(qkv[:, a:a + b]), qkv[:, a + b:]
    k, v = k.repeat_interleave(a // b, 1), v.repeat_interleave(a // b, 1)
    s = torch.einsum("ihd,jhd->hij", q.cpu(), k.cpu()).to(x.device) * d ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=x.device).triu(1), -float("inf"))
    o = (torch.softmax(s, -1) @ v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(T, a * d)
    return torch.log_softmax((norm(h + norm(o @ m.wproj.double())) @ m.head.double())[-1], -1)


def plain_search(m, prompt, beams, steps, eos):
    found = [((), 0.0, False)]
    gap = float("inf")
    for _ in range(steps):
        every = []
        for tokens, score, done in found:
            if done:
                every.append((score, tokens + (0,), True))
                continue
            p = log_probs(m, torch.cat([prompt.long(), torch.tensor(tokens, dtype=torch.long)]).to(m.device))
            best, at = p.topk(beams + 1)
            every += [(score + s, tokens + (t,), t == eos) for s, t in zip(best.tolist(), at.tolist())]
        every.sort(key=lambda e: -e[0])
        gap = min([gap] + [a[0] - b[0] for a, b in zip(every[:beams], every[1:beams + 1])])
        found = [(t, s, d) for s, t, d in every[:beams]]
    return [f[0] for f in found], [f[1] for f in found], gap


@pytest.mark.parametrize("lengths,beams,steps", [((37, 5, 64), 3, 12), ((16, 1, 31), 5, 7)])
def test_against_a_plain_search(example, lengths, beams, steps):
    model = example.Model(V=203, dtype=torch.float32, seed=5)
    gen = torch.Generator().manual_seed(11)
    prompts = [torch.randint(2, model.V, (n,), generator=gen, dtype=torch.int32) for n in lengths]
    eos = 7
    history, scores = example.search(model, prompts, beams=beams, steps=steps, eos=eos)
    for b, p in enumerate(prompts):
        tokens, want, gap = plain_search(model, p, beams, steps, eos)
        say(f"prompt of {len(p)}: scores {[round(x, 3) for x in want]}, nearest hypotheses {gap:.2e} apart")
        assert max(abs(x - y) for x, y in zip(scores[b].tolist(), want)) < 1e-3
        if gap > 2e-3:
            assert [tuple(t) for t in history[b].tolist()] == tokens


def test_example_runs(example, capsys):
    example.main()
    assert capsys.readouterr().out.count("prompt of") == 3
