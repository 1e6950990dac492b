"""gdn_beam_select and gdn_state_reorder against the fp64 oracle and indexing.

A score is off by at most its rounding 2^-24 |c| and 2^-22 of the sum of exponentials (2^-23 a term, and the sums')."""

import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, f64, say
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_03_amd as m
    m.load_library()
    return m


def select(gdn, x, s, K, finished=None, eos=-1, pad=0, ref=None):
    got = gdn.gdn_beam_select(x.to(DEV), s.to(DEV), beams=K, finished=None if finished is None else finished.to(DEV),
                              eos_token=eos, pad_token=pad)
    tokens, parents, best, over = co.beam_select(x, s, K, finished, eos, pad) if ref is None else ref
    assert np.array_equal(f64(got[0]), tokens) and np.array_equal(f64(got[1]), parents)
    b = f64(got[2])
    assert np.array_equal(np.isinf(b), np.isinf(best))
    fin = np.isfinite(best)
    assert (np.abs(b - best)[fin] <= 2.0 ** -24 * np.abs(best[fin]) + 2.0 ** -22).all()
    assert np.array_equal(got[3].cpu().numpy(), over)
    return got


def draw(seed, B, W, V, dtype, spread=2.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(spread * rng.standard_normal((B, W, V))).to(TYPES[dtype])
    s = torch.from_numpy(-5.0 * rng.random((B, W))).float()
    return x, s, torch.from_numpy(rng.random((B, W)) < 0.2)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,W,K,V", [(1, 1, 1, 1), (1, 4, 4, 2003), (3, 2, 4, 2049), (2, 5, 7, 8191), (1, 1, 64, 777),
                                     (2, 64, 64, 300), (1, 3, 6, 33000), (40, 8, 16, 8200), (2, 2, 5, 2)])
def test_against_the_oracle(gdn, B, W, K, V, dtype):
    x, s, f = draw(B * 1000 + V, B, W, V, dtype)
    select(gdn, x, s, K)
    select(gdn, x, s, K, finished=f, eos=1, pad=min(3, V - 1))


@pytest.mark.parametrize("V", [100, 5000, 9000])
@pytest.mark.parametrize("B,W,K", [(1, 3, 8), (90, 6, 8)])
def test_ties(gdn, B, W, K, V):
    """Few distinct logits, and beams that are the same: equal continuations in the order of (beam, token)."""
    rng = np.random.default_rng(V)
    one = torch.from_numpy(rng.integers(0, 3, (B, 1, V)).astype(np.float32))
    x = one.expand(B, W, V).contiguous().to(torch.bfloat16)
    s = torch.full((B, W), -1.25)
    got = gdn.gdn_beam_select(x.to(DEV), s.to(DEV), beams=K)
    for b in range(0, B, 7):
        first = np.nonzero(one[b, 0].numpy() == one[b, 0].max().item())[0]
        want = [(w, v) for w in range(W) for v in first][:K]
        assert list(zip(got[1][b].tolist(), got[0][b].tolist())) == want


@pytest.mark.parametrize("V", [3, 2500, 20000])
def test_all_equal(gdn, V):
    """Every logit the same, zeros of both signs among them."""
    x = torch.zeros(2, 2, V)
    x[:, :, 1::2] = -0.0
    got = gdn.gdn_beam_select(x.to(DEV), torch.zeros(2, 2, device=DEV), beams=min(V, 9))
    K = min(V, 9)
    assert got[0].tolist() == [list(range(K))] * 2 and got[1].tolist() == [[0] * K] * 2
    assert np.allclose(f64(got[2]), -math.log(V), atol=1e-6)


@pytest.mark.parametrize("V", [50, 10000])
def test_absent_beams_and_masked_tokens(gdn, V):
    x, s, _ = draw(5, 4, 6, V, "f32")
    x[0, 0, 7] = math.nan
    x[0, 1, 8] = math.inf
    x[0, 2] = -math.inf
    s[0, 3], s[0, 4] = -math.inf, math.nan
    x[1, :, 3:] = -math.inf                            # three continuations a beam
    x[2], s[2] = math.nan, 0.0                         # none at all
    x[3, 0] = torch.finfo(torch.float32).min           # masked with the lowest number
    x[3, 1, :10] = torch.finfo(torch.float32).min
    select(gdn, x, s, 20)
    select(gdn, x, s, 3)


def test_a_finished_beam_reads_no_logits(gdn):
    x, s, _ = draw(6, 2, 3, 3000, "bf16")
    f = torch.zeros(2, 3, dtype=torch.bool)
    f[0, 1] = f[1] = True
    x[0, 1] = math.nan
    select(gdn, x, s, 5, finished=f, pad=7)


def test_first_step_from_one_beam(gdn):
    """Only beam 0 counts at the start; K from 1 to beyond the vocabulary."""
    x, s, _ = draw(7, 3, 4, 40, "f16")
    s[:, 1:] = -math.inf
    for K in (1, 4, 50):
        select(gdn, x, s, K)


def test_padded_rows_and_odd_alignment(gdn):
    x, s, f = draw(8, 2, 3, 1001, "bf16")
    wide = torch.full((2, 3, 1007), math.nan, dtype=torch.bfloat16, device=DEV)
    wide[:, :, 3:1004] = x.to(DEV)
    got = gdn.gdn_beam_select(wide[:, :, 3:1004], s.to(DEV), finished=f.to(DEV), eos_token=4)
    want = gdn.gdn_beam_select(x.to(DEV), s.to(DEV), finished=f.to(DEV), eos_token=4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_large_offsets_and_scores(gdn):
    """Logits far from zero and very negative scores: the sums are taken against the maximum, in 64 bits."""
    x, s, _ = draw(9, 2, 3, 5000, "f32")
    select(gdn, x + 3.0e4, s - 1.0e3, 6)
    select(gdn, x * 1.0e30, s, 2)


def test_selection_is_the_same_again(gdn):
    x, s, f = draw(10, 16, 8, 30000, "bf16")
    a = [gdn.gdn_beam_select(x.to(DEV), s.to(DEV), beams=16, finished=f.to(DEV)) for _ in range(3)]
    for b in a[1:]:
        assert all(torch.equal(p, q) for p, q in zip(a[0], b))


# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("W", [1, 2, 4, 5, 8, 13, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_reorder(gdn, W, in_place):
    rng = np.random.default_rng(W)
    B = 3
    parents = rng.integers(0, W, (B, W)).astype(np.int32)
    parents[1] = rng.permutation(W)
    parents[2, 0] = -1
    parents[2, W // 2] = W                             # no parent: the row stays
    state = torch.from_numpy(rng.standard_normal((2, B * W, 3, 16, 20))).float()
    want = (state if in_place else torch.full_like(state, 7.0)).clone()
    for layer in range(2):
        for r, x in enumerate(co.reorder(state[layer].numpy(), parents)):
            if x is not None:
                want[layer, r] = torch.from_numpy(x)
    s = state.to(DEV)
    out = s if in_place else torch.full_like(s, 7.0)
    got = gdn.gdn_state_reorder(s, torch.from_numpy(parents).to(DEV), axis=1, out=out)
    assert got is out and torch.equal(got.cpu(), want)
    if not in_place:
        assert torch.equal(s.cpu(), state)


def test_reorder_to_another_number_of_beams(gdn):
    state = torch.randn(6, 4, 8, device=DEV).to(torch.bfloat16)
    parents = torch.tensor([[2, 0, 0, 1], [0, 1, 2, 2]], dtype=torch.int32, device=DEV)
    got = gdn.gdn_state_reorder(state, parents)
    assert torch.equal(got, state[[2, 0, 0, 1, 3, 4, 5, 5]])
    one = gdn.gdn_state_reorder(state, parents[:, :1].contiguous())
    assert torch.equal(one, state[[2, 3]])


def test_reorder_of_large_and_small_rows(gdn):
    for shape in ((4, 4), (4, 100003 * 4), (4, 32, 128, 128)):
        state = torch.randn(*shape, device=DEV)
        want = state[[3, 3, 1, 0]].clone()
        gdn.gdn_state_reorder(state, torch.tensor([[3, 3, 1, 0]], dtype=torch.int32, device=DEV), out=state)
        assert torch.equal(state, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_copy_pages(gdn, dtype):
    k = torch.randn(20, 2, 16, 32, device=DEV).to(TYPES[dtype])
    v = torch.randn_like(k)
    wk, wv = k.clone(), v.clone()
    src = torch.tensor([[0, 0, 3], [5, 6, 99]], dtype=torch.int32, device=DEV)
    dst = torch.tensor([[1, 3, 0], [7, -1, 8]], dtype=torch.int32, device=DEV)   # 3 -> 0 while 0 -> 3
    for a, b in ((0, 1), (0, 3), (3, 0), (5, 7)):
        wk[b], wv[b] = k[a].clone(), v[a].clone()
    for a, b in ((k, v), (v, k)):      # whichever of the two lies first in memory
        x, y = a.clone(), b.clone()
        gdn.gdn_cache_copy_pages(x, y, src, dst)
        assert torch.equal(x, wk if a is k else wv) and torch.equal(y, wv if a is k else wk)


def test_copy_pages_beyond_32_bits(gdn):
    big = torch.zeros(1200, 8, 1024, 256, dtype=torch.bfloat16, device=DEV)      # 5 GB
    other = torch.zeros_like(big)
    big[1190], other[1190] = 3.0, 4.0
    gdn.gdn_cache_copy_pages(big, other, torch.tensor([1190], dtype=torch.int32, device=DEV),
                             torch.tensor([2], dtype=torch.int32, device=DEV))
    assert (big[2] == 3.0).all() and (other[2] == 4.0).all() and not big[:2].any() and not big[3:1190].any()


def test_the_largest_vocabulary_and_beams(gdn):
    """2^24 tokens: more entries are left for the join than its threads hold; the best ones spread over all of it."""
    V, W, K = 1 << 24, 3, 64
    x = torch.zeros(1, W, V, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    at = torch.randperm(V, generator=g, device=DEV)[:100]
    x[0, 0, at[:50]], x[0, 2, at[50:]] = 8.0, 9.0
    x[0, 1, V - 1], x[0, 1, 0] = 16.0, 15.5
    s = torch.tensor([[-1.0, -3.0, -2.0]], device=DEV)
    tokens, parents, best, done = gdn.gdn_beam_select(x, s, beams=K, eos_token=V - 1)
    ls = [math.log(V - 50 + 50 * math.exp(8.0)), math.log(V - 2 + math.exp(16.0) + math.exp(15.5)),
          math.log(V - 50 + 50 * math.exp(9.0))]
    every = [(-(-1.0 - ls[0] + 8.0), 0, t) for t in at[:50].tolist()] + [(-(-2.0 - ls[2] + 9.0), 2, t) for t in at[50:].tolist()]
    every += [(-(-3.0 - ls[1] + 16.0), 1, V - 1), (-(-3.0 - ls[1] + 15.5), 1, 0)]
    every = sorted(every)[:K]
    assert tokens[0].tolist() == [t for _, _, t in every] and parents[0].tolist() == [w for _, w, _ in every]
    assert np.abs(f64(best)[0] + np.array([c for c, _, _ in every])).max() <= 2.0 ** -24 * 20 + 2.0 ** -22
    assert done[0].tolist() == [t == V - 1 for _, _, t in every]
