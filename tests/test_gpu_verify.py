"""Verification of drafted tokens: equal to the fp64 oracle, token for token."""

import numpy as np
import pytest
import torch

import gated_deltanet_03_amd as gdn
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def case(seed, B, K, V, dtype, onehot=False, sharp=2.5, noise=0.5):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, K + 1, V, generator=g)
    p = torch.softmax(logits, -1).to(TYPES[dtype])
    prob = torch.softmax(logits[:, :K] + noise * torch.randn(B, K, V, generator=g), -1)
    x = torch.multinomial(prob.reshape(B * K, V), 1, generator=g).view(B, K).int() if K else torch.zeros(B, 0).int()
    n = torch.randint(0, K + 3, (B,), generator=g).int() - 1          # idle rows and counts above K among them
    return p, None if onehot else prob.to(TYPES[dtype]), x, torch.rand(B, K + 1, generator=g), n


def check(p, q, x, u, n, **kw):
    d = [None if t is None else t.to(DEV) for t in (p, q, x, u)]
    tokens, emit = gdn.gdn_verify_drafts(*d, draft_count=None if n is None else n.to(DEV), **kw)
    tokens, emit = tokens.cpu().numpy(), emit.cpu().numpy()
    for b in range(x.shape[0]):
        want, m = oo.verify_row(p[b], None if q is None else q[b], x[b].tolist(), u[b],
                                x.shape[1] if n is None else int(n[b]))
        assert emit[b] == m and tokens[b].tolist() == want, (b, tokens[b], want, emit[b], m)
    return tokens, emit


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 2047, 2048, 2049, 5001, 32003])
@pytest.mark.parametrize("onehot", [False, True])
def test_against_oracle(dtype, V, onehot):
    check(*case(V + onehot, 9, 4, V, dtype, onehot))


@pytest.mark.parametrize("B,K", [(1, 0), (3, 0), (1, 1), (2, 7), (1, 70), (130, 2)])
def test_rows_and_drafts(B, K):
    p, q, x, u, n = case(B + K, B, K, 999, "f32", noise=0.05)
    check(p, q, x, u, None)
    check(p, q, x, u, n)


def test_large_vocabulary_in_many_tiles():
    p, q, x, u, n = case(3, 2, 2, 2 ** 21 + 5, "f32")   # above 1024 tiles of the smallest size
    check(p, q, x, u, None)


def test_uniforms_at_the_ends_and_on_borders():
    V = 4096
    p = torch.full((6, 2, V), 1.0 / V)                  # every border is exact
    q = torch.zeros(6, 1, V)
    q[:, :, 5] = 1.0
    x = torch.full((6, 1), 5, dtype=torch.int32)
    u = torch.zeros(6, 2)
    u[:, 0] = 0.9                                       # refused: the rest is p without entry 5
    u[:, 1] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 0.25, 1.0 / (V - 1), 0.75])
    tokens, _ = check(p, q, x, u, None)
    assert tokens[0, 0] == 0 and tokens[1, 0] == V - 1
    tokens, _ = check(p, q, x, u, torch.zeros(6, dtype=torch.int32))   # no drafts: c_v = (v + 1) / V > u
    assert tokens[2, 0] == V // 2 and tokens[3, 0] == V // 4
    u[:, 0] = 1.0 / V                                   # u q = p exactly: refused
    assert (check(p, q, x, u, None)[1] == 1).all()


def test_rows_without_a_rest():
    p = torch.softmax(torch.randn(5, 3, 300, generator=torch.Generator().manual_seed(1)), -1)
    q = p[:, :2].clone()
    x = torch.full((5, 2), 7, dtype=torch.int32)
    u = torch.full((5, 3), 0.5)
    q[1:, 0] *= 2                                       # p < q everywhere: nothing is left of max(p - q, 0)
    u[1:, 0] = 0.8                                      # refused: drawn from p instead
    p[2, 0] = 0.0                                       # no weight at all
    q[3, 0] = float("inf")
    tokens, emit = check(p, q, x, u, None)
    assert emit[0] == 3 and tokens[2].tolist() == [-1, -1, -1] and emit[2] == 1 and tokens[1, 0] >= 0


def test_weights_that_are_no_numbers():
    p, q, x, u, _ = case(8, 6, 2, 777, "f32")
    p[0, :, ::2] = float("nan")
    p[1, :, 5] = float("inf")
    p[2, :, 100:] = -1.0
    q[3, :, ::3] = float("nan")
    p[4] = float("nan")
    check(p, q, x, u, None)
    check(p, None, x, u, None)


def test_tokens_outside_the_vocabulary():
    p, q, x, u, _ = case(9, 4, 3, 500, "bf16")
    x[0, 0], x[1, 1], x[2, 2], x[3, 0] = -1, 500, 2 ** 31 - 1, -2 ** 31
    check(p, q, x, u, None)
    check(p, None, x, u, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padded_rows(dtype):
    p, q, x, u, n = case(10, 5, 3, 1003, dtype)
    wide = torch.full((5, 4, 1024), 9.0, dtype=p.dtype)
    wide[..., :1003] = p
    qw = torch.full((5, 3, 1011), 9.0, dtype=p.dtype)
    qw[..., :1003] = q
    wd, qd = wide.to(DEV), qw.to(DEV)
    a = gdn.gdn_verify_drafts(wd[..., :1003], qd[..., :1003], x.to(DEV), u.to(DEV), draft_count=n.to(DEV))
    b = gdn.gdn_verify_drafts(p.to(DEV), q.to(DEV), x.to(DEV), u.to(DEV), draft_count=n.to(DEV))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(p, q, x, u, n)


def test_dirty_workspace_and_graph():
    p, q, x, u, n = (t.to(DEV) for t in case(11, 7, 3, 6001, "f32"))
    ws = torch.full((gdn.load_library().gdn_verify_workspace_bytes(
        gdn.ctypes.byref(gdn.gdn_verify_shape(7, 3, 6001, 0, 6001, 6001))),), 255, dtype=torch.uint8, device=DEV)
    tokens, emit = torch.zeros(7, 4, dtype=torch.int32, device=DEV), torch.zeros(7, dtype=torch.int32, device=DEV)
    kw = dict(draft_count=n, tokens=tokens, emit_count=emit, workspace=ws)
    gdn.gdn_verify_drafts(p, q, x, u, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_verify_drafts(p, q, x, u, **kw)
    for i in range(4):
        u.copy_(torch.rand_like(u))
        graph.replay()
        torch.cuda.synchronize()
        got = tokens.clone(), emit.clone()
        check(*(t.cpu() for t in (p, q, x, u, n)))
        want = gdn.gdn_verify_drafts(p, q, x, u, draft_count=n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_row_offsets_past_32_bits():
    B, V = 9, 2 ** 24
    p = torch.zeros(B, 16, V, dtype=torch.bfloat16, device=DEV)      # 2.4e9 elements
    x = torch.full((B, 15), 3, dtype=torch.int32, device=DEV)
    u = torch.full((B, 16), 0.5, device=DEV)
    p[:, :15, 3] = 1.0
    p[:, 15, V - 1] = 1.0
    tokens, emit = gdn.gdn_verify_drafts(p, None, x, u)
    assert (emit == 16).all() and (tokens[:, 15] == V - 1).all() and (tokens[:, :15] == 3).all()
    assert np.prod(p.shape) > 2 ** 31


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [511, 512, 513, 8192, 32768, 40000, 65535, 65536, 65537, 70001])
def test_around_the_sizes_that_change_the_path(dtype, V):
    """One workgroup a row up to 65536 entries, two kernels beyond."""
    need = gdn.load_library().gdn_verify_workspace_bytes(
        gdn.ctypes.byref(gdn.gdn_verify_shape(5, 3, V, gdn._DTYPES[TYPES[dtype]], V, V)))
    assert (need > 0) == (V > 65536)
    check(*case(V, 5, 3, V, dtype))
    check(*case(V + 1, 5, 3, V, dtype, onehot=True))


def test_two_kernels_borders_rests_and_graph():
    """The small cases above again where a row takes two kernels."""
    V = 131072
    p = torch.full((6, 2, V), 1.0 / V)
    q = torch.zeros(6, 1, V)
    q[:, :, 5] = 1.0
    x = torch.full((6, 1), 5, dtype=torch.int32)
    u = torch.zeros(6, 2)
    u[:, 0] = 0.9
    u[:, 1] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 0.25, 1.0 / (V - 1), 0.75])
    tokens, _ = check(p, q, x, u, None)
    assert tokens[0, 0] == 0 and tokens[1, 0] == V - 1
    q = p[:, :1] * 2                                    # nothing is left of max(p - q, 0)
    p[2] = 0.0
    p[3, :, ::2] = float("nan")
    check(p, q, x, u, None)
    p, q, x, u, n = (t.to(DEV) for t in case(11, 7, 3, 70001, "f32"))
    ws = torch.full((gdn.load_library().gdn_verify_workspace_bytes(
        gdn.ctypes.byref(gdn.gdn_verify_shape(7, 3, 70001, 0, 70001, 70001))),), 255, dtype=torch.uint8, device=DEV)
    tokens, emit = torch.zeros(7, 4, dtype=torch.int32, device=DEV), torch.zeros(7, dtype=torch.int32, device=DEV)
    kw = dict(draft_count=n, tokens=tokens, emit_count=emit, workspace=ws)
    gdn.gdn_verify_drafts(p, q, x, u, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_verify_drafts(p, q, x, u, **kw)
    for _ in range(3):
        u.copy_(torch.rand_like(u))
        graph.replay()
        torch.cuda.synchronize()
        got = tokens.clone(), emit.clone()
        want = gdn.gdn_verify_drafts(p, q, x, u, draft_count=n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
