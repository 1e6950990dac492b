"""Verification of batches of large vocabularies: equal to the fp64 oracle, token for token.

Above 65536 entries a row takes two kernels; 64 rows of 70001 are 2240 workgroups of the first."""

import ctypes

import pytest
import torch

import gated_deltanet_03_amd as gdn
from test_gpu_verify import DEV, TYPES, case, check

pytestmark = pytest.mark.gpu


def dirty(B, K, V, dtype):
    sh = gdn.gdn_verify_shape(B, K, V, gdn._DTYPES[TYPES[dtype]], V, V)
    need = gdn.load_library().gdn_verify_workspace_bytes(ctypes.byref(sh))
    assert need == B * -(-V // 2048) * 8
    return torch.full((need,), 255, dtype=torch.uint8, device=DEV)      # NaN everywhere


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("onehot", [False, True])
@pytest.mark.parametrize("B,V", [(64, 70001), (64, 65537), (40, 131072), (33, 131071)])
def test_thousands_of_tiles(dtype, onehot, B, V):
    """Rows that end early and late in their last tile; idle rows and counts above K among them."""
    assert B * -(-V // 2048) > 2048
    p, q, x, u, n = case(V + onehot, B, 2, V, dtype, onehot)
    u[:4, 2] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.999, 0.99])       # the first and the last tiles
    check(p, q, x, u, n, workspace=dirty(B, 2, V, dtype))


@pytest.mark.parametrize("B", [8, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rests_and_weights_that_are_no_numbers(B, dtype):
    V = 70001
    p, q, x, u, _ = case(5, B, 2, V, dtype)
    q[0::8] = (p[0::8, :2].float() * 2).to(q.dtype)     # nothing is left of max(p - q, 0)
    u[0::8, 0] = 0.8
    p[1::8] = 0.0                                       # no weight at all
    p[2::8, :, ::2] = float("nan")
    p[3::8, :, 5] = float("inf")
    p[4::8, :, 100:] = -1.0
    q[5::8, :, ::3] = float("nan")
    p[6::8, :, 69000:] = float("nan")                   # a last tile without weight
    ws = dirty(B, 2, V, dtype)
    tokens, emit = check(p, q, x, u, None, workspace=ws)
    assert (tokens[1::8] == -1).all() and (emit[1::8] == 1).all()
    check(p, None, x, u, None, workspace=ws)


@pytest.mark.parametrize("B", [8, 64])
def test_tokens_outside_the_vocabulary_and_padded_rows(B):
    V = 70001
    p, q, x, u, n = case(6, B, 2, V, "bf16")
    x[0, 0], x[1, 1], x[2, 0], x[3, 0] = -1, V, 2 ** 31 - 1, -2 ** 31
    check(p, q, x, u, n)
    check(p, None, x, u, None)
    wide = torch.full((B, 3, V + 23), 9.0, dtype=p.dtype, device=DEV)
    wide[..., :V] = p.to(DEV)
    narrow = torch.full((B, 2, V + 1), 9.0, dtype=p.dtype, device=DEV)
    narrow[..., :V] = q.to(DEV)
    rest = [t.to(DEV) for t in (x, u)]
    a = gdn.gdn_verify_drafts(wide[..., :V], narrow[..., :V], *rest, draft_count=n.to(DEV))
    b = gdn.gdn_verify_drafts(p.to(DEV), q.to(DEV), *rest, draft_count=n.to(DEV))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_of_a_large_batch():
    B, V = 64, 70001
    p, q, x, u, n = (t.to(DEV) for t in case(7, B, 2, V, "f32"))
    tokens, emit = torch.zeros(B, 3, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    kw = dict(draft_count=n, tokens=tokens, emit_count=emit, workspace=dirty(B, 2, V, "f32"))
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
