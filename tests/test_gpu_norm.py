"""The block norms against the fp64 oracle.

Bounds, element by element, with e half a step of the type relative to the value
and U = 2^-24: h is rounded once, e |h|, after at most 40 roundings in fp32 (a
mean of D squares summed in a tree over 8 or 4 per vector, up to 16 vectors and
10 levels, halved by the root; the gate; the products) of its two terms,
40 U (|residual| + |scale m|).  normed adds the same of its own norm,
e |normed| + 40 U |normed|, and h's error times the factor it is scaled by.
"""

import numpy as np
import pytest
import torch

import gated_deltanet_03_amd as gdn
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24


def run(T, D, dtype, group=None, act="none", residual=True, post=True, nxt=True, eps=1e-6, scale=0.7, seed=0,
        edit=None, **kw):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]

    def n(*s):
        return torch.randn(*s, generator=g).to(t)
    c = dict(y=n(T, D), gate=n(T, D) * 2 if act != "none" else None, residual=n(T, D) * 2 if residual else None,
             post=1 + 0.2 * n(group or D) if post else None, nxt=1 + 0.2 * n(D) if nxt else None)
    if edit:
        edit(c)
    d = {k: None if v is None else v.to(DEV) for k, v in c.items()}
    h, normed = gdn.gdn_block_norm(d["y"], gate=d["gate"], gate_act=act, residual=d["residual"], residual_scale=scale,
                                   post_weight=d["post"], next_weight=d["nxt"], eps=eps, **kw)
    rh, rn, mag = oo.block_norm(c["y"], c["gate"], act, c["residual"], scale, c["post"], c["nxt"], eps)
    e = E[t]
    tiny = 2.0 ** -25 if dtype == "f16" else 1e-37
    off = np.abs(h.cpu().double().numpy() - rh)
    assert (off <= e * np.abs(rh) + 40 * U * mag + tiny).all(), (off / (np.abs(rh) + 1e-30)).max()
    assert (normed is None) == (not nxt)
    if nxt:
        factor = np.abs(c["nxt"].double().numpy()) / np.sqrt((rh ** 2).mean(-1, keepdims=True) + eps)
        off = np.abs(normed.cpu().double().numpy() - rn)
        assert (off <= (e + 40 * U) * np.abs(rn) + 40 * U * mag * factor + tiny).all(), off.max()
    return h, normed


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 3, 8, 64, 100, 127, 512, 513, 1000, 1024, 2048, 4096, 4099, 5120, 8192, 8195, 16384])
def test_widths(dtype, D):
    run(5, D, dtype, act="silu", seed=D)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("groups", [1, 3, 32, 100])
def test_groups(dtype, group, groups):
    run(7, group * groups, dtype, group=group, act="silu", residual=False, nxt=False, seed=group)
    run(3, group * groups, dtype, group=group, act="sigmoid", seed=group)


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("nxt", [False, True])
def test_parts(act, post, residual, nxt):
    for dtype in TYPES:
        run(4, 256, dtype, act=act, post=post, residual=residual, nxt=nxt)


@pytest.mark.parametrize("T", [0, 1, 2, 5, 1000])
def test_rows(T):
    h, n = run(T, 192, "bf16", act="silu", group=64)
    assert h.shape == n.shape == (T, 192)


def test_zero_rows_and_large_gates():
    def edit(c):
        c["y"][1] = 0
        c["residual"][1] = 0
        c["gate"][0] = -200.0      # act 0
        c["gate"][2] = 200.0       # silu: the gate itself
    h, n = run(4, 320, "f32", act="silu", edit=edit)
    assert (h[1] == 0).all() and (n[1] == 0).all()


def test_nan_stays_in_its_row():
    y = torch.randn(3, 512, device=DEV).to(torch.bfloat16)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    clean, cn = gdn.gdn_block_norm(y, post_weight=w, next_weight=w)
    y[1, 5] = float("nan")
    h, n = gdn.gdn_block_norm(y, post_weight=w, next_weight=w)
    assert torch.isnan(h[1]).all() and torch.isnan(n[1]).all()
    for r in (0, 2):
        assert torch.equal(h[r], clean[r]) and torch.equal(n[r], cn[r])


def test_in_place_and_other_shapes():
    t = torch.bfloat16
    y, x, z = (torch.randn(2, 3, 640, device=DEV).to(t) for _ in range(3))
    w, w2 = torch.ones(640, dtype=t, device=DEV), torch.ones(640, dtype=t, device=DEV)
    kw = dict(gate=z, residual_scale=0.5, post_weight=w, next_weight=w2)
    h, n = gdn.gdn_block_norm(y, residual=x, **kw)
    x1, y1 = x.clone(), y.clone()
    h1, n1 = gdn.gdn_block_norm(y, residual=x1, out=x1, **kw)
    assert h1 is x1 and torch.equal(h, h1) and torch.equal(n, n1)
    h2, n2 = gdn.gdn_block_norm(y1, residual=x, out=y1, **kw)
    assert h2 is y1 and torch.equal(h, h2) and torch.equal(n, n2) and h.shape == (2, 3, 640)


def test_rows_off_16_bytes():
    """Views that start inside a 16-byte line."""
    t = torch.bfloat16
    base = torch.randn(1 + 6 * 256, device=DEV).to(t)
    y = base[1:].view(6, 256)
    h, n = gdn.gdn_block_norm(y, post_weight=base[3:259], next_weight=base[5:261])
    h2, n2 = gdn.gdn_block_norm(y.clone(), post_weight=base[3:259].clone(), next_weight=base[5:261].clone())
    assert torch.equal(h, h2) and torch.equal(n, n2)


def test_graph_replays():
    t = torch.bfloat16
    y, x = (torch.randn(4, 1024, device=DEV).to(t) for _ in range(2))
    w = torch.ones(1024, dtype=t, device=DEV)
    h, n = torch.empty_like(y), torch.empty_like(y)
    kw = dict(residual=x, post_weight=w, next_weight=w, out=h, normed=n)
    gdn.gdn_block_norm(y, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_block_norm(y, **kw)
    for _ in range(4):
        y.copy_(torch.randn_like(y))
        graph.replay()
        torch.cuda.synchronize()
        got = h.clone(), n.clone()
        gdn.gdn_block_norm(y, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], h) and torch.equal(got[1], n)


def test_element_offsets_past_32_bits():
    T, D = 140000, 16384
    y = torch.ones(T, D, dtype=torch.bfloat16, device=DEV)
    y[-1] = 3.0
    h, _ = gdn.gdn_block_norm(y, residual_scale=2.0, out=y)
    assert y.numel() > 2 ** 31 and (h[-1] == 6.0).all() and (h[:3] == 2.0).all() and (h[-3:-1] == 2.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,group", [(17000, 64, 16), (4500, 1000, None), (4099, 4096, 128), (4097, 4099, None)])
def test_more_rows_than_workgroups(dtype, T, D, group):
    """Above 4096 workgroups the kernel loops over rows, keeping the weights."""
    run(T, D, dtype, group=group, act="sigmoid", seed=T)


def test_more_rows_than_workgroups_in_place():
    y = torch.randn(9000, 1024, device=DEV).to(torch.bfloat16)
    r = torch.randn_like(y)
    w = torch.ones(1024, device=DEV, dtype=torch.bfloat16)
    want = gdn.gdn_block_norm(y, residual=r, residual_scale=0.5, post_weight=w, next_weight=w)
    got = gdn.gdn_block_norm(y, residual=r, residual_scale=0.5, post_weight=w, next_weight=w, out=r)
    assert got[0] is r and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_rows_than_one_launch_takes():
    """A workgroup of 1024 threads a row: 2^22 rows are 2^32 threads."""
    T, D = 2 ** 22 + 3, 8200
    y = torch.ones(T, D, dtype=torch.bfloat16, device=DEV)
    y[-3:] = 3.0
    y[2 ** 22 - 2:2 ** 22] = 5.0
    h, _ = gdn.gdn_block_norm(y, residual_scale=2.0, out=y)
    for at, want in ((slice(0, 2), 2.0), (slice(2 ** 22 - 4, 2 ** 22 - 2), 2.0), (slice(2 ** 22 - 2, 2 ** 22), 10.0),
                     (slice(-3, None), 6.0)):
        assert (h[at] == want).all()
