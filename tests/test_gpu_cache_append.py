"""gdn_cache_append against the fp64 oracle.

Bound of a rotated element, with |x1| + |x2| the oracle's size: its rounding u |y|, and 8 e (|x1| + |x2|), e = 2^-24:
cosine and sine are off by 2^-25 of their series and 3 e of its evaluation and of the reduced angle, the products and
their sum by 2 e.  What is not rotated is equal."""

import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, f64, say
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_03_amd as m
    m.load_library()
    return m


def make(seed, new, ctx, Hq, Hkv, d, page, dtype, rotary, axes=1, far=50000):
    rng = np.random.default_rng(seed)
    T, n = TYPES[dtype], sum(new)
    need = [-(-max(x, 0) // page) for x in ctx]
    pages = sum(need) + 2
    table = np.full((len(new), max(max(need), 1)), -1, dtype=np.int32)
    order, at = rng.permutation(pages), 0
    for s in range(len(new)):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]

    def normal(*shape):
        return torch.from_numpy(rng.standard_normal(shape)).to(T)
    c = dict(q=normal(n, Hq, d), k=normal(n, Hkv, d), v=normal(n, Hkv, d), kc=normal(pages, Hkv, page, d),
             vc=normal(pages, Hkv, page, d), table=torch.from_numpy(table), lens=torch.tensor(ctx, dtype=torch.int32),
             cu=torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)), dtype=dtype,
             freq=torch.from_numpy(10000.0 ** (-np.arange(rotary // 2) / max(rotary // 2, 1))).float() if rotary else None,
             positions=None, axis=None)
    if axes > 1:
        c["positions"] = torch.from_numpy(rng.integers(-50, far, (axes, n)).astype(np.int32))
        c["axis"] = torch.from_numpy(rng.integers(-1, axes + 1, rotary // 2).astype(np.int32))
    return c


def dev(c):
    return {n: (x.to(DEV).clone() if torch.is_tensor(x) else x) for n, x in c.items()}


def oracle(c, interleaved=False, with_q=True):
    return co.append(c["k"], c["v"], c["kc"], c["vc"], c["table"], c["lens"], cu_seqlens=c["cu"],
                     q=c["q"] if with_q else None, inv_freq=c["freq"], positions=c["positions"], pair_axis=c["axis"],
                     interleaved=interleaved)


def run(gdn, c, interleaved=False, with_q=True):
    d = dev(c)
    q = gdn.gdn_cache_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["lens"], cu_seqlens=d["cu"],
                             q=d["q"] if with_q else None, inv_freq=d["freq"], positions=d["positions"],
                             pair_axis=d["axis"], interleaved=interleaved)
    return q, d["kc"], d["vc"]


def near(x, y, size, dtype, what):
    bound = U[dtype] * np.abs(y) + 8 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == "f16" else 0)
    err = np.abs(f64(x) - y)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    say(f"  {what}: worst {worst:.3f} of the bound")
    assert worst <= 1.0, what


def check(got, ref, c):
    q, kc, vc = got
    if q is not None:
        near(q, ref["q"], ref["q_size"], c["dtype"], "q")
    near(kc, ref["k_cache"], ref["k_size"], c["dtype"], "k_cache")
    assert np.array_equal(f64(vc), ref["v_cache"])


SHAPES = [
    # new, ctx, Hq, Hkv, d, page, rotary, axes
    ([1], [1], 1, 1, 32, 16, 32, 1),
    ([1], [1000], 32, 8, 128, 64, 128, 1),
    ([5, 0, 1, 70], [5, 3, 40, 100], 6, 2, 64, 16, 64, 1),
    ([9, 33], [50, 33], 4, 4, 128, 48, 32, 3),
    ([7], [300], 3, 1, 256, 32, 64, 2),
    ([7, 2], [70, 20], 2, 2, 64, 16, 6, 1),
    ([3], [17], 5, 5, 32, 16, 2, 8),
    ([1, 1, 1], [16, 17, 32], 8, 2, 256, 16, 256, 1),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[2]}.{s[3]}-{s[4]}-r{s[6]}-a{s[7]}".replace(" ", ""))
def test_against_the_oracle(gdn, shape, interleaved, dtype):
    new, ctx, Hq, Hkv, d, page, rotary, axes = shape
    c = make(3, new, ctx, Hq, Hkv, d, page, dtype, rotary, axes)
    say(f"append {dtype} {shape} interleaved={interleaved}")
    check(run(gdn, c, interleaved), oracle(c, interleaved), c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_rotation(gdn, dtype):
    c = make(5, [4, 6], [30, 6], 2, 2, 64, 16, dtype, 0)
    _, kc, vc = run(gdn, c, with_q=False)
    ref = oracle(c, with_q=False)
    assert np.array_equal(f64(kc), ref["k_cache"]) and np.array_equal(f64(vc), ref["v_cache"])


def test_keys_alone(gdn):
    c = make(5, [4, 6], [30, 6], 2, 2, 64, 16, "bf16", 64)
    check(run(gdn, c, with_q=False), oracle(c, with_q=False), c)


def test_far_positions(gdn):
    """Angles of millions of turns, in both directions."""
    c = make(7, [300], [300], 2, 1, 128, 16, "f32", 128)
    c["positions"] = torch.from_numpy(np.random.default_rng(1).integers(-(1 << 30), 1 << 30, 300).astype(np.int32))
    check(run(gdn, c), oracle(c), c)


@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 6)])
def test_slices_of_one_projection_and_in_place(gdn, d, rotary):
    new, Hq, Hkv = [5, 11], 6, 2
    c = make(9, new, [40, 11], Hq, Hkv, d, 16, "bf16", rotary)
    ref = oracle(c)
    x = dev(c)
    rows = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1)
    q, k, v = (t.unflatten(1, (-1, d)) for t in rows.split([Hq * d, Hkv * d, Hkv * d], 1))
    got = gdn.gdn_cache_append(k, v, x["kc"], x["vc"], x["table"], x["lens"], cu_seqlens=x["cu"], q=q,
                               inv_freq=x["freq"])
    check((got, x["kc"], x["vc"]), ref, c)
    x = dev(c)
    same = gdn.gdn_cache_append(x["k"], x["v"], x["kc"], x["vc"], x["table"], x["lens"], cu_seqlens=x["cu"], q=x["q"],
                                inv_freq=x["freq"], q_out=x["q"])
    assert same is x["q"] and torch.equal(same, got)


def test_dense_is_ragged(gdn):
    c = make(11, [6, 6, 6], [50, 6, 20], 4, 2, 64, 16, "f16", 64)
    a, d = run(gdn, c), dev(c)
    q = gdn.gdn_cache_append(d["k"].view(3, 6, 2, 64), d["v"].view(3, 6, 2, 64), d["kc"], d["vc"], d["table"],
                             d["lens"], q=d["q"].view(3, 6, 4, 64), inv_freq=d["freq"])
    assert torch.equal(q.view(18, 4, 64), a[0]) and torch.equal(d["kc"], a[1]) and torch.equal(d["vc"], a[2])


def test_tokens_without_a_place(gdn):
    """Places before and behind the table and numbers that are no page: nothing is written there, queries are."""
    c = make(13, [20, 20, 20], [30, 40, 40], 2, 2, 64, 16, "f32", 64)
    c["lens"] = torch.tensor([8, 60, 40], dtype=torch.int32)
    c["table"][2, 1], c["table"][2, 2] = 1 << 29, -3
    check(run(gdn, c), oracle(c), c)


def test_rows_behind_the_last_sequence_stay(gdn):
    c = make(15, [3, 4], [20, 4], 2, 2, 64, 16, "bf16", 64)
    ref, d = oracle(c), dev(c)
    pad = [torch.cat([d[n], torch.full((9, 2, 64), math.nan, dtype=torch.bfloat16, device=DEV)]) for n in ("q", "k", "v")]
    out = torch.full((16, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_cache_append(pad[1], pad[2], d["kc"], d["vc"], d["table"], d["lens"], cu_seqlens=d["cu"], q=pad[0],
                         inv_freq=d["freq"], q_out=out)
    check((out[:7], d["kc"], d["vc"]), ref, c)
    assert (out[7:] == 5.0).all()


def test_very_many_sequences(gdn):
    rng = np.random.default_rng(2)
    new = [int(x) for x in rng.integers(0, 4, 5000)]
    ctx = [n + int(x) for n, x in zip(new, rng.integers(0, 12, 5000))]
    c = make(17, new, ctx, 1, 1, 32, 16, "bf16", 32)
    check(run(gdn, c), oracle(c), c)
