"""Every key counts once, however the work is cut.

All scores are 0, so every weight is 1 and every sum a whole number below 2^24: exact in fp32, whatever its order.
Column c of the value of key j is 1 where (j / 16) mod 31 = c and 0 elsewhere, column 31 is 1: o times the number of keys
that a token sees is their count in each class, off by 3 roundings (1 / l, its product, the one here)."""

import random

import numpy as np
import pytest
import torch

from gpu_common import DEV, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_03_amd as m
    m.load_library()
    return m


def draw(rng):
    kind = rng.choice(["next", "drafts", "prompts", "mixed", "one"])
    Hkv, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    d, page = rng.choice([32, 64, 64, 128, 256]), rng.choice([16, 32, 48, 64, 256])
    far = rng.choice([100, 1000, 5000, 20000])
    if kind == "next":
        new = [1] * rng.choice([1, 3, 17, 64, 130, 300])
    elif kind == "drafts":
        new = [rng.randint(0, 8) for _ in range(rng.choice([1, 5, 20, 90]))]
    elif kind == "prompts":
        new = [rng.randint(1, 1500) for _ in range(rng.randint(1, 5))]
    elif kind == "one":
        new = [rng.randint(1, 4000)]
    else:
        new = [rng.choice([1, 1, 1, 4, rng.randint(30, 900)]) for _ in range(rng.randint(2, 40))]
    room = 60_000_000 // (Hkv * d)               # keys of a cache of 240 MB
    ctx = []
    for n in new:
        old = rng.choice([0, rng.randint(0, far), rng.randint(0, far), rng.randint(0, 30)])
        old = max(0, min(old, room - n))
        room -= n + old + page
        ctx.append(n + old if room > 0 else n)
    return dict(new=new, ctx=ctx, Hkv=Hkv, G=G, d=d, page=page, window=rng.choice([0, 0, 0, rng.randint(1, 3000)]),
                spare=rng.choice([0, 0, 7, 400]))


@pytest.mark.parametrize("seed", range(60))
def test_every_key_counts_once(gdn, seed):
    count(gdn, draw(random.Random(seed)))


@pytest.mark.parametrize("seed", range(20))
def test_tables_of_the_widest(gdn, seed):
    """Tables for 2^26 keys a sequence: work is cut in units of many keys, so that its sum stays below 2^30."""
    rng = random.Random(1000 + seed)
    c = draw(rng)
    while c["Hkv"] * c["d"] > 1024:
        c["Hkv"], c["d"] = max(c["Hkv"] // 2, 1), max(c["d"] // 2, 32)
    most = rng.choice([1, 3, 40])
    count(gdn, dict(c, new=c["new"][:most], ctx=[min(n, 9000) for n in c["ctx"][:most]], page=1024, spare=65536 - 9))


def count(gdn, c):
    new, ctx, Hkv, G, d, page = c["new"], c["ctx"], c["Hkv"], c["G"], c["d"], c["page"]
    say(f"cut {c}")
    need = [-(-n // page) for n in ctx]
    starts = np.concatenate([[0], np.cumsum(need)])
    N, most = len(new), max(max(need), 1) + c["spare"]
    j = torch.cat([torch.arange(n * page) for n in need] or [torch.zeros(0, dtype=torch.long)]).view(-1, page).to(DEV)
    v = torch.zeros(len(j), 1, page, d, device=DEV)
    v.scatter_(3, ((j >> 4) % 31)[:, None, :, None], 1.0)
    v[..., 31] = 1.0
    v = v.expand(-1, Hkv, -1, -1).contiguous()
    k = torch.zeros_like(v)
    table = np.full((N, most), -1, dtype=np.int32)
    for s in range(N):
        table[s, :need[s]] = np.arange(starts[s], starts[s + 1])
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn(int(cu[-1]), Hkv * G, d, device=DEV)
    o = torch.full_like(q, float("nan"))
    gdn.gdn_cache_attention(q, k, v, torch.from_numpy(table).to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV),
                            cu_seqlens=torch.from_numpy(cu).to(DEV), window=c["window"], o=o)
    # what each token sees
    hi = np.concatenate([np.arange(m - n, m) for n, m in zip(new, ctx)] or [np.zeros(0, int)]) + 1
    lo = np.maximum(hi - c["window"], 0) if c["window"] else np.zeros_like(hi)
    every = np.arange(max(max(ctx), 1))
    cum = np.zeros((len(every) + 1, 32))
    cum[1:, :31] = np.cumsum(((every >> 4) % 31)[:, None] == np.arange(31), 0)
    cum[1:, 31] = every + 1
    want = torch.from_numpy(cum[hi] - cum[lo]).to(DEV)[:, None]
    n = torch.from_numpy(hi - lo).to(DEV)[:, None, None].double()
    got = o[..., :32].double() * n
    off = ((got - want).abs() / want.clamp(min=1)).amax() if len(q) else 0.0
    assert not torch.isnan(o).any() and float(off) <= 3 * 2.0 ** -24, (float(off), c)
    assert not o[..., 32:].any()


@pytest.mark.parametrize("new,cols,G,dtype", [
    ([1_050_000], 64, 1, torch.float32), ([360_000], 64, 8, torch.bfloat16), ([108_000], 96, 64, torch.bfloat16),
    ([40] * 1000 + [900_000, 3], 128, 2, torch.float16), ([5, 2_000_000, 0, 70], 3, 1, torch.bfloat16)])
def test_far_more_new_tokens_than_the_table_has_keys(gdn, new, cols, G, dtype):
    """Rows behind the table's end see all of its keys, each of them once, and every row is written.

    All sequences share the table's pages; the value of key j is 1 in column (j / 16) mod 31 and in column 31.  A weight
    is 1, o a count over a count: off by 3 roundings of 2^-24 and its own to the type."""
    u = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
    room, d, N, T = cols * 16, 32, len(new), sum(new)
    say(f"behind the table: {N} sequences, {T} tokens, {room} keys")
    every = torch.arange(room, device=DEV)
    v = torch.zeros(room, d, device=DEV, dtype=dtype)
    v[every, (every >> 4) % 31] = 1.0
    v[:, 31] = 1.0
    kv = v.view(cols, 1, 16, d).contiguous()
    table = torch.arange(cols, dtype=torch.int32, device=DEV).repeat(N, 1)
    lens = torch.tensor(new, dtype=torch.int32, device=DEV)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(DEV)
    o = torch.full((T, G, d), float("nan"), device=DEV, dtype=dtype)
    gdn.gdn_cache_attention(torch.zeros_like(o), kv, kv.clone(), table, lens, cu_seqlens=cu, o=o)
    place = torch.arange(T, device=DEV) - torch.repeat_interleave(cu[:-1].long(), lens.long(), output_size=T)
    seen = place.clamp(max=room - 1) + 1
    want = torch.zeros(room + 1, d, dtype=torch.float64, device=DEV)
    want[1:] = v.double().cumsum(0) / (every + 1.0)[:, None].double()
    for t in range(0, T, 100_000):
        w, got = want[seen[t:t + 100_000]][:, None], o[t:t + 100_000].double()
        off = ((got - w).abs() / ((3 * 2.0 ** -24 + u) * w).clamp(min=1e-300)).amax()
        assert float(off) <= 1.0, (t, float(off))
