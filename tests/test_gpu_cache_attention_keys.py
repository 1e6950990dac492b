"""Every key is read from its own row, however the keys' buffers follow each other.

Key j is -1 in coordinate j mod 31 and 0 elsewhere; a query has a large number in the first 31 coordinates but one, its
class, where it has 0.  So the score of a key of the query's class is exactly 0, that of every other key so low that its
weight is exactly 0: a row of keys that is read too early or too late, or taken for another, changes which keys count
(buffers hold rows 64 or 128 keys apart in turn, which are of other classes).
Column c of the value of key j is 1 where (j / 16) mod 31 = c and 0 elsewhere, column 31 is 1.  With n keys of the class
in sight, all sums are whole numbers below 2^24 times one power of two, exact in fp32 whatever their order, and o is
count / n, off by 3 roundings in fp32 (1 / l, its product, o) and in a 16-bit type by its own one beside them.  Where
no key of the class is in sight all scores are the same; the weights, 1 but for 2^-13 at most, are the same too, and n of
them are added with n roundings above and below the line.
"""

import random

import numpy as np
import pytest
import torch

from gpu_common import DEV, say
from test_gpu_cache_attention_cuts import draw

pytestmark = pytest.mark.gpu

TYPES = {"f32": (torch.float32, 0.0), "f16": (torch.float16, 2.0 ** -11), "bf16": (torch.bfloat16, 2.0 ** -8)}
E = 2.0 ** -24
LARGE = 4096.0      # times d^-1/2: 256 and more


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_03_amd as m
    m.load_library()
    return m


def classes(gdn, new, ctx, Hkv, G, d, page, dtype, window=0, spare=0):
    kind, u = TYPES[dtype]
    need = [-(-n // page) for n in ctx]
    starts = np.concatenate([[0], np.cumsum(need)])
    N = len(new)
    j = torch.cat([torch.arange(n * page) for n in need]).view(-1, page).to(DEV)
    v = torch.zeros(len(j), 1, page, d, device=DEV, dtype=kind)
    v.scatter_(3, ((j >> 4) % 31)[:, None, :, None], 1.0)
    v[..., 31] = 1.0
    k = torch.zeros_like(v)
    k.scatter_(3, (j % 31)[:, None, :, None], -1.0)
    k, v = (x.expand(-1, Hkv, -1, -1).contiguous() for x in (k, v))
    table = np.full((N, max(max(need), 1) + spare), -1, dtype=np.int32)
    for s in range(N):
        table[s, :need[s]] = np.arange(starts[s], starts[s + 1])
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T, Hq = int(cu[-1]), Hkv * G
    mine = (torch.arange(T, device=DEV)[:, None] * 7 + torch.arange(Hq, device=DEV) * 5) % 31
    q = torch.randn(T, Hq, d, device=DEV).to(kind)
    q[..., :31] = LARGE
    q.scatter_(2, mine[..., None], 0.0)
    o = torch.full_like(q, float("nan"))
    gdn.gdn_cache_attention(q, k, v, torch.from_numpy(table).to(DEV), torch.tensor(ctx, dtype=torch.int32, device=DEV),
                            cu_seqlens=torch.from_numpy(cu).to(DEV), window=window, o=o)
    # what each row sees of its class, or of all where there is none: counts of (class, column) before each place
    hi = np.concatenate([np.arange(m - n, m) for n, m in zip(new, ctx)]) + 1
    lo = np.maximum(hi - window, 0) if window else np.zeros_like(hi)
    every = torch.arange(max(ctx), device=DEV)
    cum = torch.zeros(len(every) + 1, 31 * 31, device=DEV)
    cum[1:].scatter_(1, (every % 31 * 31 + (every >> 4) % 31)[:, None], 1.0)
    cum = cum.cumsum(0).view(-1, 31, 31)
    hi, lo = (torch.from_numpy(x).to(DEV) for x in (hi, lo))
    seen = cum[hi] - cum[lo]                                           # [T, class, column]
    want = seen.gather(1, mine[..., None].expand(-1, -1, 31)).double()   # [T, Hq, column]
    count = want.sum(-1, keepdim=True)
    none = count == 0
    want = torch.where(none, seen.sum(1)[:, None].double(), want)
    count = torch.where(none, (hi - lo)[:, None, None].double(), count)
    rel = 3 * E + u + torch.where(none, 2 * (count + 64) * E, 0.0)
    got = o.double()
    assert not torch.isnan(got).any()
    off = ((got[..., :31] - want / count).abs() / (rel * want / count).clamp(min=1e-300)).amax()
    last = ((got[..., 31:32] - 1.0).abs() / rel).amax()
    assert float(off) <= 1.0 and float(last) <= 1.0, (float(off), float(last))
    assert not got[..., 32:].any()


# Tiles of 128 rows over three blocks of keys and more, whole and cut, at every width of a key.
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("new,ctx,Hkv,G", [([300], [300], 2, 1), ([129, 500], [700, 4000], 4, 2), ([2000], [2000], 8, 4),
                                           ([513, 40, 700, 1000], [513, 3000, 6000, 1100], 2, 8)])
def test_many_rows(gdn, new, ctx, Hkv, G, d, dtype):
    say(f"keys {dtype} {d} {new} {ctx}")
    classes(gdn, new, ctx, Hkv, G, d, 32, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("seed", range(25))
def test_any_rows(gdn, seed, dtype):
    c = draw(random.Random(500 + seed))
    say(f"keys {dtype} {c}")
    ctx = [max(n, 1) for n in c["ctx"]]
    if sum(c["new"]) == 0:
        c["new"][0] = 1
    classes(gdn, c["new"], ctx, c["Hkv"], c["G"], c["d"], c["page"], dtype, c["window"], c["spare"])
