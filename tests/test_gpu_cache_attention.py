"""gdn_cache_attention against the fp64 oracle.

Bound of one output element, with A = sum w |v| / sum w (the oracle's size), u the rounding of the type (bf16 2^-8,
fp16 2^-11, fp32 2^-24) and e = 2^-24:
  * o's own rounding: u |o|;
  * weights rounded to a 16-bit type: u A;
  * a score is a sum of d products and its factor: off by at most (d + 3) e scale sum |q||k|, and its maximum's
    subtraction and the exponential add 4 e (|score| <= scale sum |q||k|) + 4 e; a factor on a weight acts above and
    below the line: twice;
  * sums over n keys in fp32, above and below: 2 (n + 64) e.
"""

import math

import numpy as np
import pytest
import torch

from gpu_common import DEV, f64, say
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = 2.0 ** -24


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_03_amd as m
    m.load_library()
    return m


def make(seed, new, ctx, Hq, Hkv, d, page, dtype, spread=1.5, cols=None):
    """Inputs on the CPU; the cache's unused rows and pages hold NaN."""
    rng = np.random.default_rng(seed)
    T = TYPES[dtype]
    need = [-(-n // page) for n in ctx]
    pages = sum(need) + 2
    table = np.full((len(new), cols or max(max(need), 1)), -1, dtype=np.int32)
    order, at = rng.permutation(pages), 0
    kc = torch.full((pages, Hkv, page, d), math.nan, dtype=T)
    vc = kc.clone()
    for s, n in enumerate(ctx):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        for p in range(need[s]):
            rows = min(page, n - p * page)
            kc[table[s, p], :, :rows] = torch.from_numpy(rng.standard_normal((Hkv, rows, d))).to(T)
            vc[table[s, p], :, :rows] = torch.from_numpy(rng.standard_normal((Hkv, rows, d))).to(T)
    q = torch.from_numpy(spread * rng.standard_normal((sum(new), Hq, d))).to(T)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, kc=kc, vc=vc, table=torch.from_numpy(table), lens=torch.tensor(ctx, dtype=torch.int32),
                cu=torch.from_numpy(cu), scale=d ** -0.5, dtype=dtype)


def oracle(c, window=0):
    return co.attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], c["scale"], cu_seqlens=c["cu"], window=window)


def call(gdn, c, window=0, dense=False, **kw):
    d = {n: (x.to(DEV) if torch.is_tensor(x) else x) for n, x in c.items()}
    q = d["q"]
    if dense:
        q = q.view(len(c["lens"]), -1, *q.shape[1:])
    o = gdn.gdn_cache_attention(q, d["kc"], d["vc"], d["table"], d["lens"], cu_seqlens=None if dense else d["cu"],
                                scale=c["scale"], window=window, **kw)
    return o.reshape(d["q"].shape)


def check(o, ref, c, what):
    d, n = c["q"].shape[-1], int(c["lens"].max()) if len(c["lens"]) else 0
    u = {"f32": E, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[c["dtype"]]
    rel = 2 * ((d + 3) * E * ref["score"] + 4 * E * (ref["score"] + 1)) + 2 * (n + 64) * E
    bound = u * np.abs(ref["o"]) + ref["size"] * (rel + (0 if c["dtype"] == "f32" else u))
    if c["dtype"] == "f16":
        bound = bound + 2.0 ** -25     # o below the normal numbers
    assert np.array_equal(np.isnan(f64(o)), np.isnan(ref["o"])), what   # rows never written hold NaN: seen or not
    err = np.nan_to_num(np.abs(f64(o) - ref["o"]))
    bound = np.nan_to_num(bound, nan=np.inf)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    say(f"  {what}: worst {worst:.3f} of the bound")
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"


SHAPES = [
    # new, ctx, Hq, Hkv, d, page
    ([1], [1], 1, 1, 32, 16),
    ([1], [301], 4, 4, 64, 16),
    ([1, 1, 1], [257, 16, 1000], 8, 2, 128, 32),
    ([1, 1], [33, 700], 6, 2, 256, 48),
    ([3, 0, 7, 1], [5, 9, 300, 64], 10, 2, 64, 64),
    ([8, 2], [520, 77], 8, 8, 32, 16),
    ([40, 1, 0, 130], [40, 300, 20, 203], 4, 2, 64, 16),
    ([129], [129], 2, 1, 128, 128),
    ([65, 33], [400, 33], 3, 1, 128, 48),
    ([90], [310], 4, 4, 256, 64),
    ([70], [95], 5, 1, 32, 32),
    ([2, 2, 2], [600, 2, 31], 16, 1, 128, 1024),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[1]}-{s[2]}.{s[3]}-{s[4]}-{s[5]}".replace(" ", ""))
def test_against_the_oracle(gdn, shape, dtype):
    new, ctx, Hq, Hkv, d, page = shape
    c = make(Hq + d + page, new, ctx, Hq, Hkv, d, page, dtype)
    say(f"attention {dtype} {shape}")
    check(call(gdn, c), oracle(c), c, "o")


# Prompts from one to many tiles of rows beside the card's workgroups, over themselves and over older text: the work is
# left whole, drawn out to whole shares, cut evenly, or cut behind whole rounds of tiles.
CUTS = [([1031], [1031], 4, 1, 64), ([520], [3000], 2, 2, 64), ([200, 900, 3], [1500, 900, 4000], 4, 1, 32),
        ([33], [6000], 4, 1, 128), ([700, 40], [700, 2500], 2, 1, 256)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d", CUTS)
def test_cuts(gdn, new, ctx, Hq, Hkv, d, dtype):
    c = make(61 + d, new, ctx, Hq, Hkv, d, 32, dtype)
    say(f"cuts {dtype} {new} {ctx}")
    check(call(gdn, c), oracle(c), c, "o")


def plain(c):
    """The formula in 64 bits on the GPU, for sizes that the oracle's loops take too long for."""
    d = {n: (x.to(DEV) if torch.is_tensor(x) else x) for n, x in c.items()}
    (N, _), ps, d_ = d["table"].shape, d["kc"].shape[2], d["kc"].shape[3]
    Hkv, cu = d["kc"].shape[1], c["cu"].tolist()
    G = c["q"].shape[1] // Hkv
    out = {"o": torch.zeros(c["q"].shape, dtype=torch.float64, device=DEV)}
    out["size"], out["score"] = torch.zeros_like(out["o"]), torch.zeros(*c["q"].shape[:2], 1, dtype=torch.float64, device=DEV)
    for s in range(N):
        L, n = cu[s + 1] - cu[s], int(c["lens"][s])
        j = torch.arange(n, device=DEV)
        page = d["table"][s].long()[j // ps]
        hidden = j > torch.arange(n - L, n, device=DEV)[:, None]
        for h in range(Hkv):
            k, v = (d[x][page, h, j % ps].double() for x in ("kc", "vc"))
            for g in range(h * G, h * G + G):
                q = d["q"][cu[s]:cu[s + 1], g].double()
                w = torch.softmax((c["scale"] * (q @ k.T)).masked_fill(hidden, -math.inf), -1)
                out["o"][cu[s]:cu[s + 1], g] = w @ v
                out["size"][cu[s]:cu[s + 1], g] = w @ v.abs()
                out["score"][cu[s]:cu[s + 1], g] = c["scale"] * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
    return {n: f64(x) for n, x in out.items()}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d", [
    ([2048, 700, 1, 63], [9000, 5000, 3000, 1031], 16, 4, 128), ([4000], [4000], 8, 8, 64),
    ([64, 1, 1, 1, 1, 1, 1, 1], [4096, 900, 700, 3000, 1500, 12000, 64, 129], 16, 4, 128),
    ([513, 300, 700, 64, 1000, 128], [513, 300, 700, 64, 1000, 128], 16, 2, 256), ([1] * 70, list(range(10, 7010, 100)), 8, 4, 64),
    ([5] * 9, [20000] + [50] * 8, 8, 2, 32)])
def test_large(gdn, new, ctx, Hq, Hkv, d, dtype):
    c = make(71, new, ctx, Hq, Hkv, d, 64, dtype)
    say(f"large {dtype} {new} {ctx}")
    check(call(gdn, c), plain(c), c, "o")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [1, 5, 16, 100, 5000])
@pytest.mark.parametrize("new,ctx", [([1, 4], [300, 90]), ([70, 3], [200, 3])])
def test_windows(gdn, new, ctx, window, dtype):
    c = make(7, new, ctx, 4, 2, 64, 16, dtype)
    say(f"window {window} {new} {dtype}")
    check(call(gdn, c, window), oracle(c, window), c, "o")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("L", [1, 5, 40])
def test_dense_is_ragged(gdn, L, dtype):
    c = make(11, [L] * 3, [L + 100, L, L + 33], 8, 2, 128, 32, dtype)
    assert torch.equal(call(gdn, c, dense=True), call(gdn, c))


@pytest.mark.parametrize("new", [[1, 1], [60, 60]])
def test_pages_that_are_none(gdn, new):
    """Page numbers outside of the cache hold no keys: in the middle, at the start, everywhere."""
    c = make(13, new, [300, 200], 4, 2, 64, 32, "bf16")
    c["table"][0, 3], c["table"][0, 0] = -1, 1 << 30
    c["table"][1, :] = -5
    ref = oracle(c)
    o = call(gdn, c)
    check(o, ref, c, "o")
    assert not o[int(c["cu"][1]):].any()


@pytest.mark.parametrize("new", [[2, 3], [50, 45]])
def test_rows_that_see_nothing(gdn, new):
    """No keys, fewer keys than new tokens, and lengths past the table and below zero."""
    c = make(17, new, [60, 60], 4, 2, 64, 16, "f32")
    for lens in ([0, 60], [1, 1], [-7, 59], [70, 1 << 30]):
        c["lens"] = torch.tensor(lens, dtype=torch.int32)
        ref = oracle(c)
        c2 = dict(c, lens=torch.tensor([60, 60]))
        o = call(gdn, c)
        check(o, ref, c2, f"lens {lens}")
        assert not o[torch.from_numpy((ref["size"] == 0).all(-1)).to(DEV)].any()


def test_rows_behind_the_last_sequence_stay(gdn):
    c = make(19, [3, 5], [40, 50], 4, 2, 64, 16, "bf16")
    q = torch.full((20, 4, 64), math.nan, dtype=torch.bfloat16)
    q[:8] = c["q"]
    ref = oracle(c)
    o = torch.full((20, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    got = call(gdn, dict(c, q=q), o=o)
    check(got[:8], ref, c, "o")
    assert (got[8:] == 7.0).all()


def test_queries_at_a_stride(gdn):
    c = make(23, [1] * 5, [100, 7, 33, 64, 250], 4, 2, 64, 16, "f16")
    wide = torch.full((5, 9, 64), math.nan, dtype=torch.float16)
    wide[:, 2:6] = c["q"]
    d = wide.to(DEV)[:, 2:6]
    o = gdn.gdn_cache_attention(d, c["kc"].to(DEV), c["vc"].to(DEV), c["table"].to(DEV), c["lens"].to(DEV),
                                cu_seqlens=c["cu"].to(DEV))
    check(o, oracle(c), c, "o")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("new", [[6], [100]])
def test_infinities_and_nan_touch_later_tokens_only(gdn, new, value, dtype):
    """One value that is no number: exactly its column of the tokens that see it is."""
    d, n = 64, 150
    c = make(29, new, [n], 4, 2, d, 16, dtype)
    at, first = n - 3, n - new[0]
    clean = call(gdn, c)
    c["vc"][c["table"][0, at // 16], 1, at % 16, 9] = value
    got = call(gdn, c)
    ref = oracle(c)["o"]
    hit = np.zeros(ref.shape, dtype=bool)
    hit[at - first:, 2:, 9] = True
    g = f64(got)
    assert np.array_equal(np.isnan(g), np.isnan(ref)) and np.array_equal(np.isinf(g), np.isinf(ref))
    assert (~np.isfinite(g) == hit).all()
    keep = torch.from_numpy(~hit).to(DEV)
    check(torch.where(keep, got, 0), dict(oracle(dict(c, vc=torch.nan_to_num(c["vc"], 0, 0, 0))), o=np.where(hit, 0, ref)),
          c, "the rest")
    assert torch.equal(got[:at - first], clean[:at - first])


@pytest.mark.parametrize("new", [[6], [100]])
def test_not_numbers_in_keys_and_queries(gdn, new):
    n = 150
    c = make(31, new, [n], 4, 2, 64, 16, "bf16")
    clean, first, at = call(gdn, c), n - new[0], n - 2
    c["kc"][c["table"][0, at // 16], 0, at % 16, 3] = math.nan
    c["q"][1, 3, 5] = math.nan
    got = call(gdn, c)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[at - first:, :2] = True
    hit[1, 3] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [[1], [40]])
def test_one_key_above_very_many(gdn, new, dtype):
    """Weights of 2^-15 of the largest that outweigh it together: none may be lost below the type's normal numbers."""
    d, n = 64, 8000
    c = make(37, new, [n], 1, 1, d, 16, dtype)
    c["q"][:] = 0
    c["q"][..., 0] = 8.0
    c["kc"][..., 0] = 0.0
    big = 15 * math.log(2.0)          # scale * 8 * k = 15 ln 2
    c["kc"][c["table"][0, 0], 0, 5, 0] = big
    c["vc"][:] = torch.where(torch.isnan(c["vc"]), c["vc"], torch.ones_like(c["vc"]))
    c["vc"][c["table"][0, 0], 0, 5] = -1.0
    ref = oracle(c)
    say(f"o = {ref['o'][-1, 0, 0]:.4f}")
    check(call(gdn, c), ref, c, "o")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [[1], [64]])
def test_rising_scores(gdn, new, dtype):
    """Scores that rise by more than 8 octaves from tile to tile, and fall again."""
    d, n = 64, 600
    c = make(41, new, [n], 2, 1, d, 16, dtype)
    for j in range(n):
        c["kc"][c["table"][0, j // 16], 0, j % 16] *= 0.1
        c["kc"][c["table"][0, j // 16], 0, j % 16, 0] = (j if j < 400 else 800 - j) / 25.0
    c["q"][..., 0] = 30.0
    check(call(gdn, c), oracle(c), c, "o")


@pytest.mark.parametrize("spread", [1e-4, 40.0])
def test_flat_and_sharp(gdn, spread):
    for new in ([1, 1], [50, 20]):
        c = make(43, new, [300, 200], 4, 2, 128, 16, "f32", spread=spread)
        check(call(gdn, c), oracle(c), c, f"spread {spread}")


def test_very_many_sequences(gdn):
    """More sequences than lanes, empty ones among them, few of them long."""
    rng = np.random.default_rng(5)
    new = [int(x) for x in rng.integers(0, 3, 150)]
    ctx = [n + int(x) for n, x in zip(new, rng.integers(0, 40, 150))]
    ctx[77] += 900
    c = make(47, new, ctx, 2, 1, 32, 16, "bf16")
    check(call(gdn, c), oracle(c), c, "o")


def test_same_results_again_and_with_another_table_width(gdn):
    """Runs are bit-identical; spare columns of the table change how the work is cut, not what it is."""
    c = make(53, [1, 2], [700, 90], 8, 2, 128, 16, "bf16")
    a = call(gdn, c)
    assert torch.equal(a, call(gdn, c))
    wide = dict(c, table=torch.cat([c["table"], torch.full((2, 3000), -1, dtype=torch.int32)], 1).contiguous())
    check(call(gdn, wide), oracle(c), c, "wide table")


def test_offsets_beyond_32_bits(gdn):
    """Pages behind 4 GiB of cache."""
    pages, Hkv, page, d = 1100, 8, 1024, 256          # 2.3e9 elements, 4.6 GB a cache
    kc = torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    gen = torch.Generator(device=DEV).manual_seed(1)
    use = torch.tensor([[1099, 3, 1098]], dtype=torch.int32)
    k = torch.randn(2100, Hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
    v = torch.randn(2100, Hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
    lens, table = torch.tensor([2100], dtype=torch.int32, device=DEV), use.to(DEV)
    cu = torch.tensor([0, 2100], dtype=torch.int32, device=DEV)
    gdn.gdn_cache_append(k, v, kc, vc, table, lens, cu_seqlens=cu)
    assert torch.equal(kc[1098, 3, 51], k[2099, 3]) and torch.equal(vc[1099, 7, 1000], v[1000, 7])
    assert not kc[1097].any() and not vc[:3].any()
    q = torch.randn(1, Hkv, d, generator=gen, device=DEV).to(torch.bfloat16)
    o = gdn.gdn_cache_attention(q[None], kc, vc, table, lens)
    small = torch.stack([kc[i].cpu() for i in use[0].tolist()]), torch.stack([vc[i].cpu() for i in use[0].tolist()])
    c = dict(q=q.cpu(), kc=small[0], vc=small[1], table=torch.tensor([[0, 1, 2]], dtype=torch.int32),
             lens=torch.tensor([2100]), cu=torch.tensor([0, 1]), scale=d ** -0.5, dtype="bf16")
    check(o[0], oracle(c), c, "o")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("octaves", [24, 25, 26])
def test_one_key_above_a_hundred_thousand(gdn, octaves, new, dtype):
    """Weights of 2^-24 to 2^-26 of the largest: 2^-7 to 2^-9 of the sum together.

    Bound: o's and the weights' rounding, u each; below fp16's normal numbers 2^-32 of the largest weight a key, above and
    below; the score of the large key, 26 octaves, through its factor and the exponential 64 e; and sums: 16 keys go into
    one addition to an accumulator (in fp32 two, but one sequence of so many keys is cut into far more than eight parts),
    so n / 16 + 64 roundings of it, above and below."""
    d, n = 32, 131072
    c = make(67, [new], [n], 1, 1, d, 1024, dtype)
    c["q"][:] = 0
    c["q"][..., 0] = 8.0
    c["kc"][:] = 0.0
    where = c["table"][0, 3]
    c["kc"][where, 0, 5, 0] = octaves * math.log(2.0) / (8.0 * c["scale"])
    c["vc"][:] = 1.0
    c["vc"][where, 0, 5] = -1.0
    gap = float(c["kc"][where, 0, 5, 0]) * 8.0 * c["scale"]                # as rounded to the type
    rest = (n - 1 - torch.arange(new - 1, -1, -1, dtype=torch.float64)) * math.exp(-gap)
    want = ((rest - 1) / (rest + 1))[:, None, None].expand(-1, 1, d).numpy()
    u = {"f32": E, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    share = float(rest.max())                                              # of the sum, where weights are rounded
    bound = u * np.abs(want) + 2 * (share * u + n * 2.0 ** -32 * (dtype == "f16") + 64 * E * share + (n / 16 + 64) * E)
    err = np.abs(f64(call(gdn, c)) - want)
    say(f"  2^-{octaves} {dtype} {new}: {err.max():.2e}, bound {bound.max():.2e}, share {share:.2e}")
    assert (err <= bound).all()


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("new", [1, 60])
def test_fp32_is_as_near_as_its_sums(gdn, new, d):
    """The error of o in fp32 as a whole, as roundings that are independent of each other add up (a third of e^2 each).

    A score of n sums (four; two for heads of 32, and where 128-row tiles are computed by one wave a SIMD, heads of 128 and
    more) has m = d / 2n roundings in each.  Scores are normal with s = 1.5, the squares of the weights lie about 2 s^2:
    the m partial sums add s^2 m / 2 by chance and (2 s^2)^2 m / 3n by their drift.  Sums over K keys, two at a time: K / 4.
    The exponential, its argument, the factor 1 / l and o's own rounding: 27."""
    ctx = [200] * 16
    c = make(73 + d, [new] * 16, ctx, 8, 2, d, 16, "f32")
    want = plain(c)["o"]
    n = 2 if d == 32 or (new > 1 and d >= 128) else 4
    m = d / (2 * n)
    bound = E * math.sqrt((1.5 ** 2 * m / 2 + 4.5 ** 2 * m / (3 * n) + ctx[0] / 4 + 27) / 3)
    err = np.linalg.norm(f64(call(gdn, c)) - want) / np.linalg.norm(want)
    say(f"  {new} tokens, d = {d}: {err:.2e} of {bound:.2e}")
    assert err <= bound


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,ctx,Hq,Hkv,d", [
    ([1], [700], 256, 1, 32), ([1, 3], [40, 900], 256, 1, 128), ([9], [400], 510, 2, 64), ([1, 1], [600, 77], 1000, 1000, 32),
    ([37, 40], [600, 40], 800, 800, 32), ([2], [300], 1537, 1537, 256)])
def test_very_many_heads(gdn, new, ctx, Hq, Hkv, d, dtype):
    """The most query heads a key head can have (more than a tile of rows), and more key heads than the card has workgroups."""
    c = make(79 + Hq, new, ctx, Hq, Hkv, d, 16, dtype)
    say(f"heads {dtype} {Hq} on {Hkv} of {d}, {new} {ctx}")
    check(call(gdn, c), oracle(c), c, "o")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_scores_of_millions(gdn, new, dtype):
    """Whole scores up to 2^23, 2^15 apart: o is the best key's value, off by the roundings of its weight, their sum, the
    factor, the product and o itself."""
    n, d = 250, 32
    c = make(83, [new], [n], 2, 1, d, 16, dtype)
    rank = np.random.default_rng(83).permutation(n)
    c["q"][:] = 0.0
    c["q"][..., 0] = 4096.0
    for j in range(n):
        c["kc"][c["table"][0, j // 16], 0, j % 16] = 0.0
        c["kc"][c["table"][0, j // 16], 0, j % 16, 0] = 8.0 * (rank[j] + 1)
    c["scale"] = 1.0
    o = f64(call(gdn, c))
    u = {"f32": E, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    for t in range(new):
        best = int(np.argmax(rank[:n - new + t + 1]))
        v = f64(c["vc"][c["table"][0, best // 16], 0, best % 16])
        assert (np.abs(o[t] - v) <= (u + 4 * E) * np.abs(v)).all(), (t, best)
