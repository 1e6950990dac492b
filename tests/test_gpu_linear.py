"""Linear attention with a decay for each head against the fp64 oracle.

Bounds, element by element, with e = half a step of the type relative to the
value (fp32 2^-24, fp16 2^-11, bf16 2^-8) and A the same sums taken over absolute
values (the oracle's ``magnitudes``):

* step: all in fp32.  A state element passes one product and one sum a token
  (plus the decay's own error of at most 3 units): (5 T + 4) 2^-24 A.  o adds the
  sum over dk and its rounding: e |o| + (5 T + dk + 4) 2^-24 A.
* prefill, state: a contribution is rounded as w v (3 units: the decay, the
  product, the remainder of the split) and summed over its 64-token chunk, then
  takes two roundings and the decay's error in each of the n later chunks or
  segments: (4 n + 80) 2^-24 A.
* prefill, o: for 16-bit inputs the state and the scores are rounded once as
  operands, e A for both together, and o once, e |o|; all else as above plus the
  sum over dk and the decays' exponentials: (4 n + 80 + dk) 2^-24 A.
Where the outputs have a pass of their own, its bf16 state is summed from two parts
of the decayed v, 2^-16 A more: 1 / 256 of e A, which no sum of roundings of mixed
signs comes near.
fp16 values below its normal range are off by up to 2^-25 instead of e |o|.
"""

import pytest
import torch

import gated_deltanet_03_amd as gdn
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24


def make(seed, lengths, Hq, Hv, dk, dv, dtype, decay="token", state=True, memory=1.0, vscale=1.0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)

    def n(*s):
        return torch.randn(*s, generator=g)
    c = dict(q=n(T, Hq, dk).to(TYPES[dtype]), k=(n(T, Hq, dk) * dk ** -0.5).to(TYPES[dtype]),
             v=(vscale * n(T, Hv, dv)).to(TYPES[dtype]), scale=dk ** -0.5, Hq=Hq, Hv=Hv)
    c["g"] = -memory * torch.rand(*((T, Hv) if decay == "token" else (Hv,)), generator=g)
    c["s0"] = vscale * n(N, Hv, dk, dv) if state else None
    cu = [0]
    for x in lengths:
        cu.append(cu[-1] + x)
    c["cu"] = torch.tensor(cu, dtype=torch.int32)
    return c


def dev(c):
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in c.items()}


def oracle(c):
    args = (c["q"], c["k"], c["v"], c["g"], c["scale"], c["Hq"], c["Hv"], c["cu"])
    return (oo.linear(*args, initial_state=c["s0"]),
            oo.linear(*args, initial_state=c["s0"], magnitudes=True))


def check(o, final, c, step=False, segs=0):
    ref, mag = oracle(c)
    e, dk = E[o.dtype], c["q"].shape[-1]
    T = int(c["cu"].diff().max()) if len(c["cu"]) > 1 else 0
    n = 5 * T + 4 if step else 4 * (T // 32 + 1 + segs) + 80
    close(o, ref["o"], e * abs(ref["o"]) + (0 if step or e == U else e) * mag["o"] + (n + dk) * U * mag["o"], "o")
    if final is not None:
        close(final, ref["final"], n * U * mag["final"], "final")


def close(x, ref, tol, what):
    x = x.detach().cpu().double().numpy()
    off = abs(x - ref)
    bad = ~(off <= tol + (2.0 ** -25 if what == "o" else 1e-37))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {off[bad].max():.3e} where {tol[bad].min():.3e}"


def prefill(c, **kw):
    d = dev(c)
    return gdn.gdn_linear_prefill(d["q"], d["k"], d["v"], d["g"], scale=d["scale"], initial_state=d["s0"],
                                  cu_seqlens=d["cu"], **kw)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_prefill_dims(dtype, dk, dv):
    c = make(dk + dv, [1, 0, 64, 63, 65, 33, 130], 2, 4, dk, dv, dtype, "token" if dk != 32 else "head")
    o, fin = prefill(c)
    check(o, fin, c)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths", [[1], [15], [16], [17], [31], [32], [33], [64], [128], [0, 0, 5], [7] * 70])
def test_prefill_lengths(dtype, lengths):
    c = make(len(lengths), lengths, 3, 3, 64, 32, dtype, state=len(lengths) > 1)
    o, fin = prefill(c)
    check(o, fin, c)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lengths,state", [([1500], True), ([900, 0, 1, 700, 128, 129], True), ([1024], False)])
@pytest.mark.parametrize("d", [(64, 64), (128, 128), (16, 128)])
def test_prefill_split_over_segments(dtype, lengths, state, d):
    """Few heads: the sequences are cut into segments (the workspace is used)."""
    c = make(5, lengths, 1, 2, *d, dtype, state=state, memory=0.02)
    sh = gdn.gdn_shape(len(lengths), sum(lengths), 1, 2, *d, 1.0, gdn._DTYPES[TYPES[dtype]])
    need = gdn.gdn_linear_workspace_bytes(sh, True)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)    # NaN everywhere
    o, fin = prefill(c, workspace=ws)
    check(o, fin, c, segs=16)


def test_prefill_split_dense_rows():
    c = make(6, [700] * 3, 2, 2, 32, 64, "bf16", memory=0.02)
    d = dev(c)
    o, fin = gdn.gdn_linear_prefill(*(d[x].view(3, 700, *d[x].shape[1:]) for x in "qkvg"), scale=c["scale"],
                                    initial_state=d["s0"])
    check(o.flatten(0, 1), fin, c, segs=16)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_decays_from_none_to_total(dtype):
    """g = 0, tiny, strong, beyond fp32's exp and -inf, next to each other: the
    differences of G that matter stay exact among sums in the thousands."""
    c = make(9, [200], 1, 4, 64, 64, dtype)
    c["g"][:, 0] = 0.0
    c["g"][::3, 1] = -60.0
    c["g"][5::50, 2] = -float("inf")
    c["g"][::7, 3] = -1000.0
    o, fin = prefill(c)
    assert torch.isfinite(o).all()
    check(o, fin, c)


@pytest.mark.parametrize("vscale", [1e-4, 1e-2, 30.0])
def test_fp16_state_out_of_fp16_range(vscale):
    """States and decayed values far below or above fp16's range keep their accuracy."""
    c = make(10, [150, 20], 1, 2, 64, 64, "f16", vscale=vscale)
    if vscale > 1:
        c["s0"] *= 3000.0           # up to 4e5
        c["q"] = c["q"] * 1e-2      # (o back in range)
    o, fin = prefill(c)
    ref, mag = oracle(c)
    close(fin, ref["final"], 100 * U * mag["final"], "final")
    close(o, ref["o"], E[torch.float16] * (abs(ref["o"]) + mag["o"]) + 150 * U * mag["o"], "o")


def test_states_given_broadcast_inplace_and_absent():
    c = make(11, [70, 3, 64], 2, 4, 32, 32, "bf16")
    d = dev(c)
    a = (d["q"], d["k"], d["v"], d["g"])
    o, fin = gdn.gdn_linear_prefill(*a, cu_seqlens=d["cu"], initial_state=d["s0"])
    inplace = d["s0"].clone()
    o2, fin2 = gdn.gdn_linear_prefill(*a, cu_seqlens=d["cu"], initial_state=inplace, final_state=inplace)
    assert fin2 is inplace and torch.equal(fin, fin2) and torch.equal(o, o2)
    one = d["s0"][:1].contiguous()
    o3, fin3 = gdn.gdn_linear_prefill(*a, cu_seqlens=d["cu"], initial_state=one)
    o4, fin4 = gdn.gdn_linear_prefill(*a, cu_seqlens=d["cu"], initial_state=one.repeat(3, 1, 1, 1))
    assert torch.equal(o3, o4) and torch.equal(fin3, fin4)
    o5, none = gdn.gdn_linear_prefill(*a, cu_seqlens=d["cu"], initial_state=d["s0"], output_final_state=False)
    assert none is None and torch.equal(o, o5)
    _, keep = gdn.gdn_linear_prefill(d["q"][:0], d["k"][:0], d["v"][:0], d["g"][:0],
                                     cu_seqlens=torch.zeros(4, dtype=torch.int32, device=DEV), initial_state=d["s0"])
    assert torch.equal(keep, d["s0"])


@pytest.mark.parametrize("split", [False, True])
def test_one_sequences_nan_stays_in_it(split):
    n = 600 if split else 40
    c = make(12, [n, 33, n], 1, 1, 32, 32, "bf16")
    clean, fin = prefill(c)
    for x in ("q", "k", "v"):
        c[x][n:n + 33] = float("nan")
    o, f = prefill(c)
    assert torch.equal(o[:n], clean[:n]) and torch.equal(o[n + 33:], clean[n + 33:])
    assert torch.equal(f[0], fin[0]) and torch.equal(f[2], fin[2]) and torch.isnan(f[1]).all()


def test_same_bits_every_time_and_on_another_stream():
    c = make(13, [2000, 77], 2, 4, 128, 128, "bf16", memory=0.05)
    o, fin = prefill(c)
    o2, fin2 = prefill(c)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3, fin3 = prefill(c)
    s.synchronize()
    assert torch.equal(o, o3) and torch.equal(fin, fin3)


def test_offsets_past_32_bits():
    """v of 2.4e9 elements; strong decays leave the last rows to the last tokens."""
    T, Hv, d = 150000, 128, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn(T, 1, d, device=DEV, generator=gen, dtype=torch.bfloat16)
    k = torch.randn(T, 1, d, device=DEV, generator=gen, dtype=torch.bfloat16)
    v = torch.randn(T, Hv, d, device=DEV, generator=gen, dtype=torch.bfloat16)
    g = torch.full((Hv,), -30.0, device=DEV)
    assert v.numel() > 2 ** 31
    o, fin = gdn.gdn_linear_prefill(q[None], k[None], v[None], g)
    n = 200
    tail = [x[-n:].contiguous()[None] for x in (q, k, v)]
    ot, ft = gdn.gdn_linear_prefill(*tail, g)
    rel = (o[0, -100:].float() - ot[0, -100:].float()).norm() / ot[0, -100:].float().norm()
    assert rel < 2 * E[torch.bfloat16]
    assert (fin - ft).norm() / ft.norm() < 1e-6
    os, fs, _ = gdn.gdn_linear_step(*(x[:, -30:].contiguous() for x in tail), g)
    assert (fs - fin).norm() / fin.norm() < 1e-6
    assert (os[0, -10:].float() - o[0, -10:].float()).norm() / os[0, -10:].float().norm() < 4 * E[torch.bfloat16]


# ---------------------------------------------------------------- step
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
def test_step_dims(dtype, dk, dv):
    c = make(dk * dv, [1, 0, 7, 8, 9, 17, 1], 2, 6, dk, dv, dtype, "token" if dv != 32 else "head")
    d = dev(c)
    o, fin, _ = gdn.gdn_linear_step(d["q"], d["k"], d["v"], d["g"], scale=c["scale"], initial_state=d["s0"],
                                    cu_seqlens=d["cu"])
    check(o, fin, c, step=True)


def test_step_single_tokens_dense_inplace_and_growing():
    c = make(21, [1] * 5, 2, 2, 64, 128, "bf16")
    c["g"] = c["g"] + 1.5          # the step takes g of any sign
    d = dev(c)
    st = d["s0"].clone()
    o, fin, _ = gdn.gdn_linear_step(*(d[x][:, None] for x in "qkvg"), scale=c["scale"], initial_state=st, final_state=st)
    assert fin is st
    check(o[:, 0], fin, c, step=True)
    o2, none, _ = gdn.gdn_linear_step(*(d[x][:, None] for x in "qkvg"), scale=c["scale"], output_final_state=False)
    assert none is None
    c["s0"] = None
    check(o2[:, 0], None, c, step=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hv,dk,dv", [(2, 4, 64, 64), (1, 3, 16, 16), (3, 3, 128, 128)])
def test_capture_and_replay(dtype, Hq, Hv, dk, dv):
    """Records hold the exact decay, key and value; what is not captured stays;
    replaying the first m records gives the state of the first m tokens bit for bit."""
    lengths, cap = [7, 3, 0, 5, 1], 6
    c = make(31, lengths, Hq, Hv, dk, dv, dtype)
    d = dev(c)
    counts = torch.tensor([9, 2, 4, -1, 1], dtype=torch.int32, device=DEV)
    R = Hv + Hq * dk + Hv * dv
    su = torch.full((5, cap, R), 7.0, device=DEV)
    a = (d["q"], d["k"], d["v"], d["g"])
    kw = dict(scale=c["scale"], initial_state=d["s0"], cu_seqlens=d["cu"])
    o, fin, rec = gdn.gdn_linear_step(*a, **kw, state_update_capacity=cap, capture_count=counts, state_update=su)
    o2, fin2, _ = gdn.gdn_linear_step(*a, **kw)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    written = [6, 2, 0, 0, 1]
    for b, n in enumerate(written):
        assert (rec[b, n:] == 7.0).all()
        for t in range(n):
            at = int(c["cu"][b]) + t
            alpha = rec[b, t, :Hv].cpu().double()
            want = c["g"][at].double().exp()
            assert ((alpha - want).abs() <= 4 * U * want).all()
            assert torch.equal(rec[b, t, Hv:Hv + Hq * dk].cpu(), c["k"][at].float().flatten())
            assert torch.equal(rec[b, t, Hv + Hq * dk:].cpu(), c["v"][at].float().flatten())
    m = torch.tensor([4, 2, 3, 5, 1], dtype=torch.int32)
    m = torch.minimum(m, torch.tensor(written, dtype=torch.int32))
    st = d["s0"].clone()
    gdn.gdn_replay_state_updates(st, rec, m.to(DEV), Hq=Hq)
    cut = [torch.cat([c[x][int(c["cu"][b]):int(c["cu"][b]) + int(m[b])] for b in range(5)]).to(DEV) for x in "qkvg"]
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), m.cumsum(0).int()]).to(DEV)
    _, want, _ = gdn.gdn_linear_step(*cut, scale=c["scale"], initial_state=d["s0"], cu_seqlens=cu)
    assert torch.equal(st, want)


def test_graph_replays_follow_their_inputs():
    """Captured step and split prefill, replayed between eager calls on other inputs."""
    c = make(41, [1500], 1, 2, 64, 64, "bf16", memory=0.02)
    d = dev(c)
    one = dev(make(42, [1] * 3, 2, 4, 64, 64, "bf16"))
    ws = torch.empty(gdn.gdn_linear_workspace_bytes(gdn.gdn_shape(1, 1500, 1, 2, 64, 64, 1.0, gdn.GDN_BF16), True),
                     dtype=torch.uint8, device=DEV)
    bufs = dict(o=torch.empty_like(d["v"]), final_state=torch.empty_like(d["s0"]))
    sb = dict(o=torch.empty_like(one["v"][:, None]), final_state=torch.empty_like(one["s0"]))

    def both():
        gdn.gdn_linear_prefill(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], cu_seqlens=d["cu"], workspace=ws,
                               **bufs)
        gdn.gdn_linear_step(*(one[x][:, None] for x in "qkvg"), initial_state=one["s0"], **sb)
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(4):
        for x in (d, one):
            x["v"].copy_(torch.randn_like(x["v"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*bufs.values(), *sb.values())]
        both()
        torch.cuda.synchronize()
        for a, b in zip(got, (*bufs.values(), *sb.values())):
            assert torch.equal(a, b), i


# ------------------------------------------------- paths chosen by size
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hv,dk,dv", [(3, 128, 128), (3, 32, 64), (2, 64, 32), (2, 128, 16), (40, 64, 128)])
def test_prefill_many_segments(dtype, Hv, dk, dv):
    """Segments by the dozen, in a sequence and beside empty and short ones, with few
    heads (half the columns a workgroup) and many."""
    c = make(51, [1700, 0, 1, 1300, 0, 65], 1, Hv, dk, dv, dtype, memory=0.01)
    o, fin = prefill(c)
    check(o, fin, c, segs=30)
    d = dev(c)
    a = (d["q"], d["k"], d["v"], d["g"])
    kw = dict(scale=d["scale"], cu_seqlens=d["cu"])
    state = d["s0"].clone()
    o2, fin2 = gdn.gdn_linear_prefill(*a, **kw, initial_state=state, final_state=state)      # in place
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    o3, none = gdn.gdn_linear_prefill(*a, **kw, initial_state=d["s0"], output_final_state=False)
    assert none is None and torch.equal(o, o3)


def test_prefill_segments_share_one_initial_state():
    c = make(52, [800, 700], 1, 2, 64, 64, "f32", memory=0.01)
    c["s0"] = c["s0"][:1].repeat(2, 1, 1, 1)
    o, fin = prefill(c)
    check(o, fin, c, segs=20)
    d = dev(c)
    o2, fin2 = gdn.gdn_linear_prefill(d["q"], d["k"], d["v"], d["g"], scale=d["scale"], cu_seqlens=d["cu"],
                                      initial_state=d["s0"][:1].contiguous())
    assert torch.equal(o, o2) and torch.equal(fin, fin2)


def test_offsets_that_are_malformed_stay_in_bounds():
    """Overlapping, reversed and out-of-range offsets give some result and touch nothing else."""
    c = make(53, [900, 900], 1, 2, 32, 32, "bf16", memory=0.01)
    d = dev(c)
    for cu in ([0, 5000, 1800], [0, 1800, 0], [900, 100, 1800], [-5, 900, 1700]):
        bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
        for f in (gdn.gdn_linear_prefill, gdn.gdn_linear_step):
            f(d["q"], d["k"], d["v"], d["g"], cu_seqlens=bad, initial_state=d["s0"])
    torch.cuda.synchronize()
    o, fin = prefill(c)
    check(o, fin, c, segs=20)
