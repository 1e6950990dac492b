"""Linear attention with inputs of any size: scores, values and states outside of a
16-bit type's range, columns of very different sizes, values that are no numbers.

Where a test derives no bound of its own, they are those of test_gpu_linear.py (e half a
step of the type relative to the value, A the same sums over absolute values): o is off
by e |o| + e A for the operands plus the fp32 sums' (4 n + 80 + dk) 2^-24 A, the state by
(4 n + 80) 2^-24 A.
"""

import pytest
import torch

from test_gpu_linear import DEV, E, TYPES, U, close, make, prefill
import gated_deltanet_03_amd as gdn

pytestmark = pytest.mark.gpu

# Heads and lengths that take the three passes: one without segments, with half the columns a
# workgroup and with all of them, and both of the split form.
SHAPES = [([40, 20, 1, 60], 2, 4, 64, 64), ([64, 30, 33], 1, 88, 128, 128), ([257, 1, 130, 64], 2, 128, 64, 128),
          ([1500], 1, 2, 128, 128), ([700, 33], 2, 40, 64, 128)]


def oracle(c):
    """The definition in 64 bits, token by token over all sequences: o, final and the same over absolute values."""
    d = {x: c[x].to(DEV).double() for x in ("q", "k", "v", "g")}
    cu, Hv = c["cu"].tolist(), c["Hv"]
    rep, N = Hv // c["Hq"], len(c["cu"]) - 1
    dk, dv, T = d["q"].shape[-1], d["v"].shape[-1], d["v"].shape[0]
    got = []
    for f in (lambda x: x, torch.abs):
        q, k, v = f(d["q"]).repeat_interleave(rep, 1), f(d["k"]).repeat_interleave(rep, 1), f(d["v"])
        a = d["g"].expand(T, Hv).exp()
        S = torch.zeros(N, Hv, dk, dv, dtype=torch.float64, device=DEV)
        if c["s0"] is not None:
            S += f(c["s0"].to(DEV).double())
        o = torch.zeros(T, Hv, dv, dtype=torch.float64, device=DEV)
        for t in range(max(cu[i + 1] - cu[i] for i in range(N))):
            live = [i for i in range(N) if cu[i] + t < cu[i + 1]]
            at = torch.tensor([cu[i] + t for i in live], device=DEV)
            i = torch.tensor(live, device=DEV)
            S[i] = a[at][:, :, None, None] * S[i] + k[at][..., None] * v[at][:, :, None, :]
            o[at] = f(torch.tensor(c["scale"], dtype=torch.float64, device=DEV)) * (q[at][..., None] * S[i]).sum(-2)
        got += [o.cpu().numpy(), S.cpu().numpy()]
    return got


def check(o, final, c, segs=0):
    ref, fin, mag, fmag = oracle(c)
    e, dk = E[o.dtype], c["q"].shape[-1]
    n = 4 * (int(c["cu"].diff().max()) // 32 + 1 + segs) + 80
    close(o, ref, e * abs(ref) + (0 if e == U else e) * mag + (n + dk) * U * mag, "o")
    close(final, fin, n * U * fmag, "final")


@pytest.mark.parametrize("lengths,Hq,Hv,dk,dv", SHAPES)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size,scale", [(300.0, 1e-6), (30.0, 1e-3), (1e-3, 1e4), (1e-4, 1e6)])
def test_scores_out_of_fp16_range(dtype, size, scale, lengths, Hq, Hv, dk, dv):
    """|q . k| up to 10^6 .. 10^7 (aligned keys) and down to 10^-7, with o in range."""
    c = make(61, lengths, Hq, Hv, dk, dv, dtype, state=False, memory=0.05)
    g = torch.Generator().manual_seed(62)
    base = torch.randn(1, Hq, dk, generator=g)
    for x in "qk":       # one direction and noise
        c[x] = (size * (base + 0.3 * torch.randn(sum(lengths), Hq, dk, generator=g))).to(TYPES[dtype])
    c["v"] = (0.1 * c["v"].float()).to(TYPES[dtype])
    c["scale"] = scale
    o, fin = prefill(c)
    assert torch.isfinite(o).all() and torch.isfinite(fin).all()
    check(o, fin, c, segs=20)


def test_equal_large_keys_agree_with_the_step():
    T, d = 40, 128
    q = torch.full((T, 1, d), 23.0, dtype=torch.float16, device=DEV)     # q . k = 67712
    v = torch.full((T, 1, d), 0.1, dtype=torch.float16, device=DEV)
    g = torch.full((1,), -20.0, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    o, fin = gdn.gdn_linear_prefill(q, q, v, g, cu_seqlens=cu)
    os, fs, _ = gdn.gdn_linear_step(q, q, v, g, cu_seqlens=cu)
    assert ((o.float() - os.float()).abs() <= 4 * E[torch.float16] * os.float().abs()).all()
    assert ((fin - fs).abs() <= 1e-5 * fs.abs()).all()


@pytest.mark.parametrize("lengths,Hq,Hv,dk,dv", SHAPES + [([600, 40], 1, 3, 16, 16)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_outputs_are_rounded_once(dtype, lengths, Hq, Hv, dk, dv):
    """The state and the scores enter o in two parts of the input type, each with what the part
    before it left: off by (2 e^2) A together, where the state of the output pass itself is summed
    from two parts of the decayed v, e^2 A more; fp16 also by its smallest step, 2^-25 where the
    largest of a column or query is at least 2^13: 2 times 2^-38 of A's largest, dk or 64 of them."""
    c = make(63, lengths, Hq, Hv, dk, dv, dtype, memory=0.05)
    o, fin = prefill(c)
    ref, _, mag, _ = oracle(c)
    e = E[o.dtype]
    n = 4 * (max(lengths) // 32 + 21) + 80 + dk
    close(o, ref, e * abs(ref) + (3 * e * e + n * U + (dk + 64) * 2.0 ** -38) * mag, "o")


@pytest.mark.parametrize("lengths,Hq,Hv,dk,dv", SHAPES + [([600, 40], 1, 3, 16, 16)])
def test_fp16_columns_of_different_sizes(lengths, Hq, Hv, dk, dv):
    """A column of v or of the state keeps its accuracy whatever stands beside it."""
    c = make(65, lengths, Hq, Hv, dk, dv, "f16", memory=0.05)
    for x in ("v", "s0"):
        c[x] = c[x].float()
        c[x][..., ::2] *= 100.0
        c[x][..., 1::2] *= 1e-5
    c["v"] = c["v"].half()
    o, fin = prefill(c)
    check(o, fin, c, segs=20)
    c["v"][..., 1::2] *= 1e5
    c["s0"][..., 1::2] *= 1e5
    c["s0"][..., ::2] *= 1e12          # these columns of o are beyond fp16
    o, fin = prefill(c)
    ref, want, mag, fmag = oracle(c)
    e, n = E[torch.float16], 4 * (max(lengths) // 32 + 21) + 80
    close(o[..., 1::2], ref[..., 1::2], (e * (abs(ref) + mag) + (n + dk) * U * mag)[..., 1::2], "o")
    close(fin, want, n * U * fmag, "final")


@pytest.mark.parametrize("lengths,Hq,Hv,dk,dv", SHAPES + [([600, 40], 1, 3, 16, 16)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_values_that_are_no_numbers_reach_later_tokens_only(dtype, value, lengths, Hq, Hv, dk, dv):
    """An infinity or NaN in v: its column of o and of the state from its token on, and nothing else."""
    c = make(66, lengths, Hq, Hv, dk, dv, dtype, memory=0.05)
    clean, fin = prefill(c)
    assert torch.isfinite(clean).all() and torch.isfinite(fin).all()
    hurt, final = torch.zeros_like(clean, dtype=torch.bool), torch.zeros_like(fin, dtype=torch.bool)
    cu = c["cu"].tolist()
    for s, (a, b) in enumerate(zip(cu, cu[1:])):
        for at, h, col in ((a + (b - a) // 2, 0, 1), (b - 1, Hv - 1, dv - 1), (a + (b - a) // 3, Hv // 2, dv // 2)):
            c["v"][at, h, col] = value
            hurt[at:b, h, col] = True
            final[s, h, :, col] = True
    o, f = prefill(c)
    assert torch.equal(o[~hurt], clean[~hurt]) and not torch.isfinite(o[hurt]).any()
    assert torch.equal(f[~final], fin[~final]) and not torch.isfinite(f[final]).any()


@pytest.mark.parametrize("which", ["q", "k"])
def test_queries_and_keys_that_are_no_numbers(which):
    c = make(67, [150, 30], 1, 2, 64, 64, "bf16", memory=0.05)
    clean, fin = prefill(c)
    c[which][70, 0, 3] = float("nan")
    o, f = prefill(c)
    last = 71 if which == "q" else 150
    assert torch.equal(o[:70], clean[:70]) and torch.equal(o[last:], clean[last:]) and torch.isnan(o[70:last]).all()
    rows = torch.tensor([r for r in range(64) if which == "q" or r != 3], device=DEV)
    assert torch.equal(f[:, :, rows], fin[:, :, rows]) and torch.equal(f[1], fin[1])
    assert which == "q" or torch.isnan(f[0, :, 3]).all()


@pytest.mark.parametrize("call,Hv,dk", [("gdn_linear_prefill", 129, 16), ("gdn_linear_step", 65, 128)])
def test_more_pairs_than_one_launch_takes(call, Hv, dk):
    """65535 one-token rows: 512 and 1024 threads a (row, head) pair are 2^32 threads and more."""
    B, dv = 65535, 128
    gen = torch.Generator(device=DEV).manual_seed(71)
    q = torch.randn(B, 1, 1, dk, device=DEV, generator=gen, dtype=torch.bfloat16)
    k = torch.randn(B, 1, 1, dk, device=DEV, generator=gen, dtype=torch.bfloat16)
    v = torch.randn(B, 1, Hv, dv, device=DEV, generator=gen, dtype=torch.bfloat16)
    o = torch.full_like(v, 7.0)
    getattr(gdn, call)(q, k, v, torch.zeros(Hv, device=DEV), scale=1.0, o=o, output_final_state=False)
    e = E[torch.bfloat16]
    for rows in torch.arange(B, device=DEV).split(4096):   # o = (q . k) v: the score in parts, products in fp32
        a, b = q[rows, 0].double(), k[rows, 0].double()
        s, size = (a * b).sum(-1, keepdim=True), (a * b).abs().sum(-1, keepdim=True)
        want, x = s * v[rows, 0].double(), v[rows, 0].double().abs()
        assert ((o[rows, 0].double() - want).abs() <= e * want.abs() + (3 * e * e + (dk + 80) * U) * size * x).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("Hq,Hv", [(61, 122), (33, 264)])
def test_one_pass_of_whole_sequences(dtype, dk, dv, Hq, Hv):
    """No segments: below 256 (sequence, head) pairs half the columns a workgroup, above 512 all of them."""
    B, T = 2, 250
    c = make(72, [T] * B, Hq, Hv, dk, dv, dtype, memory=0.05)
    sh = gdn.gdn_shape(B, T, Hq, Hv, dk, dv, 1.0, gdn._DTYPES[TYPES[dtype]])
    assert gdn.gdn_linear_workspace_bytes(sh, False) == 0
    d = {x: c[x].to(DEV).view(B, T, *c[x].shape[1:]) for x in "qkvg"}
    args, s0 = [d[x] for x in "qkvg"], c["s0"].to(DEV)
    o, fin = gdn.gdn_linear_prefill(*args, scale=c["scale"], initial_state=s0)
    check(o.flatten(0, 1), fin, c)
    state = s0.clone()
    o2, fin2 = gdn.gdn_linear_prefill(*args, scale=c["scale"], initial_state=state, final_state=state)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    one = s0[:1].contiguous()
    o3, fin3 = gdn.gdn_linear_prefill(*args, scale=c["scale"], initial_state=one)
    assert torch.equal(o[0], o3[0]) and torch.equal(fin[0], fin3[0])
    c["s0"] = c["s0"][:1].repeat(B, 1, 1, 1)
    check(o3.flatten(0, 1), fin3, c)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_one_pass_of_ragged_sequences(dtype):
    """512 pairs and more: a long sequence beside empty and short ones, in one pass."""
    lengths = [450, 0, 1, 65, 0, 31] * 3
    c = make(73, lengths, 16, 32, 128, 128, dtype, "head", memory=0.05)
    sh = gdn.gdn_shape(len(lengths), sum(lengths), 16, 32, 128, 128, 1.0, gdn._DTYPES[TYPES[dtype]])
    assert gdn.gdn_linear_workspace_bytes(sh, True) == 0
    o, fin = prefill(c)
    check(o, fin, c)
