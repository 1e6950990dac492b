"""The cache and beam operators as they are measured: cases, inputs, plain forms and exact values.

What a decoder of delta-rule blocks needs beside them to serve prompts and beams: its attention layers keep keys and
values in pages, and a beam search moves states and pages from beam to beam.

``append``   gdn_cache_append: new keys (rotated by their positions) and values into a paged cache, queries rotated
``attend``   gdn_cache_attention: new tokens against all cached keys up to their own, causal, heads sharing keys
``select``   gdn_beam_select: the best continuations over beams and vocabulary, log softmax included
``reorder``  gdn_state_reorder, gdn_cache_copy_pages: states and last pages moved from each parent to its beam

``own`` chooses between the plain forms here and the library's calls.
"""

from __future__ import annotations

import itertools
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}

# a batch of conversations: most of them some thousand tokens long, a few very long ones
CHATS = ",".join(str(n) for n in (
    32011, 811, 2700, 1200, 5003, 640, 901, 4100, 16001, 2222, 515, 1777, 700, 9000, 1300, 3500,
    1024, 600, 2048, 12345, 850, 1900, 730, 4444, 999, 2600, 1111, 7003, 560, 1650, 3900, 1450))


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one user's next token, keys and queries rotated: latency
        dict(name="append_one", op="append", dtype="bf16", new="1", ctx="1000", Hq=32, Hkv=8, d=128, page=64,
             rotary=128, axes=1, interleaved=False),
        # packed prompts of an image model: positions in time, height and width, a quarter of wide heads rotated
        dict(name="append_prompts", op="append", dtype="bf16", new="8192,5000,1031,63", ctx="8192,6000,1031,700",
             Hq=16, Hkv=2, d=256, page=64, rotary=64, axes=3, interleaved=False),
        # one user's next token after a short text, fp32 heads of a small model: latency
        dict(name="attend_one", op="attend", dtype="f32", new="1", ctx="301", Hq=4, Hkv=4, d=64, page=16, window=0),
        # one user's next token after a very long text: the cache's length is all the work there is
        dict(name="attend_long", op="attend", dtype="bf16", new="1", ctx="131001", Hq=16, Hkv=2, d=256, page=64,
             window=0),
        # a full batch's next tokens, lengths far apart
        dict(name="attend_batch", op="attend", dtype="bf16", new=",".join(["1"] * 32), ctx=CHATS, Hq=32, Hkv=8, d=128,
             page=64, window=0),
        # rows of drafted tokens to be verified, five query heads on each key head, a sliding window
        dict(name="attend_drafts", op="attend", dtype="f16", new="3,7,2,6,1,5,7,4",
             ctx="5003,900,17000,2100,333,8111,4099,64", Hq=40, Hkv=8, d=64, page=32, window=4096),
        # chunks of prompts among stored text, one of them long: the largest
        dict(name="attend_chunk", op="attend", dtype="bf16", new="2048,700,1,63", ctx="16384,5000,9000,1031", Hq=32,
             Hkv=8, d=128, page=64, window=0),
        # a prompt's only chunk in fp32, an odd length
        dict(name="attend_f32", op="attend", dtype="f32", new="1031", ctx="1031", Hq=8, Hkv=2, d=64, page=16,
             window=0),
        # one user's four beams over an odd vocabulary: latency
        dict(name="select_one", op="select", dtype="f32", B=1, W=4, K=4, V=32003),
        # a batch of beams over a large vocabulary, twice as many continuations as beams
        dict(name="select_batch", op="select", dtype="bf16", B=16, W=8, K=16, V=131072),
        # the states of four layers, moved in place
        dict(name="reorder_states", op="reorder", kind="states", layers=4, B=8, W=4, Hv=32, dk=128, dv=128),
        # each beam's last page of keys and values
        dict(name="reorder_pages", op="reorder", kind="pages", dtype="bf16", B=16, W=8, Hkv=8, page=64, d=128),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "select", "reorder"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op == "select":
        W = rng.randint(1, 12)
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 16), W=W, K=rng.randint(1, 2 * W), V=_log(rng, 200, 100000))
    if op == "reorder":
        B, W = _log(rng, 1, 12), rng.randint(2, 9)
        if rng.random() < 0.5:
            return dict(op=op, kind="states", layers=rng.randint(1, 3), B=B, W=W, Hv=rng.randint(1, 8),
                        dk=rng.choice([16, 32, 64, 128]), dv=rng.choice([16, 32, 64, 128]))
        return dict(op=op, kind="pages", dtype=dtype, B=B, W=W, Hkv=rng.randint(1, 8), page=rng.choice([16, 32, 48]),
                    d=rng.choice([32, 64, 128, 256]))
    d, Hkv = rng.choice([32, 64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    case = dict(op=op, dtype=dtype, Hq=Hq, Hkv=Hkv, d=d, page=page)
    if op == "append":
        N = _log(rng, 1, 32)
        new = [rng.choice([0, 1, 1, rng.randint(1, 7), _log(rng, 1, 9000 // N)]) for _ in range(N)]
        new[rng.randrange(N)] = rng.randint(1, 9)
        ctx = [n + rng.choice([0, _log(rng, 1, 2000)]) for n in new]
        axes = rng.choice([1, 1, 3])
        return dict(case, new=",".join(map(str, new)), ctx=",".join(map(str, ctx)), axes=axes,
                    rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.3)
    window = rng.choice([0, 0, 0, _log(rng, 16, 2000)])
    if rng.random() < 0.5:      # next tokens, or drafts
        N = _log(rng, 1, 32)
        most = rng.choice([1, 1, 8])
        new = [rng.randint(1 if most == 1 else 0, most) for _ in range(N)]
        new[rng.randrange(N)] = most
        ctx = [n + _log(rng, 1, 12000) for n in new]
    else:                       # prompts, with or without text before them
        N = rng.randint(1, 4)
        new = [_log(rng, 1, 1200) for _ in range(N)]
        ctx = [n + rng.choice([0, _log(rng, 1, 4000)]) for n in new]
    return dict(case, new=",".join(map(str, new)), ctx=",".join(map(str, ctx)), window=window)


def _numbers(text):
    return [int(x) for x in text.split(",")]


def _offsets(lengths):
    return [0, *itertools.accumulate(lengths)]


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    def below(n, *shape):
        return torch.randint(0, n, shape, generator=gen, device=dev, dtype=torch.int32)

    st = dict(case=case)
    if case["op"] == "select":
        dtype, B, W, V = DTYPES[case["dtype"]], case["B"], case["W"], case["V"]
        # a few likely tokens above a long tail, less sure in one beam than in another
        st["logits"] = (normal(B, W, V) * (1.5 + 0.8 * torch.rand(B, W, 1, generator=gen, device=dev))).to(dtype)
        st["scores"] = torch.sort(-3.0 - 6.0 * torch.rand(B, W, generator=gen, device=dev), -1, descending=True)[0]
        st["finished"] = torch.rand(B, W, generator=gen, device=dev) < 0.15
        return st
    if case["op"] == "reorder":
        B, W = case["B"], case["W"]
        parents = torch.sort(below(W, B, W), -1)[0].int()      # better beams have more children
        if case["kind"] == "states":
            st["state"] = normal(case["layers"], B * W, case["Hv"], case["dk"], case["dv"])
            st["parents"] = parents
            return st
        dtype, pages = DTYPES[case["dtype"]], 2 * B * W
        shape = (pages, case["Hkv"], case["page"], case["d"])
        st["k_cache"], st["v_cache"] = normal(*shape, dtype=dtype), normal(*shape, dtype=dtype)
        order = torch.randperm(pages, generator=gen, device=dev).int()
        mine = order[:B * W].view(B, W)
        st["src"] = mine.gather(1, parents.long())
        st["dst"] = torch.where(st["src"] == mine, -1, order[B * W:].view(B, W))
        return st
    dtype = DTYPES[case["dtype"]]
    new, ctx, page = _numbers(case["new"]), _numbers(case["ctx"]), case["page"]
    T, Hq, Hkv, d = sum(new), case["Hq"], case["Hkv"], case["d"]
    need = [-(-n // page) for n in ctx]
    pages = sum(need) + 3
    shape = (pages, Hkv, page, d)
    st["k_cache"], st["v_cache"] = normal(*shape, dtype=dtype), normal(*shape, dtype=dtype)
    order = torch.randperm(pages, generator=gen, device=dev).int()
    table = torch.full((len(new), max(max(need), 1)), -1, dtype=torch.int32, device=dev)
    starts = _offsets(need)
    for s, n in enumerate(need):
        table[s, :n] = order[starts[s]:starts[s + 1]]
    st["table"], st["lens"] = table, torch.tensor(ctx, dtype=torch.int32, device=dev)
    st["cu"] = torch.tensor(_offsets(new), dtype=torch.int32, device=dev)
    if case["op"] == "attend":
        st["q"] = normal(T, Hq, d).mul_(1.5).to(dtype)
        st["dense"] = min(new) == max(new)
        return st
    # queries, keys and values are slices of one projection's rows
    rows = normal(T, (Hq + 2 * Hkv) * d, dtype=dtype)
    st["q"] = rows[:, :Hq * d].view(T, Hq, d)
    st["k"] = rows[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    st["v"] = rows[:, (Hq + Hkv) * d:].view(T, Hkv, d)
    pairs = case["rotary"] // 2
    st["inv_freq"] = (10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)).float()
    if case["axes"] > 1:
        st["positions"] = torch.stack([below(100000, T), below(64, T), below(64, T)])
        st["axis"] = (torch.arange(pairs, device=dev) * 3 // max(pairs, 1)).int()
    else:
        st["positions"] = st["axis"] = None
    return st


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "append":
        return _append(st, case)
    if case["op"] == "attend":
        return _attend(st, case)
    if case["op"] == "select":
        return _select(st, case)
    return _reorder(st, case)


def _run_own(st, case):
    import gated_deltanet_03_amd as gdn
    if case["op"] == "append":
        q = gdn.gdn_cache_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                 cu_seqlens=st["cu"], q=st["q"], inv_freq=st["inv_freq"], positions=st["positions"],
                                 pair_axis=st["axis"], interleaved=case["interleaved"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if case["op"] == "attend":
        if st["dense"]:      # rows of equally many tokens
            q = st["q"].view(len(st["lens"]), -1, case["Hq"], case["d"])
            o = gdn.gdn_cache_attention(q, st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                        window=case["window"])
            return {"o": o.view_as(st["q"])}
        return {"o": gdn.gdn_cache_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                             cu_seqlens=st["cu"], window=case["window"])}
    if case["op"] == "select":
        tokens, parents, scores, finished = gdn.gdn_beam_select(
            st["logits"], st["scores"], beams=case["K"], finished=st["finished"], eos_token=2, pad_token=0)
        return {"tokens": tokens, "parents": parents, "scores": scores, "finished": finished}
    if case["kind"] == "states":
        return {"state": gdn.gdn_state_reorder(st["state"], st["parents"], axis=1, out=st["state"])}
    gdn.gdn_cache_copy_pages(st["k_cache"], st["v_cache"], st["src"], st["dst"])
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _append(st, case):
    """Angles in 64 bits: a position of 100000 times a frequency keeps 17 bits of its turn in 32."""
    q, k, v, cu, dev = st["q"], st["k"], st["v"], st["cu"].long(), st["q"].device
    T, page = q.shape[0], case["page"]
    N, half = len(st["lens"]), case["rotary"] // 2
    seq = torch.repeat_interleave(torch.arange(N, device=dev), cu[1:] - cu[:-1], output_size=T)
    at = st["lens"].long()[seq] - cu[1:][seq] + torch.arange(T, device=dev)
    if st["positions"] is None:
        turn = at.double()[:, None] * st["inv_freq"].double()
    else:
        turn = st["positions"].double()[st["axis"].long()].T * st["inv_freq"].double()
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]

    def rotated(x):
        f = x.float()
        rest = f[..., 2 * half:]
        if case["interleaved"]:
            a, b = f[..., 0:2 * half:2], f[..., 1:2 * half:2]
            both = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = f[..., :half], f[..., half:2 * half]
            both = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([both, rest], -1).to(x.dtype)

    where = st["table"][seq, at // page].long()
    st["k_cache"][where, :, at % page] = rotated(k)
    st["v_cache"][where, :, at % page] = v
    return {"q": rotated(q), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _attend(st, case):
    """All sequences padded to the longest."""
    q, cu, dev, d, page = st["q"], st["cu"].long(), st["q"].device, case["d"], case["page"]
    T, Hkv, G = q.shape[0], case["Hkv"], case["Hq"] // case["Hkv"]
    N, most = len(st["lens"]), max(_numbers(case["new"]))
    lens, i = st["lens"].long(), torch.arange(most, device=dev)
    idx = cu[:-1, None] + i
    live = idx < cu[1:, None]
    x = q[idx.clamp(max=T - 1)].float().view(N, most, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * most, d)
    table = st["table"].long().clamp(min=0)

    def cached(c):
        return c[table].float().transpose(1, 2).reshape(N, Hkv, -1, d)

    s = x @ cached(st["k_cache"]).transpose(-1, -2).contiguous()
    s = s.view(N, Hkv, G, most, -1).mul_(d ** -0.5)
    at = (lens - (cu[1:] - cu[:-1]))[:, None] + i
    j = torch.arange(table.shape[1] * page, device=dev)
    seen = j <= at[..., None]
    if case["window"]:
        seen = seen & (j > at[..., None] - case["window"])
    seen = seen[:, None, None]
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(N, Hkv, G * most, -1) @ cached(st["v_cache"])).view(N, Hkv, G, most, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(N, most, Hkv * G, d).to(q.dtype)
    out = torch.empty(T + 1, Hkv * G, d, dtype=q.dtype, device=dev)
    out[torch.where(live, idx, T)] = o
    return {"o": out[:T]}


def _select(st, case):
    """In 64 bits: continuations of different beams may lie 1e-7 apart."""
    x, finished = st["logits"].double(), st["finished"]
    B, W, V = x.shape
    top = x.amax(-1, keepdim=True)
    total = top + torch.exp(x - top).sum(-1, keepdim=True).log()
    c = st["scores"].double()[..., None] + (x - total)
    pad = torch.arange(V, device=x.device) == 0
    c = torch.where(finished[..., None], torch.where(pad, st["scores"].double()[..., None], -math.inf), c)
    best, at = torch.sort(c.view(B, W * V), dim=-1, descending=True, stable=True)   # equal ones in their order
    best, at = best[:, :case["K"]], at[:, :case["K"]]
    void = best == -math.inf
    tokens, parents = torch.where(void, -1, at % V), torch.where(void, -1, at // V)
    done = finished.gather(1, parents.clamp(min=0)) | (tokens == 2) | void
    return {"tokens": tokens.int(), "parents": parents.int(), "scores": best.float(), "finished": done}


def _reorder(st, case):
    if case["kind"] == "states":
        B, W = st["parents"].shape
        rows = (st["parents"].long() + W * torch.arange(B, device=st["parents"].device)[:, None]).flatten()
        st["state"].copy_(st["state"][:, rows])
        return {"state": st["state"]}
    src, dst = st["src"].long().flatten(), st["dst"].long().flatten()
    dst = torch.where(dst >= 0, dst, src)       # a beam that goes on in its own page copies it onto itself
    st["k_cache"][dst] = st["k_cache"][src]
    st["v_cache"][dst] = st["v_cache"][src]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "select":
        B, W, K, V = case["B"], case["W"], case["K"], case["V"]
        return {"bytes": B * (W * V * BYTES[case["dtype"]] + 5 * W + 13 * K), "flops": 4 * B * W * V}
    if case["op"] == "reorder":   # random parents: rows that change, and those that they come from
        B, W = case["B"], case["W"]
        moved, read = B * (W - 1.0), B * W * (1.0 - (1.0 - 1.0 / W) ** (W - 1))
        if case["kind"] == "states":
            return {"bytes": case["layers"] * (moved + read) * case["Hv"] * case["dk"] * case["dv"] * 4, "flops": 0}
        return {"bytes": 2 * (moved + read) * case["Hkv"] * case["page"] * case["d"] * BYTES[case["dtype"]],
                "flops": 0}
    es, new, ctx = BYTES[case["dtype"]], _numbers(case["new"]), _numbers(case["ctx"])
    T, Hq, Hkv, d = sum(new), case["Hq"], case["Hkv"], case["d"]
    tables = 4 * (2 * len(new) + 1) + 4 * sum(-(-n // case["page"]) for n in ctx)
    if case["op"] == "append":
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * d * es + (4 * case["axes"] * T if case["axes"] > 1 else 0) + tables,
                "flops": 3 * T * (Hq + Hkv) * case["rotary"]}
    w = case["window"]
    seen = keys = 0
    for n, m in zip(new, ctx):
        if n:
            keys += min(m, w + n - 1) if w else m
            first = m - n + 1
            if not w or m <= w:
                seen += n * (first + m) // 2
            else:
                short = max(0, w - first + 1)      # rows that see less than the window
                seen += short * (first + first + short - 1) // 2 + (n - short) * w
    return {"bytes": (2 * T * Hq + 2 * keys * Hkv) * d * es + tables, "flops": 4 * seen * Hq * d}


# ---------------------------------------------------------------------------------------------------------------
# exact values, from the definitions
# ---------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "select":
        scores = torch.empty(case["B"], case["K"], dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            every = []
            for w in range(case["W"]):
                start = st["scores"][b, w].double()
                if bool(st["finished"][b, w]):
                    every.append(start[None])
                else:
                    every.append(start + torch.log_softmax(st["logits"][b, w].double(), 0).topk(case["K"])[0])
            every.append(torch.full((case["K"],), -math.inf, dtype=torch.float64, device="cuda"))
            scores[b] = torch.cat(every).topk(case["K"])[0]
        return {"tokens": None, "parents": None, "scores": scores, "finished": None}
    if case["op"] == "reorder":
        if case["kind"] == "states":
            got = st["state"].double()
            for b, row in enumerate(st["parents"].tolist()):
                for j, p in enumerate(row):
                    got[:, b * case["W"] + j] = st["state"][:, b * case["W"] + p].double()
            return {"state": got}
        got = {n: st[n].double() for n in ("k_cache", "v_cache")}
        for s, t in zip(st["src"].flatten().tolist(), st["dst"].flatten().tolist()):
            if t >= 0:
                for n in got:
                    got[n][t] = st[n][s].double()
        return got
    new, ctx, cu, page, d = _numbers(case["new"]), _numbers(case["ctx"]), st["cu"].tolist(), case["page"], case["d"]
    G = case["Hq"] // case["Hkv"]
    if case["op"] == "append":
        got = {"q": st["q"].double(), "k_cache": st["k_cache"].double(), "v_cache": st["v_cache"].double()}
        half = case["rotary"] // 2
        for s, n in enumerate(new):
            if n == 0:
                continue
            at = torch.arange(ctx[s] - n, ctx[s], device="cuda")
            turns = torch.empty(n, half, dtype=torch.float64, device="cuda")
            for i in range(half):
                a = at if st["positions"] is None else st["positions"][int(st["axis"][i]), cu[s]:cu[s + 1]]
                turns[:, i] = a.double() * float(st["inv_freq"][i])
            z = torch.polar(torch.ones_like(turns), turns)[:, None]
            pages = st["table"][s].long()[at // page]
            for name in ("q", "k"):
                x = st[name][cu[s]:cu[s + 1]].double()
                i = torch.arange(half, device="cuda")
                first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                y = torch.complex(x[..., first], x[..., second]) * z
                x[..., first], x[..., second] = y.real, y.imag
                if name == "q":
                    got["q"][cu[s]:cu[s + 1]] = x
                else:
                    got["k_cache"][pages, :, at % page] = x
            got["v_cache"][pages, :, at % page] = st["v"][cu[s]:cu[s + 1]].double()
        return got
    o = torch.zeros(sum(new), case["Hq"], d, dtype=torch.float64, device="cuda")
    for s, n in enumerate(new):
        if n == 0:
            continue
        j = torch.arange(ctx[s], device="cuda")
        where = st["table"][s].long()[j // page]
        i = torch.arange(ctx[s] - n, ctx[s], device="cuda")[:, None]
        hidden = (j > i) | (j <= i - case["window"] if case["window"] else False)
        for h in range(case["Hkv"]):
            k, v = (st[c][where, h, j % page].double() for c in ("k_cache", "v_cache"))
            for g in range(G):
                x = st["q"][cu[s]:cu[s + 1], h * G + g].double()
                weights = torch.softmax((x @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf), -1)
                o[cu[s]:cu[s + 1], h * G + g] = weights @ v
    return {"o": o}
