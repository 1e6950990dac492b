"""Beam search over a gated-delta-rule block followed by an attention block.

    python examples/beam_search.py

A toy model with random weights continues ragged prompts with several beams each.  Its first block keeps a recurrent
state a beam (gdn_prefill_chunked, gdn_recurrent_step), its second one keys and values in pages (gdn_cache_append,
gdn_cache_attention).  After every token gdn_beam_select picks the best continuations, gdn_state_reorder moves the
states and gdn_cache_copy_pages the beams' own pages from each parent to its beam; the prompt's full pages are shared.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import gated_deltanet_03_amd as gdn  # noqa: E402


class Model:
    def __init__(self, V=503, Hq=2, Hv=4, dk=32, dv=32, heads=4, kv_heads=2, d=64, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        D = Hv * dv

        def w(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[0] ** -0.5).to(dtype)
        self.V, self.D, self.device, self.dtype = V, D, device, dtype
        self.Hq, self.Hv, self.dk, self.dv, self.heads, self.kv_heads, self.d = Hq, Hv, dk, dv, heads, kv_heads, d
        self.embedding = torch.randn(V, D, generator=gen, device=device).to(dtype)
        self.wq, self.wk, self.wv, self.wz = w(D, Hq * dk), w(D, Hq * dk), w(D, D), w(D, D)
        self.wg, self.wb, self.wo = w(D, Hv), w(D, Hv), w(D, D)
        self.wqkv, self.wproj, self.head = w(D, (heads + 2 * kv_heads) * d), w(heads * d, D), w(D, V) * 2
        self.ones, self.ones_dv = torch.ones(D, dtype=dtype, device=device), torch.ones(dv, dtype=dtype, device=device)
        self.inv_freq = 10000.0 ** (-torch.arange(d // 2, device=device, dtype=torch.float32) / (d // 2))

    def delta_inputs(self, x):
        """q, k, v, g, beta of the delta-rule block for rows [..., D]."""
        shape, unit = x.shape[:-1], torch.nn.functional.normalize
        q = unit((x @ self.wq).view(*shape, self.Hq, self.dk).float(), dim=-1).to(self.dtype)
        k = unit((x @ self.wk).view(*shape, self.Hq, self.dk).float(), dim=-1).to(self.dtype)
        v = (x @ self.wv).view(*shape, self.Hv, self.dv)
        return q, k, v, -torch.nn.functional.softplus((x @ self.wg).float()), torch.sigmoid((x @ self.wb).float())

    def close(self, x, o):
        """The delta-rule block's end: gated norm of its heads, residual, and the next block's norm."""
        y, _ = gdn.gdn_block_norm(o.reshape(-1, self.D).contiguous(), gate=(x @ self.wz).reshape(-1, self.D),
                                  gate_act="silu", post_weight=self.ones_dv)
        return gdn.gdn_block_norm(y @ self.wo, residual=x.reshape(-1, self.D).contiguous(), post_weight=self.ones,
                                  next_weight=self.ones)

    def attend(self, h, normed, cache, table, lens, cu=None, rows=None):
        """The attention block for normed rows [T, D]: packed (cu), or one token for each of `rows` sequences."""
        a, b, d = self.heads, self.kv_heads, self.d
        qkv = (normed @ self.wqkv).view(-1, a + 2 * b, d)
        if cu is None:
            qkv = qkv.view(rows, 1, a + 2 * b, d)
        q, k, v = qkv.split([a, b, b], dim=-2)
        q = gdn.gdn_cache_append(k, v, *cache, table, lens, cu_seqlens=cu, q=q, inv_freq=self.inv_freq)
        o = gdn.gdn_cache_attention(q, *cache, table, lens, cu_seqlens=cu)
        _, out = gdn.gdn_block_norm(o.reshape(-1, a * d) @ self.wproj, residual=h, post_weight=self.ones,
                                    next_weight=self.ones)
        return out


def search(model, prompts, beams=4, steps=12, page=16, eos=1):
    """The best `beams` continuations of each prompt: tokens [B, beams, steps] (0 behind the end) and scores."""
    dev, B, W = model.device, len(prompts), beams
    lengths = [len(p) for p in prompts]
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device=dev)
    # pages: a prompt's own, the full ones of which its beams share; then as many for each beam as it may fill
    full = [n // page for n in lengths]
    mine = -(-(steps + page) // page)
    first = [sum(n + 1 for n in full[:b]) for b in range(B + 1)]
    pages = first[B] + B * W * mine
    cache = [torch.zeros(pages, model.kv_heads, page, model.d, dtype=model.dtype, device=dev) for _ in range(2)]
    prompt_table = torch.full((B, max(full) + 1), -1, dtype=torch.int32)
    table = torch.full((B * W, max(full) + mine), -1, dtype=torch.int32)
    own = first[B] + torch.arange(B * W * mine, dtype=torch.int32).view(B, W, mine)
    for b in range(B):
        prompt_table[b, :full[b] + 1] = torch.arange(first[b], first[b + 1])
        for w in range(W):
            table[b * W + w, :full[b]] = torch.arange(first[b], first[b] + full[b])
            table[b * W + w, full[b]:full[b] + mine] = own[b, w]
    table, own = table.to(dev), own.to(dev)

    # the prompts, once each
    x = model.embedding[torch.cat(prompts).to(dev).long()]
    lens = torch.tensor(lengths, dtype=torch.int32, device=dev)
    o, states = gdn.gdn_prefill_chunked(*model.delta_inputs(x), cu_seqlens=cu)
    out = model.attend(*model.close(x, o), cache, prompt_table.to(dev), lens, cu=cu)
    last = out[(cu[1:] - 1).long()] @ model.head
    # every beam starts as the prompt: its state, and a copy of its last page
    tail = torch.tensor([first[b] + full[b] for b in range(B)], dtype=torch.int32, device=dev)
    gdn.gdn_cache_copy_pages(*cache, tail[:, None].expand(B, W).contiguous(), own[:, :, 0].contiguous())
    start = torch.full((B, W), -float("inf"), device=dev)
    start[:, 0] = 0.0
    states = states.repeat_interleave(W, 0)
    tokens, parents, scores, finished = gdn.gdn_beam_select(last[:, None].expand(B, W, model.V).contiguous(), start,
                                                            eos_token=eos)
    history = tokens[:, :, None]
    lens = lens.repeat_interleave(W)
    for step in range(1, steps):
        lens = lens + 1
        x = model.embedding[tokens.view(-1, 1).long()]
        o, _ = gdn.gdn_recurrent_step(*model.delta_inputs(x), initial_state=states, final_state=states)[:2]
        out = model.attend(*model.close(x, o), cache, table, lens, rows=B * W)
        tokens, parents, scores, finished = gdn.gdn_beam_select((out @ model.head).view(B, W, model.V), scores,
                                                                finished=finished, eos_token=eos)
        gdn.gdn_state_reorder(states, parents, out=states)
        # the pages written so far, page number by page number: a beam's i-th own page from its parent's i-th
        used = own[:, :, :(page + step - 1) // page + 1].transpose(1, 2).contiguous()
        source = used.gather(2, parents.long()[:, None].expand(used.shape))
        gdn.gdn_cache_copy_pages(*cache, source.view(-1, W), used.view(-1, W))
        history = torch.cat([history.gather(1, parents.long()[:, :, None].expand(history.shape)), tokens[:, :, None]], 2)
    return history, scores


def main():
    model = Model()
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(2, model.V, (n,), generator=gen, dtype=torch.int32) for n in (37, 5, 130)]
    history, scores = search(model, prompts)
    for p, h, s in zip(prompts, history.tolist(), scores.tolist()):
        print(f"prompt of {len(p)} tokens:")
        for tokens, score in zip(h, s):
            print(f"  {score:8.3f}  {tokens}")


if __name__ == "__main__":
    main()
