"""Speculative decoding over one linear-attention block with a decay for each head.

    python examples/speculative_round.py

A toy model with random weights (an embedding, one block, a head) continues ragged
prompts: gdn_linear_prefill reads them and leaves a state per row.  Then every
round a draft model (the embedding alone) proposes K tokens, gdn_linear_step runs
the last token and the drafts and records their state updates, gdn_block_norm
closes the block (the gated head norm; then residual, norm and the norm before the
head), gdn_verify_drafts accepts a prefix and draws one more token, and
gdn_replay_state_updates brings the states to exactly the accepted tokens.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import gated_deltanet_03_amd as gdn  # noqa: E402


class Model:
    def __init__(self, V=2003, Hq=2, Hv=4, dk=64, dv=64, dtype=torch.bfloat16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        D = Hv * dv

        def w(*shape):
            return (torch.randn(*shape, generator=gen, device=device) * shape[0] ** -0.5).to(dtype)
        self.V, self.Hq, self.Hv, self.D, self.device = V, Hq, Hv, D, device
        self.embedding = torch.randn(V, D, generator=gen, device=device).to(dtype)
        x = self.embedding                                      # one block: its inputs depend on the token alone
        self.q = (x @ w(D, Hq * dk)).view(V, Hq, dk)
        self.k = torch.nn.functional.normalize((x @ w(D, Hq * dk)).view(V, Hq, dk).float(), dim=-1).to(dtype)
        self.v, self.z = (x @ w(D, D)).view(V, Hv, dv), x @ w(D, D)
        self.wo, self.head = w(D, D), w(D, V) * 2
        self.ones, self.ones_dv = torch.ones(D, dtype=dtype, device=device), torch.ones(dv, dtype=dtype, device=device)
        # a fixed decay for each head, from a few tokens of memory to hundreds
        self.g = torch.log1p(-torch.exp2(-2.0 - torch.arange(Hv, device=device, dtype=torch.float32)))

    def close(self, tokens, o):
        """Probabilities after the block, from its tokens and the attention's output."""
        x, z = self.embedding[tokens], self.z[tokens]
        heads, _ = gdn.gdn_block_norm(o.reshape(-1, self.D), gate=z, gate_act="silu", post_weight=self.ones_dv)
        _, normed = gdn.gdn_block_norm(heads @ self.wo, residual=x, post_weight=self.ones, next_weight=self.ones)
        return torch.softmax((normed @ self.head).float(), -1)

    def prefill(self, tokens, cu):
        t = tokens.long()
        o, states = gdn.gdn_linear_prefill(self.q[t], self.k[t], self.v[t], self.g, cu_seqlens=cu)
        return self.close(t, o), states

    def draft(self, last, K, gen):
        """K tokens a row from the embedding alone, with its probabilities."""
        B = last.shape[0]
        tokens, probs = [last], []
        none = torch.empty(B, 0, dtype=torch.int32, device=self.device)
        for _ in range(K):
            p = torch.softmax((self.embedding[tokens[-1].long()] @ self.head).float(), -1)
            u = torch.rand(B, 1, generator=gen, device=self.device)
            t, _ = gdn.gdn_verify_drafts(p[:, None], None, none, u)      # no drafts: plain sampling
            tokens.append(t[:, 0])
            probs.append(p)
        return torch.stack(tokens, 1), torch.stack(probs, 1)


def generate(model, prompts, rounds=8, K=4, seed=1):
    """Tokens emitted for each prompt (lists), and the states after all but the last of them."""
    dev, B = model.device, len(prompts)
    gen = torch.Generator(device=dev).manual_seed(seed)
    lengths = torch.tensor([len(p) for p in prompts])
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lengths.cumsum(0)]).int().to(dev)
    probs, states = model.prefill(torch.cat(prompts).to(dev), cu)
    none = torch.empty(B, 0, dtype=torch.int32, device=dev)
    first, _ = gdn.gdn_verify_drafts(probs[(cu[1:] - 1).long()][:, None], None, none,
                                     torch.rand(B, 1, generator=gen, device=dev))
    last, out = first[:, 0].contiguous(), [first.cpu()]
    counts = torch.full((B,), K + 1, dtype=torch.int32, device=dev)
    records = None
    for _ in range(rounds):
        row, q_probs = model.draft(last, K, gen)                         # the last token and K drafts
        t = row.long()
        o, _, records = gdn.gdn_linear_step(model.q[t], model.k[t], model.v[t], model.g, initial_state=states,
                                            output_final_state=False, state_update_capacity=K + 1,
                                            capture_count=counts, state_update=records)
        p_probs = model.close(t.reshape(-1), o).view(B, K + 1, model.V)
        tokens, emitted = gdn.gdn_verify_drafts(p_probs, q_probs, row[:, 1:].contiguous(),
                                                torch.rand(B, K + 1, generator=gen, device=dev))
        gdn.gdn_replay_state_updates(states, records, emitted, Hq=model.Hq)
        last = tokens.gather(1, emitted.long()[:, None] - 1)[:, 0].contiguous()
        out.append(tokens.cpu())
    emitted = [[t for part in out for t in part[b].tolist() if t >= 0] for b in range(B)]
    return emitted, states


def main():
    model = Model()
    gen = torch.Generator().manual_seed(3)
    prompts = [torch.randint(0, model.V, (n,), generator=gen, dtype=torch.int32) for n in (37, 5, 300)]
    rounds = 8
    emitted, _ = generate(model, prompts, rounds)
    for p, e in zip(prompts, emitted):
        print(f"prompt of {len(p)} tokens: {len(e)} tokens in {rounds} rounds: {e[:12]} ...")


if __name__ == "__main__":
    main()
