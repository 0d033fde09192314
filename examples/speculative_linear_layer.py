"""Speculative decoding of a small model whose mixer is linear attention with a
decay for each head, on the library's entry points end to end.

The model is random: embedding, L blocks of

    h = norm(x);  q, k, v, z = projections of h
    o = linear attention(q, k, v, alpha)      gdn_linear_prefill / gdn_linear_recurrent
    y = gated norm(o, z) @ W_o                gdn_gated_norm
    x, h' = x + s norm(y), norm(...)          gdn_residual_norm

and an output head.  A prompt is prefilled; then every step drafts K tokens (from
the target's own embedding and head, so that some are accepted), runs the last token and
the drafts through the target in one pass with the state capture, verifies them
with gdn_accept_drafts, and commits as many captured tokens to each layer's state
as were emitted with gdn_replay_state_updates.  Nothing in a step goes through the
host; the tokens are read once at the end.

    python examples/speculative_linear_layer.py [--batch B] [--steps N] [--drafts K]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_deltanet_recurrence_02_gb300 import gdn  # noqa: E402


class Model:
    def __init__(self, layers=2, Hk=2, Hv=4, dk=64, dv=64, vocab=1000, seed=0, dtype=torch.bfloat16):
        g = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, device="cuda", generator=g) / shape[0] ** 0.5).to(dtype)

        self.Hk, self.Hv, self.dk, self.dv, self.D, self.vocab = Hk, Hv, dk, dv, Hv * dv, vocab
        self.embed = torch.randn(vocab, self.D, device="cuda", generator=g).to(dtype)
        self.head = weight(self.D, vocab)
        self.layers = [dict(
            wq=weight(self.D, Hk * dk), wk=weight(self.D, Hk * dk), wvz=weight(self.D, 2 * self.D),
            wo=weight(self.D, self.D), norm=torch.ones(dv, device="cuda"), post=torch.ones(self.D, device="cuda"),
            pre=torch.ones(self.D, device="cuda"),
            # one fixed decay for each head, from some ten tokens to some hundred
            alpha=1 - 2.0 ** -torch.linspace(3, 7, Hv, device="cuda")) for _ in range(layers)]

    def states(self, batch):
        return [torch.zeros(batch, self.Hv, self.dv, self.dk, device="cuda") for _ in self.layers]

    def run(self, tokens, batch, states, capture=0):
        """Tokens [batch * T] through the model.  Without capture the states move on;
        with it they stay, and the captures come back.  Returns probabilities
        [batch, T, vocab] and the captures."""
        T = tokens.numel() // batch
        x = self.embed[tokens].float()
        x, h = gdn.gdn_residual_norm(self.embed.new_zeros(x.shape), x, pre_weight=self.layers[0]["pre"])
        captures = []
        count = torch.full((batch,), T, dtype=torch.int32, device="cuda") if capture else None
        for i, w in enumerate(self.layers):
            q = torch.nn.functional.normalize((h @ w["wq"]).unflatten(1, (self.Hk, self.dk)), dim=-1)
            k = torch.nn.functional.normalize((h @ w["wk"]).unflatten(1, (self.Hk, self.dk)), dim=-1)
            vz = h @ w["wvz"]
            v = vz[:, :self.D].unflatten(1, (self.Hv, self.dv)).contiguous()
            z = vz[:, self.D:].unflatten(1, (self.Hv, self.dv))  # a slice of the wider rows
            how = dict(B=batch, T=T, initial_state=states[i], conventions=gdn.GDN_ALPHA_PER_HEAD,
                       scale=self.dk ** -0.5)
            if capture:
                o, _, seen = gdn.gdn_linear_recurrent(q, k, v, w["alpha"], state_update_capacity=capture,
                                                      capture_count=count, want_final_state=False, **how)
                captures.append(seen)
            else:
                o, _ = gdn.gdn_linear_prefill(q, k, v, w["alpha"], final_state=states[i], **how)
            y = gdn.gdn_gated_norm(o, z, w["norm"]).flatten(1) @ w["wo"]
            follows = self.layers[min(i + 1, len(self.layers) - 1)]["pre"]
            x, h = gdn.gdn_residual_norm(y, x, post_weight=w["post"], res_scale=0.5, pre_weight=follows,
                                         residual_out=x)
        return torch.softmax(2 * (h @ self.head).float(), -1).view(batch, T, -1), captures


def draft(model, last, K, generator):
    """K cheap drafts for each request and their distributions: a walk over the
    embedding and the head alone, without the layers."""
    probs, tokens = [], []
    for _ in range(K):
        _, h = gdn.gdn_residual_norm(model.embed[last])
        p = torch.softmax(2 * (h @ model.head).float(), -1)
        last = torch.multinomial(p, 1, generator=generator).squeeze(1)
        probs.append(p)
        tokens.append(last)
    return torch.stack(probs, 1).contiguous(), torch.stack(tokens, 1).to(torch.int32)


def generate(model, prompt, steps, K, seed=1):
    """Speculative generation from prompt [batch, T].  Returns the emitted tokens
    [batch, steps, K + 1] (-1 past the emitted ones) and the states."""
    batch = prompt.shape[0]
    g = torch.Generator("cuda").manual_seed(seed)
    states = model.states(batch)
    model.run(prompt[:, :-1].reshape(-1), batch, states)  # all but the last token
    last = prompt[:, -1]
    emitted = []
    for _ in range(steps):
        q, drafts = draft(model, last, K, g)
        tokens = torch.cat([last[:, None], drafts.long()], 1)
        p, captures = model.run(tokens.reshape(-1), batch, states, capture=K + 1)
        u = torch.rand(batch, K + 1, device="cuda", generator=g)
        out, n = gdn.gdn_accept_drafts(p, q, drafts, u)
        # the pass ran the last token and the drafts: as many of them as were emitted
        # are now part of the text
        for s, c in zip(states, captures):
            gdn.gdn_replay_state_updates(s, c, n, state_update_capacity=K + 1, Hk=model.Hk, state_out=s)
        last = out.gather(1, n.long()[:, None] - 1).squeeze(1).long()
        emitted.append(out)
    return torch.stack(emitted, 1), states


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200)
    a = ap.parse_args()
    model = Model()
    prompt = torch.randint(0, model.vocab, (a.batch, a.prompt), device="cuda",
                           generator=torch.Generator("cuda").manual_seed(2))
    emitted, _ = generate(model, prompt, a.steps, a.drafts)
    counts = (emitted >= 0).sum(-1).float()
    print(f"{a.batch} requests, {a.steps} steps of {a.drafts} drafts: {counts.mean().item():.2f} tokens a step")
    print("first request:", [t for t in emitted[0].flatten().tolist() if t >= 0])


if __name__ == "__main__":
    main()
