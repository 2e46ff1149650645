"""Speculative decoding through one recurrent layer, as a serving loop strings the calls together.

A toy model: embedding, one block, unembedding. The block is

    normed = RMS norm of the residual stream        block_norm_fwd (norm before the block)
    xbc    = normed W_in                            raw rows [x | B | C]
    prompt: conv_fwd, ssm_fwd                       drafts: ssm_step (convolution and scan in one call)
    u      = RMS norm of y per head, times silu(z)  block_norm_fwd (output norm of the core)
    out    = residual + scale * RMS norm(u W_out)   block_norm_fwd (norm after the block, and before the next)

Decoding drafts L tokens at a time (here from the model's own distribution, disturbed), verifies them in one
ssm_step that commits nothing, lets draft_verify decide how many stand and which token follows, and replays the
accepted ones at the head of the next step: first_slot and accept_len pass from one call to the next on the device.

    python examples/draft_decode.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_chunked_gb300 as kda


class Layer:
    def __init__(self, vocab=96, dim=256, heads=4, head_dim=64, groups=1, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, k=1.0: torch.randn(s, generator=gen, device=device) * k
        self.V, self.d, self.H, self.P, self.G = vocab, dim, heads, head_dim, groups
        self.inner = heads * head_dim
        self.C = self.inner + 2 * groups * 128
        self.embed = r(vocab, dim).bfloat16()
        self.w_in = r(dim, self.C + self.inner, k=dim ** -0.5).bfloat16()      # xbc and the gate z
        self.w_dt = r(dim, heads, k=dim ** -0.5).bfloat16()
        self.w_out = r(self.inner, dim, k=self.inner ** -0.5).bfloat16()
        self.unembed = r(dim, vocab, k=4 * dim ** -0.5).bfloat16()
        self.conv_w, self.conv_b = r(self.C, 4, k=0.5), r(self.C, k=0.1)
        self.a, self.d_skip, self.dt_bias = -torch.exp(r(heads)), torch.ones(heads, device=device), r(heads, k=0.5) - 2.0
        self.w1, self.w2, self.w3, self.w_core = (torch.ones(n, device=device) for n in (dim, dim, dim, head_dim))
        self.scale = torch.full((dim,), 0.7, device=device)

    def rows(self, tokens):
        """The block's inputs for tokens [...]: residual, xbc, gate, dt."""
        res = self.embed[tokens]
        _, normed, _ = kda.block_norm_fwd(res, None, w_pre=self.w1)
        proj = normed @ self.w_in
        return res, proj[..., :self.C].contiguous(), proj[..., self.C:].contiguous(), (normed @ self.w_dt).float().contiguous()

    def logits(self, res, y, z):
        lead = y.shape[:-2]
        core, _, _ = kda.block_norm_fwd(y, self.w_core, gate=z.view(y.shape), gate_act="silu")
        u = core.reshape(*lead, self.inner) @ self.w_out
        _, normed, _ = kda.block_norm_fwd(u, self.w2, residual=res, scale=self.scale, w_pre=self.w3)
        return (normed @ self.unembed).float()

    def prompt(self, tokens, lens):
        """Packed prompts: logits of every token, and the two states of every sequence."""
        cu = torch.tensor([0] + list(lens), device=tokens.device).cumsum(0).to(torch.int32)
        res, xbc, z, dt = self.rows(tokens)
        rows, conv = kda.conv_fwd(xbc, self.conv_w, self.conv_b, cu, n_seqs=len(lens))
        x, b, c = torch.split(rows, [self.inner, self.G * 128, self.G * 128], -1)
        y, state = kda.ssm_fwd(x.unflatten(-1, (self.H, self.P)), dt, self.a, b.unflatten(-1, (self.G, 128)),
                               c.unflatten(-1, (self.G, 128)), cu, d_skip=self.d_skip, dt_bias=self.dt_bias)
        return self.logits(res, y, z), conv, state

    def step(self, tokens, conv, state, accept, first=None):
        """L token slots of every sequence: logits [N, L, V]; the states advance through ``accept`` slots."""
        res, xbc, z, dt = self.rows(tokens)
        out = torch.zeros(*tokens.shape, self.H, self.P, dtype=xbc.dtype, device=xbc.device)
        y = kda.ssm_step(xbc, dt, self.a, self.conv_w, self.conv_b, conv, state, accept, groups=self.G, d_skip=self.d_skip,
                         dt_bias=self.dt_bias, first_slot=first, out=out)
        return self.logits(res, y, z)


def decode(layer, prompts, n_tokens, drafts=3, noise=0.5, seed=1):
    """Continues every prompt by at least n_tokens. Returns the tokens of each sequence and its two states, which have
    advanced through all of them but the last accepted ones still to be replayed (accept, and the tokens)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, L = len(prompts), drafts
    lens = [len(p) for p in prompts]
    logits, conv, state = layer.prompt(torch.cat(prompts), lens)
    ends = torch.tensor(lens, device="cuda").cumsum(0) - 1
    p = torch.softmax(logits[ends], -1)
    exp = lambda *s: torch.empty(*s, device="cuda").exponential_(generator=gen)
    last = (p / exp(N, layer.V)).argmax(-1).to(torch.int32)                  # the first token, and its successor's input
    texts = [[int(t)] for t in last]
    accept = torch.zeros(N, dtype=torch.int32, device="cuda")                # nothing to replay yet
    replay = torch.zeros(N, L + 1, dtype=torch.int64, device="cuda")
    all_ = torch.full((N,), L + 1, dtype=torch.int32, device="cuda")
    while min(len(t) for t in texts) < n_tokens:
        # the drafter: the layer itself, its logits disturbed, on copies of the states
        ids, dists = [], []
        dconv, dstate = conv.clone(), state.clone()
        layer.step(replay, dconv, dstate, all_, L + 1 - accept)
        tok = last.long()
        for _ in range(L):
            lg = layer.step(tok[:, None], dconv, dstate, None)[:, 0]
            q = torch.softmax(lg + noise * torch.randn(lg.shape, generator=gen, device="cuda"), -1)
            tok = (q / exp(N, layer.V)).argmax(-1)
            ids.append(tok)
            dists.append(q)
        draft, q = torch.stack(ids, 1).to(torch.int32), torch.stack(dists, 1)
        # one call: [padding | the accepted tokens of last time | last | drafts]; commits the accepted ones
        window = torch.cat([replay, last.long()[:, None]], 1)
        slots = torch.cat([window, draft.long()], 1)                         # L + 1 + 1 + L slots
        first = L + 1 - accept
        lg = layer.step(slots, conv, state, all_, first)[:, L + 1:]
        p = torch.softmax(lg, -1)                                            # after last, after draft 1, ...
        stood, _, tokens = kda.draft_verify(p.contiguous(), q, draft, torch.rand(N, L, generator=gen, device="cuda"), exp(N, layer.V))
        # the next replay: last and the accepted drafts, right-aligned in L + 1 slots
        line = torch.cat([last.long()[:, None], draft.long()], 1)
        at = torch.arange(L + 1, device="cuda")[None, :] - (L - stood.long())[:, None]
        replay = line.gather(1, at.clamp(min=0))
        accept = stood + 1
        last = tokens.gather(1, stood.long()[:, None])[:, 0]
        for i, row in enumerate(tokens.tolist()):
            texts[i] += [t for t in row if t >= 0]
    layer.step(replay, conv, state, all_, L + 1 - accept)                    # what is still to be committed
    return texts, conv, state


def main():
    layer = Layer()
    gen = torch.Generator(device="cuda").manual_seed(3)
    prompts = [torch.randint(0, layer.V, (n,), generator=gen, device="cuda") for n in (37, 5, 160)]
    texts, conv, state = decode(layer, prompts, 24)
    for p, t in zip(prompts, texts):
        print(f"{len(p)} prompt tokens -> {len(t)}: {t[:24]}")
    # the states are those of a prompt that held the decoded tokens from the start (all but the last, which is input to come)
    full = [torch.cat([p, torch.tensor(t[:-1], device="cuda")]) for p, t in zip(prompts, texts)]
    _, conv2, state2 = layer.prompt(torch.cat(full), [len(f) for f in full])
    err = ((state - state2).norm() / state2.norm()).item()
    print(f"state after drafting and replaying against one prompt: {err:.1e} relative; convolution state equal: {torch.equal(conv, conv2)}")
    return err, torch.equal(conv, conv2)


if __name__ == "__main__":
    main()
