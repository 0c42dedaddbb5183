"""Decode steps of a small hybrid stack over one page pool: a KDA layer, then a latent-attention layer.

    python examples/hybrid_decode.py [--steps N] [--batch B] [--prompt T]

A batch of sequences shares a prompt.  The prompt's latent rows are appended once, into pages that every sequence's
attention reads as the shared prefix; a snapshot of the KDA state at its end sits in pages of the same pool and starts
every sequence.  Each step then runs, per layer, what a serving engine runs:

  KDA layer        kda_decode_step_fused: ShortConv, L2Norm, gates and one step of the recurrence, states in place
  attention layer  kda_mla_append (normalise, rotate, write the token's row and rotate its queries), then
                   kda_mla_decode over the shared prefix and the sequence's own pages

The weights are random; the projections around the operators are plain matrix products.  After the last step the
attention of every sequence is recomputed over its whole history in fp64 and the largest difference is printed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from kda_delta_rule_gb300 import kda as K  # noqa: E402

D, H, DK, DV = 512, 8, 64, 64            # model width, heads, KDA head sizes
DC, DR, PAGE = 256, 32, 64               # latent row, position part, tokens per page


class Weights:
    def __init__(self, gen):
        def w(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") / shape[0] ** 0.5).bfloat16()
        c = H * (2 * DK + DV)
        self.qkv, self.conv = w(D, c), (torch.randn(c, 4, generator=gen, device="cuda") / 2).bfloat16()
        self.gate, self.beta, self.kda_out = w(D, H * DK), w(D, H), w(H * DV, D)
        self.kv, self.kv_norm = w(D, DC + DR), (1 + 0.1 * torch.randn(DC, generator=gen, device="cuda")).bfloat16()
        self.q, self.q_pe, self.mla_out = w(D, H * DC), w(D, H * DR), w(H * DC, D)


def rope_table(n):
    ang = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(DR // 2, device="cuda", dtype=torch.float64) / (DR // 2))
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def slot(pages, t):
    return pages[t // PAGE] * PAGE + t % PAGE


def run(steps=80, batch=6, prompt=300, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = Weights(gen)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # one pool for both kinds of pages
    page_bytes = max(PAGE * (DC + DR) * 2, H * DK * DV * 4)
    pool = K.PagePool(page_bytes, 1 + -(-prompt // PAGE) + batch * -(-steps // PAGE))
    state_page = pool.alloc(1, K.PAGE_KDA_STATE)[0]
    prefix = pool.alloc(-(-prompt // PAGE), K.PAGE_MLA_KV)
    own = [[] for _ in range(batch)]
    rope, scale = rope_table(prompt + steps), (DK + DR) ** -0.5

    # the shared prompt: its latent rows, once, and a snapshot of the recurrent state
    x = torch.randn(prompt, D, generator=gen, device="cuda").bfloat16()
    kv = x @ w.kv
    K.kda_mla_append(pool.pages, PAGE, i32([slot(prefix, t) for t in range(prompt)]), i32(list(range(prompt))), rope,
                     kv[:, :DC], kv[:, DC:], norm_weight=w.kv_norm)
    pool.store_kda(state_page, 0.05 * torch.randn(1, H, DK, DV, generator=gen, device="cuda"))
    state = torch.empty(1, H, DK, DV, device="cuda")
    pool.load_kda(state_page, state)
    state = state.repeat(batch, 1, 1, 1)
    conv = torch.zeros(batch, 3, H * (2 * DK + DV), device="cuda", dtype=torch.bfloat16)

    table = torch.full((batch, -(-steps // PAGE)), -1, dtype=torch.int32, device="cuda")
    for t in range(steps):
        if t % PAGE == 0:                                   # a fresh page for every sequence
            for b, page in enumerate(pool.alloc(batch, K.PAGE_MLA_KV)):
                own[b].append(page)
            table[:, t // PAGE] = i32([p[-1] for p in own])
        h = torch.randn(batch, D, generator=gen, device="cuda").bfloat16()
        o = K.kda_decode_step_fused(state, conv, h @ w.qkv, w.conv, (h @ w.gate).view(batch, H, DK), h @ w.beta)
        h = h + o.reshape(batch, H * DV) @ w.kda_out
        kv = h @ w.kv
        q_pe = K.kda_mla_append(pool.pages, PAGE, i32([slot(p, t) for p in own]), i32([prompt + t] * batch), rope,
                                kv[:, :DC], kv[:, DC:], q_pe=(h @ w.q_pe).view(batch, H, DR), norm_weight=w.kv_norm)
        q = (h @ w.q).view(batch, 1, H, DC)
        o, lse = K.kda_mla_decode(q, q_pe.view(batch, 1, H, DR), pool.pages, PAGE, table, i32([t + 1] * batch), scale,
                                  prefix_pages=i32(prefix), prefix_len=prompt)
        h = h + o.reshape(batch, H * DC) @ w.mla_out
    assert K.kda_device_errors() == 0

    # the last step's attention again, over each sequence's whole history
    rows = pool.pages[:, :PAGE * (DC + DR) * 2].view(torch.bfloat16).view(pool.n_pages, PAGE, DC + DR)
    worst = 0.0
    for b in range(batch):
        keys = torch.cat([rows[prefix].flatten(0, 1)[:prompt], rows[own[b]].flatten(0, 1)[:steps]]).double()
        s = torch.cat([q[b, 0], q_pe[b]], -1).double() @ keys.T * scale
        ref = torch.softmax(s, -1) @ keys[:, :DC]
        worst = max(worst, float((o[b, 0].double() - ref).abs().max() / ref.abs().max()))
    return worst, h


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=80)
    ap.add_argument("--batch", type=int, default=6)
    ap.add_argument("--prompt", type=int, default=300)
    args = ap.parse_args()
    worst, h = run(args.steps, args.batch, args.prompt)
    print(f"{args.steps} steps of {args.batch} sequences behind {args.prompt} shared tokens: attention within {worst:.1e} "
          f"of fp64, |h| = {float(h.float().norm()):.3f}")


if __name__ == "__main__":
    main()
