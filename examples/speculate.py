"""Text with drafted tokens: the network of generate.py takes a tree of them a
step, through the library's calls for drafted tokens.

The draft is the network without its layers (embedding, last norm, vocabulary).
Each step, for every text that goes on,

    a tree below the last token, level by level, from the draft's logits
    mt_tree_layout                      positions and visibility bits
    the layers, as in generate.py, with mt_tree_attention
    mt_token_probs -> mt_tree_verify    the accepted tokens and the one after them
    mt_cache_keep                       their keys and values, in all layers

The weights are random, so the text means nothing; its tokens are those that the
network alone would take (temperature 0), or are distributed as if it drew them
one by one.

    python examples/speculate.py --tokens 32 --temperature 0.7 --drawn
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from generate import EPS, Config, Model, Runner, mt, reference  # noqa: E402, F401


def tree_of(widths):
    """(parents, first token of each level): each token of level k has widths[k] children."""
    parent, level, starts = [-1], [0], [0]
    for w in widths:
        starts.append(len(parent))
        level = [len(parent) + i for i in range(len(level) * w)]
        parent += [starts[-2] + i // w for i in range(len(level))]
    return parent, starts + [len(parent)]


class TreeRunner(Runner):
    def draft(self, tokens):
        """The draft's logits after each of the tokens."""
        x = self.m.embed[tokens.long()]
        return self._linear(self._norm(x, torch.zeros_like(x), self.m.norm)[1], self.m.head, torch.float32)

    def tree(self, tokens, parent, q_start, kv_len, longest):
        """The logits after every one of the trees' tokens."""
        c, m = self.m.cfg, self.m
        D, H, KV, T = c.head_dim, c.q_heads, c.kv_heads, tokens.numel()
        i32 = dict(dtype=torch.int32, device="cuda")
        positions, visible = torch.empty(T, **i32), torch.empty(T, (longest + 31) // 32, **i32)
        mt.mt_tree_layout(parent, q_start, kv_len, positions, visible)
        space = torch.empty(mt.mt_paged_attention_workspace_bytes(T, self.texts, H, KV, D), dtype=torch.uint8, device="cuda")
        x = m.embed[tokens.long()]
        zero = torch.zeros_like(x)
        for layer, (kc, vc) in zip(m.layers, self.cache):
            residual, n = self._norm(x, zero, layer["n1"])
            q, k, v = self._linear(n, layer["qkv"]).split([H * D, KV * D, KV * D], 1)
            q, k, v = q.unflatten(1, (H, D)), k.unflatten(1, (KV, D)), v.unflatten(1, (KV, D))
            mt.mt_rope_append(q, k, v, positions, m.inv_freq, q, kc, vc, self.pages, q_start, kv_len, q_norm=layer["qn"],
                              k_norm=layer["kn"], eps=EPS)
            a = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
            mt.mt_tree_attention(q, kc, vc, self.pages, q_start, kv_len, visible, longest, 1 / math.sqrt(D), a, space, window=c.window,
                                 sinks=c.sinks)
            residual, n = self._norm(self._linear(a.view(T, H * D), layer["o"]), residual, layer["n2"])
            x = self._mlp(n, residual, layer)
        return self._linear(self._norm(x, zero, m.norm)[1], m.head, torch.float32)


def generate(model: Model, prompts: list[list[int]], tokens: int, temperature: float = 0.0, widths=(3, 2, 1), drawn: bool = False,
             seed: int = 0):
    """Continues the prompts by at least `tokens` tokens.  widths: children of a
    token at each level of the drafted trees; drawn: children drawn from the
    draft's distribution under the temperature, not its most probable tokens.
    Returns the texts, and of every step the accepted tokens' logits, as
    (text, tokens that they follow, logits)."""
    B, c = len(prompts), model.cfg
    if not all(prompts) or tokens < 1 or not widths or min(widths) < 1 or (drawn and not temperature > 0):
        raise ValueError("prompts of a token or more, a token or more to make, trees, and a temperature to draw at are required")
    tree, level = tree_of(widths)
    n, depth = len(tree), len(widths)
    run = TreeRunner(model, max(map(len, prompts)) + tokens + depth + n, B)
    g = torch.Generator(device="cuda").manual_seed(seed)
    texts, raw = [list(p) for p in prompts], []
    if any(len(p) > 1 for p in prompts):
        run.step([p[:-1] for p in prompts])  # all but the last token, the first tree's root
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    while True:
        on = [b for b in range(B) if len(texts[b]) < len(prompts[b]) + tokens]
        if not on:
            return texts, raw
        A = len(on)
        # ---- the trees, all texts' level by level
        drafted = torch.empty(A, n, **i32)
        drafted[:, 0] = torch.tensor([texts[b][-1] for b in on], **i32)
        q = torch.zeros(A, n, c.vocab, **f32) if drawn else None
        for k, w in enumerate(widths):
            above, here = slice(level[k], level[k + 1]), slice(level[k + 1], level[k + 2])
            logits = run.draft(drafted[:, above].reshape(-1))
            if drawn:
                p = torch.empty_like(logits)
                mt.mt_token_probs(logits, p, torch.full((p.shape[0],), temperature, **f32))
                q[:, above] = p.view(A, -1, c.vocab)
                picked = torch.multinomial(p, w, replacement=True, generator=g)
            else:
                picked = logits.topk(w, 1).indices
            drafted[:, here] = picked.view(A, -1).to(torch.int32)
        # ---- the network takes them all; texts that are done have none
        starts = [0]
        for b in range(B):
            starts.append(starts[-1] + (n if b in on else 0))
        ids, parent = drafted.view(-1), torch.tensor(tree * A, **i32)
        q_start = torch.tensor(starts, **i32)
        kv_len = torch.tensor([run.lens[b] + (n if b in on else 0) for b in range(B)], **i32)
        logits = run.tree(ids, parent, q_start, kv_len, n)
        # ---- the accepted path and the token after it
        target = torch.empty_like(logits)
        mt.mt_token_probs(logits, target, torch.full((A * n,), temperature, **f32))
        out, path = torch.empty(B, depth + 1, **i32), torch.empty(B, depth + 1, **i32)
        count, kept = torch.empty(B, **i32), torch.empty(B, **i32)
        mt.mt_tree_verify(target, ids, parent, torch.rand(A * n, generator=g, device="cuda"), q_start, out, path, count,
                          draft=q.view(A * n, c.vocab) if drawn else None)
        mt.mt_cache_keep(run.cache, run.pages, q_start, kv_len, path, count, new_len=kept)
        for b, m, t, where in zip(range(B), count.tolist(), out.tolist(), path.tolist()):
            for i in range(m):
                raw.append((b, len(texts[b]) + i, logits[starts[b] + where[i]]))
            texts[b] += t[:m]
        run.lens = kept.tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--drawn", action="store_true")
    a = ap.parse_args()
    model = Model(Config())
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (5, 37, 130)]
    texts, raw = generate(model, prompts, a.tokens, a.temperature, drawn=a.drawn)
    for p, t in zip(prompts, texts):
        print(f"prompt of {len(p)} tokens, then", t[len(p):])
    print(f"{sum(len(t) - len(p) for p, t in zip(prompts, texts))} tokens of {len(texts)} texts")


if __name__ == "__main__":
    main()
