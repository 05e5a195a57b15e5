"""A small transformer that generates text through the library's calls alone.

Every step of a batch - prompts of several lengths, then single tokens - runs

    mt_add_rmsnorm -> q/k/v projection -> mt_rope_append -> mt_paged_attention
    -> o projection -> mt_add_rmsnorm -> mt_swiglu_gateup -> mt_down_residual

per layer (the mt_prefill_* calls where there are more than eight rows), then
the vocabulary projection, mt_logit_penalties and an argmax.  The weights are
random bf16, so the text means nothing; the same network in plain torch
operations (``reference``) gives the same logits up to bf16 rounding.

    python examples/generate.py --tokens 32
"""
from __future__ import annotations

import argparse
import math
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_gemv_epilogues_gb300 as mt  # noqa: E402

BF = mt.MT_W_BF16
EPS = 1e-6


@dataclass
class Config:
    layers: int = 2
    hidden: int = 512
    ffn: int = 1408
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    vocab: int = 5003
    page: int = 16
    window: int = 0       # 0: full attention
    sinks: int = 0
    theta: float = 10000.0


class Model:
    def __init__(self, cfg: Config, seed: int = 0, device: str = "cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g) / math.sqrt(shape[-1])).to(torch.bfloat16).to(device)

        def gain(n):
            return (1 + 0.1 * torch.randn(n, generator=g)).to(torch.bfloat16).to(device)

        c, D = cfg, cfg.head_dim
        self.cfg = cfg
        self.embed = torch.randn(c.vocab, c.hidden, generator=g).to(torch.bfloat16).to(device)
        self.head = w(c.vocab, c.hidden)
        self.norm = gain(c.hidden)
        # q, k and v of a layer stacked: one projection, and rows whose parts the rotary call takes as views
        self.layers = [dict(n1=gain(c.hidden), qkv=w((c.q_heads + 2 * c.kv_heads) * D, c.hidden), qn=gain(D), kn=gain(D),
                            o=w(c.hidden, c.q_heads * D), n2=gain(c.hidden), gate=w(c.ffn, c.hidden), up=w(c.ffn, c.hidden),
                            down=w(c.hidden, c.ffn)) for _ in range(c.layers)]
        self.inv_freq = (c.theta ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(device)


def last_rows(new: list[list[int]]) -> list[int]:
    """The row of the last new token of every text that has any."""
    rows, at = [], 0
    for n in new:
        at += len(n)
        if n:
            rows.append(at - 1)
    return rows


class Runner:
    """The paged cache of up to ``len(texts)`` texts and the buffers of a step."""

    def __init__(self, model: Model, max_tokens: int, texts: int):
        c = model.cfg
        self.m, self.texts = model, texts
        self.width = -(-max_tokens // c.page)
        pages = self.width * texts
        shape = (pages, c.page, c.kv_heads, c.head_dim)
        self.cache = [(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
                      for _ in range(c.layers)]
        # pages in no particular order, as a server's free list hands them out
        self.pages = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(texts, self.width).cuda()
        self.lens = [0] * texts

    def _rows(self, call, x, *rest):
        """mt_add_rmsnorm takes up to eight rows a call."""
        for i in range(0, x.shape[0], 8):
            call(i, min(i + 8, x.shape[0]))

    def _norm(self, x, residual, weight):
        total, normed = torch.empty_like(x), torch.empty_like(x)
        self._rows(lambda i, j: mt.mt_add_rmsnorm(x[i:j], residual[i:j], weight, EPS, total[i:j], normed[i:j]), x)
        return total, normed

    def _space(self, M, K, N):
        return torch.empty(mt.mt_prefill_workspace_bytes(M, K, N, 0), dtype=torch.uint8, device="cuda")

    def _linear(self, x, w, dtype=torch.bfloat16):
        (M, K), N = x.shape, w.shape[0]
        y = torch.empty(M, N, dtype=dtype, device="cuda")
        if M <= 8:
            mt.mt_linear_bias(x, w, None, None, 0, None, y, fmt=BF)
        else:
            mt.mt_prefill_linear_bias(x, w, None, None, 0, None, y, self._space(M, K, N), fmt=BF)
        return y

    def _mlp(self, x, residual, layer):
        (M, d), f = x.shape, layer["gate"].shape[0]
        h, y = torch.empty(M, f, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
        if M <= 8:
            mt.mt_swiglu_gateup(x, layer["gate"], layer["up"], None, None, 0, h, fmt=BF)
            mt.mt_down_residual(h, layer["down"], None, None, 0, residual, y, fmt=BF)
        else:
            mt.mt_prefill_swiglu_gateup(x, layer["gate"], layer["up"], None, None, 0, h, self._space(M, d, f), fmt=BF)
            mt.mt_prefill_down_residual(h, layer["down"], None, None, 0, residual, y, self._space(M, f, d), fmt=BF)
        return y

    def step(self, new: list[list[int]]):
        """Takes each text's new tokens (none for a text that waits); returns
        the fp32 logits after the last token of every text that has new ones,
        in their order, [those texts, vocab]."""
        c, m = self.m.cfg, self.m
        if len(new) != self.texts or not any(new):
            raise ValueError(f"new tokens of {self.texts} texts, at least one of them with some, are required")
        for b, n in enumerate(new):
            if self.lens[b] + len(n) > self.width * c.page:
                raise ValueError(f"text {b}: the cache has room for {self.width * c.page} tokens")
        D, H, KV = c.head_dim, c.q_heads, c.kv_heads
        starts = [0]
        for n in new:
            starts.append(starts[-1] + len(n))
        T = starts[-1]
        place = [self.lens[b] + i for b, n in enumerate(new) for i in range(len(n))]
        self.lens = [a + len(n) for a, n in zip(self.lens, new)]
        ids = torch.tensor([t for n in new for t in n]).cuda()
        i32 = dict(dtype=torch.int32, device="cuda")
        q_start, kv_len, positions = torch.tensor(starts, **i32), torch.tensor(self.lens, **i32), torch.tensor(place, **i32)
        longest = max(len(n) for n in new)
        space = torch.empty(mt.mt_paged_attention_workspace_bytes(T, self.texts, H, KV, D), dtype=torch.uint8, device="cuda")

        x = m.embed[ids]
        zero = torch.zeros_like(x)
        for layer, (kc, vc) in zip(m.layers, self.cache):
            residual, n = self._norm(x, zero, layer["n1"])
            q, k, v = self._linear(n, layer["qkv"]).split([H * D, KV * D, KV * D], 1)
            q, k, v = q.unflatten(1, (H, D)), k.unflatten(1, (KV, D)), v.unflatten(1, (KV, D))
            # in place for q; k and v go to their pages
            mt.mt_rope_append(q, k, v, positions, m.inv_freq, q, kc, vc, self.pages, q_start, kv_len, q_norm=layer["qn"],
                              k_norm=layer["kn"], eps=EPS)
            a = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
            mt.mt_paged_attention(q, kc, vc, self.pages, q_start, kv_len, longest, 1 / math.sqrt(D), a, space, window=c.window,
                                  sinks=c.sinks)
            residual, n = self._norm(self._linear(a.view(T, H * D), layer["o"]), residual, layer["n2"])
            x = self._mlp(n, residual, layer)
        last = last_rows(new)
        _, n = self._norm(x[last], zero[last], m.norm)
        return self._linear(n, m.head, torch.float32)


def reference(model: Model, text: list[int]) -> torch.Tensor:
    """The last token's logits of one text in plain fp32 operations."""
    c = model.cfg
    D, H, KV = c.head_dim, c.q_heads, c.kv_heads
    n, dev = len(text), model.embed.device
    place = torch.arange(n, device=dev)
    angle = place[:, None].double() * model.inv_freq.double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def norm(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    def turn(x):
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    seen = place[None] <= place[:, None]
    if c.window:
        seen &= (place[None] > place[:, None] - c.window) | (place[None] < c.sinks)
    x = model.embed[torch.tensor(text, device=dev)].float()
    for layer in model.layers:
        w = {k: v.float() for k, v in layer.items()}
        q, k, v = (norm(x, layer["n1"]) @ w["qkv"].t()).split([H * D, KV * D, KV * D], 1)
        q, k = turn(norm(q.unflatten(1, (H, D)), layer["qn"])), turn(norm(k.unflatten(1, (KV, D)), layer["kn"]))
        k, v = k.repeat_interleave(H // KV, 1), v.unflatten(1, (KV, D)).repeat_interleave(H // KV, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(D)
        p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        x = x + torch.einsum("hij,jhd->ihd", p, v).flatten(1) @ w["o"].t()
        h = norm(x, layer["n2"])
        x = x + (torch.nn.functional.silu(h @ w["gate"].t()) * (h @ w["up"].t())) @ w["down"].t()
    return norm(x[-1:], model.norm) @ model.head.float().t()


def generate(model: Model, prompts: list[list[int]], tokens: int, repetition: float = 1.3, banned: int | None = None):
    """Greedy continuation of the prompts under a repetition penalty, without
    the token `banned`; returns the texts and each step's raw logits."""
    c, B = model.cfg, len(prompts)
    if not all(prompts):
        raise ValueError("a prompt needs at least one token")
    run = Runner(model, max(map(len, prompts)) + tokens, B)
    texts, new, raw = [list(p) for p in prompts], [list(p) for p in prompts], []
    words = torch.full((B, (c.vocab + 31) // 32), -1, dtype=torch.int32)
    if banned is not None:
        bit = 1 << (banned % 32)
        words[:, banned // 32] = ~(bit - (1 << 32) if bit >> 31 else bit)
    words = words.cuda()
    f32 = dict(dtype=torch.float32, device="cuda")
    for _ in range(tokens):
        logits = run.step(new)
        raw.append(logits.clone())
        flat, starts = [t for x in texts for t in x], [0]
        for x in texts:
            starts.append(starts[-1] + len(x))
        i32 = dict(dtype=torch.int32, device="cuda")
        mt.mt_logit_penalties(logits, logits, history=torch.tensor(flat, **i32), history_start=torch.tensor(starts, **i32),
                              prompt_len=torch.tensor([len(p) for p in prompts], **i32), repetition=torch.full((B,), repetition, **f32),
                              presence=torch.full((B,), 0.2, **f32), frequency=torch.full((B,), 0.1, **f32), allowed=words)
        new = [[t] for t in logits.argmax(1).tolist()]
        for x, t in zip(texts, new):
            x.extend(t)
    return texts, raw


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=4)
    a = ap.parse_args()
    model = Model(Config(window=a.window, sinks=a.sinks if a.window else 0))
    g = torch.Generator().manual_seed(2)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist() for n in (5, 37, 130)]
    texts, raw = generate(model, prompts, a.tokens)
    for p, t in zip(prompts, texts):
        print(f"prompt of {len(p)} tokens, then", t[len(p):])
    want = torch.cat([reference(model, t[:-1]) for t in texts])
    off = float((raw[-1] - want).norm() / want.norm())
    print(f"last step's logits against plain fp32 operations: {off:.1e} of their norm")


if __name__ == "__main__":
    main()
