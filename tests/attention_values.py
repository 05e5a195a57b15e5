"""Values and bounds for paged attention that show the loss of any one key.

Each page's values lie in one column of the head (the page's number modulo the
head size), 1 or -1 by key, and scores are small, so that all keys weigh about
the same.  A column then adds up a few hundred terms of both signs: the roundings
of its weights add up to a fraction of one term, and a key, page or block that is
left out, taken twice or taken from elsewhere shows."""
import math

import torch

from paged_util import HALF, Paged


def coded(lens, hq, hkv, d, page, order="nhd", seed=0):
    p = Paged(lens, hq, hkv, d, page, order=order, seed=seed, q_scale=0.1)
    g = torch.Generator().manual_seed(seed + 1)
    for b, (_, kv) in enumerate(lens):
        j = torch.arange(kv)
        vb = torch.zeros(kv, hkv, d)
        vb[j, :, (j // page) % d] = torch.randint(0, 2, (kv, hkv), generator=g).float() * 2 - 1
        p.values[b] = vb.to(torch.bfloat16)
        for i in range(-(-kv // page)):
            n = min(page, kv - i * page)
            p.v[p.pages[b, i], :n] = p.values[b][i * page:i * page + n]
    return p


def reference(p, scale, window, sinks, rounding, dtype):
    """(out, tolerance, margin) in 64 bits: margin is the least, over the visible
    keys of all rows, of how far leaving the key out moves its column, in units
    of that column's tolerance.

    The weights' roundings are independent: six times the root of their sum of
    squares, at the most that each can be.  fp32: a product of 16 keys is one
    addition to the sum, taken as two roundings of it (tensor cores may cut
    rather than round), beside a score's error."""
    rows = int(p.q_start[-1])
    out = torch.zeros(rows, p.hq, p.d, dtype=torch.float64)
    tol = torch.zeros_like(out)
    margin = math.inf
    g, step = p.hq // p.hkv, 2.0 ** -23
    for b, (n, kv) in enumerate(p.lens):
        r0 = int(p.q_start[b])
        j = torch.arange(kv)
        pos = torch.arange(n)[:, None] + kv - n
        seen = j <= pos
        if window:
            seen &= (j > pos - window) | (j < sinks)
        for h in range(p.hq):
            q, k, v = p.q[r0:r0 + n, h].double(), p.keys[b][:, h // g].double(), p.values[b][:, h // g].double()
            score = (q.abs() @ k.abs().t() * scale).max(1).values
            w = torch.softmax((q @ k.t() * scale).masked_fill(~seen, -math.inf), 1)
            o, spread = w @ v, w @ v.abs()
            rel = 2 * (p.d + 32) * step * (score + 1.0) + (kv / 8 + 64) * step
            t = HALF[dtype] * o.abs() + 6 * rounding * (w.square() @ v.square()).sqrt() + rel[:, None] * spread + 1e-30
            out[r0:r0 + n, h], tol[r0:r0 + n, h] = o, t
            column = (j // p.page) % p.d
            margin = min(margin, float((w / t[:, column])[seen].min()))
    return out, tol, margin


# (sequences, heads, page, window, sinks): a text and a chunk split over the
# whole GPU, single tokens of many lengths, a mixed batch, a window
CASES = {"one text of 20011": ([(1, 20011)], (4, 1, 128), 16, 0, 0),
         "two texts, head size 64": ([(1, 9973), (2, 5001)], (14, 2, 64), 16, 0, 0),
         "chunk of 40 after 8960": ([(40, 9000)], (4, 1, 128), 64, 0, 0),
         "ragged texts": ([(1, 1 + 397 * b) for b in range(12)], (8, 2, 128), 16, 0, 0),
         "mixed": ([(90, 700), (1, 3000), (1, 65), (33, 33), (1, 1100)], (6, 2, 64), 16, 0, 0),
         "window and sinks": ([(1, 9000), (70, 5000), (1, 300)], (8, 2, 64), 16, 700, 20),
         "pages of 12": ([(1, 7000), (20, 1500)], (4, 2, 64), 12, 0, 0),
         "head size 256": ([(1, 7000), (20, 1500)], (4, 2, 256), 16, 0, 0)}
