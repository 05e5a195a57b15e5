"""Trees, 64-bit and exact references for the tests of the calls for drafted
tokens."""
import math
from fractions import Fraction

import torch

from paged_util import Paged


def mixed_tree(n, seed=0, roots=1):
    """Parents of n tokens: early tokens have more children; -1 for the first `roots`."""
    g = torch.Generator().manual_seed(seed)
    u = torch.rand(n, generator=g).tolist()
    return [-1 if i < roots else int(u[i] ** 1.5 * i) for i in range(n)]


def ancestors(parent, i):
    """Token i and its ancestors; a parent that is not an earlier token is none."""
    got = [i]
    while 0 <= parent[got[-1]] < got[-1]:
        got.append(parent[got[-1]])
    return got


def seen_of(parent):
    """[n, n] bool: i sees j."""
    n = len(parent)
    m = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        m[i, ancestors(parent, i)] = True
    return m


def bit_rows(rows, T, words, fill=0):
    """int32 [T, words] of bool rows [n_i, m_i], one matrix after another; `fill` in rows of no sequence."""
    out = torch.full((T, words), fill, dtype=torch.int64)
    at = 0
    for m in rows:
        n = m.shape[0]
        wide = torch.zeros(n, words * 32, dtype=torch.int64)
        k = min(m.shape[1], words * 32)
        wide[:, :k] = m[:, :k].long()
        out[at:at + n] = (wide.view(n, words, 32) << torch.arange(32)).sum(2)
        at += n
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)


def tree_attention_ref(p: Paged, seen, scale, window=0, sinks=0):
    """As paged_util.attention_ref; seen: a bool matrix [n, n] a sequence."""
    n_rows = int(p.q_start[-1])
    out = torch.zeros(n_rows, p.hq, p.d, dtype=torch.float64)
    spread = torch.zeros_like(out)
    lse = torch.full((n_rows, p.hq), -math.inf, dtype=torch.float64)
    score = torch.zeros(n_rows, p.hq, dtype=torch.float64)
    g = p.hq // p.hkv
    for b, (n, kv) in enumerate(p.lens):
        r0 = int(p.q_start[b])
        if n == 0 or kv == 0:
            continue
        base = kv - n
        bits = seen[b][:, :n]
        j = torch.arange(kv)
        pos = base + bits.sum(1).clamp(min=1)[:, None] - 1
        mask = (j < base).expand(n, kv).clone()
        if window:
            mask &= (j > pos - window) | (j < sinks)
        at = (j - base).clamp(0, max(bits.shape[1] - 1, 0))
        mask |= bits[:, at] & ((j >= base) & (j - base < bits.shape[1]))
        for h in range(p.hq):
            q = p.q[r0:r0 + n, h].double()
            k, v = p.keys[b][:, h // g].double(), p.values[b][:, h // g].double()
            s = (q @ k.t() * scale).masked_fill(~mask, -math.inf)
            z = torch.logsumexp(s, 1)
            w = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            out[r0:r0 + n, h], spread[r0:r0 + n, h], lse[r0:r0 + n, h] = w @ v, w @ v.abs(), z
            score[r0:r0 + n, h] = (q.abs() @ k.abs().t() * scale).max(1).values
    return out, lse, spread, score


def probability(x):
    """A row's entry as the call takes it: above 1 as 1, below 0 and NaN as 0."""
    return Fraction(min(x, 1.0)) if x > 0 else Fraction(0)


def verify_ref(target, draft, tokens, parent, random, starts, cols):
    """(tokens, path, count) in rationals: the definition, without rounding."""
    V = target.shape[1]
    out_t, out_p, out_c = [], [], []
    tokens, parent, random = tokens.tolist(), parent.tolist(), [min(max(x, 0.0), 1 - 2.0 ** -24) if x == x else 0.0 for x in random.tolist()]
    for a, z in zip(starts[:-1], starts[1:]):
        n = z - a
        if n == 0:
            out_t.append([-1] * cols)
            out_p.append([-1] * cols)
            out_c.append(0)
            continue
        node, path, said = 0, [0], []
        while True:
            p = [probability(x) for x in target[a + node].tolist()]
            q = [probability(x) for x in draft[a + node].tolist()] if draft is not None else None
            left, mass, cut, found = list(p), Fraction(1), Fraction(0), None
            if len(path) < cols:
                for c in range(node + 1, n):
                    if parent[a + c] != node:
                        continue
                    x, u = tokens[a + c], Fraction(random[a + c])
                    r = left[x] if 0 <= x < V else Fraction(0)
                    qx = (q[x] if 0 <= x < V else Fraction(0)) if q is not None else 1
                    if u * mass * qx < r:
                        found = c
                        break
                    if q is None:
                        mass = max(Fraction(0), mass - r)
                        if 0 <= x < V:
                            left[x] = Fraction(0)
                    else:
                        cut += mass
                        left = [max(Fraction(0), s - cut * t) for s, t in zip(p, q)]
                        mass = sum(left)
            if found is None:
                break
            node = found
            path.append(node)
            said.append(tokens[a + node])
        if sum(left) == 0:
            left = p
        total, run, drawn = sum(left), Fraction(0), -1
        limit = Fraction(random[a]) * total
        for v, s in enumerate(left):
            run += s
            if run > limit:
                drawn = v
                break
        said.append(drawn)
        out_t.append(said + [-1] * (cols - len(said)))
        out_p.append(path + [-1] * (cols - len(path)))
        out_c.append(len(path))
    return out_t, out_p, out_c
