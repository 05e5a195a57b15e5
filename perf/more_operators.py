"""The operators of a step that checks drafted tokens, as cases to measure.

A small model drafts a tree of tokens for every text; the large one takes all
of them in one pass.  Five calls around that pass: the tree's positions and
visibility bits from its parents ("layout"); attention of the tree's tokens over
the paged cache and over their own ancestors ("attention"); probabilities of
logits under a temperature ("probs"); the walk that accepts drafted tokens
against the target's probabilities from given random numbers and draws the token
after them ("verify"); the accepted tokens' keys and values moved together in
every layer's cache ("keep").  ``run`` computes them in elementary torch
operations, or, where ``own`` is true, through the library's calls.
"""
import math
import random

import torch

own = False

# Head layouts (query heads, key/value heads, head size): the library's
# attention-projection workloads, and generic ones.
HEADS = {"32x8x128": (32, 8, 128), "32x8x64": (32, 8, 64), "14x2x64": (14, 2, 64), "16x16x128": (16, 16, 128),
         "40x8x128": (40, 8, 128), "24x8x96": (24, 8, 96), "64x4x128": (64, 4, 128)}


def listed():
    return [
        # one user's drafted tree, laid out on the device: the smallest call
        layout("layout, one tree of 60", B=1, n=60, shape="mixed"),
        # a large serving batch with large trees
        layout("layout, 128 trees of up to 500", B=128, n=500, shape="mixed"),
        # one user's step on a short text: latency
        attention("tree of 25, one short text", B=1, n=25, kv=1203, heads="32x8x128", page=16, shape="mixed"),
        # a serving batch's step on texts of many lengths, a tree each
        attention("trees of up to 64, 24 texts", B=24, n=64, kv=9100, heads="32x8x128", page=16, shape="mixed"),
        # few users with very long texts: the keys' axis is all there is to split
        attention("trees of 16, 3 texts of 80 000", B=3, n=16, kv=80011, heads="14x2x64", page=64, shape="wide"),
        # long texts kept by a window and first tokens; the pages between are given back
        attention("trees, window and sinks", B=32, n=32, kv=30000, heads="32x8x64", page=32, shape="mixed", window=4096, sinks=4),
        # one user's tree after the penalties: fp32 logits
        probs("probs, 9 rows", R=9, V=151936, dtype="float32"),
        # a serving batch's trees
        probs("probs, 448 rows", R=448, V=128256, dtype="bfloat16"),
        # one user's tree of the draft's most probable tokens
        verify("verify, one tree of 25", B=1, n=25, V=151936, shape="mixed", draft=False),
        # a serving batch: chains drawn from the draft's probabilities
        verify("verify, 64 chains of 6", B=64, n=7, V=128256, shape="chain", draft=True),
        # one user's accepted tokens, all layers
        keep("keep, one text", B=1, n=25, cols=6, L=36, kv=700, heads="32x8x128", page=16),
        # a serving batch's, all layers
        keep("keep, 64 texts", B=64, n=64, cols=8, L=36, kv=330, heads="32x8x128", page=16),
    ]


def layout(name, B, n, shape):
    return {"name": name, "op": "layout", "B": B, "n": n, "shape": shape, "kv": 3000 + n}


def attention(name, B, n, kv, heads, page, shape, window=0, sinks=0):
    return {"name": name, "op": "attention", "B": B, "n": n, "kv": kv, "heads": heads, "page": page, "shape": shape, "window": window,
            "sinks": sinks}


def probs(name, R, V, dtype):
    return {"name": name, "op": "probs", "R": R, "V": V, "dtype": dtype}


def verify(name, B, n, V, shape, draft):
    return {"name": name, "op": "verify", "B": B, "n": n, "V": V, "shape": shape, "draft": draft, "kv": n + 1, "cols": 9}


def keep(name, B, n, cols, L, kv, heads, page):
    return {"name": name, "op": "keep", "B": B, "n": n, "cols": cols, "L": L, "kv": kv, "heads": heads, "page": page}


def draw(rng):
    def spread(lo, hi):  # over the logarithm, odd sizes as likely as even ones
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["layout", "attention", "attention", "attention", "probs", "verify", "verify", "keep"])
    heads, page = rng.choice(sorted(HEADS)), rng.choice([16, 32, 48, 64, 128])
    shape = rng.choice(["mixed", "mixed", "wide", "chain", "forest"])
    if kind == "layout":
        n = spread(1, 1000)
        c = layout("", spread(1, max(1, min(256, 30000000 // (n * n)))), n, shape)
    elif kind == "attention":
        n = spread(1, 300)
        kv = n + spread(1, 40000)
        window, sinks = (spread(300, 4096), rng.choice([0, 1, 4, 17, 64])) if rng.random() < 0.4 else (0, 0)
        most = min(64, 600000 // (n * 16 + kv), 1000000000 // (n * kv * HEADS[heads][0]))
        c = attention("", spread(1, max(1, most)), n, kv, heads, page, shape, window, sinks)
    elif kind == "probs":
        c = probs("", spread(1, 448), spread(1000, 160000), rng.choice(["float32", "bfloat16"]))
    elif kind == "verify":
        n, draft = spread(1, 60), rng.random() < 0.5
        V = spread(1000, 160000)
        c = verify("", spread(1, max(1, min(100, 57000000 // (n * V)))), n, V, "mixed" if shape == "forest" else shape, draft)
    else:
        n, L = spread(1, 200), rng.choice([1, 7, 16, 28, 36, 48])
        kv = n + spread(1, 400)
        c = keep("", spread(1, max(1, min(64, 500000 // (kv * L)))), n, min(n, spread(1, 24)), L, kv, heads, page)
    del c["name"]
    return c


def lengths(case):
    """(new tokens, tokens in the cache with them) of each text: the first as long as the case says, the others spread."""
    got = []
    for b in range(case["B"]):
        a, c = (b * 0.6180339887 % 1.0, b * 0.7548776662 % 1.0)
        n = case["n"] - int(a * 0.6 * case["n"]) if case.get("shape") != "chain" else case["n"]
        kv = case["kv"] - int(c * 0.8 * case["kv"])
        got.append((n, max(n, kv)))
    return got


def parents(case, n, b):
    """The tree of text b: each token's parent, -1 for none."""
    shape = case["shape"]
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "wide":  # three children each
        return [(i - 1) // 3 if i else -1 for i in range(n)]
    first = min(n, 4) if shape == "forest" else 1  # several first tokens hang on the text itself
    # the earlier tokens, which a draft holds for likelier, have more children
    return [-1 if i < first else int(((i + 7 * b) * 0.6180339887 % 1.0) ** 1.5 * i) for i in range(n)]


def trees(case):
    return [parents(case, n, b) for b, (n, _) in enumerate(lengths(case))]


def depths(tree):
    got = []
    for p in tree:
        got.append(0 if p < 0 else got[p] + 1)
    return got


def prepare(case, seed):
    """The inputs of one case, made from the seed."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return {"layout": prepare_layout, "attention": prepare_attention, "probs": prepare_probs, "verify": prepare_verify,
            "keep": prepare_keep}[case["op"]](case, g, random.Random(int(seed)))


def normal(g, *shape, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, scale, generator=g)


def whole(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def starts_of(lens):
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    return starts


def prepare_layout(case, g, rng):
    # the texts' lengths and the order of equally deep tokens come from the seed
    lens = lengths(case)
    flat = []
    for tree in trees(case):
        n = len(tree)
        at = rng.randrange(n)  # one token hangs elsewhere
        if tree[at] > 0:
            tree[at] = rng.randrange(at)
        flat += tree
    starts = starts_of(lens)
    T, most = starts[-1], max(n for n, _ in lens)
    return {"case": case, "B": case["B"], "T": T, "most": most, "parent": whole(flat), "q_start": whole(starts),
            "kv_len": whole([kv + rng.randrange(500) for _, kv in lens]),
            "positions": torch.empty(T, dtype=torch.int32, device="cuda"),
            "visible": torch.empty(T, (most + 31) // 32, dtype=torch.int32, device="cuda")}


def paged(case, lens, g):
    """The page table of the texts: pages in no order, as a server's free list hands them out; unused entries are -1."""
    page = case["page"]
    need = [-(-kv // page) for _, kv in lens]
    most, count = max(need), sum(need) + 3
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["B"], most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        if case.get("window"):
            # pages that no token sees any more are given back
            first, last = -(-case["sinks"] // page), (lens[b][1] - lens[b][0] - case["window"] + 1) // page
            if last > first:
                table[b, first:last] = -1
    return table, most, count


def prepare_attention(case, g, rng):
    hq, hkv, d = HEADS[case["heads"]]
    lens, page, B = lengths(case), case["page"], case["B"]
    starts = starts_of(lens)
    T, most_n = starts[-1], max(n for n, _ in lens)
    words = (most_n + 31) // 32
    rows = []
    for tree in trees(case):
        seen = []
        for i, p in enumerate(tree):
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        for m in seen:
            every = [(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)]
            rows.append([x - (1 << 32) if x >> 31 else x for x in every])
    table, most, count = paged(case, lens, g)
    s = {"case": case, "T": T, "B": B, "hq": hq, "hkv": hkv, "d": d, "page": page, "pages": table, "most": most * page, "max_q": most_n,
         "q_start": whole(starts), "kv_len": whole([kv for _, kv in lens]), "visible": whole(rows), "words": words,
         "k_cache": normal(g, count, page, hkv, d), "v_cache": normal(g, count, page, hkv, d)}
    # scores of a standard deviation of about 2, and values with a mean, as trained heads have them
    s["q"] = normal(g, T, hq, d, scale=2.0)
    s["v_cache"] += 0.25
    s["scale"] = 1.0 / math.sqrt(d)
    return s


def prepare_probs(case, g, rng):
    R, V = case["R"], case["V"]
    x = torch.randn(R, V, generator=g, device="cuda") * 3.0
    # a grammar's mask leaves a third of the tokens of every third row
    few = (torch.arange(R, device="cuda")[:, None] % 3 == 2) & (torch.rand(R, V, generator=g, device="cuda") > 0.33)
    x = x.masked_fill_(few, -math.inf).to(getattr(torch, case["dtype"]))
    t = 0.4 + torch.rand(R, generator=g, device="cuda")
    t[torch.arange(R, device="cuda") % 8 == 5] = 0.0  # texts that take the most probable token
    return {"case": case, "logits": x, "temperature": t}


def prepare_verify(case, g, rng):
    B, V, n = case["B"], case["V"], case["n"]
    lens = lengths(case)
    starts = starts_of(lens)
    T, made = starts[-1], trees(case)
    x = torch.randn(T, V, generator=g, device="cuda") * 5.0
    s = {"case": case, "B": B, "T": T, "V": V, "target": torch.softmax(x, 1), "q_start": whole(starts),
         "parent": whole([p for tree in made for p in tree]), "random": torch.rand(T, generator=g, device="cuda")}
    # the draft is a coarser model of the same text
    q = torch.softmax(x + torch.randn(T, V, generator=g, device="cuda") * 1.5, 1)
    count = [[tree[:i].count(p) for i, p in enumerate(tree)] for tree in made]  # earlier siblings
    width = 1 + max(max(c) for c in count)
    row = whole([a + max(p, 0) for a, tree in zip(starts, made) for p in tree], torch.int64)
    nth = whole([k for c in count for k in c], torch.int64)
    if case["draft"]:
        picked = torch.multinomial(q, width, replacement=True, generator=g)
        s["draft"] = q
    else:
        picked = torch.topk(q, width, 1).indices
        s["draft"] = None
    s["tokens"] = picked[row, nth].to(torch.int32)
    cols = case["cols"]
    s["out"] = {"tokens": torch.empty(B, cols, dtype=torch.int32, device="cuda"), "path": torch.empty(B, cols, dtype=torch.int32, device="cuda"),
                "count": torch.empty(B, dtype=torch.int32, device="cuda")}
    return s


def kept(case):
    """How many tokens each text keeps."""
    return [1 + int((b + 1) * 0.5698402910 % 1.0 * min(case["cols"], n)) for b, (n, _) in enumerate(lengths(case))]


def prepare_keep(case, g, rng):
    hq, hkv, d = HEADS[case["heads"]]
    lens, B, cols = lengths(case), case["B"], case["cols"]
    table, most, count = paged(case, lens, g)
    # every layer's keys and values, [layers, 2, pages, page, heads, dim]
    cache = normal(g, case["L"], 2, count, case["page"], hkv, d)
    path = [[0] + sorted(rng.sample(range(1, n), m - 1)) + [-1] * (cols - m) for (n, _), m in zip(lens, kept(case))]
    return {"case": case, "B": B, "cache": cache, "layers": [(x[0], x[1]) for x in cache], "pages": table, "page": case["page"],
            "q_start": whole(starts_of(lens)), "kv_len": whole([kv for _, kv in lens]), "path": whole(path),
            "count": whole(kept(case)), "new_len": torch.empty(B, dtype=torch.int32, device="cuda")}


def run(state):
    return {"layout": run_layout, "attention": run_attention, "probs": run_probs, "verify": run_verify,
            "keep": run_keep}[state["case"]["op"]](state)


def ancestors(parent, n, N):
    """[B, N, N]: token j is token i or one of its ancestors; `parent` [B, N] holds -1 where there is none."""
    i = torch.arange(N, device=parent.device)
    seen = (i[:, None] == i) & (i < n[:, None])[:, :, None]
    up = parent
    for _ in range(max(1, (N - 1).bit_length())):  # twice as far up each time
        there = up >= 0
        at = up.clamp(min=0)
        seen = seen | (there[:, :, None] & seen.gather(1, at[:, :, None].expand(-1, -1, N)))
        up = torch.where(there, up.gather(1, at), up)
    return seen


def by_text(s, N):
    """Each text's rows as [B, N], their number, and the parents there."""
    start = s["q_start"].long()
    n, i = start[1:] - start[:-1], torch.arange(N, device=start.device)
    row = (start[:-1, None] + i).clamp(max=s["T"] - 1)
    parent = s["parent"].long()[row]
    parent = torch.where((parent >= 0) & (parent < i) & (i < n[:, None]), parent, -1)
    return row, n, i, parent


def run_layout(s):
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        mt.mt_tree_layout(s["parent"], s["q_start"], s["kv_len"], s["positions"], s["visible"])
        return {"positions": s["positions"], "visible": s["visible"]}
    N = s["most"]
    row, n, i, parent = by_text(s, N)
    seen = ancestors(parent, n, N)
    place = (s["kv_len"].long() - n)[:, None] + seen.sum(2) - 1
    words = (N + 31) // 32
    bits = torch.nn.functional.pad(seen, (0, 32 * words - N)).view(*seen.shape[:2], words, 32)
    bits = (bits.long() << torch.arange(32, device=row.device)).sum(3)
    bits = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32)
    there = i < n[:, None]
    return {"positions": place[there].to(torch.int32), "visible": bits[there]}


def run_attention(s):
    c = s["case"]
    q = s["q"]
    T, B, hq, hkv, d = s["T"], s["B"], s["hq"], s["hkv"], s["d"]
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        if "out" not in s:
            s["out"] = torch.empty_like(q)
            s["lse"] = torch.empty(T, hq, dtype=torch.float32, device=q.device)
            s["workspace"] = torch.empty(mt.mt_paged_attention_workspace_bytes(T, B, hq, hkv, d), dtype=torch.uint8, device=q.device)
        mt.mt_tree_attention(q, s["k_cache"], s["v_cache"], s["pages"], s["q_start"], s["kv_len"], s["visible"], s["max_q"], s["scale"],
                             s["out"], s["workspace"], lse=s["lse"], window=c["window"], sinks=c["sinks"])
        return {"out": s["out"], "lse": s["lse"]}
    group, Q, K = hq // hkv, s["max_q"], s["most"]
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    key = torch.arange(K, device=q.device)
    there = key < kv_len[:, None]                                                     # [B, K]
    page = s["pages"].long()[:, key // s["page"]].clamp(min=0)
    slot = page * s["page"] + key % s["page"]

    def gathered(cache):
        x = cache.view(-1, hkv, d)[slot].float()
        return torch.where(there[:, :, None, None], x, 0.0).permute(0, 2, 1, 3)         # [B, hkv, K, d]

    i = torch.arange(Q, device=q.device)
    row = (start[:-1, None] + i).clamp(max=T - 1)
    x = q[row].float().view(B, Q, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, group * Q, d)
    score = torch.matmul(x, gathered(s["k_cache"]).transpose(2, 3)).view(B, hkv, group, Q, K)
    n = start[1:] - start[:-1]
    base = kv_len - n
    bits = (s["visible"][row][..., None] >> torch.arange(32, device=q.device, dtype=torch.int32)) & 1
    bits = bits.reshape(B, Q, -1) != 0                                                # [B, Q, 32 words]
    j = key - base[:, None]                                                           # [B, K] which new token a key is
    fresh = bits.gather(2, j.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, Q, -1))
    old = (j < 0)[:, None].expand(-1, Q, -1)
    if c["window"]:
        place = base[:, None] + (bits & (torch.arange(bits.shape[2], device=q.device) < n[:, None])[:, None]).sum(2).clamp(min=1) - 1
        old = old & ((key > place[:, :, None] - c["window"]) | (key < c["sinks"]))
    seen = there[:, None, :] & torch.where((j < 0)[:, None], old, fresh)
    score = score.mul_(s["scale"]).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, hkv, group * Q, K), gathered(s["v_cache"])).view(B, hkv, group, Q, d)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, Q, hq, d)
    lse = (total.log() + top).permute(0, 3, 1, 2, 4).reshape(B, Q, hq)
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(start[1:], t, right=True)
    return {"out": out[b, t - start[b]].to(torch.bfloat16), "lse": lse[b, t - start[b]].contiguous()}


def run_probs(s):
    x, t = s["logits"], s["temperature"]
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        if "probs" not in s:
            s["probs"] = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        mt.mt_token_probs(x, s["probs"], temperature=t)
        return s["probs"]
    x = x.float()
    top = x.amax(1, keepdim=True)
    v = torch.arange(x.shape[1], device=x.device)
    first = torch.where(x == top, v, x.shape[1]).amin(1, keepdim=True)
    warm = t[:, None] > 0
    e = ((x - top) / torch.where(warm, t[:, None], 1.0)).exp()
    return torch.where(warm, e / e.sum(1, keepdim=True), (v == first).float())


def run_verify(s):
    c, out = s["case"], s["out"]
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        mt.mt_tree_verify(s["target"], s["tokens"], s["parent"], s["random"], s["q_start"], out["tokens"], out["path"], out["count"],
                          draft=s["draft"])
        return out
    B, V, N, cols = s["B"], s["V"], c["n"], c["cols"]
    p, q = s["target"], s["draft"]
    row, n, i, parent = by_text(s, N)
    has = parent >= 0
    up = row.gather(1, parent.clamp(min=0))
    token, u = s["tokens"].long()[row], s["random"].double()[row]
    before = has[:, :, None] & (parent[:, :, None] == parent[:, None, :]) & (i < i[:, None])  # [B, N, N]: j is an earlier sibling of i
    rank, children = before.sum(2), (parent[:, :, None] == i).sum(1)
    p_at = torch.where(has, p[up, token].double(), 0.0)
    if q is None:
        p_at = torch.where((before & (token[:, :, None] == token[:, None, :])).any(2), 0.0, p_at)
        rest = (1.0 - (before * p_at[:, None, :]).sum(2)).clamp(min=0.0)
        taken = has & (u * rest < p_at)
    else:
        width = int(c_width(c))
        # of every row, by the number of its refused children: S, and the sum of max(p - S q, 0)
        cut, mass = torch.zeros(s["T"], width + 1, dtype=torch.float64, device=p.device), torch.ones(s["T"], width + 1, dtype=torch.float64, device=p.device)
        for k in range(1, width + 1):
            cut[:, k] = cut[:, k - 1] + mass[:, k - 1]
            if k < width:
                mass[:, k] = (p.double() - cut[:, k, None] * q.double()).clamp(min=0.0).sum(1)
        q_at = q[up, token].double()
        left = (p_at - cut[up, rank] * q_at).clamp(min=0.0)
        taken = has & (u * q_at * mass[up, rank] < left)
    first = taken & ~(before & taken[:, None, :]).any(2)
    seen = ancestors(parent, n, N)
    depth = seen.sum(2) - 1
    good = first | (i == 0)
    on = seen[:, :, 0] & (seen <= good[:, None, :]).all(2) & (depth < cols) & (i < n[:, None])
    count = on.sum(1)
    end = torch.where(on, i, 0).amax(1)
    refused = torch.where(count < cols, children.gather(1, end[:, None])[:, 0], 0)
    at = row.gather(1, end[:, None])[:, 0]
    left = p[at].double()
    if q is None:
        gone = has & (parent == end[:, None]) & (count < cols)[:, None]
        mask = torch.zeros(B, V, device=p.device).scatter_add_(1, token, gone.float())
        left = torch.where(mask > 0, 0.0, left)
    else:
        left = (left - cut[at, refused][:, None] * q[at].double()).clamp(min=0.0)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, p[at].double())
    total = left.cumsum(1)
    drawn = (total <= s["random"].double()[s["q_start"].long()[:-1]][:, None] * total[:, -1:]).sum(1)
    # where the threshold is the sum itself, rounded, the last token that has a share
    drawn = torch.minimum(drawn, torch.where(left > 0, torch.arange(V, device=p.device), -1).amax(1))
    slot = torch.arange(cols, device=p.device)
    path = torch.full((B, cols + 1), -1, device=p.device).scatter_(1, torch.where(on, depth, cols), torch.where(on, i, -1))[:, :cols]
    next_node = torch.nn.functional.pad(path, (0, 1), value=-1)[:, 1:]
    tokens = torch.where(next_node >= 0, token.gather(1, next_node.clamp(min=0)), -1)
    tokens = torch.where(slot == count[:, None] - 1, drawn[:, None], tokens)
    return {"tokens": tokens.to(torch.int32), "path": path.to(torch.int32), "count": count.to(torch.int32)}


def c_width(case):
    """The most children of a token."""
    return max(max(tree.count(p) if p >= 0 else 1 for p in set(tree)) for tree in trees(case))


def run_keep(s):
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        mt.mt_cache_keep(s["layers"], s["pages"], s["q_start"], s["kv_len"], s["path"], s["count"], new_len=s["new_len"])
        return {"cache": s["cache"].view(torch.int16), "new_len": s["new_len"]}
    start, cache, page = s["q_start"].long(), s["cache"], s["page"]
    base = s["kv_len"].long() - (start[1:] - start[:-1])
    count, path = s["count"].long(), s["path"].long()
    b, i = (torch.arange(path.shape[1], device=path.device) < count[:, None]).nonzero(as_tuple=True)
    to, come = base[b] + i, base[b] + path[b, i]
    table = s["pages"].long()
    cache[:, :, table[b, to // page], to % page] = cache[:, :, table[b, come // page], come % page]
    return {"cache": cache.view(torch.int16), "new_len": (base + count).to(torch.int32)}


def work(case):
    op = case["op"]
    if op == "probs":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["R"] * case["V"] * (size + 4), "flops": 4 * case["R"] * case["V"]}
    lens = lengths(case)
    T = sum(n for n, _ in lens)
    if op == "layout":
        return {"bytes": 8 * T + 4 * T * ((max(n for n, _ in lens) + 31) // 32), "flops": 0}
    if op == "verify":
        # a text draws from one row; where tokens were drafted at random and one was refused, the draft's row is read too
        rows = case["B"] * (1.8 if case["draft"] else 1.0)
        return {"bytes": rows * case["V"] * 4 + 16 * T, "flops": 2 * rows * case["V"]}
    hq, hkv, d = HEADS[case["heads"]]
    if op == "keep":
        moved = sum(m - 1 for m in kept(case))
        return {"bytes": 2 * 2 * 2 * case["L"] * moved * hkv * d + 16 * case["B"], "flops": 0}
    keys = pairs = 0
    for (n, kv), tree in zip(lens, trees(case)):
        base, w = kv - n, case["window"]
        first = max(0, base - w + 1) if w else 0  # the first key in the first token's window
        keys += kv - first + min(case["sinks"], first)
        for depth in depths(tree):
            lo = max(0, base + depth - w + 1) if w else 0
            pairs += base - min(base, lo) + min(case["sinks"], lo, base) + depth + 1
    words = (max(n for n, _ in lens) + 31) // 32
    return {"bytes": 2 * 2 * keys * hkv * d + 2 * 2 * T * hq * d + 4 * T * hq + 4 * T * words + 4 * sum(-(-kv // case["page"]) for _, kv in lens),
            "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """run()'s outputs in 64 bits, text by text."""
    s = prepare(case, seed)
    return {"layout": exact_layout, "attention": exact_attention, "probs": exact_probs, "verify": exact_verify,
            "keep": exact_keep}[case["op"]](s)


def up_from(tree, i):
    """Token i and its ancestors."""
    got = [i]
    while 0 <= tree[got[-1]] < got[-1]:
        got.append(tree[got[-1]])
    return got


def exact_layout(s):
    start, flat, kv = s["q_start"].tolist(), s["parent"].tolist(), s["kv_len"].tolist()
    place, bits = [], []
    words = s["visible"].shape[1]
    for b in range(s["B"]):
        tree = flat[start[b]:start[b + 1]]
        for i in range(len(tree)):
            line = up_from(tree, i)
            place.append(kv[b] - len(tree) + len(line) - 1)
            row = [0] * words
            for j in line:
                row[j // 32] |= 1 << (j % 32)
            bits.append([x - (1 << 32) if x >= 1 << 31 else x for x in row])
    return {"positions": whole(place), "visible": whole(bits)}


def exact_attention(s):
    case, hq, hkv, d, page = s["case"], s["hq"], s["hkv"], s["d"], s["page"]
    dev, group, w = s["q"].device, hq // hkv, case["window"]
    out = torch.zeros(s["T"], hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], hq), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, ((n, kv), tree) in enumerate(zip(lengths(case), trees(case))):
        hidden = torch.ones(n, kv, dtype=torch.bool)
        for i in range(n):
            line = up_from(tree, i)
            p = kv - n + len(line) - 1
            hidden[i, max(0, p - w + 1) if w else 0:kv - n] = False
            hidden[i, :min(case["sinks"], kv - n)] = False
            hidden[i, [kv - n + j for j in line]] = False
        hidden = hidden.to(dev)
        used = s["pages"][b, :-(-kv // page)].long().clamp(min=0)
        keys, values = (x[used].reshape(-1, hkv, d)[:kv] for x in (s["k_cache"], s["v_cache"]))
        for h in range(hq):
            k, v = keys[:, h // group].double(), values[:, h // group].double()
            x = (s["q"][at:at + n, h].double() @ k.t() * s["scale"]).masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[at:at + n, h] = z
            out[at:at + n, h] = torch.exp(x - z[:, None]) @ v
        at += n
    return {"out": out, "lse": lse}


def exact_probs(s):
    got = torch.zeros(s["logits"].shape, dtype=torch.float64, device=s["logits"].device)
    for r, t in enumerate(s["temperature"].tolist()):
        x = s["logits"][r].double()
        if t > 0:
            got[r] = torch.exp(x / t - torch.logsumexp(x / t, 0))
        else:
            got[r, int((x == x.max()).nonzero()[0])] = 1.0
    return got


def exact_verify(s):
    case, V, cols = s["case"], s["V"], s["case"]["cols"]
    start, flat, token, u = s["q_start"].tolist(), s["parent"].tolist(), s["tokens"].tolist(), s["random"].double().tolist()
    tokens, paths, counts = [], [], []
    for b in range(s["B"]):
        a, n = start[b], start[b + 1] - start[b]
        tree, node, path, said = flat[a:a + n], 0, [0], []
        while True:
            p = s["target"][a + node].double()
            q = s["draft"][a + node].double() if s["draft"] is not None else None
            left, mass, cut, found = p.clone(), 1.0, 0.0, None
            for child in range(node + 1, n) if len(path) < cols else ():
                if tree[child] != node:
                    continue
                x = token[a + child]
                if u[a + child] * mass * (1.0 if q is None else float(q[x])) < float(left[x]):
                    found = child
                    break
                if q is None:
                    mass = max(0.0, mass - float(left[x]))
                    left[x] = 0.0
                else:
                    cut += mass
                    left = torch.relu(p - cut * q)
                    mass = float(left.sum())
            if found is None:
                break
            node = found
            path.append(node)
            said.append(token[a + node])
        if float(left.sum()) <= 0:
            left = p
        total = torch.cumsum(left, 0)
        over = (total > u[a] * total[-1]).nonzero()
        said.append(int(over[0]) if over.numel() else int((left > 0).nonzero()[-1]))
        tokens.append(said + [-1] * (cols - len(said)))
        paths.append(path + [-1] * (cols - len(path)))
        counts.append(len(path))
    return {"tokens": whole(tokens), "path": whole(paths), "count": whole(counts)}


def exact_keep(s):
    cache, page, table = s["cache"].clone(), s["page"], s["pages"].tolist()
    start, kv, path, count = s["q_start"].tolist(), s["kv_len"].tolist(), s["path"].tolist(), s["count"].tolist()
    news = []
    for b in range(s["B"]):
        base = kv[b] - (start[b + 1] - start[b])
        for i in range(count[b]):
            a, z = base + path[b][i], base + i
            cache[:, :, table[b][z // page], z % page] = s["cache"][:, :, table[b][a // page], a % page]
        news.append(base + count[b])
    return {"cache": cache.view(torch.int16), "new_len": whole(news)}
