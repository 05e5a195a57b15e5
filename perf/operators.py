"""The operators of a decode or prompt step around the library's projections, as cases to measure.

Three calls: rotary positions with several axes, with the per-head RMSNorm
before them and the write of K and V into the paged cache after them
("rope"); attention of each sequence's new tokens over its paged cache, full
or with a sliding window and first tokens that stay visible ("attention");
penalties, biases and allowed-token masks on the vocabulary's logits
("logits").  ``run`` computes them in elementary torch operations, or, where
``own`` is true, through the library's calls.
"""
import math

import torch

own = False

# Head layouts (query heads, key/value heads, head size): the library's
# attention-projection workloads, and generic ones.
HEADS = {"32x8x128": (32, 8, 128), "32x8x64": (32, 8, 64), "14x2x64": (14, 2, 64), "16x16x128": (16, 16, 128),
         "40x8x128": (40, 8, 128), "24x8x96": (24, 8, 96), "64x4x128": (64, 4, 128)}


def listed():
    return [
        # one user's decode step with a text position: the smallest call
        rope("rope, one token", B=1, q=1, kv=900, heads="32x8x128", axes=1, norm=True),
        # the new tokens of a picture and its question, for a small model without per-head norms
        rope("rope, picture of 1531 tokens", B=1, q=1531, kv=1531, heads="14x2x64", axes=3, norm=False),
        # prompts of a batch, text and pictures
        rope("rope, prompts of 11 000 tokens", B=3, q=5000, kv=9000, heads="32x8x128", axes=3, norm=True),
        # one user's decode step on a short text: latency
        attention("decode, one short text", B=1, q=1, kv=777, heads="32x8x128", page=16),
        # a serving batch's decode step on texts of many lengths
        attention("decode, 48 ragged texts", B=48, q=1, kv=9100, heads="32x8x128", page=16),
        # few users with very long texts: the keys' axis is all there is to split
        attention("decode, 2 texts of 100 000", B=2, q=1, kv=100001, heads="14x2x64", page=64),
        # long texts kept by a window and first tokens; the pages between are given back
        attention("decode, window and sinks", B=32, q=1, kv=30000, heads="32x8x64", page=32, window=4096, sinks=4),
        # one step of a mixed batch: a chunk of one prompt beside other users' single tokens
        attention("mixed, chunk of 384", B=16, q=384, kv=6100, heads="32x8x128", page=16, mixed=True),
        # a whole prompt
        attention("prompt of 8000", B=1, q=8000, kv=8000, heads="32x8x128", page=64),
        # prompts under a window
        attention("prompts, window and sinks", B=4, q=3900, kv=5000, heads="32x8x64", page=16, window=1024, sinks=16),
        # one user's logits, long text, the grammar of a tool call
        logits("logits, one text", B=1, V=151936, hist=6000, dtype="float32", mask=True),
        # a large serving batch
        logits("logits, 200 texts", B=200, V=128256, hist=3000, dtype="bfloat16", mask=True),
    ]


def rope(name, B, q, kv, heads, axes, norm, page=16, adjacent=False, part=1.0):
    return {"name": name, "op": "rope", "B": B, "q": q, "kv": kv, "heads": heads, "axes": axes, "norm": norm, "page": page,
            "adjacent": adjacent, "part": part, "mixed": False}


def attention(name, B, q, kv, heads, page, window=0, sinks=0, mixed=False):
    return {"name": name, "op": "attention", "B": B, "q": q, "kv": kv, "heads": heads, "page": page, "window": window,
            "sinks": sinks, "mixed": mixed}


def logits(name, B, V, hist, dtype, mask):
    return {"name": name, "op": "logits", "B": B, "V": V, "hist": hist, "dtype": dtype, "mask": mask}


def draw(rng):
    def spread(lo, hi):  # over the logarithm, odd sizes as likely as even ones
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["rope", "decode", "decode", "prompt", "prompt", "mixed", "logits"])
    heads = rng.choice(sorted(HEADS))
    page = rng.choice([16, 32, 48, 64, 128])
    if kind == "rope":
        q = spread(1, 5000)
        B = spread(1, max(1, min(64, 10000 // q)))
        c = rope("", B, q, q + spread(1, 4000), heads, rng.choice([1, 2, 3]), rng.random() < 0.5, page, rng.random() < 0.3,
                 rng.choice([1.0, 1.0, 0.5]))
    elif kind == "logits":
        c = logits("", spread(1, 200), spread(30000, 200000), spread(1, 8000), rng.choice(["float32", "bfloat16"]),
                   rng.random() < 0.7)
    else:
        window, sinks = (spread(64, 4096), rng.choice([0, 1, 4, 17, 64])) if rng.random() < 0.5 else (0, 0)
        if kind == "decode":
            kv = spread(1, 60000)
            c = attention("", spread(1, max(1, min(64, 400000 // kv))), rng.choice([1, 1, 1, 2, 5]), kv, heads, page, window, sinks)
        elif kind == "prompt":
            q = spread(20, 4000)
            kv = q + rng.choice([0, spread(1, 2900)])
            c = attention("", spread(1, max(1, min(8, 12000000 // (q * kv)))), q, kv, heads, page, window, sinks)
        else:
            c = attention("", spread(2, 16), spread(20, 384), spread(400, 6000), heads, page, window, sinks, True)
    del c["name"]
    return c


def lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence: the first as long as the case says, the others spread."""
    got = []
    for b in range(case["B"]):
        a, c = (b * 0.6180339887 % 1.0, b * 0.7548776662 % 1.0)
        q = case["q"] - int(a * 0.8 * case["q"])
        if case["mixed"] and b:
            q = 1
        kv = case["kv"] - int(c * 0.8 * case["kv"])
        got.append((q, max(q, kv)))
    return got


def prepare(case, seed):
    """The inputs of one case, made from the seed."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return prepare_logits(case, g) if case["op"] == "logits" else prepare_paged(case, g)


def normal(g, *shape, scale=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, scale, generator=g)


def whole(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def prepare_paged(case, g):
    hq, hkv, d = HEADS[case["heads"]]
    lens, page, B = lengths(case), case["page"], case["B"]
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    T = starts[-1]
    need = [-(-kv // page) for _, kv in lens]
    most, count = max(need), sum(need) + 3
    # pages in no order, as a server's free list hands them out; the table's unused entries are -1
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        if case["op"] == "attention" and case["window"] and not case["mixed"]:
            # pages that no new token sees any more are given back
            first, last = -(-case["sinks"] // page), (lens[b][1] - lens[b][0] - case["window"] + 1) // page
            if last > first:
                table[b, first:last] = -1
    s = {"case": case, "T": T, "B": B, "hq": hq, "hkv": hkv, "d": d, "page": page, "pages": table, "most": most * page,
         "max_q": max(n for n, _ in lens), "q_start": whole(starts), "kv_len": whole([kv for _, kv in lens]),
         "k_cache": normal(g, count, page, hkv, d), "v_cache": normal(g, count, page, hkv, d)}
    if case["op"] == "attention":
        # scores of a standard deviation of about 2, and values with a mean, as trained heads have them
        s["q"] = normal(g, T, hq, d, scale=2.0)
        s["v_cache"] += 0.25
        s["scale"] = 1.0 / math.sqrt(d)
        return s
    # one projection's rows hold a token's queries, keys and values side by side
    s["qkv"] = normal(g, T, (hq + 2 * hkv) * d)
    rot = int(d * case["part"]) // 16 * 16
    s["inv_freq"] = (1000000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(torch.float32).cuda()
    # time, height and width take contiguous sections of the frequencies
    s["axis"] = (torch.arange(rot // 2) * case["axes"] // (rot // 2)).to(torch.uint8).cuda()
    place = torch.arange(T, device="cuda", dtype=torch.int32)
    side = max(1, int(math.sqrt(case["q"])))
    every = [place + int(case["kv"]), place // side % side, place % side]
    s["positions"] = torch.stack(every[:case["axes"]]).contiguous()
    s["q_norm"] = 1.0 + normal(g, d, scale=0.1) if case["norm"] else None
    s["k_norm"] = 1.0 + normal(g, d, scale=0.1) if case["norm"] else None
    return s


def prepare_logits(case, g):
    B, V = case["B"], case["V"]
    dtype = getattr(torch, case["dtype"])
    hist = [case["hist"] - int(b * 0.6180339887 % 1.0 * 0.9 * case["hist"]) for b in range(B)]
    starts = [0]
    for n in hist:
        starts.append(starts[-1] + n)
    u = torch.rand(starts[-1], generator=g, device="cuda", dtype=torch.float64)
    s = {"case": case, "B": B, "V": V, "logits": (torch.randn(B, V, generator=g, device="cuda") * 3.0).to(dtype)}
    # tokens of a text: few are very frequent
    s["history"] = (V * u ** 5).to(torch.int32).clamp(max=V - 1)
    s["history_start"] = whole(starts)
    s["prompt_len"] = whole([n * 2 // 3 for n in hist])
    row = torch.rand(3, B, generator=g, device="cuda")
    s["repetition"], s["presence"], s["frequency"] = 1.0 + 0.3 * row[0], row[1].contiguous(), 0.5 * row[2]
    each = 40  # biased tokens of each text, no token twice in a text
    s["bias_start"] = whole([each * b for b in range(B + 1)])
    step = V // each
    s["bias_ids"] = (torch.arange(each, device="cuda") * step + torch.randint(step, (B, each), generator=g, device="cuda")).reshape(-1).to(torch.int32)
    s["bias_values"] = torch.randn(B * each, generator=g, device="cuda") * 5.0
    if case["mask"]:
        words = (V + 31) // 32
        bits = torch.randint(-2 ** 31, 2 ** 31, (3, B, words), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        few = torch.arange(B, device="cuda")[:, None] % 3
        # texts in a grammar that leaves few tokens, in one that leaves half, and without one
        s["allowed"] = torch.where(few == 0, bits[0] & bits[1] & bits[2], torch.where(few == 1, bits[0], -1)).to(torch.int32)
    else:
        s["allowed"] = None
    return s


def run(state):
    op = state["case"]["op"]
    if op == "rope":
        return run_rope(state)
    if op == "attention":
        return run_attention(state)
    return run_logits(state)


def heads_of(s):
    """q, k and v as views of the projection's rows."""
    T, hq, hkv, d = s["T"], s["hq"], s["hkv"], s["d"]
    q, k, v = s["qkv"].split([hq * d, hkv * d, hkv * d], dim=1)
    return q.view(T, hq, d), k.view(T, hkv, d), v.view(T, hkv, d)


def run_rope(s):
    q, k, v = heads_of(s)
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        if "q_out" not in s:
            s["q_out"] = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        mt.mt_rope_append(q, k, v, s["positions"], s["inv_freq"], s["q_out"], s["k_cache"], s["v_cache"], s["pages"],
                          s["q_start"], s["kv_len"], axis=s["axis"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
                          pairing=mt.MT_ROPE_ADJACENT if s["case"]["adjacent"] else mt.MT_ROPE_HALF)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    adjacent = s["case"]["adjacent"]
    angle = s["positions"].double()[s["axis"].long()].t() * s["inv_freq"].double()  # [T, rot / 2]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        n = 2 * cos.shape[-1]
        r, rest = x[..., :n], x[..., n:]
        a, b = (r[..., 0::2], r[..., 1::2]) if adjacent else (r[..., :n // 2], r[..., n // 2:])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack([a, b], -1).flatten(-2) if adjacent else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1).to(torch.bfloat16)

    t = torch.arange(s["T"], device=q.device)
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    at = s["kv_len"].long()[b] - (s["q_start"].long()[b + 1] - t)
    page = s["pages"].long()[b, at // s["page"]]
    s["k_cache"][page, at % s["page"]] = turned(k, s["k_norm"])
    s["v_cache"][page, at % s["page"]] = v
    return {"q": turned(q, s["q_norm"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
        mt.mt_paged_attention(q, s["k_cache"], s["v_cache"], s["pages"], s["q_start"], s["kv_len"], s["max_q"], s["scale"],
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
    place = (kv_len - (start[1:] - start[:-1]))[:, None] + i                          # [B, Q] position of each new token
    seen = there[:, None, :] & (key <= place[:, :, None])
    if c["window"]:
        seen = seen & ((key > place[:, :, None] - c["window"]) | (key < c["sinks"]))
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


def run_logits(s):
    if own:
        import quantized_gemv_epilogues_gb300 as mt
        if "out" not in s:
            s["out"] = torch.empty_like(s["logits"])
        mt.mt_logit_penalties(s["logits"], s["out"], history=s["history"], history_start=s["history_start"],
                              prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                              frequency=s["frequency"], bias_ids=s["bias_ids"], bias_values=s["bias_values"],
                              bias_start=s["bias_start"], allowed=s["allowed"])
        return s["out"]
    B, V, dev = s["B"], s["V"], s["logits"].device
    start = s["history_start"].long()
    n = torch.arange(s["history"].numel(), device=dev)
    b = torch.searchsorted(start[1:], n, right=True)
    at = b * V + s["history"].long()
    made = (n - start[b] >= s["prompt_len"].long()[b]).float()
    count = torch.zeros(B * V, device=dev).index_add_(0, at, made).view(B, V)
    known = torch.zeros(B * V, device=dev).index_fill_(0, at, 1.0).view(B, V) > 0
    n = torch.arange(s["bias_ids"].numel(), device=dev)
    b = torch.searchsorted(s["bias_start"][1:].long(), n, right=True)
    bias = torch.zeros(B, V, device=dev)
    bias[b, s["bias_ids"].long()] = s["bias_values"]
    x = s["logits"].float() + bias
    r = s["repetition"][:, None]
    x = torch.where(known, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0).float()
    if s["allowed"] is not None:
        t = torch.arange(V, device=dev)
        x = torch.where((s["allowed"][:, t // 32] >> (t % 32).int()) & 1 != 0, x, -math.inf)
    return x.to(s["logits"].dtype)


def visible(case, place):
    """How many keys the token at `place` sees."""
    n, w = place + 1, case["window"]
    return n if not w or n <= w else w + min(case["sinks"], n - w)


def work(case):
    if case["op"] == "logits":
        B, V = case["B"], case["V"]
        size = 4 if case["dtype"] == "float32" else 2
        hist = sum(case["hist"] - int(b * 0.6180339887 % 1.0 * 0.9 * case["hist"]) for b in range(B))
        return {"bytes": 2 * B * V * size + (B * ((V + 31) // 32) * 4 if case["mask"] else 0) + 4 * hist + 320 * B,
                "flops": 4 * B * V}
    hq, hkv, d = HEADS[case["heads"]]
    lens = lengths(case)
    T = sum(n for n, _ in lens)
    if case["op"] == "rope":
        return {"bytes": 2 * 2 * T * (hq + 2 * hkv) * d + 4 * case["axes"] * T, "flops": T * (hq + hkv) * d * (7 if case["norm"] else 3)}
    keys = pairs = 0
    for n, kv in lens:
        pairs += sum(visible(case, kv - n + i) for i in range(n))
        first = kv - n - case["window"] + 1 if case["window"] else 0  # the first key in the first token's window
        keys += kv - max(0, first) + min(case["sinks"], max(0, first)) if case["window"] else kv
    return {"bytes": 2 * 2 * keys * hkv * d + 2 * 2 * T * hq * d + 4 * T * hq + 4 * sum(-(-kv // case["page"]) for _, kv in lens),
            "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """run()'s outputs in 64 bits, sequence by sequence and head by head."""
    s = prepare(case, seed)
    return {"rope": exact_rope, "attention": exact_attention, "logits": exact_logits}[case["op"]](s)


def exact_rope(s):
    q, k, v = heads_of(s)
    case, rot = s["case"], 2 * s["inv_freq"].numel()
    T, dev = s["T"], q.device
    turn = torch.zeros(T, rot // 2, dtype=torch.complex128, device=dev)
    for i, (a, f) in enumerate(zip(s["axis"].tolist(), s["inv_freq"].double().tolist())):
        turn[:, i] = torch.polar(torch.ones(T, dtype=torch.float64, device=dev), s["positions"][a].double() * f)
    sides = []
    for x, w in ((q, s["q_norm"]), (k, s["k_norm"])):
        x = x.double()
        if w is not None:
            x = x * (x.square().mean(2) + 1e-6).rsqrt()[:, :, None] * w.double()
        y = x.clone()
        lo, hi = (torch.arange(0, rot, 2), torch.arange(1, rot, 2)) if case["adjacent"] else (torch.arange(rot // 2), torch.arange(rot // 2, rot))
        z = torch.complex(x[:, :, lo.to(dev)], x[:, :, hi.to(dev)]) * turn[:, None, :]
        y[:, :, lo.to(dev)], y[:, :, hi.to(dev)] = z.real, z.imag
        sides.append(y)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    at, table = 0, s["pages"].tolist()
    for b, (n, kv) in enumerate(lengths(case)):
        places = range(kv - n, kv)
        page = torch.tensor([table[b][p // s["page"]] for p in places], device=dev)
        row = torch.tensor([p % s["page"] for p in places], device=dev)
        kc[page, row], vc[page, row] = sides[1][at:at + n], v[at:at + n].double()
        at += n
    return {"q": sides[0], "k_cache": kc, "v_cache": vc}


def exact_attention(s):
    case, hq, hkv, d, page = s["case"], s["hq"], s["hkv"], s["d"], s["page"]
    dev, group = s["q"].device, hq // hkv
    out = torch.zeros(s["T"], hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((s["T"], hq), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, (n, kv) in enumerate(lengths(case)):
        used = s["pages"][b, :-(-kv // page)].long().clamp(min=0)
        keys, values = (x[used].reshape(-1, hkv, d)[:kv] for x in (s["k_cache"], s["v_cache"]))
        j = torch.arange(kv, device=dev)
        for lo in range(0, n, 2048):
            i = torch.arange(lo, min(n, lo + 2048), device=dev)[:, None] + kv - n
            hidden = j > i
            if case["window"]:
                hidden |= (i - j >= case["window"]) & (j >= case["sinks"])
            rows = slice(at + lo, at + min(n, lo + 2048))
            for h in range(hq):
                k, v = keys[:, h // group].double(), values[:, h // group].double()
                w = (s["q"][rows, h].double() @ k.t() * s["scale"]).masked_fill(hidden, -math.inf)
                z = torch.logsumexp(w, 1)
                lse[rows, h] = z
                out[rows, h] = torch.exp(w - z[:, None]) @ v
        at += n
    return {"out": out, "lse": lse}


def exact_logits(s):
    B, V = s["B"], s["V"]
    got = s["logits"].double()
    hs, bs, prompt = s["history_start"].tolist(), s["bias_start"].tolist(), s["prompt_len"].tolist()
    for b in range(B):
        row = got[b]
        row[s["bias_ids"][bs[b]:bs[b + 1]].long()] += s["bias_values"][bs[b]:bs[b + 1]].double()
        text = s["history"][hs[b]:hs[b + 1]].long()
        known, r = torch.unique(text), s["repetition"][b].double()
        old = row[known]
        row[known] = torch.where(old > 0, old / r, old * r)
        made, times = torch.unique(text[prompt[b]:], return_counts=True)
        row[made] -= s["frequency"][b].double() * times + s["presence"][b].double()
        if s["allowed"] is not None:
            bit = torch.arange(32, device=row.device, dtype=torch.int32)
            row[((s["allowed"][b][:, None] >> bit) & 1).reshape(-1)[:V] == 0] = -math.inf
    return got
