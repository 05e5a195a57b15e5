"""Inputs, 64-bit references and error bounds for the tests of the calls
around the projections: rotary positions, paged attention, logit penalties."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


class Paged:
    """A paged cache and a batch on it, made on the CPU; ``lens`` holds each
    sequence's (new tokens, tokens in the cache with them).

    order: "nhd" pages of [token][head], "hnd" of [head][token], "kv" with K and
    V of a page side by side.  Slots that hold no token are NaN, and so are the
    pages that no sequence has; entries past a sequence's last page are -1."""

    def __init__(self, lens, hq, hkv, d, page, order="nhd", seed=0, q_scale=1.0, spare=2, width=None, q_pad=0, rows_pad=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.d, self.page = lens, hq, hkv, d, page
        need = [-(-max(kv, 0) // page) for _, kv in lens]
        self.num_pages = sum(need) + spare
        width = width or max(1, max(need))
        self.pages = torch.full((len(lens), width), -1, dtype=torch.int32)
        ids = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.pages[b, :n] = ids[at:at + n]
            at += n
        starts = [0]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        self.T = starts[-1] + rows_pad
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.kv_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32)
        shape = (self.num_pages, page, hkv, d)
        self.keys, self.values = [], []
        k = torch.full(shape, math.nan, dtype=torch.bfloat16)
        v = torch.full(shape, math.nan, dtype=torch.bfloat16)
        for b, (_, kv) in enumerate(lens):
            kb = torch.randn(kv, hkv, d, generator=g).to(torch.bfloat16)
            vb = (torch.randn(kv, hkv, d, generator=g) + 0.25).to(torch.bfloat16)
            for p in range(need[b]):
                n = min(page, kv - p * page)
                k[self.pages[b, p], :n] = kb[p * page:p * page + n]
                v[self.pages[b, p], :n] = vb[p * page:p * page + n]
            self.keys.append(kb)
            self.values.append(vb)
        self.order = order
        self.k, self.v = self._laid_out(k, v, "cpu")
        q = torch.randn(self.T, hq * d + q_pad, generator=g) * q_scale
        self.q_rows = q.to(torch.bfloat16)
        self.q = self.q_rows[:, :hq * d].unflatten(1, (hq, d))

    def _laid_out(self, k, v, device):
        if self.order == "kv":
            both = torch.stack([k, v], 1).to(device)  # [pages, 2, page, heads, d]
            return both[:, 0], both[:, 1]
        if self.order == "hnd":
            return tuple(x.permute(0, 2, 1, 3).contiguous().to(device).permute(0, 2, 1, 3) for x in (k, v))
        return k.to(device), v.to(device)

    def cuda(self):
        """(q, k, v, pages, q_start, kv_len) on the GPU, in the chosen layout."""
        k, v = self._laid_out(self.k.contiguous(), self.v.contiguous(), "cuda")
        q = self.q_rows.cuda()[:, :self.hq * self.d].unflatten(1, (self.hq, self.d))
        return q, k, v, self.pages.cuda(), self.q_start.cuda(), self.kv_len.cuda()

    @property
    def max_q(self):
        return max(n for n, _ in self.lens)


def attention_ref(p, scale, window=0, sinks=0):
    """(out, lse, spread, score) in 64 bits for the rows of the sequences:
    spread = sum_j w_j |v_j| and score = the largest sum |q_i k_i| scale, which
    the error bounds need."""
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
        pos = torch.arange(n)[:, None] + kv - n
        j = torch.arange(kv)
        seen = j <= pos
        if window:
            seen &= (j > pos - window) | (j < sinks)
        for h in range(p.hq):
            q = p.q[r0:r0 + n, h].double()
            k, v = p.keys[b][:, h // g].double(), p.values[b][:, h // g].double()
            s = (q @ k.t() * scale).masked_fill(~seen, -math.inf)
            z = torch.logsumexp(s, 1)
            w = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            out[r0:r0 + n, h], spread[r0:r0 + n, h], lse[r0:r0 + n, h] = w @ v, w @ v.abs(), z
            score[r0:r0 + n, h] = (q.abs() @ k.abs().t() * scale).max(1).values
    return out, lse, spread, score


def attention_bounds(p, ref, weight_rounding, dtype):
    """How far out and lse may be off: the weights' rounding, fp32 sums of d
    and of n products (a step of 2^-23 each, as tensor cores may truncate)
    with their effect on the scores, and the output's own rounding."""
    out, lse, spread, score = ref
    n = max([kv for _, kv in p.lens] + [1])
    step = 2.0 ** -23
    ds = (p.d + 32) * step * (score + 1.0)                     # error of a score, and of exp2
    rel = weight_rounding + 2 * ds + (n + 64) * step
    tol_out = HALF[dtype] * out.abs() + spread * rel[..., None] * (1 + HALF[dtype]) + 1e-30
    shown = torch.where(lse == -math.inf, torch.zeros_like(lse), lse.abs())
    return tol_out, ds + (n + 64) * step + 4 * step * (shown + score)


def check(got, ref, tol, what=""):
    got, ref = got.detach().cpu().double(), ref.double()
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    assert bool(torch.isfinite(got[~inf]).all()), f"{what}: non-finite output"
    excess = ((got - ref).abs() - tol)[~inf]
    assert excess.numel() == 0 or float(excess.max()) <= 0, \
        f"{what}: {int((excess > 0).sum())} of {excess.numel()} off, worst by {float(excess.max()):.3e}"
