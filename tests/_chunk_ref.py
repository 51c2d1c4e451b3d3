"""Plain 64-bit forms of the chunk attention, the received weights and the eviction,
and the inputs their tests use (tests only; shares no code with the library)."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24   # half a step of fp32, relative
H8 = 2.0 ** -8   # half a step of bf16, relative


class Chunk:
    """Requests of (cached, new) tokens with their offsets and slots.  page: slots come in runs of that many."""

    def __init__(self, lens, seed, page=1, spare=7):
        rng = np.random.default_rng(seed)
        self.lens = lens
        self.P = np.array([p for p, _ in lens], np.int64)
        self.T = np.array([t for _, t in lens], np.int64)
        self.N = self.P + self.T
        self.B = len(lens)
        self.qo = np.concatenate([[0], np.cumsum(self.T)]).astype(np.int32)
        self.kv = np.concatenate([[0], np.cumsum(self.N)]).astype(np.int32)
        self.total_q, self.total_kv = int(self.qo[-1]), int(self.kv[-1])
        pages = (self.N + page - 1) // page
        places = rng.permutation(int(pages.sum()) + spare)
        self.rows = len(places) * page
        slots, at = [], 0
        for n, k in zip(self.N, pages):
            slots.append((places[at: at + k, None] * page + np.arange(page)).reshape(-1)[:n])
            at += k
        self.slots = np.concatenate(slots).astype(np.int32) if slots else np.zeros(0, np.int32)
        self.max_q, self.max_kv = int(self.T.max(initial=0)), int(self.N.max(initial=0))

    def device(self, dev="cuda:0"):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        return dict(kv_indices=t(self.slots), kv_indptr=t(self.kv), qo_indptr=t(self.qo))


def visible(c, b, window, full):
    """[T, N] truth values of request b."""
    p = (c.P[b] + np.arange(c.T[b]))[:, None]
    j = np.arange(c.N[b])[None, :]
    seen = j <= p
    if window:
        seen &= j > p - window
    if full is not None:
        seen |= j < full[b]
    return torch.from_numpy(seen)


def scores(x, K, p, cap, slope, scale):
    """Scores of rows x at positions p against K's rows, and how far fp32 may be off: D products and
    sums (2^-24 of sum |q||k| each), the roundings of the scale, the bias, the sum and the reference (their own
    size each; the reference is the largest score, moved by 53 ln 2, and may lie 28 ln 2 below a later one),
    and of a capped score cap 2^-20: e^2u and a reciprocal to 2 ulp, an argument to 2 roundings."""
    D = x.shape[-1]
    z = scale * (x @ K.T)
    ds = (D + 2) * U * scale * (x.abs() @ K.abs().T)
    if cap:
        z = cap * torch.tanh(z / cap)
        ds = ds + cap * 2.0 ** -20
    j = torch.arange(len(K), dtype=torch.float64)
    z = z - slope * (p[:, None] - j).abs()
    top = z.abs() if not slope else z.abs() + slope * (p[:, None] - j).abs()
    return z, ds + 4 * U * (top + z.max(1, keepdim=True).values.abs() + 60)


def attention(q, k_pool, v_pool, c, scale, cap=0.0, slopes=None, window=0, full=None):
    """(out, lse, bound_out, bound_lse) in float64, for a bf16 result computed in fp32 with bf16 weights:
    a score off by ds is a factor e^ds in its weight and in their sum; 2^x to 2 ulp and one bf16 rounding of
    every weight (their sum is taken before that); N terms in the sums (twice: truncating adders); one bf16
    rounding of the result."""
    H, D = q.shape[1:]
    G = k_pool.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(c.B):
        if c.T[b] == 0:
            continue
        rows = torch.from_numpy(c.slots[c.kv[b]: c.kv[b + 1]].astype(np.int64))
        seen = visible(c, b, window, full)
        p = torch.from_numpy((c.P[b] + np.arange(c.T[b])).astype(np.float64))
        tok = slice(int(c.qo[b]), int(c.qo[b + 1]))
        for h in range(H):
            K, V = k_pool[rows, h // (H // G)].double(), v_pool[rows, h // (H // G)].double()
            z, ds = scores(q[tok, h].double(), K, p, cap, float(slopes[h]) if slopes is not None else 0.0, scale)
            w = torch.softmax(z.masked_fill(~seen, -torch.inf), 1)
            lse[tok, h] = torch.logsumexp(z.masked_fill(~seen, -torch.inf), 1)
            used = seen.any(0)
            Vs = torch.where(used[:, None], V, 0.0)
            out[tok, h] = w @ Vs
            size, away = w @ Vs.abs(), (w * torch.where(seen, ds, 0.0)) @ Vs.abs()
            mean_ds = (w * torch.where(seen, ds, 0.0)).sum(1, keepdim=True)
            n = 2 * len(rows) + 64
            b_out[tok, h] = H8 * out[tok, h].abs() + size * (H8 * (1 + H8) + n * U + 2 * mean_ds) + 2 * away
            b_lse[tok, h] = mean_ds[:, 0] + n * U + 8 * U * (lse[tok, h].abs() + 60)
    return out, lse, b_out, b_lse


def received(q, k_pool, lse, c, scale, cap=0.0, slopes=None, window=0, full=None, last_rows=0, prev=None, prev_lens=None,
             decay=0.0):
    """(weights, bound) in float64: fp32 sums of e^(z - lse), each off by its score's error, 4 roundings of
    2^x and its argument (of the size of z and lse), and of up to as many additions as there are terms."""
    H = q.shape[1]
    G = k_pool.shape[1]
    w = torch.zeros(c.total_kv, dtype=torch.float64)
    bound = torch.zeros_like(w)
    at = 0
    for b in range(c.B):
        cols = slice(int(c.kv[b]), int(c.kv[b + 1]))
        if prev is not None:
            n = int(prev_lens[b])
            w[int(c.kv[b]): int(c.kv[b]) + n] += decay * prev[at: at + n].double()
            at += n
        first = max(0, int(c.T[b]) - last_rows) if last_rows else 0
        if c.T[b] == 0:
            continue
        rows = torch.from_numpy(c.slots[cols].astype(np.int64))
        seen = visible(c, b, window, full)[first:]
        p = torch.from_numpy((c.P[b] + np.arange(c.T[b])).astype(np.float64))[first:]
        tok = slice(int(c.qo[b]) + first, int(c.qo[b + 1]))
        for h in range(H):
            z, ds = scores(q[tok, h].double(), k_pool[rows, h // (H // G)].double(), p, cap,
                           float(slopes[h]) if slopes is not None else 0.0, scale)
            ls = lse[tok, h].double()[:, None]
            e = torch.where(seen, torch.exp(z - ls), 0.0)
            w[cols] += e.sum(0)
            bound[cols] += (e * (ds + 4 * U * (z.abs() + ls.abs()) + 8 * U)).sum(0)
    terms = H * int(c.T.max(initial=0)) + 8
    return w, bound + (bound + w.abs()) * U * terms


def evict(weights, slots, lens, budget, sinks, recent):
    """(slots that stay, offsets, their weights, slots that go) as lists: the first `sinks` and the last
    `recent` columns of a request count as +inf, NaN as -inf, and ties go to the lower column."""
    stay, go, indptr, kept_w, at = [], [], [0], [], 0
    for n, c in zip(lens, budget):
        def key(j):
            x = float(weights[at + j])
            if j < sinks or j >= n - recent:
                x = np.inf
            return (-(-np.inf if np.isnan(x) else x), j)
        keep = set(sorted(range(n), key=key)[: max(0, int(c))])
        for j in range(n):
            (stay if j in keep else go).append(int(slots[at + j]))
            if j in keep:
                kept_w.append(float(weights[at + j]))
        at += n
        indptr.append(len(stay))
    return stay, indptr, kept_w, go
