"""Plain 64-bit forms of the grouped-query layer and the cache-row calls, and
the inputs their tests use (tests only; shares no code with the library).

Everything is a loop over requests and heads on CPU tensors in float64.
"""
from __future__ import annotations

import numpy as np
import torch

MAX_DEPTH = 7


# ---------------------------------------------------------------- inputs
def random_tree(rng, T, chain=False):
    """(parent, depth) of T nodes, parents first, depth at most 7 (a chain: any)."""
    par, dep = [-1], [0]
    for i in range(1, T):
        p = i - 1 if chain else int(rng.integers(0, i))
        while not chain and dep[p] >= MAX_DEPTH:
            p = par[p]
        par.append(p)
        dep.append(dep[p] + 1)
    return par[:T], dep[:T]


def tree_visibility(P, parent):
    """[T, P + T] truth values: the prefix, the node's ancestors and the node."""
    T = len(parent)
    vis = np.zeros((T, P + T), bool)
    vis[:, :P] = True
    for i in range(T):
        n = i
        while n >= 0:
            vis[i, P + n] = True
            n = parent[n]
    return vis


def pack_bits(vis):
    """Rows of truth values as little-endian uint32 words (padding bits zero)."""
    T, N = vis.shape
    W = (N + 31) // 32
    full = np.zeros((T, W * 32), bool)
    full[:, :N] = vis
    return np.packbits(full, axis=1, bitorder="little").view("<u4").reshape(-1)


class Batch:
    """Requests of (prefix, new tokens) with their offsets, slots, trees and masks.  mask: 'tree',
    'chain' or 'random' (every third row of a random mask sees nothing)."""

    def __init__(self, lens, seed, mask="tree", rows=None, slot_lo=0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens = rng, lens
        self.P = np.array([p for p, _ in lens], np.int64)
        self.T = np.array([t for _, t in lens], np.int64)
        self.B = len(lens)
        self.qo = np.concatenate([[0], np.cumsum(self.T)]).astype(np.int32)
        self.kv = np.concatenate([[0], np.cumsum(self.P + self.T)]).astype(np.int32)
        self.total_q, self.total_kv = int(self.qo[-1]), int(self.kv[-1])
        self.rows = rows or self.total_kv + 7
        self.slots = (slot_lo + rng.permutation(self.rows - slot_lo)[: self.total_kv]).astype(np.int32)
        self.parent, self.depth, self.vis, words, start = [], [], [], [], [0]
        for p, t in lens:
            par, dep = random_tree(rng, t, mask == "chain")
            vis = tree_visibility(p, par)
            if mask == "random":
                vis = rng.random((t, p + t)) < 0.6
                vis[2::3] = False
            self.parent.append(par)
            self.depth.append(dep)
            self.vis.append(vis)
            words.append(pack_bits(vis))
            start.append(start[-1] + words[-1].size)
        self.words = np.concatenate(words) if words else np.zeros(0, np.uint32)
        self.mask_indptr = np.array(start, np.int32)
        self.max_q, self.max_kv = int(self.T.max(initial=0)), int((self.P + self.T).max(initial=0))

    def device(self, dev="cuda:0"):
        """The integer arrays on the device, as the library takes them."""
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.d = dict(kv_indices=t(self.slots), kv_indptr=t(self.kv), qo_indptr=t(self.qo),
                      mask=t(self.words.view(np.int32)), mask_indptr=t(self.mask_indptr),
                      depth=t(np.concatenate(self.depth).astype(np.int32)))
        return self.d


# ---------------------------------------------------------------- forms
def attention(q, k_pool, v_pool, batch, scale):
    """(out, lse, bound_out, bound_lse) in float64.

    The bounds follow from the roundings of a bf16 result computed in fp32 with
    bf16 softmax weights, u = 2^-24 and h = 2^-8 half a bf16 step:
      scores   D products and sums: |ds| <= (D + 2) u scale sum|q||k| (each row's
               largest), a factor e^ds in every weight and in their sum;
      weights  2^x to 2 ulp, one bf16 rounding each: h sum p|v| (their sum is
               taken before the rounding);
      sums     N terms: N u relative to sum p|v| (twice: truncating adders);
      output   one bf16 rounding: h |out|."""
    H, D = q.shape[1:]
    G = k_pool.shape[1]
    u, h8 = 2.0 ** -24, 2.0 ** -8
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -torch.inf, dtype=torch.float64)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(batch.B):
        rows = torch.from_numpy(batch.slots[batch.kv[b]: batch.kv[b + 1]].astype(np.int64))
        N = len(rows)
        for i in range(int(batch.T[b])):
            t = int(batch.qo[b]) + i
            seen = rows[torch.from_numpy(batch.vis[b][i])]
            if len(seen) == 0:
                continue
            for h in range(H):
                K, V = k_pool[seen, h // (H // G)].double(), v_pool[seen, h // (H // G)].double()
                x = q[t, h].double()
                s = scale * (K @ x)
                ds = (D + 2) * u * scale * float((K.abs() @ x.abs()).max()) + 4 * u * float(s.abs().max())
                m = s.max()
                w = torch.exp(s - m)
                lse[t, h] = m + torch.log(w.sum())
                p = w / w.sum()
                out[t, h] = p @ V
                away = p @ V.abs()
                b_out[t, h] = h8 * out[t, h].abs() + away * (h8 * (1 + h8) + 2 * ds + (2 * N + 32) * u)
                b_lse[t, h] = ds + (N + 32) * u + 8 * u * abs(float(lse[t, h]))
    return out, lse, b_out, b_lse


def norm_rope(x, weight, eps, table, pos, interleaved):
    """x: [n, heads, D]; table: float32 [max_pos, R] or None; pos: [n].  (y, bound)"""
    x = x.double()
    D = x.shape[-1]
    if weight is not None:
        x = x * (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt() * weight.double()
    y, size = x.clone(), x.abs()
    if table is not None:
        R = table.shape[1]
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
            c = table[pos, i].double()[:, None]
            s = table[pos, R // 2 + i].double()[:, None]
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., b] * c + x[..., a] * s
            size[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
            size[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    # mean of D squares (D u / 2 after the root), four more fp32 roundings, then one to bf16
    return y, 2.0 ** -8 * y.abs() + size * (D / 2 + 16) * 2.0 ** -24


def compact(slots, pool_rows):
    """(new slots, live, come): come[r] is the row that row r's values come from."""
    live = sorted({int(r) for r in slots if 0 <= r < pool_rows})
    n, named = len(live), set(live)
    holes = [r for r in range(n) if r not in named]
    to = dict(zip([r for r in live if r >= n], holes))
    come = list(range(pool_rows))
    for r, hole in to.items():
        come[hole] = r
    return [to.get(int(r), int(r)) for r in slots], n, come
