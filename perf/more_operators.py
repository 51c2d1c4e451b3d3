"""Chunks over a paged cache, and a cache that keeps its heaviest rows, as measured cases: inputs, plain
forms and the library's calls.

A grouped-query layer keeps one K row and one V row of ``num_kv_heads x head_dim`` bf16 values per token in
paged pools whose rows are named by ``kv_indices``: per request the cached tokens' rows, then those of the
chunk of new tokens.  Three operators run on such a cache:

  attn     attention of a chunk of any length (a prompt, a part of one, a single token).  Token i of a request
           with P cached ones is at position p = P + i, column j at position j.  With z = scale <q, k_j>, capped
           to cap tanh(z / cap) where there is a cap, less slope_h |p - j| where heads have slopes, it is softmax
           attention over the columns j < full_b (a prefix that everyone sees) and those with p - window < j <= p
  weights  how much attention every column received: the sum of the softmax's weights over heads and tokens (all
           of the chunk, or its last ones), added to what the columns had received before
  evict    per request the columns that stay when the cache may hold `budget` of them: the first ones and the
           latest, then those that received most; the rest leaves.  Order is kept

Sizes follow the verify step's workloads (prefixes of 4096 and 131072, from [1024, 16384] and [2048, 8192])
and generic head layouts.
"""
import zlib

import torch

own = False

DEV = "cuda"
WORKSPACE = 160 << 20


# ---------------------------------------------------------------- cases
_HEADS = {"heads": 64, "kv_heads": 8, "dim": 128}
_PLAIN = {"cap": 0.0, "bias": False, "window": 0, "full_hi": 0}


def listed():
    return [
        # one user's next token under capped scores: latency
        {"name": "attn_decode_1", "op": "attn", "batch": 1, "prefix_lo": 4095, "prefix_hi": 4095, "q_lo": 1, "q_hi": 1,
         **_HEADS, **_PLAIN, "cap": 50.0, "page": 1},
        # a full batch's next tokens in a layer with a window of 4096 and a few first tokens that stay visible
        {"name": "attn_decode_64_window", "op": "attn", "batch": 64, "prefix_lo": 1024, "prefix_hi": 16384, "q_lo": 1,
         "q_hi": 1, **_HEADS, **_PLAIN, "window": 4096, "full_hi": 8, "page": 16},
        # a whole prompt
        {"name": "attn_prompt_8192", "op": "attn", "batch": 1, "prefix_lo": 0, "prefix_hi": 0, "q_lo": 8192, "q_hi": 8192,
         **_HEADS, **_PLAIN, "page": 64},
        # the last chunk of a long document, scores capped, rows in any order
        {"name": "attn_capped_after_30720", "op": "attn", "batch": 1, "prefix_lo": 30720, "prefix_hi": 30720, "q_lo": 2048,
         "q_hi": 2048, "heads": 32, "kv_heads": 4, "dim": 128, **_PLAIN, "cap": 50.0, "page": 1},
        # chunks of every length for a model whose heads weigh distance
        {"name": "attn_bias_16", "op": "attn", "batch": 16, "prefix_lo": 0, "prefix_hi": 8192, "q_lo": 1, "q_hi": 500,
         "heads": 16, "kv_heads": 16, "dim": 64, **_PLAIN, "bias": True, "page": 16},
        # a layer with a window, and a system prompt that every token sees whole
        {"name": "attn_window_prefix_4", "op": "attn", "batch": 4, "prefix_lo": 0, "prefix_hi": 4096, "q_lo": 1500,
         "q_hi": 2000, "heads": 40, "kv_heads": 8, "dim": 128, **_PLAIN, "window": 1024, "full_hi": 300, "page": 64},
        # what a batch's next tokens attended to, added to the columns' sums
        {"name": "weights_decode_32", "op": "weights", "batch": 32, "prefix_lo": 2048, "prefix_hi": 8192, "q_lo": 1,
         "q_hi": 1, **_HEADS, **_PLAIN, "page": 1, "last_rows": 0, "decay": 1.0},
        # the last 32 tokens of a long prompt's last chunk as observers of all columns
        {"name": "weights_observers_32", "op": "weights", "batch": 1, "prefix_lo": 24576, "prefix_hi": 24576, "q_lo": 8192,
         "q_hi": 8192, **_HEADS, **_PLAIN, "page": 64, "last_rows": 32, "decay": 0.0},
        # two chunks in full, scores capped
        {"name": "weights_chunk_2048", "op": "weights", "batch": 2, "prefix_lo": 4096, "prefix_hi": 8192, "q_lo": 2048,
         "q_hi": 2048, "heads": 32, "kv_heads": 4, "dim": 128, **_PLAIN, "cap": 30.0, "page": 16, "last_rows": 0, "decay": 0.9},
        # one conversation that has outgrown its budget: latency
        {"name": "evict_one", "op": "evict", "batch": 1, "n_lo": 4097, "n_hi": 4097, "budget_lo": 2048, "budget_hi": 2048,
         "sinks": 4, "recent": 256},
        # a batch of ragged conversations, budgets of their own
        {"name": "evict_batch_64", "op": "evict", "batch": 64, "n_lo": 1024, "n_hi": 16384, "budget_lo": 1024,
         "budget_hi": 4096, "sinks": 4, "recent": 128},
        # long documents cut down to an eighth
        {"name": "evict_long_8", "op": "evict", "batch": 8, "n_lo": 131072, "n_hi": 131072, "budget_lo": 16384,
         "budget_hi": 16384, "sinks": 16, "recent": 1024},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random())) - 1))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "weights", "weights", "evict"])
    if op == "evict":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(131072, 1048576 // batch))
        most = _log_int(rng, 1, 16384)
        recent = rng.randint(0, most // 4)
        return {"op": op, "batch": batch, "n_lo": rng.randint(0, hi), "n_hi": hi, "budget_lo": rng.randint(1, most),
                "budget_hi": most, "sinks": rng.randint(0, 16), "recent": recent}
    heads, kv_heads = rng.choice([(8, 2), (16, 16), (32, 4), (64, 8), (40, 8), (12, 1), (28, 4), (5, 5), (128, 8), (64, 1)])
    dim = rng.choice([64, 128, 128])
    batch = _log_int(rng, 1, 64)
    kind = rng.choice(["one", "short", "chunk", "chunk"])
    # no more score entries or padded rows than the largest listed cases have, nor longer than these
    most_q = max(1, min(8192, int((2_000_000_000 / (batch * heads)) ** 0.5)))
    q_hi = {"one": 1, "short": rng.randint(2, 65), "chunk": _log_int(rng, min(65, most_q), most_q)}[kind]
    q_lo = rng.randint(1, q_hi)
    columns = min(131072, 2_000_000_000 // (batch * q_hi * heads), 500_000_000 // (batch * kv_heads * dim))
    hi = _log_int(rng, 0, max(1, columns - q_hi))
    case = {"op": op, "batch": batch, "prefix_lo": rng.randint(0, hi), "prefix_hi": hi, "q_lo": q_lo, "q_hi": q_hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "cap": rng.choice([0.0, 0.0, 0.0, 20.0, 30.0, 50.0]),
            "bias": rng.random() < 0.25, "window": rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]),
            "full_hi": rng.choice([0, 0, _log_int(rng, 1, 2048)]), "page": rng.choice([1, 1, 16, 64])}
    if op == "weights":
        case.update(last_rows=rng.choice([0, 0, rng.randint(1, 64)]), decay=rng.choice([0.0, 1.0, 0.9]))
    return case


# ---------------------------------------------------------------- inputs
def _ragged(case, *names):
    """Lengths of the batch's requests, the first one's the largest (host tensors).  They belong to the
    case: its outputs have one shape, whatever the seed of the values."""
    sizes = sorted((k, v) for k, v in case.items() if isinstance(v, int))
    g = torch.Generator().manual_seed(zlib.crc32(repr(sizes).encode()))
    out = []
    for name in names:
        x = torch.randint(case[name + "_lo"], case[name + "_hi"] + 1, (case["batch"],), generator=g)
        x[0] = case[name + "_hi"]
        out.append(x)
    return out


def _starts(lens):
    return torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])


def _full_lens(case, N):
    """Columns that all tokens of a request see, whatever their position."""
    g = torch.Generator().manual_seed(7 + case["batch"])
    return torch.minimum(torch.randint(0, case["full_hi"] + 1, (case["batch"],), generator=g), N)


def _normal(shape, gg, scale=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return out.normal_(0.0, scale, generator=gg)


def _i32(t):
    return t.to(torch.int32).to(DEV)


def prepare(case, seed):
    gg = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "evict":
        N, C = _ragged(case, "n", "budget")
        total, kept = int(N.sum()), torch.minimum(N, C)
        s["kv_indptr"], s["budget"] = _i32(_starts(N)), _i32(C)
        s["kv_indices"] = torch.randperm(total + 64, generator=gg, device=DEV)[:total].to(torch.int32)
        # sums of attention weights are far apart, and columns that nobody saw have the same
        w = torch.empty(total, dtype=torch.float32, device=DEV).normal_(0.0, 2.0, generator=gg).exp_()
        s["weights"] = w.masked_fill_(torch.rand(total, generator=gg, device=DEV) < 0.1, 0.0)
        s["max_kv"] = int(N.max())
        s["new_indices"] = torch.empty(int(kept.sum()), dtype=torch.int32, device=DEV)
        s["new_weights"] = torch.empty(int(kept.sum()), dtype=torch.float32, device=DEV)
        s["new_indptr"] = torch.empty(case["batch"] + 1, dtype=torch.int32, device=DEV)
        s["evicted"] = torch.empty(total - int(kept.sum()), dtype=torch.int32, device=DEV)
        return s
    T, P = _ragged(case, "q", "prefix")
    N = P + T
    H, G, D, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    s.update(qo_indptr=_i32(_starts(T)), kv_indptr=_i32(_starts(N)), max_q=int(T.max()), max_kv=int(N.max()), scale=D ** -0.5)
    # every request has whole pages of the pool, in any order
    pages = (N + page - 1) // page
    many = int(pages.sum())
    places = torch.randperm(many + many // 8 + 4, generator=gg, device=DEV)
    rows = places.numel() * page
    slots = (places[:many, None] * page + torch.arange(page, device=DEV)).flatten()
    at = torch.repeat_interleave(_starts(pages * page)[:-1] - _starts(N)[:-1], N).to(DEV)
    s["kv_indices"] = slots[torch.arange(int(N.sum()), device=DEV) + at].to(torch.int32)
    s["k_pool"] = _normal((rows, G, D), gg)
    s["q"] = _normal((int(T.sum()), H, D), gg, 6.0 if case["cap"] else 1.5)
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H) if case["bias"] else None
    s["full_len"] = _i32(_full_lens(case, N)) if case["full_hi"] else None
    s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)
    if case["op"] == "attn":
        s["v_pool"] = _normal((rows, G, D), gg)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    else:
        # what the attention left: each row's log of its sum (of the rows that are counted)
        s["lse"] = torch.zeros(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        z, tok, in_q = _scores(s, case["last_rows"])
        lse = z.amax(-1)
        lse = lse + z.sub_(lse[..., None]).exp_().sum(-1).log_()
        s["lse"][tok[in_q]] = lse.permute(0, 2, 1)[in_q]
        # what the columns but the new ones had before
        s["prev"] = torch.rand(int(P.sum()), generator=gg, device=DEV) * 4.0
        s["prev_indptr"] = _i32(_starts(P))
        s["weights"] = torch.empty(int(N.sum()), dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _scores(s, last_rows=0):
    """Scores of every head, token and column in 32 bits, [batch, heads, tokens, columns], -inf where a token
    does not see a column; the tokens' places, and which of them there are.  last_rows: of the last tokens alone."""
    case, q, idx = s["case"], s["q"], s["kv_indices"].long()
    kv, qo = s["kv_indptr"].long(), s["qo_indptr"].long()
    H, D = q.shape[1:]
    Hk = s["k_pool"].shape[1]
    B, Nm = kv.numel() - 1, s["max_kv"]
    N, T = kv[1:] - kv[:-1], qo[1:] - qo[:-1]
    rows = torch.clamp(T, max=last_rows) if last_rows else T
    Tm = min(s["max_q"], last_rows) if last_rows else s["max_q"]
    col, row = torch.arange(Nm, device=q.device), torch.arange(Tm, device=q.device)
    in_kv, in_q = col < N[:, None], row < rows[:, None]
    slots = idx[torch.where(in_kv, kv[:-1, None] + col, 0)]                       # [B, Nm]
    tok = torch.where(in_q, (qo[1:] - rows)[:, None] + row, 0)                    # [B, Tm]
    pos = (N - rows)[:, None] + row
    away = pos[:, :, None] - col                                                  # [B, Tm, Nm]
    seen = away >= 0
    if case["window"]:
        seen &= away < case["window"]
    if s["full_len"] is not None:
        seen |= (col < s["full_len"].long()[:, None])[:, None, :]
    seen &= in_kv[:, None, :]
    qf = q[tok].float().view(B, Tm, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    z = torch.matmul(qf, s["k_pool"][slots].float().permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, H, Tm, Nm)
    if case["cap"]:
        z = z.div_(case["cap"]).tanh_().mul_(case["cap"])
    if s["slopes"] is not None:
        z = z.addcmul_(away.abs().float()[:, None], s["slopes"][:, None, None], value=-1.0)
    return z.masked_fill_(~seen[:, None], float("-inf")), tok, in_q


def _plain_attn(s):
    z, tok, in_q = _scores(s)
    B, H, Tm, Nm = z.shape
    kv, idx = s["kv_indptr"].long(), s["kv_indices"].long()
    Hk, D = s["v_pool"].shape[1:]
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    col = torch.arange(Nm, device=z.device)
    slots = idx[torch.where(col < (kv[1:] - kv[:-1])[:, None], kv[:-1, None] + col, 0)]
    v = s["v_pool"][slots].float().permute(0, 2, 1, 3)
    o = torch.matmul(p.view(B, Hk, -1, Nm), v).view(B, H, Tm, D) / l
    lse = (m + l.log()).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3)[in_q].to(torch.bfloat16), "lse": lse.permute(0, 2, 1)[in_q].contiguous()}


def _plain_weights(s):
    z, tok, in_q = _scores(s, s["case"]["last_rows"])
    lse = torch.where(in_q[:, :, None], s["lse"][tok], float("inf")).permute(0, 2, 1)
    got = z.sub_(lse[..., None]).exp_().sum((1, 2))                               # [B, Nm]
    kv, pv = s["kv_indptr"].long(), s["prev_indptr"].long()
    out = got[torch.arange(got.shape[1], device=got.device) < (kv[1:] - kv[:-1])[:, None]]
    if s["case"]["decay"]:
        at = torch.arange(s["prev"].numel(), device=got.device)
        b = torch.searchsorted(pv[1:].contiguous(), at, right=True)
        out[kv[b] + at - pv[b]] += s["case"]["decay"] * s["prev"]
    return {"weights": out}


def _plain_evict(s):
    case, kv = s["case"], s["kv_indptr"].long()
    N, Nm = kv[1:] - kv[:-1], s["max_kv"]
    col = torch.arange(Nm, device=kv.device)
    there = col < N[:, None]
    at = torch.where(there, kv[:-1, None] + col, 0)
    if Nm == 0:
        keep = there
    else:
        held = (col < case["sinks"]) | (col >= (N - case["recent"])[:, None])
        w = torch.where(there, torch.where(held, float("inf"), s["weights"][at]), float("-inf"))
        order = w.sort(dim=1, descending=True, stable=True).indices
        place = torch.empty_like(order).scatter_(1, order, col.expand_as(order))
        keep = there & (place < s["budget"].long()[:, None])
    kept = torch.minimum(N, s["budget"].long())
    indptr = torch.cat([kept.new_zeros(1), kept.cumsum(0)]).to(torch.int32)
    stay, go = at[keep], at[there & ~keep]
    return {"indices": s["kv_indices"][stay], "indptr": indptr, "weights": s["weights"][stay], "evicted": s["kv_indices"][go]}


PLAIN = {"attn": _plain_attn, "weights": _plain_weights, "evict": _plain_evict}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from tree_speculative_decoding_gb300 import ddt
    op, case = s["op"], s["case"]
    if op == "attn":
        ddt.ddt_gqa_chunk_attn(s["q"], s["k_pool"], s["v_pool"], s["kv_indices"], s["kv_indptr"], s["qo_indptr"], s["scale"],
                               s["out"], s["lse"], max_q_len=s["max_q"], max_kv_len=s["max_kv"], score_cap=case["cap"],
                               slopes=s["slopes"], window=case["window"], full_len=s["full_len"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        ddt.ddt_gqa_chunk_weights(s["q"], s["k_pool"], s["lse"], s["kv_indices"], s["kv_indptr"], s["qo_indptr"], s["scale"],
                                  s["weights"], prev=s["prev"] if case["decay"] else None, prev_indptr=s["prev_indptr"],
                                  decay=case["decay"], last_rows=case["last_rows"], max_q_len=s["max_q"],
                                  max_kv_len=s["max_kv"], score_cap=case["cap"], slopes=s["slopes"], window=case["window"],
                                  full_len=s["full_len"], workspace=s["workspace"])
        return {"weights": s["weights"]}
    ddt.ddt_cache_evict(s["weights"], s["kv_indices"], s["kv_indptr"], s["budget"], s["new_indices"], s["new_indptr"],
                        s["new_weights"], s["evicted"], sinks=case["sinks"], recent=case["recent"], max_kv_len=s["max_kv"])
    return {"indices": s["new_indices"], "indptr": s["new_indptr"], "weights": s["new_weights"], "evicted": s["evicted"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ---------------------------------------------------------------- work
def _seen(case):
    """Per request: pairs of a token and a column that it sees, and columns that a token sees (of the tokens
    that count)."""
    T, P = _ragged(case, "q", "prefix")
    N, W = P + T, case["window"]
    full = _full_lens(case, N) if case["full_hi"] else torch.zeros_like(N)
    pairs, columns = [], []
    for t, n, f in zip(T.tolist(), N.tolist(), full.tolist()):
        r = min(t, case.get("last_rows") or t)
        p = torch.arange(n - r, n, dtype=torch.float64)
        lo = (p - W + 1).clamp(min=0) if W else torch.zeros_like(p)
        pairs.append(float((f + (p + 1 - lo.clamp(min=f)).clamp(min=0)).sum()))
        columns.append(f + max(0, n - max(f, int(lo[0]))))
    return T.double(), torch.tensor(pairs, dtype=torch.float64), torch.tensor(columns, dtype=torch.float64)


def work(case):
    if case["op"] == "evict":
        N, C = _ragged(case, "n", "budget")
        n, k = float(N.sum()), float(torch.minimum(N, C).sum())
        return {"bytes": 8 * n + 8 * k + 4 * (n - k) + 12 * case["batch"], "flops": 0}
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    T, pairs, columns = _seen(case)
    if case["op"] == "attn":
        return {"bytes": float(columns.sum()) * (4 * G * D + 4) + float(T.sum()) * H * (4 * D + 4),
                "flops": 4.0 * H * D * float(pairs.sum())}
    rows = float(T.clamp(max=case["last_rows"]).sum() if case["last_rows"] else T.sum())
    n = sum(float(x.double().sum()) for x in _ragged(case, "q", "prefix"))
    return {"bytes": float(columns.sum()) * (2 * G * D + 4) + rows * H * (2 * D + 4) + n * (8 if case["decay"] else 4),
            "flops": 2.0 * H * D * float(pairs.sum())}


# ---------------------------------------------------------------- 64 bits
def _exact_heads(s):
    """For every request, head and block of 2048 tokens: the request, the head, its K/V head, the tokens and
    their scores in 64 bits, and which columns they see."""
    case = s["case"]
    kv, qo = s["kv_indptr"].tolist(), s["qo_indptr"].tolist()
    H = s["q"].shape[1]
    per = H // s["k_pool"].shape[1]
    for b in range(len(kv) - 1):
        rows = s["kv_indices"][kv[b]: kv[b + 1]].long()
        n, t = len(rows), qo[b + 1] - qo[b]
        first = max(0, t - case["last_rows"]) if case.get("last_rows") else 0
        K = s["k_pool"][rows].double()
        j = torch.arange(n, device=DEV, dtype=torch.float64)
        for lo in range(first, t, 2048):
            i = torch.arange(lo, min(t, lo + 2048), device=DEV, dtype=torch.float64)
            d = (n - t) + i[:, None] - j
            hide = d < 0
            if case["window"]:
                hide = hide | (d >= case["window"])
            if s["full_len"] is not None:
                hide = hide & (j >= int(s["full_len"][b]))
            tok = slice(qo[b] + lo, qo[b] + lo + len(i))
            for h in range(H):
                x = s["scale"] * (s["q"][tok, h].double() @ K[:, h // per].T)
                if case["cap"]:
                    e = torch.expm1(x * (-2.0 / case["cap"]))
                    x = torch.where(torch.isinf(e), -1.0, -e / (e + 2.0)) * case["cap"]
                if s["slopes"] is not None:
                    x = x - float(s["slopes"][h]) * d.abs()
                yield b, h, h // per, tok, rows, x.masked_fill(hide, float("-inf"))


def exact(case, seed):
    if case["op"] != "evict":
        T, P = (x.double() for x in _ragged(case, "q", "prefix"))
        r = T.clamp(max=case["last_rows"]) if case.get("last_rows") else T
        if float((r * (P + T)).sum()) * case["heads"] * case["dim"] > 1.2e12:
            return None
    s = prepare(case, seed)
    if case["op"] == "attn":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
        for b, h, g, tok, rows, x in _exact_heads(s):
            lse[tok, h] = torch.logsumexp(x, 1)
            out[tok, h] = torch.exp(x - lse[tok, h][:, None]) @ s["v_pool"][rows, g].double()
        return {"out": out, "lse": lse}
    if case["op"] == "weights":
        kv, pv = s["kv_indptr"].tolist(), s["prev_indptr"].tolist()
        w = torch.zeros(kv[-1], dtype=torch.float64, device=DEV)
        for b in range(len(kv) - 1):
            w[kv[b]: kv[b] + pv[b + 1] - pv[b]] = s["prev"][pv[b]: pv[b + 1]].double() * case["decay"]
        for b, h, g, tok, rows, x in _exact_heads(s):
            w[kv[b]: kv[b + 1]] += torch.exp(x - s["lse"][tok, h].double()[:, None]).sum(0)
        return {"weights": w}
    kv, budget = s["kv_indptr"].tolist(), s["budget"].tolist()
    w, idx = s["weights"].tolist(), s["kv_indices"].tolist()
    stay, go, indptr = [], [], [0]
    for b in range(len(kv) - 1):
        n = kv[b + 1] - kv[b]
        held = [j < case["sinks"] or j >= n - case["recent"] for j in range(n)]
        order = sorted(range(n), key=lambda j: (not held[j], 0.0 if held[j] else -w[kv[b] + j], j))
        keep = set(order[: budget[b]])
        stay += [kv[b] + j for j in range(n) if j in keep]
        go += [kv[b] + j for j in range(n) if j not in keep]
        indptr.append(len(stay))
    i32 = torch.int32
    return {"indices": torch.tensor([idx[i] for i in stay], dtype=i32), "indptr": torch.tensor(indptr, dtype=i32),
            "weights": torch.tensor([w[i] for i in stay], dtype=torch.float64), "evicted": torch.tensor([idx[i] for i in go], dtype=i32)}
