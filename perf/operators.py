"""The grouped-query cache operators as measured cases: inputs, plain forms and the library's calls.

A grouped-query layer of a verify step keeps one K row and one V row of ``num_kv_heads x head_dim``
bf16 values per token in paged pools whose rows are named by ``kv_indices`` (prefix rows, then the
tree nodes' rows).  Five operators run on such pools:

  attn     tree attention of the new tokens over their request's rows under a bit-packed mask
  append   per-head RMS norm and rotation of q and k, and the write of k and v into the pools
  copy     rows of every layer's pool copied to other rows (forking, moving a request)
  commit   the accepted nodes' rows gathered behind the prefix, in every layer's pool at once
  compact  the live rows moved to the front of every pool, and the row numbers rewritten

Sizes follow the verify step's own workloads (prefix 4096 and 131072, prefixes from [1024, 16384] and
[2048, 8192], budgets of 8 to 64, 576-wide rows, pools of 65536 rows) and generic head layouts.
"""
import zlib

import torch

own = False

DEV = "cuda"
MAX_DEPTH = 7
EPS = 1e-6
WORKSPACE = 96 << 20


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the tree step of a short conversation: 21 cached tokens, 8 drafted ones; latency
        {"name": "attn_short_tree", "op": "attn", "batch": 1, "prefix_lo": 21, "prefix_hi": 21, "q_lo": 9, "q_hi": 9,
         "heads": 8, "kv_heads": 2, "dim": 64, "mask": "tree", "shuffled": True},
        # many users at once, 16 or 32 drafted tokens each after 2048 to 8192 cached ones
        {"name": "attn_mixed_32", "op": "attn", "batch": 32, "prefix_lo": 2048, "prefix_hi": 8192, "q_lo": 17, "q_hi": 33,
         "heads": 32, "kv_heads": 4, "dim": 128, "mask": "tree", "shuffled": True},
        # one user with a very long document and a wide tree
        {"name": "attn_long_tree", "op": "attn", "batch": 1, "prefix_lo": 131072, "prefix_hi": 131072, "q_lo": 65, "q_hi": 65,
         "heads": 64, "kv_heads": 8, "dim": 128, "mask": "tree", "shuffled": True},
        # plain decoding of a full batch: one new token per request
        {"name": "attn_decode_64", "op": "attn", "batch": 64, "prefix_lo": 1024, "prefix_hi": 16384, "q_lo": 1, "q_hi": 1,
         "heads": 64, "kv_heads": 8, "dim": 128, "mask": "tree", "shuffled": True},
        # one token of one request through a layer: latency
        {"name": "append_decode_1", "op": "append", "batch": 1, "prefix_lo": 4096, "prefix_hi": 4096, "q_lo": 1, "q_hi": 1,
         "heads": 64, "kv_heads": 8, "dim": 128, "rope_dim": 128, "interleaved": False, "norm": True},
        # prefill chunks of 128 tokens of 32 requests
        {"name": "append_prefill_32", "op": "append", "batch": 32, "prefix_lo": 0, "prefix_hi": 8192, "q_lo": 128, "q_hi": 128,
         "heads": 64, "kv_heads": 8, "dim": 128, "rope_dim": 128, "interleaved": False, "norm": True},
        # the nodes of one tree copied within the 576-wide pool of one layer
        {"name": "copy_tree_33", "op": "copy", "pools": 1, "rows": 65536, "width": 576, "n": 33},
        # a 16384-token request copied in all layers' K and V pools
        {"name": "copy_request_16384", "op": "copy", "pools": 32, "rows": 40000, "width": 1024, "n": 16384},
        # one request's accepted path, one layer
        {"name": "commit_1", "op": "commit", "batch": 1, "pools": 1, "width": 576, "prefix_hi": 4096, "q_hi": 33},
        # a batch's accepted paths in the K and V pools of 32 layers
        {"name": "commit_64_layers_32", "op": "commit", "batch": 64, "pools": 64, "width": 1024, "prefix_hi": 256, "q_hi": 33},
        # a small pool after a few requests ended
        {"name": "compact_small", "op": "compact", "pools": 1, "rows": 4096, "width": 576, "live": 1500, "shared": 0},
        # a full-size pool of 8 layers, half of its rows freed, some prefixes shared between requests
        {"name": "compact_65536", "op": "compact", "pools": 16, "rows": 65536, "width": 1024, "live": 32768, "shared": 8192},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** rng.random())) - 1))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "copy", "commit", "compact"])
    if op in ("attn", "append"):
        heads, kv_heads = rng.choice([(8, 2), (16, 16), (32, 4), (64, 8), (40, 8), (12, 1), (28, 4), (5, 5), (128, 8), (64, 1)])
        dim = rng.choice([64, 128])
        batch = _log_int(rng, 1, 64)
        kind = rng.choice(["one", "tree", "any", "most"])
        q_hi = {"one": 1, "tree": rng.randint(2, 65), "any": rng.randint(1, 128), "most": 128}[kind]
        q_lo = rng.randint(1, q_hi)
        if op == "append":
            hi = _log_int(rng, 0, 16384)
            return {"op": op, "batch": batch, "prefix_lo": rng.randint(0, hi), "prefix_hi": hi, "q_lo": q_lo, "q_hi": q_hi,
                    "heads": heads, "kv_heads": kv_heads, "dim": dim, "rope_dim": rng.choice([dim, dim, dim // 2, 48]),
                    "interleaved": rng.random() < 0.3, "norm": rng.random() < 0.8}
        # no more score entries, cache values or padded rows than the largest listed cases have
        most = min(131072, 500_000_000 // (batch * q_hi * heads), 1_000_000_000 // (batch * kv_heads * dim))
        hi = _log_int(rng, 0, max(1, most - 128))
        return {"op": op, "batch": batch, "prefix_lo": rng.randint(0, hi), "prefix_hi": hi, "q_lo": q_lo, "q_hi": q_hi,
                "heads": heads, "kv_heads": kv_heads, "dim": dim, "mask": rng.choice(["tree", "tree", "chain", "random"]),
                "shuffled": rng.random() < 0.8}
    width = rng.choice([576, 128, 512, 1024, 1288])
    pools = _log_int(rng, 1, 32)
    if op == "copy":
        rows = _log_int(rng, 1000, 40000)
        return {"op": op, "pools": pools, "rows": rows, "width": width, "n": _log_int(rng, 1, min(16384, rows // 2))}
    if op == "commit":
        return {"op": op, "batch": _log_int(rng, 1, 64), "pools": _log_int(rng, 1, 64), "width": width,
                "prefix_hi": rng.randint(0, 256), "q_hi": rng.randint(1, 128)}
    rows = _log_int(rng, 1000, 65536)
    pools = _log_int(rng, 1, 16)
    live = rng.randint(1, rows)
    return {"op": op, "pools": pools, "rows": rows, "width": width, "live": live, "shared": rng.randint(0, live // 2)}


# ---------------------------------------------------------------- inputs
def _layout(case):
    """Lengths of the batch's requests: new tokens and cached ones (host tensors).  They belong to the
    case: its outputs have one shape, whatever the seed of the values."""
    B = case["batch"]
    sizes = sorted((k, v) for k, v in case.items() if isinstance(v, int))
    g = torch.Generator().manual_seed(zlib.crc32(repr(sizes).encode()))
    T = torch.randint(case.get("q_lo", 1), case["q_hi"] + 1, (B,), generator=g)
    T[0] = case["q_hi"]
    P = torch.randint(case.get("prefix_lo", 0), case["prefix_hi"] + 1, (B,), generator=g)
    zero = torch.zeros(1, dtype=torch.int64)
    qo = torch.cat([zero, T.cumsum(0)])
    kv = torch.cat([zero, (P + T).cumsum(0)])
    return T, P, qo, kv


def _trees(T, g, chain):
    """Parent and depth of every node: parents before children, depth at most 7 (a chain: any)."""
    parents, depths = [], []
    for t in T.tolist():
        par, dep = [-1], [0]
        pick = torch.rand(t, generator=g).tolist()
        for i in range(1, t):
            p = i - 1 if chain else int(pick[i] * i)
            while not chain and dep[p] >= MAX_DEPTH:
                p = par[p]
            par.append(p)
            dep.append(dep[p] + 1)
        parents.append(par)
        depths.append(dep)
    return parents, depths


def _tree_bits(parent):
    """[T, T] truth values: node j is node i or one of its ancestors."""
    t = len(parent)
    vis = torch.zeros(t, t, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            vis[i] = vis[p]
        vis[i, i] = True
    return vis


def _pack(bits):
    """Rows of truth values as 32-bit words, lowest bit first, padding bits zero."""
    t, n = bits.shape
    w = (n + 31) // 32
    full = torch.zeros(t, w * 32, dtype=torch.bool, device=bits.device)
    full[:, :n] = bits
    place = torch.ones(32, dtype=torch.int64, device=bits.device) << torch.arange(32, device=bits.device)
    words = (full.view(t, w, 32).to(torch.int64) * place).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _normal(shape, gg, scale=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return out.normal_(0.0, scale, generator=gg)


def _i32(t):
    return t.to(torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gg = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op in ("attn", "append"):
        T, P, qo, kv = _layout(case)
        total_q, total_kv = int(qo[-1]), int(kv[-1])
        H, G, D = case["heads"], case["kv_heads"], case["dim"]
        rows = total_kv + total_kv // 8 + 64
        order = torch.randperm(rows, generator=gg, device=DEV) if case.get("shuffled", True) else torch.arange(rows, device=DEV)
        s.update(kv_indices=order[:total_kv].to(torch.int32).contiguous(), kv_indptr=_i32(kv), qo_indptr=_i32(qo),
                 max_q=int(T.max()), max_kv=int((P + T).max()))
        chain = case["mask"] == "chain" if op == "attn" else case["q_lo"] == 128
        parents, depths = _trees(T, g, chain)
        s["depth"] = _i32(torch.tensor([d for ds in depths for d in ds]))
        s["k_pool"] = _normal((rows, G, D), gg)
        s["v_pool"] = _normal((rows, G, D), gg)
    if op == "attn":
        words, start = [], [0]
        for b in range(len(T)):
            t, p = int(T[b]), int(P[b])
            if case["mask"] == "random":  # 70 of 100 columns seen; every fifth node sees nothing
                bits = torch.rand(t, p + t, generator=gg, device=DEV) < 0.7
                bits[4::5] = False
            else:
                bits = torch.ones(t, p + t, dtype=torch.bool, device=DEV)
                bits[:, p:] = _tree_bits(parents[b]).to(DEV)
            words.append(_pack(bits).reshape(-1))
            start.append(start[-1] + words[-1].numel())
        s.update(mask=torch.cat(words), mask_indptr=_i32(torch.tensor(start)), scale=D ** -0.5)
        s["q"] = _normal((total_q, H, D), gg, 1.5)
        s["out"] = torch.empty(total_q, H, D, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(total_q, H, dtype=torch.float32, device=DEV)
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)
    elif op == "append":
        R = case["rope_dim"]
        qkv = _normal((total_q, (H + 2 * G) * D), gg, 2.0)  # one projection's output
        s["q"] = qkv[:, : H * D].unflatten(1, (H, D))
        s["k"] = qkv[:, H * D: (H + G) * D].unflatten(1, (G, D))
        s["v"] = qkv[:, (H + G) * D:].unflatten(1, (G, D))
        s["q_weight"] = _normal((D,), gg, 0.2).add_(1.0) if case["norm"] else None
        s["k_weight"] = _normal((D,), gg, 0.2).add_(1.0) if case["norm"] else None
        far = int((P + T).max()) + 1
        angle = torch.arange(far, device=DEV, dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R))
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        s["q_out"] = torch.empty(total_q, H, D, dtype=torch.bfloat16, device=DEV)
    elif op == "copy":
        s["pool"] = _normal((case["pools"], case["rows"], case["width"]), gg)
        order = torch.randperm(case["rows"], generator=gg, device=DEV).to(torch.int32)
        s["src"] = order[: case["n"]].contiguous()
        s["dst"] = order[case["n"]: 2 * case["n"]].contiguous()
    elif op == "commit":
        T, P, qo, kv = _layout(case)
        rows = int(kv[-1]) + 64
        s["pool"] = _normal((case["pools"], rows, case["width"]), gg)
        s.update(kv_indices=torch.randperm(rows, generator=gg, device=DEV)[: int(kv[-1])].to(torch.int32).contiguous(),
                 kv_indptr=_i32(kv), qo_indptr=_i32(qo))
        parents, _ = _trees(T, g, False)
        lens, nodes = [], []
        for par in parents:  # the path to a node drawn at random
            n = int(torch.randint(0, len(par), (1,), generator=g))
            path = []
            while n >= 0:
                path.append(n)
                n = par[n]
            lens.append(len(path))
            nodes.append(path[::-1] + [-1] * (MAX_DEPTH + 1 - len(path)))
        s["accept_len"], s["accepted_nodes"] = _i32(torch.tensor(lens)), _i32(torch.tensor(nodes))
        s["new_len"] = torch.empty(len(T), dtype=torch.int32, device=DEV)
    else:
        s["pool"] = _normal((case["pools"], case["rows"], case["width"]), gg)
        rows = torch.randperm(case["rows"], generator=gg, device=DEV)[: case["live"]]
        shared = rows[torch.randint(0, case["live"], (case["shared"],), generator=gg, device=DEV)]
        s["kv_indices"] = torch.cat([rows, shared]).to(torch.int32)
        s["new_indices"] = torch.empty_like(s["kv_indices"])
        s["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_attn(s):
    q, idx = s["q"], s["kv_indices"].long()
    kv, qo, mi = s["kv_indptr"].long(), s["qo_indptr"].long(), s["mask_indptr"].long()
    total_q, H, D = q.shape
    Hk = s["k_pool"].shape[1]
    B, Tm, Nm = kv.numel() - 1, s["max_q"], s["max_kv"]
    N, T = kv[1:] - kv[:-1], qo[1:] - qo[:-1]
    col, row = torch.arange(Nm, device=q.device), torch.arange(Tm, device=q.device)
    in_kv, in_q = col < N[:, None], row < T[:, None]
    slots = idx[torch.where(in_kv, kv[:-1, None] + col, 0)]                       # [B, Nm]
    tok = torch.where(in_q, qo[:-1, None] + row, 0)                               # [B, Tm]
    W = (N + 31) // 32
    word = mi[:-1, None, None] + row[None, :, None] * W[:, None, None] + (col // 32)[None, None, :]
    ok = in_q[:, :, None] & in_kv[:, None, :]
    vis = ((s["mask"][torch.where(ok, word, 0)] >> (col % 32).to(torch.int32)) & 1).bool() & ok  # [B, Tm, Nm]
    # [B, Hk, group * Tm, Nm]
    qf = q[tok].float().view(B, Tm, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    k = s["k_pool"][slots].float()
    sc = torch.matmul(qf, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(B, Hk, H // Hk, Tm, Nm)
    del k
    sc = sc.masked_fill_(~vis[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = s["v_pool"][slots].float().permute(0, 2, 1, 3)
    o = torch.matmul(p.view(B, Hk, -1, Nm), v).view(B, Hk, H // Hk, Tm, D) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + l.log()).squeeze(-1)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, Tm, H, D)[in_q].to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, Tm, H)[in_q].contiguous()}


def _norm_rope(x, weight, cos, sin, interleaved):
    """x: [tokens, heads, D] in 32 bits; cos, sin: [tokens, 1, R / 2]."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    r = cos.shape[-1]
    a, b = (x[..., 0: 2 * r: 2], x[..., 1: 2 * r: 2]) if interleaved else (x[..., :r], x[..., r: 2 * r])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., 2 * r:]], -1)


def _plain_append(s):
    qo, kv = s["qo_indptr"].long(), s["kv_indptr"].long()
    total = s["q"].shape[0]
    t = torch.arange(total, device=qo.device)
    b = torch.searchsorted(qo[1:].contiguous(), t, right=True)
    P = (kv[1:] - kv[:-1] - (qo[1:] - qo[:-1]))[b]
    slot = s["kv_indices"][kv[b] + P + (t - qo[b])].long()
    cs = s["cos_sin"][P + s["depth"].long()][:, None, :]
    cos, sin = cs.chunk(2, -1)
    il = s["case"]["interleaved"]
    q = _norm_rope(s["q"].float(), s["q_weight"], cos, sin, il).to(torch.bfloat16)
    k = _norm_rope(s["k"].float(), s["k_weight"], cos, sin, il).to(torch.bfloat16)
    s["k_pool"][slot] = k
    s["v_pool"][slot] = s["v"]
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_copy(s):
    s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return {"pool": s["pool"]}


def _plain_commit(s):
    kv, qo = s["kv_indptr"].long(), s["qo_indptr"].long()
    first = kv[1:] - (qo[1:] - qo[:-1])                                           # place of each root's row
    k = torch.arange(MAX_DEPTH + 1, device=kv.device)
    taken = k < s["accept_len"][:, None]
    idx = s["kv_indices"].long()
    src = idx[first[:, None] + torch.where(taken, s["accepted_nodes"].long(), 0)]
    dst = idx[first[:, None] + torch.where(taken, k, 0)]                          # the rest: the root onto itself
    s["pool"][:, dst.reshape(-1)] = s["pool"][:, src.reshape(-1)]
    new_len = (first - kv[:-1]).to(torch.int32) + s["accept_len"]
    return {"pool": s["pool"], "new_len": new_len}


def _plain_compact(s):
    idx, rows = s["kv_indices"].long(), s["pool"].shape[1]
    used = torch.zeros(rows, dtype=torch.bool, device=idx.device)
    used[idx] = True
    n = used.sum()
    row = torch.arange(rows, device=idx.device)
    holes = (~used & (row < n)).nonzero().squeeze(1)
    movers = (used & (row >= n)).nonzero().squeeze(1)
    to = row.clone()
    to[movers] = holes
    s["pool"][:, holes] = s["pool"][:, movers]
    return {"pool": s["pool"], "indices": to[idx].to(torch.int32), "live": n.to(torch.int32).reshape(1)}


PLAIN = {"attn": _plain_attn, "append": _plain_append, "copy": _plain_copy, "commit": _plain_commit, "compact": _plain_compact}


# ---------------------------------------------------------------- the library's calls
def _own(s):
    from tree_speculative_decoding_gb300 import ddt
    op = s["op"]
    if op == "attn":
        ddt.ddt_gqa_verify_attn(s["q"], s["k_pool"], s["v_pool"], s["kv_indices"], s["kv_indptr"], s["qo_indptr"], s["mask"],
                                s["mask_indptr"], s["scale"], s["out"], s["lse"], max_q_len=s["max_q"], max_kv_len=s["max_kv"],
                                workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        ddt.ddt_gqa_norm_rope_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["cos_sin"], s["depth"],
                                     s["qo_indptr"], s["kv_indices"], s["kv_indptr"], s["q_out"], s["k_pool"], s["v_pool"],
                                     interleaved=s["case"]["interleaved"])
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "copy":
        ddt.ddt_cache_copy(s["pool"], s["pool"], s["src"], s["dst"])
        return {"pool": s["pool"]}
    if op == "commit":
        ddt.ddt_cache_commit(s["pool"], s["kv_indices"], s["kv_indptr"], s["qo_indptr"], s["accept_len"], s["accepted_nodes"],
                             MAX_DEPTH, s["new_len"])
        return {"pool": s["pool"], "new_len": s["new_len"]}
    ddt.ddt_cache_compact(s["pool"], s["kv_indices"], s["new_indices"], s["live"], workspace=s["workspace"])
    return {"pool": s["pool"], "indices": s["new_indices"], "live": s["live"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("attn", "append"):
        H, G, D = case["heads"], case["kv_heads"], case["dim"]
        T, P, qo, kv = (x.double() for x in _layout(case))
        tokens = float(qo[-1])
        if op == "attn":
            # a tree node sees its ancestors, about the square root of the nodes; a random mask 56 of 100 columns
            seen = {"tree": P + T.sqrt(), "chain": P + (T + 1) / 2, "random": 0.56 * (P + T)}[case["mask"]]
            bytes_ = float(kv[-1]) * (4 * G * D + 4) + tokens * H * (4 * D + 4) + float((T * (P + T)).sum()) / 8
            return {"bytes": bytes_, "flops": 4.0 * H * D * float((T * seen).sum())}
        R = case["rope_dim"]
        return {"bytes": tokens * ((H + 2 * G) * D * 4 + 4 * R + 8), "flops": tokens * (H + G) * (5.0 * D + 3 * R)}
    row = case["pools"] * case["width"] * 2
    if op == "copy":
        return {"bytes": case["n"] * (2.0 * row + 8), "flops": 0}
    if op == "commit":
        T = _layout(case)[0].double()
        moved = float((T.sqrt().clamp(max=MAX_DEPTH + 1) / 2).sum())  # half of a path's nodes, at a guess, have moved
        return {"bytes": moved * 2 * row + 64.0 * case["batch"], "flops": 0}
    gone = 1 - case["live"] / case["rows"]
    return {"bytes": case["live"] * gone * 2 * row + 8.0 * (case["live"] + case["shared"]) + case["rows"] / 8, "flops": 0}


# ---------------------------------------------------------------- 64 bits
def _exact_attn(s):
    kv, qo, mi = (s[n].tolist() for n in ("kv_indptr", "qo_indptr", "mask_indptr"))
    total, H, D = s["q"].shape
    Hk = s["k_pool"].shape[1]
    per = H // Hk
    out = torch.zeros(total, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((total, H), float("-inf"), dtype=torch.float64, device=DEV)
    bit = torch.arange(32, device=DEV, dtype=torch.int32)
    for b in range(len(kv) - 1):
        t, n = qo[b + 1] - qo[b], kv[b + 1] - kv[b]
        rows = s["kv_indices"][kv[b]: kv[b + 1]].long()
        words = s["mask"][mi[b]: mi[b + 1]].view(t, -1)
        seen = (((words[:, :, None] >> bit) & 1) != 0).flatten(1)[:, :n]
        K, V = s["k_pool"][rows].double(), s["v_pool"][rows].double()
        for h in range(H):
            if h % per == 0:
                Kh, Vh = K[:, h // per], V[:, h // per]
            z = (s["q"][qo[b]: qo[b + 1], h].double() * s["scale"]) @ Kh.t()
            z[~seen] = float("-inf")
            le = torch.logsumexp(z, 1)
            lse[qo[b]: qo[b + 1], h] = le
            some = le > float("-inf")
            out[qo[b]: qo[b + 1], h] = torch.where(some[:, None], torch.exp(z - torch.where(some, le, 0.0)[:, None]) @ Vh, 0.0)
    return {"out": out, "lse": lse}


def _exact_append(s):
    kv, qo = s["kv_indptr"].tolist(), s["qo_indptr"].tolist()
    il, R = s["case"]["interleaved"], s["case"]["rope_dim"]
    D = s["q"].shape[2]
    place = torch.arange(R // 2, device=DEV)
    first, second = (2 * place, 2 * place + 1) if il else (place, place + R // 2)

    def turned(x, w, pos):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        z = torch.complex(x[..., first], x[..., second])
        table = s["cos_sin"][pos].double()
        z = z * torch.complex(table[:, None, : R // 2], table[:, None, R // 2:])
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    for b in range(len(kv) - 1):
        a, e = qo[b], qo[b + 1]
        pos = (kv[b + 1] - kv[b] - (e - a)) + s["depth"][a:e].long()
        q[a:e] = turned(s["q"][a:e], s["q_weight"], pos)
        rows = s["kv_indices"][kv[b + 1] - (e - a): kv[b + 1]].long()
        kp[rows] = turned(s["k"][a:e], s["k_weight"], pos)
        vp[rows] = s["v"][a:e].double()
    return {"q": q, "k_pool": kp, "v_pool": vp}


def _exact_rows(s):
    """copy, commit, compact: which row each row of the new pool comes from."""
    op = s["op"]
    come = list(range(s["pool"].shape[1]))
    more = {}
    if op == "copy":
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            come[b] = a
    elif op == "commit":
        kv, qo, idx = s["kv_indptr"].tolist(), s["qo_indptr"].tolist(), s["kv_indices"].tolist()
        lens = []
        for b, n in enumerate(s["accept_len"].tolist()):
            root = kv[b + 1] - (qo[b + 1] - qo[b])
            lens.append(root - kv[b] + n)
            for k, node in enumerate(s["accepted_nodes"][b].tolist()[:n]):
                come[idx[root + k]] = idx[root + node]
        more["new_len"] = torch.tensor(lens, dtype=torch.int32)
    else:
        idx = s["kv_indices"].tolist()
        live = sorted(set(idx))
        taken = set(live)
        free = [r for r in range(len(live)) if r not in taken]
        late = [r for r in live if r >= len(live)]
        new = dict(zip(late, free))
        for r, hole in new.items():
            come[hole] = r
        more["indices"] = torch.tensor([new.get(r, r) for r in idx], dtype=torch.int32)
        more["live"] = torch.tensor([len(live)], dtype=torch.int32)
    return {"pool": s["pool"].index_select(1, torch.tensor(come, device=DEV)), **more}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_rows(s)
