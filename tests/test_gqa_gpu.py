"""The grouped-query layer and the cache-row calls on the GPU, against plain
64-bit forms (tests/_gqa_ref.py, which also derives every tolerance)."""
import numpy as np
import pytest
import torch

from tests import _gqa_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ddt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_decoding_gb300 import _build
    _build.build()
    from tree_speculative_decoding_gb300 import ddt as m
    m.ddt_get_error()
    return m


def clean(ddt):
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (0, 0)


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


# ---------------------------------------------------------------- attention
def attn_inputs(batch, H, G, D, seed, strided=False, q_scale=1.5):
    q = normal((batch.total_q, H, D), seed, q_scale)
    k, v = normal((batch.rows, G, D), seed + 1), normal((batch.rows, G, D), seed + 2)
    if strided:   # one pool with a token's K and V next to each other
        kv = torch.stack([k, v], 1).to(DEV)
        return q, k, v, kv[:, 0], kv[:, 1]
    return q, k, v, k.to(DEV), v.to(DEV)


def run_attn(ddt, batch, q, kd, vd, scale, num_ctas=0, lse=True, **kw):
    d = batch.device()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV) if lse else None
    ddt.ddt_gqa_verify_attn(q.to(DEV), kd, vd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], d["mask"],
                            d["mask_indptr"], scale, out, ls, max_q_len=batch.max_q, max_kv_len=batch.max_kv,
                            num_ctas=num_ctas, **kw)
    return out, ls


def check_attn(out, ls, q, k, v, batch, scale):
    o, l, bo, bl = ref.attention(q, k, v, batch, scale)
    err = (out.double().cpu() - o).abs() - bo
    assert float(err.max()) <= 0, f"out over its bound by {float(err.max())}"
    if ls is not None:
        got = ls.double().cpu()
        empty = torch.isinf(l)
        assert torch.equal(torch.isinf(got) & (got < 0), empty)
        err = (got - l).abs()[~empty] - bl[~empty]
        assert err.numel() == 0 or float(err.max()) <= 0, f"lse over its bound by {float(err.max())}"


ATTN = [
    # heads, kv heads, dim, (prefix, new tokens) per request, mask
    (8, 2, 64, [(21, 9)], "tree"),
    (8, 2, 128, [(21, 9)], "tree"),
    (5, 5, 128, [(0, 1), (1, 1), (63, 1), (64, 1), (127, 1), (200, 1)], "tree"),
    (16, 16, 64, [(62, 1), (63, 2), (61, 3), (0, 7)], "tree"),
    (40, 8, 128, [(127, 33), (3, 17), (250, 1)], "tree"),
    (12, 1, 128, [(130, 30), (64, 11)], "random"),
    (28, 4, 64, [(95, 40), (300, 1), (0, 64)], "random"),
    (64, 8, 128, [(400, 17), (129, 33)], "tree"),
    (64, 1, 64, [(70, 5), (10, 2)], "tree"),
    (128, 1, 128, [(40, 3)], "tree"),
    (4, 2, 128, [(100, 128), (0, 128)], "chain"),
    (2, 1, 64, [(31, 128), (5, 65), (900, 2)], "random"),
    (1, 1, 128, [(1500, 1)], "tree"),
]


@pytest.mark.parametrize("H,G,D,lens,mask", ATTN)
@pytest.mark.parametrize("ctas", [0, 1, 3, 29])
def test_attention(ddt, H, G, D, lens, mask, ctas):
    batch = ref.Batch(lens, 11 + H + len(lens), mask)
    q, k, v, kd, vd = attn_inputs(batch, H, G, D, 5 * H + D)
    out, ls = run_attn(ddt, batch, q, kd, vd, D ** -0.5, ctas)
    clean(ddt)
    check_attn(out, ls, q, k, v, batch, D ** -0.5)


@pytest.mark.parametrize("ctas", [2, 5, 7, 16, 64, 128, 512])
@pytest.mark.parametrize("H,T,D", [(8, 1, 128), (16, 20, 128), (16, 33, 64)])
def test_attention_dealt_to_any_number_of_ctas(ddt, ctas, H, T, D):
    # shares that cut the long request many times, and that hold its end, whole requests and a start
    batch = ref.Batch([(1900, T), (40, T), (0, T), (700, max(1, T // 2))], 3, "tree")
    q, k, v, kd, vd = attn_inputs(batch, H, 2, D, 9)
    out, ls = run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    clean(ddt)
    check_attn(out, ls, q, k, v, batch, 0.1)


def test_attention_peaked_scores_and_a_rising_maximum(ddt):
    # scores far apart (a few columns hold all the weight), the largest ones last
    batch = ref.Batch([(700, 4)], 8, "tree")
    q, k, v, kd, vd = attn_inputs(batch, 4, 1, 128, 2)
    ramp = torch.linspace(0.0, 6.0, batch.total_kv).to(torch.bfloat16)
    k[torch.from_numpy(batch.slots.astype(np.int64))] *= ramp[:, None, None]
    kd.copy_(k)
    for ctas in (1, 3):
        out, ls = run_attn(ddt, batch, q, kd, vd, 1.0, ctas)
        clean(ddt)
        check_attn(out, ls, q, k, v, batch, 1.0)


def test_attention_strided_pool_and_no_lse(ddt):
    batch = ref.Batch([(150, 9), (33, 1)], 4, "tree")
    q, k, v, kd, vd = attn_inputs(batch, 16, 4, 128, 3, strided=True)
    assert not kd.is_contiguous()
    out, ls = run_attn(ddt, batch, q, kd, vd, 0.09, lse=False)
    clean(ddt)
    check_attn(out, ls, q, k, v, batch, 0.09)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctas,H", [(0, 8), (3, 8), (0, 64), (5, 64)])
def test_attention_unseen_rows_may_hold_anything(ddt, D, ctas, H):
    # prefix columns hidden from every row, others from some, with NaN and infinities in their K
    # and V rows and in the pool's unnamed rows; one row sees nothing
    batch = ref.Batch([(180, 6), (70, 1)], 21, "tree")
    for b in range(batch.B):
        batch.vis[b][:, 3:50:7] = False
        batch.vis[b][0, 60] = False
    batch.vis[0][4] = False
    batch.words = np.concatenate([ref.pack_bits(x) for x in batch.vis])
    q, k, v, kd, vd = attn_inputs(batch, H, 2, D, 6)
    clean_k, clean_v = k.clone(), v.clone()
    named = torch.from_numpy(batch.slots.astype(np.int64))
    unnamed = torch.ones(batch.rows, dtype=torch.bool)
    unnamed[named] = False
    bad = [float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min]
    hidden = [named[int(batch.kv[b]) + c] for b in range(batch.B) for c in range(3, 50, 7)]
    for n, r in enumerate(hidden + list(unnamed.nonzero().flatten())):
        k[r], v[r] = bad[n % 4], bad[(n + 1) % 4]
    # the column hidden from one row only: finite for the rows that see it, so its K may not be NaN
    kd.copy_(k)
    vd.copy_(v)
    out, ls = run_attn(ddt, batch, q, kd, vd, 0.125, ctas)
    clean(ddt)
    assert torch.isfinite(out).all()
    check_attn(out, ls, q, clean_k, clean_v, batch, 0.125)
    # a V row with NaN that one node sees: that node's rows are NaN, the others' are not
    r = named[int(batch.kv[0]) + 60]
    vd[r] = float("nan")
    out2, ls2 = run_attn(ddt, batch, q, kd, vd, 0.125, ctas)
    clean(ddt)
    assert torch.equal(ls2, ls)
    assert torch.isfinite(out2[0]).all() and torch.isfinite(out2[4]).all() and torch.isfinite(out2[6]).all()
    assert torch.isnan(out2[1:4]).all() and torch.isnan(out2[5]).all()
    o, _, bo, _ = ref.attention(q, clean_k, clean_v, batch, 0.125)
    assert ((out2[0].double().cpu() - o[0]).abs() <= bo[0]).all()


def test_attention_padded_batch_leaves_the_rest_alone(ddt):
    # a request without new tokens, and rows of q behind the last request
    batch = ref.Batch([(40, 3), (12, 0), (0, 0), (9, 5)], 31, "tree")
    q, k, v, kd, vd = attn_inputs(batch, 8, 4, 128, 14)
    pad = torch.cat([q, torch.full((6, 8, 128), float("nan"), dtype=torch.bfloat16)])
    for ctas in (0, 1, 5):
        out, ls = run_attn(ddt, batch, pad, kd, vd, 0.1, ctas)
        clean(ddt)
        check_attn(out[: batch.total_q], ls[: batch.total_q], q, k, v, batch, 0.1)
        assert (out[batch.total_q:] == 7).all() and (ls[batch.total_q:] == 7).all()


def test_attention_bad_offsets_latch_and_write_nothing(ddt):
    batch = ref.Batch([(40, 3), (30, 4)], 32, "tree")
    q, k, v, kd, vd = attn_inputs(batch, 4, 2, 64, 15)
    good = {n: getattr(batch, n).copy() for n in ("qo", "kv", "mask_indptr")}
    for field, index, value, bit in (("qo", 2, batch.total_q + 1, 0x1), ("qo", 1, -1, 0x1), ("kv", 2, batch.total_kv + 1, 0x2),
                                     ("kv", 1, 5000, 0x2), ("mask_indptr", 2, int(batch.mask_indptr[2]) + 1, 0x8),
                                     ("mask_indptr", 2, 10 ** 6, 0x8)):
        for n, a in good.items():
            setattr(batch, n, a.copy())
        getattr(batch, field)[index] = value
        out, ls = run_attn(ddt, batch, q, kd, vd, 0.1)
        torch.cuda.synchronize()
        st, bits = ddt.ddt_get_error()
        assert st == 5 and bits & bit, (field, bits)
        lo = 0 if index == 1 else 3   # the broken request's rows
        hi = batch.total_q
        assert (out[lo:hi][-1] == 7).all()


def test_attention_slot_outside_the_pool_latches(ddt):
    batch = ref.Batch([(40, 3)], 33, "tree")
    q, k, v, kd, vd = attn_inputs(batch, 4, 2, 64, 15)
    for slot in (-1, batch.rows, 2 ** 31 - 1):
        batch.slots[17] = slot
        run_attn(ddt, batch, q, kd, vd, 0.1)
        torch.cuda.synchronize()
        assert ddt.ddt_get_error() == (5, 0x4)


def test_attention_is_the_same_on_every_run_on_a_stream_and_in_a_graph(ddt):
    batch = ref.Batch([(500, 17), (30, 3)], 34, "tree")
    q, k, v, kd, vd = attn_inputs(batch, 16, 2, 128, 16)
    d = batch.device()
    qd = q.to(DEV)
    out, ls = torch.zeros_like(qd), torch.zeros(q.shape[:2], device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    # the longer bounds of a graph that is replayed for growing requests
    call = lambda stream=None: ddt.ddt_gqa_verify_attn(  # noqa: E731
        qd, kd, vd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], d["mask"], d["mask_indptr"], 0.1, out, ls,
        max_q_len=32, max_kv_len=1000, workspace=ws, stream=stream)
    call()
    clean(ddt)
    check_attn(out, ls, q, k, v, batch, 0.1)
    first = out.clone()
    for _ in range(5):
        out.zero_()
        call()
        assert torch.equal(out, first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    q2 = normal(q.shape, 99)
    qd.copy_(q2)
    g.replay()
    clean(ddt)
    check_attn(out, ls, q2, k, v, batch, 0.1)


def test_attention_rows_past_32_bit_offsets(ddt):
    # K and V rows behind 2^31 elements of their pools
    H, G, D = 16, 8, 128
    rows = (1 << 21) + 3000
    batch = ref.Batch([(300, 5)], 35, "tree", rows=rows, slot_lo=(1 << 21) + 5)
    small = ref.Batch([(300, 5)], 35, "tree", rows=rows, slot_lo=(1 << 21) + 5)
    lo = (1 << 21) + 5
    small.slots = small.slots - lo
    q = normal((batch.total_q, H, D), 1)
    k, v = normal((rows - lo, G, D), 2), normal((rows - lo, G, D), 3)
    kd = torch.zeros(rows, G, D, dtype=torch.bfloat16, device=DEV)
    vd = torch.zeros(rows, G, D, dtype=torch.bfloat16, device=DEV)
    kd[lo:], vd[lo:] = k.to(DEV), v.to(DEV)
    for ctas in (0, 1, 5):
        out, ls = run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
        clean(ddt)
        check_attn(out, ls, q, k, v, small, 0.1)


# ---------------------------------------------------------------- norm, rotation, append
def append_inputs(batch, H, G, D, R, norm, seed, far=None):
    N = batch.total_q
    qkv = normal((N, (H + 2 * G) * D), seed, 2.0)
    w = [(normal((D,), seed + i, 0.3) + 1.0).to(torch.bfloat16) if norm else None for i in (1, 2)]
    far = far or batch.max_kv + 1
    table = None
    if R:
        ang = np.arange(far)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
        table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    return qkv, w, table


def positions(batch, chain):
    return torch.from_numpy(np.concatenate(
        [p + (np.arange(t) if chain else np.array(dep, np.int64)) for (p, t), dep in zip(batch.lens, batch.depth)]
    ).astype(np.int64))


APPEND = [
    # heads, kv heads, dim, rope_dim, interleaved, norm, (prefix, new) per request, depth given
    (8, 2, 64, 64, False, True, [(21, 9)], True),
    (64, 8, 128, 128, False, True, [(4096, 1)], True),
    (40, 8, 128, 64, False, True, [(5, 17), (0, 1), (300, 33)], True),
    (5, 5, 128, 48, False, False, [(5, 3), (7, 0), (0, 0), (9, 4)], False),
    (12, 1, 64, 32, True, True, [(100, 128), (0, 128)], False),
    (16, 16, 128, 128, True, False, [(k, 1 + k % 3) for k in range(40)], True),
    (128, 8, 128, 0, False, True, [(3, 4)], True),
    (1, 1, 64, 16, False, False, [(0, 1)], False),
    (4, 2, 64, 64, False, True, [(2, 1)] * 1100, True),
]


def run_append(ddt, batch, qkv, w, table, H, G, D, interleaved, depth, pools, q_out=None, eps=1e-6):
    d = batch.device()
    x = qkv.to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([H * D, G * D, G * D], 1))
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    q_out = torch.full((qkv.shape[0], H, D), 7.0, dtype=torch.bfloat16, device=DEV) if q_out is None else q_out
    dep = None
    if depth:
        dep = torch.zeros(qkv.shape[0], dtype=torch.int32, device=DEV)
        dep[: batch.total_q] = d["depth"]
    ddt.ddt_gqa_norm_rope_append(q, k, v, dev(w[0]), dev(w[1]), eps, dev(table), dep, d["qo_indptr"], d["kv_indices"],
                                 d["kv_indptr"], q_out, pools[0], pools[1], interleaved=interleaved)
    return q_out


def check_append(batch, qkv, w, table, H, G, D, interleaved, depth, before, q_out, pools, eps=1e-6):
    pos = positions(batch, not depth)
    N = batch.total_q
    q, k, v = (t[:N].unflatten(1, (-1, D)) for t in qkv.split([H * D, G * D, G * D], 1))
    y, tol = ref.norm_rope(q, w[0], eps, table, pos, interleaved)
    assert ((q_out[:N].double().cpu() - y).abs() <= tol).all()
    want, tk = ref.norm_rope(k, w[1], eps, table, pos, interleaved)
    new = torch.cat([torch.from_numpy(batch.slots[batch.kv[b + 1] - t: batch.kv[b + 1]].astype(np.int64))
                     for b, (_, t) in enumerate(batch.lens)])
    kp, vp = pools[0].cpu(), pools[1].cpu()
    assert ((kp[new].double() - want).abs() <= tk).all()
    assert torch.equal(vp[new], v)
    rest = torch.ones(batch.rows, dtype=torch.bool)
    rest[new] = False
    assert torch.equal(kp[rest], before[0][rest]) and torch.equal(vp[rest], before[1][rest])


@pytest.mark.parametrize("H,G,D,R,il,norm,lens,depth", APPEND)
def test_append(ddt, H, G, D, R, il, norm, lens, depth):
    batch = ref.Batch(lens, 77 + H, "tree" if depth else "chain")
    qkv, w, table = append_inputs(batch, H, G, D, R, norm, 3 * H + D)
    before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
    pools = [t.to(DEV) for t in before]
    q_out = run_append(ddt, batch, qkv, w, table, H, G, D, il, depth, pools)
    clean(ddt)
    check_append(batch, qkv, w, table, H, G, D, il, depth, before, q_out, pools)


def test_append_one_norm_weight_and_zero_rows(ddt):
    # a row of zeros stays zero (eps keeps its norm finite); q normed, k not
    batch = ref.Batch([(3, 5)], 6, "tree")
    qkv, w, table = append_inputs(batch, 4, 2, 128, 128, True, 5)
    qkv[2] = 0
    w[1] = None
    before = normal((batch.rows, 2, 128), 1), normal((batch.rows, 2, 128), 2)
    pools = [t.to(DEV) for t in before]
    q_out = run_append(ddt, batch, qkv, w, table, 4, 2, 128, False, True, pools)
    clean(ddt)
    check_append(batch, qkv, w, table, 4, 2, 128, False, True, before, q_out, pools)
    assert (q_out[2] == 0).all()


def test_append_in_place_padded_and_strided_pool(ddt):
    H, G, D = 8, 2, 64
    batch = ref.Batch([(30, 4), (11, 2)], 7, "tree")
    qkv, w, table = append_inputs(batch, H, G, D, 64, True, 8)
    pad = torch.cat([qkv, torch.full((3, qkv.shape[1]), 5.0, dtype=torch.bfloat16)])
    d = batch.device()
    q = pad[:, : H * D].unflatten(1, (H, D)).contiguous().to(DEV)
    k, v = (t.unflatten(1, (G, D)).to(DEV) for t in pad[:, H * D:].split(G * D, 1))
    kv = normal((batch.rows, 2, G, D), 9).to(DEV)
    before = kv[:, 0].cpu(), kv[:, 1].cpu()
    dep = torch.zeros(len(pad), dtype=torch.int32, device=DEV)
    dep[: batch.total_q] = d["depth"]
    ddt.ddt_gqa_norm_rope_append(q, k, v, w[0].to(DEV), w[1].to(DEV), 1e-6, table.to(DEV), dep, d["qo_indptr"],
                                 d["kv_indices"], d["kv_indptr"], q, kv[:, 0], kv[:, 1])
    clean(ddt)
    check_append(batch, qkv, w, table, H, G, D, False, True, before, q, (kv[:, 0], kv[:, 1]))
    assert (q[batch.total_q:] == 5).all()


def test_append_device_checks(ddt):
    H, G, D = 4, 2, 64
    lens = [(6, 3), (4, 2)]
    for what, bit in (("slot", 0x4), ("position", 0x800), ("qo", 0x1), ("kv", 0x2)):
        batch = ref.Batch(lens, 12, "tree")
        qkv, w, table = append_inputs(batch, H, G, D, 64, True, 8, far=64)
        first = int(batch.slots[7])     # the first request's second token
        if what == "slot":
            batch.slots[7] = batch.rows
        elif what == "position":
            batch.depth[0][1] = -8
        elif what == "qo":
            batch.qo[0] = -4
        else:
            batch.kv[1], batch.kv[2] = 13, batch.total_kv + 5
        before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
        pools = [t.to(DEV) for t in before]
        q_out = run_append(ddt, batch, qkv, w, table, H, G, D, False, True, pools)
        torch.cuda.synchronize()
        st, bits = ddt.ddt_get_error()
        assert st == 5 and bits == bit, (what, bits)
        if what in ("slot", "position"):
            assert torch.equal(pools[0][first].cpu(), before[0][first])
            assert (q_out[1] == 7).all() == (what == "position")


# ---------------------------------------------------------------- cache rows
def slab(pools, rows, width, seed, gap=0):
    """[pools, rows, width] with `gap` elements between pools."""
    flat = normal((pools, rows * width + gap), seed).to(DEV)
    return flat[:, : rows * width].view(pools, rows, width) if gap == 0 else flat[:, : rows * width].unflatten(1, (rows, width))


@pytest.mark.parametrize("pools,rows,width,n,gap", [
    (1, 100, 576, 33, 0), (3, 50, 128, 25, 64), (70, 40, 8, 17, 0), (2, 400, 1288, 200, 8), (2, 9, 20000, 4, 0),
    (1, 2, 64, 1, 0), (5, 3000, 64, 1500, 0)])
def test_copy(ddt, pools, rows, width, n, gap):
    g = torch.Generator().manual_seed(rows)
    order = torch.randperm(rows, generator=g)
    src, dst = order[:n].clone(), order[n: 2 * n]
    src[n // 2:] = src[: n - n // 2].clone()    # the same source more than once
    p = slab(pools, rows, width, 3, gap)
    want = p.cpu()
    want[:, dst] = want[:, src]
    ddt.ddt_cache_copy(p, p, src.int().to(DEV), dst.int().to(DEV))
    clean(ddt)
    assert torch.equal(p.cpu(), want)
    # into another slab with other rows, a row onto its own number among them
    other = slab(pools, rows + 5, width, 4)
    want2 = other.cpu()
    want2[:, dst + 5] = want[:, src]
    ddt.ddt_cache_copy(p, other, src.int().to(DEV), (dst + 5).int().to(DEV))
    same = torch.arange(rows, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_copy(p, p, same, same)
    clean(ddt)
    assert torch.equal(other.cpu(), want2) and torch.equal(p.cpu(), want)


def test_copy_skips_slots_outside(ddt):
    p = slab(2, 20, 64, 1)
    want = p.cpu()
    want[:, 3] = want[:, 4]
    src = torch.tensor([4, -1, 5, 20], dtype=torch.int32, device=DEV)
    dst = torch.tensor([3, 1, 20, 2], dtype=torch.int32, device=DEV)
    ddt.ddt_cache_copy(p, p, src, dst)
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (5, 0x4)
    assert torch.equal(p.cpu(), want)


def commit_inputs(batch, seed):
    rng = np.random.default_rng(seed)
    lens, nodes = [], []
    for par in batch.parent:
        path, n = [], int(rng.integers(0, len(par))) if par else -1
        while n >= 0:
            path.append(n)
            n = par[n]
        lens.append(len(path))
        nodes.append(path[::-1] + [-1] * (8 - len(path)))
    return np.array(lens, np.int32), np.array(nodes, np.int32)


@pytest.mark.parametrize("pools,width,lens", [
    (1, 576, [(20, 33)]), (6, 128, [(0, 9), (5, 128), (3, 1), (2, 0)]), (64, 1024, [(k % 5, 1 + 3 * k % 40) for k in range(40)]),
    (3, 3000, [(1, 20), (2, 60)])])
def test_commit(ddt, pools, width, lens):
    batch = ref.Batch(lens, 50 + pools, "tree")
    alen, nodes = commit_inputs(batch, pools)
    p = slab(pools, batch.rows, width, 5)
    come = torch.arange(batch.rows)
    for b, n in enumerate(alen):
        root = int(batch.kv[b + 1] - batch.T[b])
        for k in range(n):
            come[batch.slots[root + k]] = int(batch.slots[root + nodes[b][k]])
    want = p.cpu()[:, come]
    d = batch.device()
    new_len = torch.empty(batch.B, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_commit(p, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], torch.from_numpy(alen).to(DEV),
                         torch.from_numpy(nodes).to(DEV), 7, new_len)
    clean(ddt)
    assert torch.equal(p.cpu(), want)
    assert new_len.cpu().tolist() == (batch.P + alen).tolist()


def test_commit_of_one_latent_pool_equals_commit_kv(ddt):
    batch = ref.Batch([(20, 33), (0, 12)], 51, "tree")
    alen, nodes = commit_inputs(batch, 3)
    a = slab(1, batch.rows, 576, 5)
    b = a[0].clone()
    d = batch.device()
    al, nd = torch.from_numpy(alen).to(DEV), torch.from_numpy(nodes).to(DEV)
    ddt.ddt_cache_commit(a, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], al, nd, 7)
    ddt.ddt_commit_kv(b, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], al, nd, 7)
    clean(ddt)
    assert torch.equal(a[0], b)


@pytest.mark.parametrize("alen,nodes,bit", [
    (3, [0, 2, 2], 0x200), (3, [1, 2, 3], 0x200), (2, [0, 9], 0x200), (9, [0, 1, 2], 0x200), (0, [0], 0x200),
    (2, [0, 4], 0x4)])
def test_commit_refuses_what_is_not_a_path(ddt, alen, nodes, bit):
    batch = ref.Batch([(4, 9), (3, 9)], 52, "tree")
    if bit == 0x4:
        batch.slots[4 + 4] = batch.rows   # the first request's node 4
    p = slab(2, batch.rows, 128, 5)
    want = p.cpu()
    d = batch.device()
    al = torch.tensor([alen, 1], dtype=torch.int32, device=DEV)
    nd = torch.tensor([nodes + [-1] * (8 - len(nodes)), [0] + [-1] * 7], dtype=torch.int32, device=DEV)
    new_len = torch.full((2,), -5, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_commit(p, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], al, nd, 7, new_len)
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (5, bit)
    assert torch.equal(p.cpu(), want) and new_len.cpu().tolist() == [-5, 4]


@pytest.mark.parametrize("pools,rows,width,live,shared", [
    (1, 4096, 576, 1500, 0), (3, 100, 64, 50, 30), (2, 33, 8, 33, 0), (2, 64, 8, 1, 0), (1, 1, 16, 1, 5), (4, 70000, 16, 35000, 9000),
    (2, 32, 8, 32, 3), (2, 1000, 1288, 999, 0), (1, 2000, 8, 0, 0), (2, 40000, 8, 39000, 0)])
def test_compact(ddt, pools, rows, width, live, shared):
    g = torch.Generator().manual_seed(rows + live)
    named = torch.randperm(rows, generator=g)[:live]
    slots = torch.cat([named, named[torch.randint(0, max(live, 1), (shared if live else 0,), generator=g)]]).int()
    want_slots, n, come = ref.compact(slots.tolist(), rows)
    p = slab(pools, rows, width, 6)
    before = p.cpu()
    want = before[:, torch.tensor(come)]
    idx = slots.to(DEV)
    new, cnt = torch.empty_like(idx), torch.full((1,), -1, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_compact(p, idx, new, cnt)
    clean(ddt)
    assert cnt.item() == n == len(set(slots.tolist()))
    assert new.cpu().tolist() == want_slots and torch.equal(idx.cpu(), slots)
    assert torch.equal(p.cpu(), want)
    # every slot still names its values, all below n; again, in place: nothing more to do
    if live:
        assert int(new.max()) < n and torch.equal(p.cpu()[:, new.cpu().long()], before[:, slots.long()])
    again = new.clone()
    ws = torch.empty(ddt.ddt_cache_compact_workspace_size(rows), dtype=torch.uint8, device=DEV)
    ddt.ddt_cache_compact(p, again, again, cnt, workspace=ws)
    clean(ddt)
    assert torch.equal(again, new) and cnt.item() == n and torch.equal(p.cpu(), want)


def test_compact_keeps_slots_outside_and_latches(ddt):
    p = slab(1, 50, 64, 7)
    slots = torch.tensor([40, -3, 7, 50, 2 ** 31 - 1, 40], dtype=torch.int32)
    want_slots, n, come = ref.compact(slots.tolist(), 50)
    want = p.cpu()[:, torch.tensor(come)]
    new, cnt = torch.empty(6, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_compact(p, slots.to(DEV), new, cnt)
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (5, 0x4)
    assert cnt.item() == n == 2 and new.cpu().tolist() == want_slots == [1, -3, 0, 50, 2 ** 31 - 1, 1]
    assert torch.equal(p.cpu(), want)


def test_cache_calls_capture_and_replay(ddt):
    rows = 500
    p = slab(2, rows, 128, 8)
    first = p.cpu()
    g = torch.Generator().manual_seed(1)
    idx = torch.randperm(rows, generator=g)[:200].int().to(DEV)
    new, cnt = torch.empty_like(idx), torch.empty(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(ddt.ddt_cache_compact_workspace_size(rows), dtype=torch.uint8, device=DEV)
    src, dst = torch.arange(0, 10, dtype=torch.int32, device=DEV), torch.arange(300, 310, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ddt.ddt_cache_compact(p, idx, new, cnt, workspace=ws)
        ddt.ddt_cache_copy(p, p, src, dst)
    for seed in (2, 3):
        g.manual_seed(seed)
        slots = torch.randperm(rows, generator=g)[:200].int()
        idx.copy_(slots)
        p.copy_(first)
        graph.replay()
        clean(ddt)
        want_slots, n, come = ref.compact(slots.tolist(), rows)
        want = first[:, torch.tensor(come)]
        want[:, 300:310] = want[:, 0:10]
        assert new.cpu().tolist() == want_slots and cnt.item() == n and torch.equal(p.cpu(), want)
