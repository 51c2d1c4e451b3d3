"""The grouped-query layer and the cache-row calls where the documentation
allows what the other tests do not call: small workspaces, large batches, the
largest head counts, several streams at once, shared workspaces, values at the
ends of the type, indices named twice."""
import numpy as np
import pytest
import torch

from tests import _gqa_ref as ref
from tests import test_gqa_gpu as base

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ddt = base.ddt   # the fixture
clean, normal = base.clean, base.normal


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("H,G,D", [(16, 4, 128), (32, 1, 64)])
def test_attention_within_any_workspace(ddt, H, G, D):
    # num_ctas = 0 takes what the workspace holds, down to none; a given count is refused below its size
    batch = ref.Batch([(600, 9), (200, 5)], 61, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 62)
    size = lambda n: ddt.ddt_gqa_verify_attn_workspace_size(2, H, G, D, batch.max_q, n)  # noqa: E731
    for nbytes in (0, 256, size(1) - 256, size(1), size(7), size(7) + 255, size(512)):
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=DEV)[:nbytes]
        out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, 0, workspace=ws)
        clean(ddt)
        base.check_attn(out, ls, q, k, v, batch, 0.1)
    with pytest.raises(ddt.DDTError):
        base.run_attn(ddt, batch, q, kd, vd, 0.1, 7, workspace=torch.empty(size(7) - 256, dtype=torch.uint8, device=DEV))
    clean(ddt)


@pytest.mark.parametrize("B,T,H,G,D", [(256, 1, 4, 2, 64), (257, 1, 4, 2, 64), (300, 3, 2, 1, 128), (256, 2, 128, 1, 64)])
def test_attention_of_many_requests(ddt, B, T, H, G, D):
    # up to 256 requests are dealt, more have a CTA per request and K/V head
    rng = np.random.default_rng(B)
    lens = [(int(rng.integers(0, 40)), T) for _ in range(B - 2)] + [(290, T), (0, T)]
    batch = ref.Batch(lens, 63, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 64)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5)
    clean(ddt)
    base.check_attn(out, ls, q, k, v, batch, D ** -0.5)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_of_the_most_rows(ddt, D):
    # 128 heads on one K/V head and 128 new tokens: 64 tile groups
    batch = ref.Batch([(37, 128)], 65, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, 128, 1, D, 66)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5)
    again, _ = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5, 300)
    clean(ddt)
    # every 37th token against the 64-bit form, the rest against the other split's result
    some = list(range(0, 128, 37))
    part = ref.Batch([(37, 128)], 65, "tree")
    part.vis[0] = part.vis[0].copy()
    keep = np.zeros(128, bool)
    keep[some] = True
    part.vis[0][~keep] = False
    o, l, bo, bl = ref.attention(q, k, v, part, D ** -0.5)
    assert ((out.double().cpu() - o).abs() <= bo)[some].all()
    assert ((ls.double().cpu() - l).abs() <= bl)[some].all()
    # two results within their bounds differ by at most both: 2 (2 h p|v| + h |out|), p|v| <= max |v|
    top = float(v.abs().max())
    assert float((out - again).abs().max()) <= 2 * 3 * 2.0 ** -8 * top * 1.05


@pytest.mark.parametrize("H,T,lone", [(4, 4, False), (64, 3, False), (64, 5, True)])
@pytest.mark.parametrize("ctas", [1, 3, 0])
def test_attention_reference_moves(ddt, H, T, lone, ctas):
    """Scores that rise by thousands along the cache, so that the reference moves many times: in
    both halves of a block, in both outputs of a lone tile, and in late shares.  (64 heads on one
    K/V head: two tiles of rows; 5 x 64 rows leave a third, lone one.)"""
    batch = ref.Batch([(1100, T)], 67, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, 1, 128, 68)
    steps = torch.from_numpy(np.repeat(np.arange(batch.total_kv // 37 + 1), 37)[: batch.total_kv].astype(np.float32) * 2.0)
    at = torch.from_numpy(batch.slots.astype(np.int64))
    k[at, 0, 0] = steps.to(torch.bfloat16)       # one value that every query weighs alike
    q[:, :, 0] = 32.0
    kd.copy_(k)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 1.0, ctas)
    clean(ddt)
    base.check_attn(out, ls, q, k, v, batch, 1.0)
    # the same falling: the reference stays where the first columns put it
    k[at, 0, 0] = steps.flip(0).to(torch.bfloat16)
    kd.copy_(k)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 1.0, ctas)
    clean(ddt)
    base.check_attn(out, ls, q, k, v, batch, 1.0)


@pytest.mark.parametrize("H,T", [(8, 3), (64, 5)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("ctas", [1, 4, 0])
def test_attention_values_that_are_seen_come_out(ddt, H, T, bad, ctas):
    # a value that is NaN or infinite in a seen V row is in the output of the rows that see it, in
    # its place alone; a NaN in a seen K row makes the whole row NaN
    batch = ref.Batch([(500, T)], 71, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, 2, 64, 72, q_scale=0.5)
    col = 500 + T - 1                       # the last node: it sees itself, no other node does
    row = int(batch.slots[col])
    vd[row, 1, 5] = bad
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    clean(ddt)
    hit = torch.zeros(out.shape, dtype=torch.bool)
    hit[T - 1, H // 2:, 5] = True
    got = out.cpu()
    want = torch.full((H // 2,), bad, dtype=torch.bfloat16)
    assert torch.equal(got[T - 1, H // 2:, 5].isnan(), want.isnan())
    if bad == bad:
        assert torch.equal(got[T - 1, H // 2:, 5], want)
    o, l, bo, bl = ref.attention(q, k, v, batch, 0.1)
    assert ((got.double() - o).abs() <= bo)[~hit].all() and ((ls.double().cpu() - l).abs() <= bl).all()
    kd[row, 0, 3] = float("nan")
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    clean(ddt)
    hit[T - 1, : H // 2] = True
    assert out.cpu()[T - 1, : H // 2].isnan().all() and ls.cpu()[T - 1, : H // 2].isnan().all()
    assert ((out.double().cpu() - o).abs() <= bo)[~hit].all()


@pytest.mark.parametrize("H,G,T,D", [(8, 2, 5, 64), (64, 2, 4, 64), (64, 2, 5, 64), (8, 1, 17, 128), (16, 2, 33, 128)])
@pytest.mark.parametrize("ctas", [1, 4, 0])
def test_attention_of_a_query_that_is_nan(ddt, H, G, T, D, ctas):
    # its row is NaN whole, no other one is; in tiles, lone tiles and the few rows behind a tile
    batch = ref.Batch([(700, T)], 101, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 102, q_scale=0.5)
    o, l, bo, bl = ref.attention(q, k, v, batch, 0.1)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool)
    hit[0, 0] = hit[T - 1, H - 1] = hit[T // 2, H // 2] = True
    q[hit] = float("nan")
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    clean(ddt)
    assert out.cpu()[hit].isnan().all() and ls.cpu()[hit].isnan().all()
    assert ((out.double().cpu() - o).abs() <= bo)[~hit].all() and ((ls.double().cpu() - l).abs() <= bl)[~hit].all()


@pytest.mark.parametrize("H,G,D,lens", [
    # shapes that are dealt or not, with one tile of rows at a time or two
    (64, 8, 128, [(300, 33)] * 6), (64, 8, 128, [(1500, 33)]), (32, 4, 128, [(600, 32)] * 16), (32, 4, 64, [(500, 17)] * 24),
    (64, 8, 64, [(2500, 17), (100, 33)]), (128, 8, 64, [(400, 33), (100, 20), (700, 1)]), (16, 16, 128, [(300, 9)] * 10),
    (32, 2, 128, [(1300, 16), (40, 5), (900, 16)]),
])
@pytest.mark.parametrize("room", ["none", "some", "all"])
def test_attention_chooses_its_way(ddt, H, G, D, lens, room):
    batch = ref.Batch(lens, 109 + H, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 110)
    n = ddt.ddt_gqa_verify_attn_num_ctas(batch.B, H, G, batch.max_q, batch.max_kv)
    assert n > 0
    n = {"none": 0, "some": 9, "all": n}[room]
    nbytes = ddt.ddt_gqa_verify_attn_workspace_size(batch.B, H, G, D, batch.max_q, n)
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=DEV)[:nbytes]
    out, ls = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5, workspace=ws)
    clean(ddt)
    base.check_attn(out, ls, q, k, v, batch, D ** -0.5)


FEW = [
    # heads, kv heads, dim, (prefix, new tokens) per request: 1 to 8 rows behind one or two tiles
    (8, 1, 128, [(300, 17), (40, 33), (1000, 33)]), (16, 2, 64, [(500, 33), (0, 17), (129, 65), (600, 3)]),
    (1, 1, 128, [(400, 128)]), (4, 1, 64, [(700, 33), (511, 65), (200, 34), (60, 97)]), (43, 1, 128, [(300, 3), (20, 6)]),
    (43, 1, 64, [(290, 6)]), (128, 1, 128, [(270, 1), (10, 2)]), (5, 1, 128, [(257, 26), (400, 52), (300, 27)]),
]


@pytest.mark.parametrize("H,G,D,lens", FEW)
@pytest.mark.parametrize("mask", ["tree", "random"])
@pytest.mark.parametrize("ctas", [0, 1, 2, 5, 40])
def test_attention_of_a_few_rows_behind_a_tile(ddt, H, G, D, lens, mask, ctas):
    batch = ref.Batch(lens, 103 + H, mask)
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 104)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5, ctas)
    clean(ddt)
    base.check_attn(out, ls, q, k, v, batch, D ** -0.5)


@pytest.mark.parametrize("ctas", [0, 3])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_of_a_few_rows_with_unseen_nan_and_rising_scores(ddt, D, ctas):
    batch = ref.Batch([(900, 33)], 105, "tree")
    H = 8
    q, k, v, kd, vd = base.attn_inputs(batch, H, 1, D, 106)
    steps = torch.from_numpy(np.repeat(np.arange(batch.total_kv // 37 + 1), 37)[: batch.total_kv].astype(np.float32) * 2.0)
    at = torch.from_numpy(batch.slots.astype(np.int64))
    k[at, 0, 0] = steps.to(torch.bfloat16)
    q[:, :, 0] = 32.0
    kd.copy_(k)
    # a node that the last one does not see holds anything
    hidden = [n for n in range(33) if not batch.vis[0][32, 900 + n]]
    for n, bad in zip(hidden, (float("nan"), float("inf"), float("-inf"))):
        others = [i for i in range(33) if batch.vis[0][i, 900 + n]]
        kd[int(batch.slots[900 + n])] = bad
        vd[int(batch.slots[900 + n])] = bad
        batch.vis[0][others] = False     # rows that see it are not compared
    keep = torch.from_numpy(batch.vis[0].any(1))
    assert keep[32] and int(keep.sum()) > 3
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 1.0, ctas)
    clean(ddt)
    o, l, bo, bl = ref.attention(q, k, v, batch, 1.0)
    assert ((out.double().cpu() - o).abs() <= bo)[keep].all() and ((ls.double().cpu() - l).abs() <= bl)[keep].all()


def test_attention_on_two_streams_at_once(ddt):
    batches = [ref.Batch([(3000, 9)], 73, "tree"), ref.Batch([(2500, 33)], 74, "tree")]
    made = [base.attn_inputs(b, 16, 2, 128, 75 + i) for i, b in enumerate(batches)]
    calls, outs, firsts = [], [], []
    for b, (q, k, v, kd, vd) in zip(batches, made):
        d = {n: t for n, t in b.device().items()}
        n = ddt.ddt_gqa_verify_attn_num_ctas(1, 16, 2, b.max_q, b.max_kv)
        ws = torch.empty(ddt.ddt_gqa_verify_attn_workspace_size(1, 16, 2, 128, b.max_q, n), dtype=torch.uint8, device=DEV)
        qd, out = q.to(DEV), torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        calls.append(lambda s, b=b, d=d, ws=ws, qd=qd, out=out, kd=kd, vd=vd: ddt.ddt_gqa_verify_attn(
            qd, kd, vd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], d["mask"], d["mask_indptr"], 0.1, out,
            max_q_len=b.max_q, max_kv_len=b.max_kv, workspace=ws, stream=s))
        outs.append(out)
        calls[-1](None)
        torch.cuda.synchronize()
        base.check_attn(out, None, q, k, v, b, 0.1)
        firsts.append(out.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(s)
    clean(ddt)
    assert all(torch.equal(o, f) for o, f in zip(outs, firsts))


def test_attention_without_a_workspace_on_another_stream(ddt):
    # the call's own workspace belongs to the call's stream: what the current stream allocates and
    # writes meanwhile is other memory
    batch = ref.Batch([(4000, 16)], 77, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, 32, 2, 128, 78)
    d, qd = batch.device(), q.to(DEV)
    s = torch.cuda.Stream()
    outs = [torch.empty(q.shape, dtype=torch.bfloat16, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    for out in outs:
        ddt.ddt_gqa_verify_attn(qd, kd, vd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], d["mask"], d["mask_indptr"],
                                0.1, out, max_q_len=16, max_kv_len=4016, stream=s)
        torch.full((8 << 20,), 255, dtype=torch.uint8, device=DEV)
    clean(ddt)
    base.check_attn(outs[0], None, q, k, v, batch, 0.1)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_two_graphs_share_a_workspace_in_turn(ddt):
    batch = ref.Batch([(900, 9), (50, 20)], 79, "tree")
    d = batch.device()
    n = ddt.ddt_gqa_verify_attn_num_ctas(2, 32, 2, batch.max_q, batch.max_kv)
    ws = torch.empty(ddt.ddt_gqa_verify_attn_workspace_size(2, 32, 2, 128, batch.max_q, n), dtype=torch.uint8, device=DEV)
    graphs, made, outs = [], [], []
    for i in range(2):
        q, k, v, kd, vd = base.attn_inputs(batch, 32, 2, 128, 80 + 5 * i)
        qd, out = q.to(DEV), torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            ddt.ddt_gqa_verify_attn(qd, kd, vd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], d["mask"],
                                    d["mask_indptr"], 0.1, out, max_q_len=batch.max_q, max_kv_len=batch.max_kv, workspace=ws)
        graphs.append(g)
        made.append((q, k, v, kd, vd, qd))
        outs.append(out)
    for _ in range(3):
        for g in graphs:
            g.replay()
    clean(ddt)
    for (q, k, v, *_), out in zip(made, outs):
        base.check_attn(out, None, q, k, v, batch, 0.1)


@pytest.mark.parametrize("H,T", [(4, 9), (64, 3)])
def test_attention_ignores_bits_past_the_last_column(ddt, H, T):
    # kv_len 309, 70, 31: the last word's bits past it are set, and the slots there are another request's
    batch = ref.Batch([(309 - T, T), (70 - T, T), (31 - T, T)], 85, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, 1, 64, 86)
    for b in range(3):
        W, N = -(-int(batch.P[b] + T) // 32), int(batch.P[b] + T)
        lo = int(batch.mask_indptr[b])
        batch.words[lo + W - 1: lo + T * W: W] |= np.uint32((0xffffffff << (N % 32)) & 0xffffffff)
    for ctas in (0, 1, 4):
        out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
        clean(ddt)
        base.check_attn(out, ls, q, k, v, batch, 0.1)


def test_attention_reads_a_slot_named_twice(ddt):
    # two columns of one request, and two requests' prefixes, on the same rows
    batch = ref.Batch([(300, 4), (300, 3)], 83, "tree")
    batch.slots[batch.kv[1]: batch.kv[1] + 300] = batch.slots[:300]
    batch.slots[10:20] = batch.slots[30:40]
    q, k, v, kd, vd = base.attn_inputs(batch, 8, 2, 64, 84)
    for ctas in (0, 5):
        out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
        clean(ddt)
        base.check_attn(out, ls, q, k, v, batch, 0.1)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("B", [1, 30, 31, 32, 33, 70])
def test_append_finds_its_request(ddt, B):
    # 31 requests are looked up in one round, more by a search; empty ones at both ends and between
    lens = [(3 * k, 0 if k % 4 == 0 else 1 + k % 3) for k in range(B)] if B > 1 else [(5, 2)]
    batch = ref.Batch(lens, 85, "tree")
    qkv, w, table = base.append_inputs(batch, 4, 2, 64, 64, True, 86)
    before = normal((batch.rows, 2, 64), 1), normal((batch.rows, 2, 64), 2)
    pools = [t.to(DEV) for t in before]
    q_out = base.run_append(ddt, batch, qkv, w, table, 4, 2, 64, False, True, pools)
    clean(ddt)
    base.check_append(batch, qkv, w, table, 4, 2, 64, False, True, before, q_out, pools)


def test_append_of_tiny_values_and_nan(ddt):
    # squares that underflow leave the norm to eps; a NaN stays in its own row
    batch = ref.Batch([(4, 3)], 87, "tree")
    H, G, D = 2, 1, 64
    qkv, w, table = base.append_inputs(batch, H, G, D, 0, True, 88)
    qkv[0, :D], qkv[1, :D], qkv[2, :D] = 2.0 ** 60, 2.0 ** -126, float("nan")
    before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
    pools = [t.to(DEV) for t in before]
    q_out = base.run_append(ddt, batch, qkv, w, table, H, G, D, False, True, pools).cpu()
    clean(ddt)
    assert q_out[2, 0].isnan().all()
    y, tol = ref.norm_rope(qkv[:, : H * D].unflatten(1, (H, D)), w[0], 1e-6, None, None, False)
    ok = torch.ones(3, H, dtype=torch.bool)
    ok[2, 0] = False
    assert ((q_out.double() - y).abs() <= tol)[ok].all()


def test_append_and_attention_follow_each_other_at_once(ddt):
    """Each kernel may start before the one ahead has ended; what it reads has to be complete all
    the same: the rows just appended, the mask just built, the q just rotated."""
    H, G, D = 8, 2, 128
    batch = ref.Batch([(700, 9), (20, 5), (333, 16)], 89, "tree")
    d = batch.device()
    qkv, w, table = base.append_inputs(batch, H, G, D, 128, True, 90)
    wd, td = [t.to(DEV) for t in w], table.to(DEV)
    kd, vd = normal((batch.rows, G, D), 1).to(DEV), normal((batch.rows, G, D), 2).to(DEV)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.to(DEV).split([H * D, G * D, G * D], 1))
    mask = torch.zeros_like(d["mask"])
    outs = []
    for wait in (True, False, False, False):
        kp, vp, qo, out = kd.clone(), vd.clone(), torch.zeros_like(q).contiguous(), torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
        parent = torch.from_numpy(np.concatenate(batch.parent).astype(np.int32)).to(DEV)
        prefix = torch.from_numpy(batch.P.astype(np.int32)).to(DEV)
        mask.zero_()
        torch.cuda.synchronize()
        ddt.ddt_compile_visibility(parent, d["qo_indptr"], prefix, d["mask_indptr"], mask)
        if wait:
            torch.cuda.synchronize()
        ddt.ddt_gqa_norm_rope_append(q, k, v, wd[0], wd[1], 1e-6, td, d["depth"], d["qo_indptr"], d["kv_indices"],
                                     d["kv_indptr"], qo, kp, vp)
        if wait:
            torch.cuda.synchronize()
        ddt.ddt_gqa_verify_attn(qo, kp, vp, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], mask, d["mask_indptr"],
                                0.1, out, max_q_len=batch.max_q, max_kv_len=batch.max_kv)
        outs.append(out)
    clean(ddt)
    assert torch.equal(mask, d["mask"])
    assert all(torch.equal(o, outs[0]) for o in outs)


# ---------------------------------------------------------------- cache rows
def test_copy_of_one_row_of_many_bytes_and_many_pools(ddt):
    p = base.slab(1, 3, 1 << 20, 91)        # rows of 2 MB
    want = p.cpu()
    want[:, 2] = want[:, 0]
    ddt.ddt_cache_copy(p, p, torch.tensor([0], dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV))
    clean(ddt)
    assert torch.equal(p.cpu(), want)
    p = base.slab(70000, 2, 8, 92)          # more pools than a grid has rows
    want = p.cpu()
    want[:, 1] = want[:, 0]
    ddt.ddt_cache_copy(p, p, torch.tensor([0], dtype=torch.int32, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV))
    clean(ddt)
    assert torch.equal(p.cpu(), want)


def test_commit_and_compact_of_many_pools(ddt):
    batch = ref.Batch([(2, 9), (0, 4)], 93, "tree")
    alen, nodes = base.commit_inputs(batch, 5)
    p = base.slab(66000, batch.rows, 8, 94)
    come = torch.arange(batch.rows)
    for b, n in enumerate(alen):
        root = int(batch.kv[b + 1] - batch.T[b])
        for k in range(n):
            come[batch.slots[root + k]] = int(batch.slots[root + nodes[b][k]])
    want = p.cpu()[:, come]
    d = batch.device()
    ddt.ddt_cache_commit(p, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], torch.from_numpy(alen).to(DEV),
                         torch.from_numpy(nodes).to(DEV), 7)
    clean(ddt)
    assert torch.equal(p.cpu(), want)
    slots = d["kv_indices"][: 9].clone()
    want_slots, n, come = ref.compact(slots.cpu().tolist(), batch.rows)
    live = torch.empty(1, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_compact(p, slots, slots, live)
    clean(ddt)
    assert slots.cpu().tolist() == want_slots and live.item() == n
    assert torch.equal(p.cpu(), want[:, torch.tensor(come)])


def test_compact_of_nothing_and_of_everything(ddt):
    for rows in (1, 31, 32, 33, 1024 * 32, 1024 * 32 + 1):
        p = base.slab(1, rows, 8, 95)
        before = p.cpu()
        live = torch.full((1,), -1, dtype=torch.int32, device=DEV)
        none = torch.empty(0, dtype=torch.int32, device=DEV)
        ddt.ddt_cache_compact(p, none, none, live)
        clean(ddt)
        assert live.item() == 0 and torch.equal(p.cpu(), before)
        every = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device=DEV)
        new = torch.empty_like(every)
        ddt.ddt_cache_compact(p, every, new, live)
        clean(ddt)
        assert live.item() == rows and torch.equal(new, every) and torch.equal(p.cpu(), before)
        last = torch.tensor([rows - 1], dtype=torch.int32, device=DEV)     # one row, the last
        ddt.ddt_cache_compact(p, last, last, live)
        clean(ddt)
        assert live.item() == 1 and last.item() == 0 and torch.equal(p.cpu()[:, 0], before[:, rows - 1])


def test_compact_of_the_most_rows(ddt):
    rows = 1 << 24
    p = base.slab(1, 16, 8, 96)[0].repeat(rows // 16, 1)[None]
    p[0, :, 0] = (torch.arange(rows, device=DEV) % 256).to(torch.bfloat16)
    idx = torch.arange(rows - 5, 3, -7, dtype=torch.int32, device=DEV)
    before = p.clone()
    new, live = torch.empty_like(idx), torch.empty(1, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_compact(p, idx, new, live)
    clean(ddt)
    n = idx.numel()
    assert live.item() == n and new.sort().values.equal(torch.arange(n, dtype=torch.int32, device=DEV))
    assert torch.equal(p[0, new.long()], before[0, idx.long()])
    with pytest.raises(ddt.DDTError):
        ddt.ddt_cache_compact(torch.empty(1, rows + 1, 8, dtype=torch.bfloat16, device=DEV), idx, new, live)


def test_cache_calls_on_another_stream(ddt):
    rows = 4000
    p = base.slab(4, rows, 512, 97)
    before = p.cpu()
    idx = torch.randperm(rows, generator=torch.Generator().manual_seed(3))[:1500].int()
    slots, live = idx.to(DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    src, dst = torch.arange(1500, 1600, dtype=torch.int32, device=DEV), torch.arange(3000, 3100, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ddt.ddt_cache_compact(p, slots, slots, live, stream=s)
    torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)     # on the current stream
    ddt.ddt_cache_copy(p, p, src, dst, stream=s)
    clean(ddt)
    want_slots, n, come = ref.compact(idx.tolist(), rows)
    want = before[:, torch.tensor(come)]
    want[:, 3000:3100] = want[:, 1500:1600]
    assert slots.cpu().tolist() == want_slots and torch.equal(p.cpu(), want)
