"""Chunk attention on the GPU, against a plain 64-bit form (tests/_chunk_ref.py,
which also derives the tolerances)."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref

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


def inputs(c, H, G, D, seed, q_scale=1.5):
    return normal((c.total_q, H, D), seed, q_scale), normal((c.rows, G, D), seed + 1), normal((c.rows, G, D), seed + 2)


def slopes_of(H):
    return 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H)


def run(ddt, c, q, k, v, scale, cap=0.0, slopes=None, window=0, full=None, lse=True, **kw):
    d = c.device()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV) if lse else None
    ddt.ddt_gqa_chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), d["kv_indices"], d["kv_indptr"], d["qo_indptr"], scale, out, ls,
                           max_q_len=c.max_q, max_kv_len=c.max_kv, score_cap=cap,
                           slopes=None if slopes is None else slopes.to(DEV), window=window,
                           full_len=None if full is None else torch.tensor(full, dtype=torch.int32, device=DEV), **kw)
    return out, ls


def check(out, ls, want):
    o, l, bo, bl = want
    err = (out.double().cpu() - o).abs() - bo
    assert float(err.max()) <= 0, f"out over its bound by {float(err.max())}"
    if ls is not None:
        err = (ls.double().cpu() - l).abs() - bl
        assert float(err.max()) <= 0, f"lse over its bound by {float(err.max())}"


CASES = [
    # heads, kv heads, dim, (cached, new) per request, cap, slopes, window, full, page
    (8, 2, 64, [(21, 1)], 0.0, False, 0, None, 1),
    (8, 2, 128, [(21, 9)], 0.0, False, 0, None, 1),
    (5, 5, 128, [(0, 1), (1, 1), (63, 1), (64, 1), (127, 1), (200, 1)], 30.0, False, 0, None, 1),
    (16, 16, 64, [(62, 1), (63, 2), (61, 3), (0, 7)], 0.0, True, 0, None, 16),
    (8, 1, 128, [(0, 300)], 0.0, False, 0, None, 64),
    (8, 1, 64, [(0, 300), (5, 0), (130, 65)], 0.0, False, 0, None, 16),
    (16, 2, 128, [(700, 33), (0, 1), (64, 200)], 0.0, False, 100, None, 1),
    (12, 1, 128, [(130, 130), (64, 11)], 20.0, True, 0, None, 64),
    (40, 8, 128, [(500, 150), (3, 17), (250, 1)], 50.0, False, 64, [40, 3, 0], 1),
    (28, 4, 64, [(95, 140), (600, 1), (0, 64)], 0.0, True, 200, [7, 64, 60], 16),
    (4, 2, 128, [(10, 129)], 0.0, False, 1, None, 1),
    (4, 1, 128, [(300, 40), (0, 200)], 0.0, True, 33, [400, 128], 1),
    (64, 1, 64, [(70, 5), (10, 2)], 0.0, False, 0, None, 1),
    (128, 1, 128, [(40, 3)], 15.0, False, 0, None, 64),
    (2, 2, 128, [(0, 513)], 0.0, True, 0, [513], 64),
    (1, 1, 128, [(1500, 1)], 0.0, False, 0, None, 1),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("ctas", [0, 1, 3, 29])
def test_attention(ddt, case, ctas):
    H, G, D, lens, cap, bias, window, full, page = case
    c = ref.Chunk(lens, 11 + H + len(lens), page)
    q, k, v = inputs(c, H, G, D, 5 * H + D, 6.0 if cap else 1.5)
    kw = dict(cap=cap, slopes=slopes_of(H) if bias else None, window=window, full=full)
    out, ls = run(ddt, c, q, k, v, D ** -0.5, num_ctas=ctas, **kw)
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, D ** -0.5, **kw))


@pytest.mark.parametrize("ctas", [2, 5, 7, 16, 64, 128, 512])
@pytest.mark.parametrize("H,T,D", [(8, 1, 128), (16, 70, 128), (16, 33, 64)])
def test_dealt_to_any_number_of_ctas(ddt, ctas, H, T, D):
    # shares that cut the long request many times, and that hold its end, whole requests and a start
    c = ref.Chunk([(1900, T), (40, T), (0, 0), (700, max(1, T // 2))], 3)
    q, k, v = inputs(c, H, 2, D, 9)
    out, ls = run(ddt, c, q, k, v, 0.1, num_ctas=ctas, window=1200, full=[100, 0, 0, 5])
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, 0.1, window=1200, full=[100, 0, 0, 5]))


SPREAD = [(8, 1, 128, [(200, 70), (0, 140)]), (4, 4, 64, [(90, 40), (0, 3)]), (16, 2, 128, [(300, 1)])]


@pytest.mark.parametrize("H,G,D,lens", SPREAD)
@pytest.mark.parametrize("ctas", [0, 5])
def test_columns_that_a_token_does_not_see_may_hold_anything(ddt, H, G, D, lens, ctas):
    # K rows of NaN and infinities, V rows of NaN, +-infinity: each in a column that some tokens of the
    # chunk see (later ones) and others do not; rows that nobody sees are behind the window
    c = ref.Chunk(lens, 31, 16)
    q, k, v = inputs(c, H, G, D, 77)
    full, window = [3, 0][: c.B], 60
    for b in range(c.B):
        rows = c.slots[c.kv[b]: c.kv[b + 1]].astype(np.int64)
        if c.N[b] > 130:
            v[rows[5]], k[rows[6]], k[rows[7]] = torch.nan, torch.nan, torch.inf   # seen by the first tokens, or by none
        last = rows[c.N[b] - 1 - min(1, c.T[b] - 1):]
        v[last[0], :, 3], v[last[0], :, 4], v[last[0], :, 5] = torch.inf, -torch.inf, torch.nan
        if len(last) > 1:
            v[last[1], :, 3], v[last[1], :, 4] = -torch.inf, -torch.inf
    out, ls = run(ddt, c, q, k, v, D ** -0.5, window=window, full=full, num_ctas=ctas)
    clean(ddt)
    # the formula, row by row over what the row sees
    for b in range(c.B):
        rows = torch.from_numpy(c.slots[c.kv[b]: c.kv[b + 1]].astype(np.int64))
        seen = ref.visible(c, b, window, full)
        for i in range(int(c.T[b])):
            r, t = rows[seen[i]], int(c.qo[b]) + i
            for h in range(H):
                z = D ** -0.5 * (k[r, h // (H // G)].double() @ q[t, h].double())
                want = torch.softmax(z, 0) @ v[r, h // (H // G)].double()
                got = out[t, h].double().cpu()
                assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, i, h)
                assert torch.equal(torch.isinf(got), torch.isinf(want)) and torch.equal(got[torch.isinf(got)], want[torch.isinf(want)])
                ok = torch.isfinite(want)
                # weights and result rounded to bf16, the rest in fp32
                size = torch.softmax(z, 0) @ torch.where(torch.isfinite(v[r, h // (H // G)]), v[r, h // (H // G)], 0.0).double().abs()
                assert bool(((got - want).abs()[ok] <= (2.5 * ref.H8 * size + 1e-4)[ok]).all()) or bool(torch.isnan(z).any())


@pytest.mark.parametrize("size", [1e30, 3e38, 1e-20])
@pytest.mark.parametrize("ctas", [0, 3])
def test_values_of_any_size_stay_finite(ddt, size, ctas):
    c = ref.Chunk([(500, 70), (40, 1)], 5)
    q, k, v = inputs(c, 8, 2, 128, 4)
    v = (torch.tanh(v.float()) * size).to(torch.bfloat16)
    out, ls = run(ddt, c, q, k, v, 0.1, num_ctas=ctas)
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, 0.1))


@pytest.mark.parametrize("H,T", [(2, 1), (8, 100)])
def test_peaked_scores_that_rise_against_the_order_of_the_columns(ddt, H, T):
    # columns are taken from the latest on: scores that grow towards the first ones move the reference often
    c = ref.Chunk([(900, T)], 8)
    q, k, v = inputs(c, H, 1, 128, 2)
    ramp = torch.linspace(9.0, 0.0, c.total_kv).to(torch.bfloat16)
    k[torch.from_numpy(c.slots.astype(np.int64))] *= ramp[:, None, None]
    for ctas in (0, 1, 3):
        out, ls = run(ddt, c, q, k, v, 1.0, num_ctas=ctas)
        clean(ddt)
        check(out, ls, ref.attention(q, k, v, c, 1.0))


def test_steep_slopes_and_slopes_below_zero(ddt):
    c = ref.Chunk([(700, 90), (0, 30)], 9)
    q, k, v = inputs(c, 6, 2, 128, 12)
    for slopes in (torch.tensor([4.0, 1.0, 0.0, 30.0, 0.5, 1e-3]), torch.tensor([-0.5, 0.25, -2.0, 0.0, -0.01, 1.0])):
        for full in (None, [64, 30]):
            out, ls = run(ddt, c, q, k, v, 0.1, slopes=slopes, full=full)
            clean(ddt)
            check(out, ls, ref.attention(q, k, v, c, 0.1, slopes=slopes, full=full))


def test_scores_of_minus_infinity_alone_give_an_empty_row(ddt):
    c = ref.Chunk([(150, 2)], 9)
    q, k, v = inputs(c, 2, 2, 64, 12)
    q = q.abs() + 1
    k[torch.from_numpy(c.slots.astype(np.int64))] = -torch.inf
    for ctas in (0, 1, 3):
        out, ls = run(ddt, c, q, k, v, 0.1, num_ctas=ctas)
        clean(ddt)
        assert not out.any() and bool((ls == -torch.inf).all())


def test_capped_scores_of_infinite_products(ddt):
    # a product of -inf is a score of -cap, one of +inf a score of cap; the first request has nothing but those
    c = ref.Chunk([(150, 2), (90, 3)], 9)
    q, k, v = inputs(c, 2, 2, 64, 12)
    q = q.abs() + 1
    rows = c.slots.astype(np.int64)
    k[rows[: c.N[0]]] = -torch.inf
    k[rows[c.N[0] + 5]] = torch.inf
    k[rows[c.N[0] + 60:]] = -torch.inf
    out, ls = run(ddt, c, q, k, v, 0.1, cap=6.0)
    clean(ddt)
    kk = k.clone()
    kk[torch.isinf(k)] = torch.sign(k[torch.isinf(k)]) * 1e4
    check(out, ls, ref.attention(q, kk, v, c, 0.1, cap=6.0))


def test_strided_pools_rows_left_alone_and_no_lse(ddt):
    c = ref.Chunk([(150, 40), (0, 0), (33, 1)], 4)
    H, G, D, extra = 16, 4, 128, 5
    q, k, v = inputs(c, H, G, D, 3)
    kv = torch.stack([k, v], 1).to(DEV)   # a token's K and V next to each other
    d = c.device()
    qd = torch.cat([q, q[:extra]]).to(DEV)
    out = torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ddt.ddt_gqa_chunk_attn(qd, kv[:, 0], kv[:, 1], d["kv_indices"], d["kv_indptr"], d["qo_indptr"], 0.1, out)
    clean(ddt)
    assert bool((out[c.total_q:] == 7.0).all())
    check(out[: c.total_q], None, ref.attention(q, k, v, c, 0.1))


def test_offsets_that_start_behind_zero(ddt):
    c = ref.Chunk([(64, 20), (10, 150)], 6)
    q, k, v = inputs(c, 8, 2, 64, 8)
    want, wl, _, _ = ref.attention(q, k, v, c, 0.1)
    d = c.device()
    for skip in (1, 33):
        qd = torch.cat([q[:1].expand(skip, -1, -1), q]).to(DEV)
        out = torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full(qd.shape[:2], 7.0, device=DEV)
        idx = torch.cat([torch.full((skip,), -5, dtype=torch.int32, device=DEV), d["kv_indices"]])
        ddt.ddt_gqa_chunk_attn(qd, k.to(DEV), v.to(DEV), idx, d["kv_indptr"] + skip, d["qo_indptr"] + skip, 0.1, out, lse)
        clean(ddt)
        assert bool((out[:skip] == 7.0).all()) and bool((lse[:skip] == 7.0).all())
        check(out[skip:], lse[skip:], ref.attention(q, k, v, c, 0.1))


def test_more_requests_than_can_be_dealt(ddt):
    lens = [(i % 90, i % 5) for i in range(300)] + [(0, 40), (700, 9)]
    c = ref.Chunk(lens, 2)
    for H, G in ((2, 1), (32, 2)):
        q, k, v = inputs(c, H, G, 64, 8)
        out, ls = run(ddt, c, q, k, v, 0.1, window=50)
        clean(ddt)
        check(out, ls, ref.attention(q, k, v, c, 0.1, window=50))


def test_bad_data_is_latched_and_the_rest_is_right(ddt):
    c = ref.Chunk([(64, 20), (300, 30), (10, 5)], 6)
    q, k, v = inputs(c, 8, 2, 64, 8)
    want = ref.attention(q, k, v, c, 0.1)
    d = c.device()

    def go(max_q=None, ctas=0, **change):
        e = dict(d, **change)
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        ddt.ddt_gqa_chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), e["kv_indices"], e["kv_indptr"], e["qo_indptr"], 0.1, out,
                               max_q_len=max_q or c.max_q, max_kv_len=c.max_kv, num_ctas=ctas)
        torch.cuda.synchronize()
        return out, ddt.ddt_get_error()[1]

    for ctas in (0, 4):
        out, bits = go(max_q=20, ctas=ctas)   # the second request's 30 tokens are more than was said
        assert bits == 0x1 and bool((out[20:50] == 7.0).all())
        ok = torch.cat([torch.arange(20), torch.arange(50, 55)])
        check(out[ok.to(DEV)], None, tuple(x[ok] for x in want))
        bad = d["kv_indptr"].clone()
        bad[1] = 10   # fewer columns than tokens, and a request that starts too early
        out, bits = go(ctas=ctas, kv_indptr=bad)
        assert bits == 0x2 and bool((out[:20] == 7.0).all())
        slots = d["kv_indices"].clone()
        slots[3], slots[100] = -1, c.rows
        out, bits = go(ctas=ctas, kv_indices=slots)
        assert bits == 0x4
        check(out[50:], None, tuple(x[50:] for x in want))


def test_graph_and_streams(ddt):
    c = ref.Chunk([(300, 150), (40, 1)], 6)
    q, k, v = inputs(c, 16, 2, 128, 8)
    d = c.device()
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    want = ref.attention(q, k, v, c, 0.1, window=90)
    nbytes = ddt.ddt_gqa_chunk_attn_workspace_size(16, 2, 128, c.max_q, ddt.ddt_gqa_chunk_attn_num_ctas(2, 16, 2, c.max_q, c.max_kv))
    outs = []

    def call(stream, ws):
        out = torch.zeros_like(qd)
        lse = torch.zeros(qd.shape[:2], device=DEV)
        outs.append((out, lse))
        return lambda: ddt.ddt_gqa_chunk_attn(qd, kd, vd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], 0.1, out, lse,
                                              max_q_len=c.max_q, max_kv_len=c.max_kv, window=90, workspace=ws, stream=stream)

    wss = [torch.empty(nbytes, dtype=torch.uint8, device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    a, b = call(None, wss[0]), call(side, wss[1])
    torch.cuda.synchronize()
    for _ in range(20):   # at the same time, a workspace each
        a()
        b()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    f = call(None, wss[0])
    with torch.cuda.graph(g):
        f()
    outs[-1][0].zero_()
    for _ in range(3):
        g.replay()
    clean(ddt)
    for out, lse in outs:
        check(out, lse, want)
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_slots_past_two_billion_bytes(ddt):
    # rows whose places in the pool pass 32 bits
    rows, G, D = 9_000_000, 2, 128
    pool = torch.zeros(rows, 2, G, D, dtype=torch.bfloat16, device=DEV)
    c = ref.Chunk([(300, 40)], 1)
    q, k, v = inputs(c, 4, G, D, 3)
    far = torch.from_numpy(c.slots.astype(np.int64)) + (rows - c.rows)
    pool[far.to(DEV), 0] = k[far - (rows - c.rows)].to(DEV)
    pool[far.to(DEV), 1] = v[far - (rows - c.rows)].to(DEV)
    d = c.device()
    out = torch.zeros_like(q, device=DEV)
    ddt.ddt_gqa_chunk_attn(q.to(DEV), pool[:, 0], pool[:, 1], far.to(torch.int32).to(DEV), d["kv_indptr"], d["qo_indptr"], 0.1, out)
    clean(ddt)
    check(out, None, ref.attention(q, k, v, c, 0.1))


def test_any_workspace_and_one_that_is_too_small(ddt):
    # without a count the work is dealt to what the workspace holds, down to none; with one it is refused
    c = ref.Chunk([(900, 40), (10, 70)], 6)
    q, k, v = inputs(c, 16, 2, 64, 8)
    want = ref.attention(q, k, v, c, 0.1)
    for ctas in (0, 1, 2, 7, 100):
        nbytes = max(256, ddt.ddt_gqa_chunk_attn_workspace_size(16, 2, 64, c.max_q, ctas))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        out, ls = run(ddt, c, q, k, v, 0.1, workspace=ws)
        clean(ddt)
        check(out, ls, want)
        with pytest.raises(ddt.DDTError, match="DDT_ERR_WORKSPACE"):
            run(ddt, c, q, k, v, 0.1, workspace=ws, num_ctas=ctas + 1)
    clean(ddt)


def test_windows_and_prefixes_at_their_limits(ddt):
    c = ref.Chunk([(200, 30), (0, 9)], 6)
    q, k, v = inputs(c, 4, 4, 64, 8)
    for window, full in ((2 ** 31 - 1, None), (230, [-5, 2 ** 31 - 1]), (229, [-2 ** 31, 3]), (1, [0, 0]), (2 ** 30, [230, 9])):
        out, ls = run(ddt, c, q, k, v, 0.1, window=window, full=full)
        clean(ddt)
        check(out, ls, ref.attention(q, k, v, c, 0.1, window=window, full=full))


def test_nothing_to_do(ddt):
    c = ref.Chunk([(20, 0), (0, 0)], 6)
    q, k, v = inputs(c, 4, 4, 64, 8)
    run(ddt, c, q, k, v, 0.1)
    c = ref.Chunk([(20, 0), (0, 3), (5, 0)], 6)
    q, k, v = inputs(c, 4, 4, 64, 8)
    out, ls = run(ddt, c, q, k, v, 0.1)
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, 0.1))


@pytest.mark.parametrize("H,G", [(8, 1), (128, 1), (6, 6)])
def test_a_long_chunk(ddt, H, G):
    # more items than CTAs, and items whose columns differ a lot; checked on some of the rows
    T = 20000 // H
    c = ref.Chunk([(300, T), (1, 5)], 3, 16)
    q, k, v = inputs(c, H, G, 128, 8)
    out, ls = run(ddt, c, q, k, v, 0.09, window=700, full=[40, 2])
    clean(ddt)
    few = ref.Chunk([(300, T), (1, 5)], 3, 16)
    rng = np.random.default_rng(1)
    for i in sorted({0, 1, T - 1, *rng.integers(0, T, 12).tolist()}):   # one row: a chunk of one behind all before it
        one = ref.Chunk([(300 + i, 1)], 3)
        one.slots = few.slots[: 300 + i + 1]
        want = ref.attention(q[i: i + 1], k, v, one, 0.09, window=700, full=[40])
        check(out[i: i + 1], ls[i: i + 1], want)
