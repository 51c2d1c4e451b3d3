"""Received weights on the GPU, against a plain 64-bit form (tests/_chunk_ref.py, which also
derives the tolerances)."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import CASES, DEV, clean, ddt, normal, slopes_of  # noqa: F401  (ddt: the fixture)

pytestmark = pytest.mark.gpu


def inputs(c, H, G, D, seed, q_scale=1.5):
    return normal((c.total_q, H, D), seed, q_scale), normal((c.rows, G, D), seed + 1)


def row_sums(q, k, c, scale, **kw):
    """The rows' lse in fp32, as the attention leaves them (its own test says how near they are)."""
    v = torch.zeros(c.rows, k.shape[1], k.shape[2], dtype=torch.bfloat16)
    return ref.attention(q, k, v, c, scale, **kw)[1].float()


def run(ddt, c, q, k, lse, scale, cap=0.0, slopes=None, window=0, full=None, prev=None, prev_lens=None, **kw):  # noqa: F811
    d = c.device()
    w = torch.full((c.total_kv,), 7.0, device=DEV)
    if prev is not None:
        kw.update(prev=prev.to(DEV), prev_indptr=torch.tensor(np.concatenate([[0], np.cumsum(prev_lens)]), dtype=torch.int32, device=DEV))
    ddt.ddt_gqa_chunk_weights(q.to(DEV), k.to(DEV), lse.to(DEV), d["kv_indices"], d["kv_indptr"], d["qo_indptr"], scale, w,
                              max_q_len=c.max_q, max_kv_len=c.max_kv, score_cap=cap,
                              slopes=None if slopes is None else slopes.to(DEV), window=window,
                              full_len=None if full is None else torch.tensor(full, dtype=torch.int32, device=DEV), **kw)
    return w


def check(w, want):
    err = (w.double().cpu() - want[0]).abs() - want[1]
    assert float(err.max()) <= 0, f"over its bound by {float(err.max())} at {int(err.argmax())}"


@pytest.mark.parametrize("case", CASES + [
    (8, 1, 128, [(600, 2), (255, 1), (256, 2), (257, 1)], 0.0, True, 100, [0, 3, 256, 500], 64),
    (16, 16, 128, [(900, 16), (100, 1)], 30.0, False, 0, None, 1)])
@pytest.mark.parametrize("ctas,last_rows", [(0, 0), (1, 3), (3, 0), (29, 40)])
def test_received(ddt, case, ctas, last_rows):  # noqa: F811
    H, G, D, lens, cap, bias, window, full, page = case
    c = ref.Chunk(lens, 11 + H + len(lens), page)
    q, k = inputs(c, H, G, D, 5 * H + D, 6.0 if cap else 1.5)
    kw = dict(cap=cap, slopes=slopes_of(H) if bias else None, window=window, full=full)
    lse = row_sums(q, k, c, D ** -0.5, **kw)
    prev_lens = [int(p) - (int(p) > 20) * 3 for p in c.P]   # the chunk's own columns have no sums yet
    prev = torch.rand(sum(prev_lens), generator=torch.Generator().manual_seed(1))
    more = dict(last_rows=last_rows, prev=prev, prev_lens=prev_lens, decay=0.75)
    w = run(ddt, c, q, k, lse, D ** -0.5, num_ctas=ctas, **kw, **more)
    clean(ddt)
    check(w, ref.received(q, k, lse, c, D ** -0.5, **kw, **more))


@pytest.mark.parametrize("ctas", [2, 7, 64, 512])
@pytest.mark.parametrize("H,T,D", [(8, 1, 128), (16, 200, 128), (16, 33, 64)])
def test_dealt_to_any_number_of_ctas(ddt, ctas, H, T, D):  # noqa: F811
    c = ref.Chunk([(1900, T), (40, T), (0, 0), (300, 0), (700, max(1, T // 2))], 3)
    q, k = inputs(c, H, 2, D, 9)
    kw = dict(window=1200, full=[100, 0, 0, 9, 5])
    lse = row_sums(q, k, c, 0.1, **kw)
    w = run(ddt, c, q, k, lse, 0.1, num_ctas=ctas, **kw)
    clean(ddt)
    check(w, ref.received(q, k, lse, c, 0.1, **kw))


def test_layers_add_up_in_place_and_rows_add_up_to_one(ddt):  # noqa: F811
    # the sums of a step: every row gives each of its heads one in all, whatever the masks
    c = ref.Chunk([(300, 40), (0, 129), (77, 1)], 7, 16)
    H, G, D = 8, 2, 128
    d = c.device()
    w = torch.zeros(c.total_kv, device=DEV)
    for layer in range(3):
        q, k = inputs(c, H, G, D, 100 + layer)
        qd, kd = q.to(DEV), k.to(DEV)
        out, lse = torch.empty_like(qd), torch.empty(qd.shape[:2], device=DEV)
        ddt.ddt_gqa_chunk_attn(qd, kd, kd, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], 0.1, out, lse, window=50)
        ddt.ddt_gqa_chunk_weights(qd, kd, lse, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], 0.1, w,
                                  prev=w if layer else None, window=50)
    clean(ddt)
    for b in range(c.B):
        got = float(w[int(c.kv[b]): int(c.kv[b + 1])].double().sum())
        assert abs(got - 3 * H * int(c.T[b])) <= 3 * H * int(c.T[b]) * 2.0 ** -14   # lse and scores: 2^-17 of a weight at most


def test_unseen_values_rows_left_alone_and_empty_rows(ddt):  # noqa: F811
    c = ref.Chunk([(300, 40), (10, 3)], 5)
    H, G, D = 4, 2, 64
    q, k = inputs(c, H, G, D, 8)
    lse = row_sums(q, k, c, 0.1, window=60)
    rows = c.slots[: c.N[0]].astype(np.int64)
    k[rows[:200]] = torch.nan           # behind every token's window
    bad = lse.clone()
    bad[5, 1] = -torch.inf              # a row that saw nothing
    w = run(ddt, c, q, k, bad, 0.1, window=60)
    clean(ddt)
    k[rows[:200]] = 0.0
    want, bound = ref.received(q, k, bad.clamp(min=-1e30).masked_fill(bad == -torch.inf, 1e30), c, 0.1, window=60)
    check(w, (want, bound))
    assert not w[:200].any()


def test_bad_data_is_latched(ddt):  # noqa: F811
    c = ref.Chunk([(64, 20), (300, 30), (10, 5)], 6)
    q, k = inputs(c, 8, 2, 64, 8)
    lse = row_sums(q, k, c, 0.1)
    d = c.device()
    prev = torch.ones(int(c.P.sum()), device=DEV)
    want = ref.received(q, k, lse, c, 0.1, prev=prev.cpu(), prev_lens=list(c.P), decay=1.0)

    def go(indptr, **change):
        e = dict(d, **change)
        w = torch.full((c.total_kv,), 7.0, device=DEV)
        ddt.ddt_gqa_chunk_weights(q.to(DEV), k.to(DEV), lse.to(DEV), e["kv_indices"], e["kv_indptr"], e["qo_indptr"], 0.1, w, prev=prev,
                                  prev_indptr=torch.tensor(indptr, dtype=torch.int32, device=DEV), max_q_len=c.max_q, max_kv_len=c.max_kv)
        torch.cuda.synchronize()
        return w, ddt.ddt_get_error()[1]

    w, bits = go([0, 64, 364, 374])
    assert bits == 0
    check(w, want)
    for bad in ([0, 64, 364, 380], [0, 64, 340, 374], [0, 64, -3, 374]):   # past the end, too many, backwards
        w, bits = go(bad)
        assert bits == 0x2
        n = int(c.kv[1])
        assert float((w.double().cpu() - want[0]).abs()[:n].sub(want[1][:n]).max()) <= 0
        assert bool((w[int(c.kv[2]):] == 7.0).all())
    slots = d["kv_indices"].clone()
    slots[3] = c.rows
    w, bits = go([0, 64, 364, 374], kv_indices=slots)
    assert bits == 0x4


def test_graph_and_more_requests_than_can_be_dealt(ddt):  # noqa: F811
    c = ref.Chunk([(i % 300, i % 4) for i in range(280)], 2)
    q, k = inputs(c, 4, 2, 64, 8)
    lse = row_sums(q, k, c, 0.1)
    d = c.device()
    qd, kd, ld = q.to(DEV), k.to(DEV), lse.to(DEV)
    w = torch.zeros(c.total_kv, device=DEV)
    f = lambda: ddt.ddt_gqa_chunk_weights(qd, kd, ld, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], 0.1, w,  # noqa: E731
                                          max_q_len=c.max_q, max_kv_len=c.max_kv)
    f()
    clean(ddt)
    want = ref.received(q, k, lse, c, 0.1)
    check(w, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    w.zero_()
    g.replay()
    clean(ddt)
    check(w, want)


def test_requests_without_new_tokens_decay(ddt):  # noqa: F811
    c = ref.Chunk([(300, 0), (0, 0), (40, 0)], 2)
    prev = torch.rand(340, generator=torch.Generator().manual_seed(3))
    empty = torch.zeros(0, 4, 64, dtype=torch.bfloat16)
    k = normal((c.rows, 2, 64), 1)
    w = run(ddt, c, empty, k, torch.zeros(0, 4), 0.1, prev=prev, prev_lens=[300, 0, 40], decay=0.5)
    clean(ddt)
    assert torch.equal(w.cpu(), prev * 0.5)
    w = run(ddt, c, empty, k, torch.zeros(0, 4), 0.1)
    clean(ddt)
    assert not w.any()


def test_without_a_workspace_and_with_less(ddt):  # noqa: F811
    c = ref.Chunk([(700, 40), (10, 70)], 6)
    q, k = inputs(c, 16, 2, 64, 8)
    lse = row_sums(q, k, c, 0.1)
    want = ref.received(q, k, lse, c, 0.1)
    for nbytes in (256, 4096, 100000):
        w = run(ddt, c, q, k, lse, 0.1, workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV))
        clean(ddt)
        check(w, want)
    with pytest.raises(ddt.DDTError, match="DDT_ERR_WORKSPACE"):
        run(ddt, c, q, k, lse, 0.1, workspace=torch.empty(256, dtype=torch.uint8, device=DEV), num_ctas=2)


def test_a_row_that_is_not_a_number_stays_in_its_columns(ddt):  # noqa: F811
    # the last rows of a tile are the last token's again where there are no more
    c = ref.Chunk([(100, 5)], 6)
    q, k = inputs(c, 4, 2, 64, 8)
    lse = row_sums(q, k, c, 0.1, window=30)
    q[4] = torch.nan
    w = run(ddt, c, q, k, lse, 0.1, window=30).cpu()
    clean(ddt)
    seen = ref.visible(c, 0, 30, None)[4]
    assert torch.equal(torch.isnan(w), seen)
