"""GqaChunkStep with what its other tests leave out: layers that are not observed, norm and rotation on a cache
that rows have left, eviction of weights that the caller gives, captures."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref, _gqa_ref
from tests.test_chunk_gpu import DEV, check, clean, ddt, normal  # noqa: F401  (ddt: the fixture)
from tests.test_chunk_step_gpu import Placed
from tests.test_chunk_weights_gpu import check as check_weights
from tests.test_gqa_step_gpu import table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("observed", [[1, 3], [2], [0, 3]])
@pytest.mark.parametrize("with_prev", [False, True])
def test_some_layers_are_observed(ddt, observed, with_prev):  # noqa: F811
    # the first observed layer starts the sums, whichever it is, and does so again when the step runs again
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    H, G, D, layers = 4, 2, 64, 4
    c = ref.Chunk([(120, 30), (0, 9)], 3)
    kv = torch.zeros(2 * layers, c.rows, G, D, dtype=torch.bfloat16, device=DEV)
    prev = torch.rand(c.total_kv, generator=torch.Generator().manual_seed(1)) if with_prev else None
    step = GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, H, prev=None if prev is None else prev.to(DEV), decay=0.5)
    step._weights.fill_(torch.nan)   # what nobody has written
    x = [[normal((c.total_q, h, D), 10 * n + i).to(DEV) for i, h in enumerate((H, G, G))] for n in range(layers)]
    for _ in range(2):
        want, bound = torch.zeros(c.total_kv, dtype=torch.float64), 0.0
        for n in range(layers):
            step.layer(n, *x[n], observe=n in observed)
            clean(ddt)
            if n in observed:
                first = n == observed[0] and with_prev
                w, e = ref.received(x[n][0].cpu(), kv[2 * n].cpu(), step.lse.cpu(), c, D ** -0.5, prev=prev if first else None,
                                    prev_lens=c.N, decay=0.5)
                want, bound = want + w, bound + e + (want + w).abs() * 4 * ref.U
        check_weights(step._weights, (want, bound))


def test_layers_captured_one_by_one(ddt):  # noqa: F811
    # every layer runs once before its capture: a layer's graph adds to the sums unless it is the lowest
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    H, G, D, layers = 4, 2, 64, 3
    c = ref.Chunk([(120, 30), (0, 9)], 3)
    kv = torch.zeros(2 * layers, c.rows, G, D, dtype=torch.bfloat16, device=DEV)
    x = [[normal((c.total_q, h, D), 10 * n + i).to(DEV) for i, h in enumerate((H, G, G))] for n in range(layers)]
    make = lambda: GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, H, observe=True)  # noqa: E731
    plain, step, graphs = make(), make(), []
    outs = [plain.layer(n, *x[n]).clone() for n in range(layers)]
    for n in range(layers):
        step.layer(n, *x[n])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step.layer(n, *x[n])
    for _ in range(2):
        for n in range(layers):
            graphs[n].replay()
            assert torch.equal(step.out, outs[n])
    clean(ddt)
    assert torch.equal(step.weights, plain.weights)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_and_rotation_behind_an_eviction(ddt, interleaved):  # noqa: F811
    # what has left moves the columns but not the rotation: tokens behind an eviction are rotated by their place in
    # the conversation, in the chunk step and in the verify step
    from tree_speculative_decoding_gb300 import workloads
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep, GqaVerifyStep
    H, G, D, new = 8, 2, 128, 9
    cs = table(400, D)
    wq, wk = ((normal((D,), 50 + i, 0.3) + 1.0).to(torch.bfloat16) for i in range(2))
    how = dict(cos_sin=cs.to(DEV), interleaved=interleaved)
    kv = torch.zeros(2, 400, G, D, dtype=torch.bfloat16, device=DEV)
    lens = [150, 60]
    c = ref.Chunk([(0, n) for n in lens], 4)
    step = GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, H, observe=True, **how)
    q, k, v = (normal((c.total_q, h, D), 60 + i) for i, h in enumerate((H, G, G)))
    step.layer(0, *(x.to(DEV) for x in (q, k, v)), wq.to(DEV), wk.to(DEV))
    clean(ddt)

    def rotated(x, w, pos):
        y, bound = _gqa_ref.norm_rope(x, w, 1e-6, cs, pos, interleaved)
        return y, bound

    pos = torch.cat([torch.arange(n) for n in lens])
    for got, x, w in ((step.q, q, wq), (kv[0][torch.from_numpy(c.slots.astype(np.int64)).to(DEV)], k, wk)):
        y, bound = rotated(x, w, pos)
        assert bool(((got.double().cpu() - y).abs() <= bound).all())
    left, indptr, _, _ = step.evict([70, 33], 4, 10)
    kept = step.new_len
    gone = np.asarray(lens) - kept
    free = np.setdiff1d(np.arange(400), left.cpu().numpy())
    slots = np.concatenate([np.concatenate([left.cpu().numpy()[indptr[b]: indptr[b + 1]], free[b * new: (b + 1) * new]]) for b in range(2)])
    c2 = Placed([(int(n), new) for n in kept], slots, 400)
    place = torch.from_numpy(np.concatenate([np.arange(new) + g for g in gone]).astype(np.int32)).to(DEV)
    q, k, v = (normal((2 * new, h, D), 70 + i) for i, h in enumerate((H, G, G)))
    args = [x.to(DEV) for x in (q, k, v, wq, wk)]
    step2 = GqaChunkStep(kv, torch.from_numpy(c2.slots).to(DEV), c2.P, c2.T, H, position=place, **how)
    out = step2.layer(0, *args).clone()
    clean(ddt)
    pos = torch.cat([torch.arange(n, n + new) for n in lens])
    at = torch.from_numpy(np.concatenate([c2.slots[c2.kv[b + 1] - new: c2.kv[b + 1]] for b in range(2)]).astype(np.int64)).to(DEV)
    for got, x, w in ((step2.q, q, wq), (kv[0][at], k, wk)):
        y, bound = rotated(x, w, pos)
        assert bool(((got.double().cpu() - y).abs() <= bound).all())
    want = ref.attention(step2.q.cpu(), kv[0].cpu(), kv[1].cpu(), c2, D ** -0.5)
    check(out, None, want)

    # the same tokens as a chain of the verify step (the new rows of its cache are written again)
    wl = workloads.make_workload("gqa", 5, 2, 1, [int(n) for n in kept], [new - 1, new - 1], 6, 256, 1.5, pool_rows=400, fill_pool=False)
    wl.kv_indices = c2.slots
    verify = GqaVerifyStep(wl, 1, H, G, D, device=DEV, position=place, **how)
    verify.kv = kv
    kv[0][at] = 0
    verify.build_chain_visibility()
    other = verify.layer(0, *args)
    clean(ddt)
    assert torch.equal(verify.q, step2.q)
    check(other, None, want)


def test_evict_by_weights_of_the_caller(ddt):  # noqa: F811
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    c = ref.Chunk([(70, 4), (9, 1)], 7)
    kv = torch.zeros(2, c.rows, 2, 64, dtype=torch.bfloat16, device=DEV)
    given = normal((c.total_kv,), 5).float()
    for way in ("filled", "set"):
        step = GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, 4)
        if way == "set":
            step.weights = given.to(DEV)
        else:
            step.weights.copy_(given)
        left, indptr, weights, gone = step.evict([30, 4], 2, 3)
        clean(ddt)
        stay, want_indptr, want_w, want_gone = ref.evict(given, c.slots, c.N, [30, 4], 2, 3)
        assert left.tolist() == stay and indptr.tolist() == want_indptr and gone.tolist() == want_gone and weights.tolist() == want_w


def test_evict_refuses_a_capture(ddt):  # noqa: F811
    # its budgets are the host's: a replay would copy from memory that is long somebody else's
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    c = ref.Chunk([(70, 4)], 7)
    kv = torch.zeros(2, c.rows, 2, 64, dtype=torch.bfloat16, device=DEV)
    step = GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, 4)
    step.weights.zero_()
    step.evict([30])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(RuntimeError, match="captured"):
            step.evict([20])
    assert step.new_len.tolist() == [30]
    left, indptr, _, _ = step.evict([20])
    clean(ddt)
    assert left.numel() == 20 and indptr.tolist() == [0, 20]


@pytest.mark.parametrize("side", [False, True])
def test_evict_without_requests(ddt, side):  # noqa: F811
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    i32 = lambda n, x: torch.full((n,), x, dtype=torch.int32, device=DEV)  # noqa: E731
    indptr = i32(1, -7)
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    ddt.ddt_cache_evict(torch.zeros(0, device=DEV), i32(0, 0), i32(1, 0), i32(0, 0), i32(0, 0), indptr, stream=stream)
    clean(ddt)
    assert indptr.tolist() == [0]
    kv = torch.zeros(2, 10, 2, 64, dtype=torch.bfloat16, device=DEV)
    step = GqaChunkStep(kv, i32(0, 0), [], [], 4)
    step.weights.zero_()
    left, indptr, weights, gone = step.evict([])
    clean(ddt)
    assert indptr.tolist() == [0] and left.numel() == weights.numel() == gone.numel() == 0
