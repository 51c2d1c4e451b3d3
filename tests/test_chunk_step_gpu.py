"""Chunks through GqaChunkStep as a model would run them: a prompt in two chunks, what its tokens received,
eviction, compaction, then single tokens on what is left, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import DEV, check, clean, ddt, normal, slopes_of  # noqa: F401  (ddt: the fixture)
from tests.test_chunk_weights_gpu import check as check_weights

pytestmark = pytest.mark.gpu


class Placed(ref.Chunk):
    """Requests whose slots are given."""

    def __init__(self, lens, slots, rows):
        super().__init__(lens, 0)
        self.slots, self.rows = np.asarray(slots, np.int32), rows


@pytest.mark.parametrize("H,G,D,cap,bias,window", [(8, 2, 128, 0.0, False, 0), (4, 4, 64, 20.0, True, 90)])
def test_prompt_evict_compact_decode(ddt, H, G, D, cap, bias, window):  # noqa: F811
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    layers, rows, rng = 2, 900, np.random.default_rng(3)
    how = dict(cap=cap, slopes=slopes_of(H) if bias else None, window=window)
    mine = dict(score_cap=cap, slopes=slopes_of(H).to(DEV) if bias else None, window=window)
    kv = torch.zeros(2 * layers, rows, G, D, dtype=torch.bfloat16, device=DEV)
    free = [int(s) for s in rng.permutation(rows)]
    lens = [(0, 150), (0, 40)]
    slots = [[], []]
    prev, prev_lens, prev_indptr = None, None, None

    for number, new in enumerate([[150, 40], [100, 1], [1, 1], [1, 3]]):
        for b, n in enumerate(new):
            slots[b] += [free.pop() for _ in range(n)]
        lens = [(len(s) - n, n) for s, n in zip(slots, new)]
        c = Placed(lens, slots[0] + slots[1], rows)
        idx = torch.from_numpy(c.slots).to(DEV)
        step = GqaChunkStep(kv, idx, c.P, c.T, H, observe=True, last_rows=0 if number else 16, prev=prev,
                            prev_indptr=prev_indptr, decay=0.5, **mine)
        want, bound = torch.zeros(c.total_kv, dtype=torch.float64), 0.0
        for n in range(layers):
            q, k, v = normal((c.total_q, H, D), 100 * number + n, 1.5), normal((c.total_q, G, D), 7 + n), normal((c.total_q, G, D), 9 + n)
            out = step.layer(n, q.to(DEV), k.to(DEV), v.to(DEV)).clone()
            clean(ddt)
            kp, vp = kv[2 * n].cpu(), kv[2 * n + 1].cpu()
            at = torch.from_numpy(np.concatenate([c.slots[c.kv[b + 1] - t: c.kv[b + 1]] for b, t in enumerate(new)]).astype(np.int64))
            assert torch.equal(kp[at], k) and torch.equal(vp[at], v) and torch.equal(step.q.cpu(), q)
            o, l, bo, bl = ref.attention(q, kp, vp, c, D ** -0.5, **how)
            check(out, step.lse, (o, l, bo, bl))
            first = n == 0 and prev is not None
            w, e = ref.received(q, kp, step.lse.cpu(), c, D ** -0.5, **how, last_rows=step.last_rows,
                                prev=prev.cpu() if first else None, prev_lens=prev_lens, decay=0.5)
            want, bound = want + w, bound + e + (want + w).abs() * 4 * ref.U
        check_weights(step.weights, (want, bound))

        budget, sinks, recent = [60 + 40 * number, 30], 3, 5
        left, indptr, weights, gone = step.evict(budget, sinks, recent)
        clean(ddt)
        stay, want_indptr, want_w, want_gone = ref.evict(step.weights.cpu(), c.slots, c.N, budget, sinks, recent)
        assert left.tolist() == stay and indptr.tolist() == want_indptr and gone.tolist() == want_gone
        assert weights.cpu().tolist() == want_w and step.new_len.tolist() == np.diff(want_indptr).tolist()
        before = kv.clone()
        step.compact(left)
        clean(ddt)
        assert torch.equal(kv[:, left.long()], before[:, torch.tensor(stay, device=DEV)])
        assert step.live.item() == len(stay) and sorted(left.tolist()) == list(range(len(stay)))
        now = left.tolist()
        slots = [now[want_indptr[b]: want_indptr[b + 1]] for b in range(2)]
        free = [s for s in range(rows) if s not in set(now)]
        prev, prev_lens, prev_indptr = weights, step.new_len, indptr


def test_verify_step_after_a_prompt(ddt):  # noqa: F811
    # a prompt longer than a tree through the chunk calls, into the cache of a verify step: the tree's
    # attention then reads the rows that the chunk wrote
    from tree_speculative_decoding_gb300 import workloads
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep, GqaVerifyStep
    H, G, D = 8, 2, 128
    wl = workloads.make_workload("gqa", 5, 1, 1, [300], [8], 6, 256, 1.5, pool_rows=400, fill_pool=False)
    verify = GqaVerifyStep(wl, 1, H, G, D, device=DEV)
    chunk = GqaChunkStep(verify.kv, verify.kv_indices[:300].contiguous(), [0], [300], H)
    q, k, v = (normal((300, h, D), 20 + i).to(DEV) for i, h in enumerate((H, G, G)))
    chunk.layer(0, q, k, v)
    verify.build_chain_visibility()
    q2, k2, v2 = (normal((9, h, D), 30 + i).to(DEV) for i, h in enumerate((H, G, G)))
    out = verify.layer(0, q2, k2, v2).clone()
    again = GqaChunkStep(verify.kv, verify.kv_indices, [300], [9], H)
    other = again.layer(0, q2, k2, v2)
    clean(ddt)
    c = Placed([(300, 9)], verify.kv_indices.cpu().numpy(), 400)
    o, l, bo, bl = ref.attention(q2.cpu(), verify.kv[0].cpu(), verify.kv[1].cpu(), c, D ** -0.5)
    check(out, None, (o, l, bo, bl))
    check(other, None, (o, l, bo, bl))


def test_chunk_step_as_a_graph(ddt):  # noqa: F811
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    H, G, D, layers = 8, 2, 64, 2
    kv = torch.zeros(2 * layers, 500, G, D, dtype=torch.bfloat16, device=DEV)
    idx = torch.randperm(500, generator=torch.Generator().manual_seed(1))[:400].to(torch.int32).to(DEV)
    step = GqaChunkStep(kv, idx, [200, 0], [60, 140], H, observe=True, window=70)
    x = [[normal((200, h, D), 10 * n + i).to(DEV) for i, h in enumerate((H, G, G))] for n in range(layers)]

    def run():
        return [step.layer(n, *x[n]).clone() for n in range(layers)]

    first = run()
    torch.cuda.synchronize()
    sums = step.weights.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    step.weights.zero_()
    g.replay()
    g.replay()
    clean(ddt)
    assert all(torch.equal(a, b) for a, b in zip(first, outs)) and torch.equal(step.weights, sums)


def test_evict_on_another_stream(ddt):  # noqa: F811
    # the budgets' copy is read when the stream gets there: the current stream may not have its memory before
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    c = ref.Chunk([(700, 4), (90, 1), (30, 0)], 7)
    kv = torch.zeros(2, c.rows, 2, 64, dtype=torch.bfloat16, device=DEV)
    step = GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, 4)
    step.weights.copy_(normal((c.total_kv,), 5).float())
    side = torch.cuda.Stream()
    for sleep in (1000, 50_000_000):  # (the first time for what is loaded with the first call)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(sleep)
        out = step.evict([300, 1 << 40, 11], 2, 3, stream=side)
        others = [torch.zeros(n, dtype=torch.int32, device=DEV) for n in (3, 4, 402) for _ in range(40)]
        pending = not side.query()
    torch.cuda.synchronize()
    assert pending  # else nothing is tested
    left, indptr, weights, gone = out
    clean(ddt)
    stay, want_indptr, want_w, want_gone = ref.evict(step.weights.cpu(), c.slots, c.N, [300, 1 << 20, 11], 2, 3)
    assert indptr.tolist() == want_indptr and left.tolist() == stay and gone.tolist() == want_gone
    assert weights.cpu().tolist() == want_w and all(int(x.sum()) == 0 for x in others)


@pytest.mark.parametrize("lens", [[(40, 0), (300, 0)], []])
def test_step_without_new_tokens(ddt, lens):  # noqa: F811
    # the earlier sums decay; there is nothing else to do
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    c = ref.Chunk(lens, 7)
    kv = torch.zeros(4, c.rows, 2, 64, dtype=torch.bfloat16, device=DEV)
    prev = normal((c.total_kv,), 5).float().to(DEV)
    step = GqaChunkStep(kv, torch.from_numpy(c.slots).to(DEV), c.P, c.T, 4, observe=True, prev=prev, decay=0.5)
    none = lambda heads: torch.empty(0, heads, 64, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    for n in range(2):
        assert step.layer(n, none(4), none(2), none(2)).shape == (0, 4, 64)
    clean(ddt)
    assert torch.equal(step.weights, 0.5 * prev)
    left, indptr, weights, gone = step.evict([20] * len(lens))
    clean(ddt)
    assert weights.numel() == 20 * len(lens) and indptr[1:].tolist() == [20 * (b + 1) for b in range(len(lens))]
