"""GqaChunkStep with what its other tests leave out: layers that are not observed, norm and rotation on a cache
that rows have left, eviction of weights that the caller gives, captures."""
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import DEV, clean, ddt, normal  # noqa: F401  (ddt: the fixture)
from tests.test_chunk_weights_gpu import check as check_weights

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
