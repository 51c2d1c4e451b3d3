"""GqaChunkStep with what its other tests leave out: layers that are not observed, norm and rotation on a cache
that rows have left, eviction of weights that the caller gives, captures."""
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import DEV, clean, ddt, normal  # noqa: F401  (ddt: the fixture)

pytestmark = pytest.mark.gpu


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
