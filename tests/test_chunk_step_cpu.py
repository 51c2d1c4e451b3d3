"""Refusals of GqaChunkStep that reach no kernel."""
import pytest
import torch

from tests.test_gqa_cpu import lib  # noqa: F401  (builds the library)


def step(**kw):
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    kv = torch.zeros(2, 50, 2, 64, dtype=torch.bfloat16)
    return GqaChunkStep(kv, torch.arange(20, dtype=torch.int32), [10], [10], 4, **kw)


@pytest.mark.parametrize("observe", [False, True])
def test_evict_without_sums_is_refused(lib, observe):  # noqa: F811
    # no layer has run (or was observed), and nobody has given weights: there is nothing to rank by
    with pytest.raises(ValueError, match="nothing to evict by"):
        step(observe=observe).evict([5])


def test_slots_of_another_number_are_refused(lib):  # noqa: F811
    from tree_speculative_decoding_gb300.pipeline import GqaChunkStep
    with pytest.raises(ValueError, match="prefix_len"):
        GqaChunkStep(torch.zeros(2, 50, 2, 64, dtype=torch.bfloat16), torch.arange(19, dtype=torch.int32), [10], [10], 4)
