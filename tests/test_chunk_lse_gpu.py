"""The rows' log of their sum, to fp32's own precision."""
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import DEV, clean, ddt, inputs, run  # noqa: F401  (ddt: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H,cap,bias", [(64, 2, 0.0, False), (128, 8, 0.0, False), (128, 16, 30.0, False), (64, 2, 0.0, True)])
def test_lse_of_equal_scores(ddt, D, H, cap, bias):  # noqa: F811
    # scores of 0: weights of a power of two, so a row of n columns has n of them exactly, and what is left is the
    # logarithm (CUDA's log2f: 1 ulp), ln 2 as a float and one product: 4 half steps of the result; and
    # cap 2^-20 of a capped score
    c = ref.Chunk([(0, 300), (900, 3)], 3)
    q, k, v = inputs(c, H, 2, D, 1)
    q.zero_()
    n = torch.cat([torch.arange(1, 301), torch.arange(901, 904)]).double()[:, None]
    slopes = torch.zeros(H) if bias else None
    _, ls = run(ddt, c, q, k, v, 0.1, cap=cap, slopes=slopes, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))  # items whole
    clean(ddt)
    want = n.log().expand(-1, H)
    assert bool(((ls.double().cpu() - want).abs() <= 4 * ref.U * want + cap * 2.0 ** -20).all())
    # cut into parts: every part's lse so, its weight 2^(x - 9) of an argument rounded by 16's size and to 2 ulp of
    # 2^x, the same four and one more for their sum
    for ctas in (3, 7):
        _, ls = run(ddt, c, q, k, v, 0.1, cap=cap, slopes=slopes, num_ctas=ctas)
        clean(ddt)
        assert bool(((ls.double().cpu() - want).abs() <= 10 * ref.U * want + 2.0 ** -21 + 2.0 ** -22 + cap * 2.0 ** -20).all())
