"""Slopes with a prefix that reaches far behind the tokens' own positions: the scores of such columns rise from
the prefix's end towards the token, against which the attention takes its blocks."""
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import check, clean, ddt, inputs, run  # noqa: F401  (ddt: the fixture)

pytestmark = pytest.mark.gpu

STEEP = [0.25, 0.5, 0.70710678, 1.0]


@pytest.mark.parametrize("H,G,D", [(4, 4, 64), (4, 4, 128), (4, 1, 64), (4, 2, 128)])
@pytest.mark.parametrize("lens,full", [([(0, 512)], [512]), ([(0, 700), (0, 65)], [650, 65]), ([(500, 530)], [1000]),
                                       ([(0, 130), (3, 40)], [2000, 2000])])
@pytest.mark.parametrize("ctas", [0, 1, 5])
def test_prefix_ahead_of_the_tokens(ddt, H, G, D, lens, full, ctas):  # noqa: F811
    c = ref.Chunk(lens, 21, 16)
    q, k, v = inputs(c, H, G, D, 4 * H + D)
    kw = dict(slopes=torch.tensor(STEEP), full=full)
    out, ls = run(ddt, c, q, k, v, D ** -0.5, num_ctas=ctas, **kw)
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, D ** -0.5, **kw))


@pytest.mark.parametrize("slopes", [[0.25, 1.0], [-0.5, 30.0], [1000.0, -0.01], [8192.0, 1e-4]])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_long_prefix_and_slopes_of_any_size(ddt, slopes, cap):  # noqa: F811
    c = ref.Chunk([(0, 2048)], 22)
    q, k, v = inputs(c, 2, 1, 64, 5, 6.0 if cap else 1.5)
    kw = dict(cap=cap, slopes=torch.tensor(slopes), full=[2048])
    out, ls = run(ddt, c, q, k, v, 0.125, **kw)
    clean(ddt)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(ls).all())
    check(out, ls, ref.attention(q, k, v, c, 0.125, **kw))


def test_products_that_outweigh_the_distance(ddt):  # noqa: F811
    # columns behind the row's position whose products exceed the others' by more than the slope takes
    c = ref.Chunk([(10, 300)], 23)
    q, k, v = inputs(c, 2, 2, 128, 6)
    q = q.abs() + 1
    k[torch.from_numpy(c.slots[150:].astype("int64"))] = 8.0
    k[torch.from_numpy(c.slots[:150].astype("int64"))] = -8.0
    kw = dict(slopes=torch.tensor([3.0, 0.5]), full=[310])
    for ctas in (0, 1, 4):
        out, ls = run(ddt, c, q, k, v, 1.0, num_ctas=ctas, **kw)
        clean(ddt)
        check(out, ls, ref.attention(q, k, v, c, 1.0, **kw))
