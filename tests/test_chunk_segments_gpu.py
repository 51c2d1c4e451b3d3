"""Many short requests in few CTAs: a CTA goes through segment after segment of a single block, each with
rows, poison and tiles of its own."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import check, clean, ddt, inputs, run  # noqa: F401  (ddt: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,D", [(2, 2, 64), (2, 2, 128), (16, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("ctas", [1, 2])
def test_values_that_are_not_finite_stay_in_their_requests(ddt, H, G, D, ctas):  # noqa: F811
    # every other request has a column of V that is not finite and that its last tokens alone see
    rng = np.random.default_rng(H + D)
    c = ref.Chunk([(0, int(t)) for t in rng.integers(2, 41, 70)], 8)
    q, k, v = inputs(c, H, G, D, 17)
    for b in range(0, c.B, 2):
        rows = c.slots[c.kv[b]: c.kv[b + 1]].astype(np.int64)
        j = int(rng.integers(1, c.T[b]))
        v[rows[j], :, int(rng.integers(D))] = [torch.nan, torch.inf, -torch.inf][b // 2 % 3]
    out, ls = run(ddt, c, q, k, v, D ** -0.5, num_ctas=ctas)
    again, _ = run(ddt, c, q, k, v, D ** -0.5, num_ctas=ctas)
    clean(ddt)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    got = out.double().cpu()
    bad = ~torch.isfinite(v)
    plain = ref.attention(q, k, v.masked_fill(bad, 0.0), c, D ** -0.5)
    want, special = plain[0].clone(), torch.zeros(got.shape, dtype=torch.bool)
    for b in range(c.B):
        rows = torch.from_numpy(c.slots[c.kv[b]: c.kv[b + 1]].astype(np.int64))
        for j, g, e in zip(*(x.tolist() for x in torch.nonzero(bad[rows], as_tuple=True))):
            heads = slice(g * (H // G), (g + 1) * (H // G))
            want[int(c.qo[b]) + j: int(c.qo[b + 1]), heads, e] = float(v[rows[j], g, e])
            special[int(c.qo[b]) + j: int(c.qo[b + 1]), heads, e] = True
    assert torch.equal(torch.nan_to_num(got[special], 5.5), torch.nan_to_num(want[special], 5.5))
    zero = torch.zeros_like(got)
    check(torch.where(special, zero, got), ls, (torch.where(special, zero, plain[0]), *plain[1:]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7])
def test_single_blocks_of_one_tile_between_two_tiles(ddt, D, ctas):  # noqa: F811
    rng = np.random.default_rng(D)
    lens = [(int(rng.integers(0, 90)), int(rng.integers(17, 33) if b % 3 == 0 else rng.integers(1, 17))) for b in range(120)]
    c = ref.Chunk(lens, 9)
    q, k, v = inputs(c, 16, 2, D, 5)
    out, ls = run(ddt, c, q, k, v, D ** -0.5, num_ctas=ctas)
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, D ** -0.5))
