"""The grouped-query calls on values at the ends of what the types hold: finite
ones whose sums against a reference overflow, infinities and NaN in rows that
are seen and that are not."""
import numpy as np
import pytest
import torch

from tests import _gqa_ref as ref
from tests import test_gqa_gpu as base

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ddt = base.ddt   # the fixture
clean, normal = base.clean, base.normal


# ---------------------------------------------------------------- finite values
def rising(batch, H, D, first, power, seed):
    """Scores of ~0 in the first columns and ~33 log2 units above them behind: 64 such weights sum
    to less than 2^40, so the reference stays.  Values of about 2^power."""
    q, k, v, kd, vd = base.attn_inputs(batch, H, 1, D, seed, q_scale=0.01)
    at = torch.from_numpy(batch.slots.astype(np.int64))
    k[at, 0, 0] = 0.0
    for b in range(batch.B):
        k[at[int(batch.kv[b]) + first: int(batch.kv[b + 1])], 0, 0] = 0.71484375   # x 32: 33.0 log2 units
    q[:, :, 0] = 32.0
    v = (v.float() * 2.0 ** power).to(torch.bfloat16)
    kd.copy_(k)
    vd.copy_(v)
    return q, k, v, kd, vd


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,T", [(4, 4), (64, 3), (64, 5)])   # one tile; two; two and a lone third
@pytest.mark.parametrize("ctas", [0, 1, 3])
@pytest.mark.parametrize("first,power", [(64, 90), (128, 90), (128, 120), (300, 120)])
def test_attention_of_large_finite_values_is_finite(ddt, D, H, T, ctas, first, power):
    batch = ref.Batch([(600, T), (40, T)], 151, "tree")
    q, k, v, kd, vd = rising(batch, H, D, first, power, 152)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 1.0, ctas)
    clean(ddt)
    assert torch.isfinite(out).all()
    base.check_attn(out, ls, q, k, v, batch, 1.0)


@pytest.mark.parametrize("H,T", [(4, 4), (64, 33)])   # few rows and many: both forms of the join
@pytest.mark.parametrize("ctas", [0, 1, 12, 40])
def test_attention_joins_parts_of_the_largest_values(ddt, H, T, ctas):
    # every value 1.5 * 2^127: so is the result, and a sum of parts before its division is above the type
    batch = ref.Batch([(2500, T)], 153, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, 1, 64, 154, q_scale=0.1)
    v[:] = 1.5 * 2.0 ** 127
    vd.copy_(v)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    clean(ddt)
    # weights that sum to 1 within a bf16 rounding each: half a step of a result below 2^128
    assert ((out.double().cpu() / (1.5 * 2.0 ** 127) - 1).abs() <= 2.0 ** -8 * (1 + 2.0 ** -8) + 2.0 ** -8).all()
