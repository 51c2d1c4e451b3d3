"""Offsets of the grouped-query calls and of the cache rows that name part of
the rows, or that are broken: what is not a request's own stays as it was."""
import numpy as np
import pytest
import torch

from tests import _gqa_ref as ref
from tests import test_gqa_gpu as base

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ddt = base.ddt   # the fixture
clean, normal = base.clean, base.normal


# ---------------------------------------------------------------- append
def append_at(ddt, batch, qkv, w, table, H, G, D, depth, pools):
    """The append with `depth` per token as it is (or None); q_out is 7 before the call."""
    d = batch.device()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.to(DEV).split([H * D, G * D, G * D], 1))
    q_out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ddt.ddt_gqa_norm_rope_append(q, k, v, w[0].to(DEV), w[1].to(DEV), 1e-6, table.to(DEV),
                                 None if depth is None else depth.to(DEV), d["qo_indptr"], d["kv_indices"],
                                 d["kv_indptr"], q_out, pools[0], pools[1])
    return q_out


@pytest.mark.parametrize("B", [1, 3, 31, 32, 70])
@pytest.mark.parametrize("prefix,ahead", [(40, 5), (2, 5), (0, 5), (3, 60)])
@pytest.mark.parametrize("tree", [True, False])
def test_append_leaves_tokens_ahead_of_the_first_request(ddt, B, prefix, ahead, tree):
    # the offsets of a sub-batch: its first token is not the projection's first
    H, G, D = 4, 2, 64
    batch = ref.Batch([(prefix + k % 3, 1 + k % 4) for k in range(B)], 131, "tree" if tree else "chain")
    qkv, w, table = base.append_inputs(batch, H, G, D, 64, True, 132)
    wide = torch.cat([normal((ahead, qkv.shape[1]), 133), qkv])
    depth = torch.cat([torch.zeros(ahead, dtype=torch.int32), torch.from_numpy(np.concatenate(batch.depth).astype(np.int32))])
    batch.qo += ahead
    before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
    pools = [t.to(DEV) for t in before]
    q_out = append_at(ddt, batch, wide, w, table, H, G, D, depth if tree else None, pools)
    clean(ddt)
    assert (q_out[:ahead] == 7).all()
    base.check_append(batch, qkv, w, table, H, G, D, False, tree, before, q_out[ahead:], pools)


@pytest.mark.parametrize("more,index,value,bits", [(0, 1, 9, 0x1), (40, 4, 4, 0x3)])
def test_append_refuses_offsets_that_fall(ddt, more, index, value, bits):
    # few requests: qo 0 9 4 12, and the tokens 4 .. 8 count one offset up to them, which is request
    # 1's: it starts at 9.  Many: qo 0 4 9 12 4 14 .., and the search for them ends at request 2,
    # which starts at 9 (those behind it end at request 4, whose prefix would be negative)
    H, G, D = 4, 2, 64
    batch = ref.Batch([(20, 4), (20, 5), (20, 3)] + [(2, 1)] * more, 134, "chain")
    qkv, w, table = base.append_inputs(batch, H, G, D, 64, True, 135)
    before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
    if more == 0:
        batch.qo[2] = 4
    batch.qo[index] = value
    pools = [t.to(DEV) for t in before]
    q_out = append_at(ddt, batch, qkv, w, table, H, G, D, None, pools)
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (5, bits)
    assert (q_out[4:9] == 7).all()
    second = torch.from_numpy(batch.slots[24: 49].astype(np.int64))
    for pool, old in zip(pools, before):
        assert torch.equal(pool.cpu()[second], old[second])
