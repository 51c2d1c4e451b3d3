"""Offsets of the grouped-query calls and of the cache rows that name part of
the rows, or that are broken: what is not a request's own stays as it was."""
import functools

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


LOW, HIGH = -2 ** 31, 2 ** 31 - 1   # their differences do not fit 32 bits
LENS = [(300, 9), (40, 5), (280, 3), (500, 7)]
# field, index, value (None: one more), and the latched bits; a border breaks the requests at both sides
BROKEN = [("qo", 2, LOW, 0x1), ("qo", 2, -1, 0x1), ("qo", 2, HIGH, 0x1), ("qo", 2, None, 0x8), ("qo", 4, LOW, 0x1),
          ("kv", 2, LOW, 0x2), ("kv", 2, -1, 0x2), ("kv", 2, HIGH, 0x2), ("kv", 2, 5000, 0x2), ("kv", 4, LOW, 0x2), ("kv", 4, HIGH, 0x2),
          ("mask_indptr", 2, LOW, 0x8), ("mask_indptr", 2, HIGH, 0x8), ("mask_indptr", 2, None, 0x8), ("mask_indptr", 4, LOW, 0x8)]


def broken(batch, field, index, value):
    """The requests and the tokens that the changed offset leaves alone."""
    good = [b for b in range(batch.B) if b not in (index - 1, index)]
    keep = torch.zeros(batch.total_q, dtype=torch.bool)
    for b in good:
        keep[int(batch.qo[b]): int(batch.qo[b + 1])] = True
    offsets = getattr(batch, field)
    offsets[index] = offsets[index] + 1 if value is None else value
    return good, keep


@functools.lru_cache
def attention_case(H):
    batch = ref.Batch(LENS, 136, "tree")
    made = base.attn_inputs(batch, H, 2, 64, 137)
    return made, ref.attention(*made[:3], batch, 0.1)


@pytest.mark.parametrize("field,index,value,bits", BROKEN)
@pytest.mark.parametrize("ctas", [0, 1, 5])
@pytest.mark.parametrize("H", [4, 64])
@pytest.mark.parametrize("bound", [False, True])
def test_attention_of_broken_offsets_leaves_the_request_and_serves_the_others(ddt, field, index, value, bits, ctas, H, bound):
    batch = ref.Batch(LENS, 136, "tree")
    (q, _, _, kd, vd), (o, l, bo, bl) = attention_case(H)
    if bound:       # the caller's bound leaves all to the offsets
        batch.max_kv = HIGH
    good, keep = broken(batch, field, index, value)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    torch.cuda.synchronize()
    st, latched = ddt.ddt_get_error()
    assert st == 5 and latched & bits and not latched & ~0xb, latched
    out, ls = out.cpu(), ls.cpu()
    assert (out[~keep] == 7).all() and (ls[~keep] == 7).all()
    assert ((out.double() - o).abs() <= bo)[keep].all() and ((ls.double() - l).abs() <= bl)[keep].all()


@pytest.mark.parametrize("qo,kv", [((HIGH, LOW), (0, 300)), ((0, 9), (1, LOW)), ((LOW, HIGH), (0, 300)), ((0, 9), (LOW, HIGH)),
                                   ((0, 9), (HIGH, HIGH)), ((HIGH, HIGH), (0, 300))])
@pytest.mark.parametrize("ctas", [0, 1])
def test_attention_of_one_request_between_extremes(ddt, qo, kv, ctas):
    batch = ref.Batch([(291, 9)], 138, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, 4, 2, 64, 139)
    batch.qo[:], batch.kv[:], batch.max_kv = qo, kv, HIGH
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1, ctas)
    torch.cuda.synchronize()
    st, bits = ddt.ddt_get_error()
    assert st == 5 and bits & 0xb and not bits & ~0xb
    assert (out == 7).all() and (ls == 7).all()


def test_attention_counts_mask_words_beyond_32_bits(ddt):
    # 128 rows of 2^25 words are 2^32 words, which 32 bits take for none
    N = 1 << 30
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    idx = torch.zeros(N, dtype=torch.int32, device=DEV)
    q = torch.ones(128, 4, 64, dtype=torch.bfloat16, device=DEV)
    pool = torch.ones(8, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 7.0)
    for ctas in (0, 3):
        ddt.ddt_gqa_verify_attn(q, pool, pool, idx, i32(0, N), i32(0, 128), i32(-1), i32(0, 0), 0.1, out,
                                max_q_len=128, max_kv_len=N, num_ctas=ctas)
        torch.cuda.synchronize()
        assert ddt.ddt_get_error() == (5, 0x8)
        assert (out == 7).all()


@pytest.mark.parametrize("field,index,value,bits", [b for b in BROKEN if b[0] != "mask_indptr" and b[2] is not None])
def test_append_of_broken_offsets_leaves_the_request_and_serves_the_others(ddt, field, index, value, bits):
    H, G, D = 4, 2, 64
    batch = ref.Batch(LENS, 140, "chain")
    qkv, w, table = base.append_inputs(batch, H, G, D, 64, True, 141)
    before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
    # what the call does with whole offsets
    whole = [t.to(DEV) for t in before]
    want = append_at(ddt, batch, qkv, w, table, H, G, D, None, whole).cpu()
    clean(ddt)
    base.check_append(batch, qkv, w, table, H, G, D, False, False, before, want, whole)
    new = [torch.from_numpy(batch.slots[batch.kv[b + 1] - t: batch.kv[b + 1]].astype(np.int64)) for b, (_, t) in enumerate(LENS)]
    good, keep = broken(batch, field, index, value)
    pools = [t.to(DEV) for t in before]
    q_out = append_at(ddt, batch, qkv, w, table, H, G, D, None, pools).cpu()
    torch.cuda.synchronize()
    st, latched = ddt.ddt_get_error()
    assert (st, latched) == (5, bits)
    # A token's request is the number of offsets up to it, so a border below all others sends
    # every token ahead of it one request on, and one above all others every token behind one back:
    # both to a request that does not have them.
    if field == "qo":
        good = [b for b in good if (b > index if value < 0 else b < index)]
        for b in set(range(batch.B)) - set(good):
            keep[sum(t for _, t in LENS[:b]): sum(t for _, t in LENS[:b + 1])] = False
    assert torch.equal(q_out[keep], want[keep]) and (q_out[~keep] == 7).all()
    for pool, old, full in zip(pools, before, whole):
        mine = old.clone()
        for b in good:
            mine[new[b]] = full.cpu()[new[b]]
        assert torch.equal(pool.cpu(), mine)


@pytest.mark.parametrize("field,value", [("qo", LOW), ("qo", HIGH), ("kv", LOW), ("kv", HIGH), ("kv", -1)])
def test_commit_of_broken_offsets_leaves_the_request_and_serves_the_others(ddt, field, value):
    batch = ref.Batch(LENS, 142, "tree")
    alen, nodes = base.commit_inputs(batch, 5)
    p = base.slab(3, batch.rows, 64, 143)
    come, new = torch.arange(batch.rows), (batch.P + alen).tolist()
    good, _ = broken(ref.Batch(LENS, 142, "tree"), field, 2, value)
    for b in range(batch.B):
        root = int(batch.kv[b + 1] - batch.T[b])
        for k in range(alen[b] if b in good else 0):
            come[batch.slots[root + k]] = int(batch.slots[root + nodes[b][k]])
        if b not in good:
            new[b] = -5
    want = p.cpu()[:, come]
    broken(batch, field, 2, value)
    d = batch.device()
    new_len = torch.full((batch.B,), -5, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_commit(p, d["kv_indices"], d["kv_indptr"], d["qo_indptr"], torch.from_numpy(alen).to(DEV),
                         torch.from_numpy(nodes).to(DEV), 7, new_len)
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (5, 0x200)
    assert torch.equal(p.cpu(), want) and new_len.cpu().tolist() == new


# ---------------------------------------------------------------- nothing to do
@pytest.mark.parametrize("cached", [0, 300])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_a_batch_without_new_tokens_is_left_alone(ddt, B, cached):
    # padding: rows of q that belong to no request; the mask, and without cached rows the slots, are empty
    batch = ref.Batch([(cached, 0)] * B, 144, "tree")
    H, G, D = 8, 2, 64
    q = normal((5, H, D), 145)
    pool = normal((max(batch.rows, 1), G, D), 146).to(DEV)
    before = pool.clone()
    assert batch.words.size == 0 and (cached > 0 or batch.slots.size == 0)
    for ctas, max_q in ((0, 0), (0, 4), (3, 4)):
        batch.max_q, batch.max_kv = max_q, cached + 8
        out, ls = base.run_attn(ddt, batch, q, pool, pool, 0.1, ctas)
        clean(ddt)
        assert (out == 7).all() and (ls == 7).all()
    qkv, w, table = torch.ones(5, (H + 2 * G) * D, dtype=torch.bfloat16), [torch.ones(D, dtype=torch.bfloat16)] * 2, torch.ones(9, 64)
    q_out = append_at(ddt, batch, qkv, w, table, H, G, D, None, [pool, pool.clone()])
    clean(ddt)
    assert (q_out == 7).all() and torch.equal(pool, before)
    d = batch.device()
    zero, new_len = torch.zeros(B, dtype=torch.int32, device=DEV), torch.full((B,), -5, dtype=torch.int32, device=DEV)
    ddt.ddt_cache_commit(pool[None], d["kv_indices"], d["kv_indptr"], d["qo_indptr"], zero, zero[:, None].expand(-1, 8).contiguous(), 7, new_len)
    clean(ddt)
    assert torch.equal(pool, before) and (new_len == cached).all()


def test_a_call_takes_an_empty_array_for_none(ddt):
    # one request has new tokens, and the arrays say that it has no slots: refused on the device
    batch = ref.Batch([(0, 2)], 147, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, 4, 2, 64, 148)
    batch.slots, batch.words = batch.slots[:0], batch.words[:0]
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 0.1)
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (5, 0x2)
    assert (out == 7).all() and (ls == 7).all()


# ---------------------------------------------------------------- another stream
def test_attention_reads_its_bounds_on_the_calls_stream(ddt):
    # offsets that the call's stream writes late, without the host's bounds
    batch = ref.Batch([(300, 4), (20, 9)], 149, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, 8, 2, 64, 150)
    d, qd = batch.device(), q.to(DEV)
    late = {n: torch.zeros_like(d[n]) for n in ("qo_indptr", "kv_indptr")}
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    call = lambda **kw: ddt.ddt_gqa_verify_attn(  # noqa: E731
        qd, kd, vd, d["kv_indices"], late["kv_indptr"], late["qo_indptr"], d["mask"], d["mask_indptr"], 0.1, out, **kw)
    call()      # of requests without tokens; loads what the calls below run
    with torch.cuda.stream(s):
        torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    assert (out == 7).all()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
        for n, t in late.items():
            t.copy_(d[n])
    call(stream=s)
    clean(ddt)
    base.check_attn(out, None, q, k, v, batch, 0.1)
