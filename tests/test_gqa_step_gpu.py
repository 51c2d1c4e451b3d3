"""A verify step of a stack of grouped-query layers through GqaVerifyStep, as a
model would run it, against the CPU oracle (tree, mask, accept) and plain
64-bit forms (layers and cache rows)."""
import numpy as np
import pytest
import torch

from tests import _gqa_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_decoding_gb300 import _build
    _build.build()
    from tree_speculative_decoding_gb300 import ddt
    ddt.ddt_get_error()
    return ddt


def workload(seed, prefix, budget):
    from tree_speculative_decoding_gb300 import workloads
    return workloads.make_workload("gqa", seed, len(prefix), 1, prefix, budget, 6, 256, 1.5,
                                   pool_rows=sum(prefix) + sum(budget) + 60, fill_pool=False)


def as_batch(wl, parent, depth):
    """The workload's requests, slots and given trees as a ref.Batch."""
    batch = ref.Batch([(int(p), int(t)) for p, t in zip(wl.prefix_len, wl.q_len)], 0, rows=wl.pool_rows)
    batch.slots = wl.kv_indices
    cut = lambda a: [a[lo:hi].tolist() for lo, hi in zip(wl.qo_indptr[:-1], wl.qo_indptr[1:])]  # noqa: E731
    batch.parent, batch.depth = cut(parent), cut(depth)
    batch.vis = [ref.tree_visibility(int(p), par) for p, par in zip(wl.prefix_len, batch.parent)]
    return batch


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def table(rows, R):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))


@pytest.mark.parametrize("H,G,D,layers,prefix,budget", [
    (8, 2, 128, 2, [21, 300, 0], [8, 16, 3]),      # one tile of rows per K/V head
    (16, 2, 64, 3, [200, 517], [32, 0]),           # two tiles, and an item dealt to several CTAs
])
def test_step(lib, oracle_mod, H, G, D, layers, prefix, budget):
    from tree_speculative_decoding_gb300.pipeline import GqaVerifyStep
    wl = workload(0x6A0 + H, prefix, budget)
    tok, par, dep = oracle_mod.build_tree(wl.topk_logp, wl.topk_ids, wl.root_id, wl.budget, wl.qo_indptr,
                                          wl.max_depth, wl.K)
    batch = as_batch(wl, par, dep)
    argmax = oracle_mod.best_child_argmax(par, wl.qo_indptr, tok, np.ones(wl.total_q, bool), wl.argmax_random)
    cs = table(max(prefix) + wl.max_depth + 1, D)
    step = GqaVerifyStep(wl, layers, H, G, D, cos_sin=cs.to(DEV), device=DEV)
    cache = normal(step.kv.shape, 1)
    weights = [(normal((D,), 50 + i, 0.3) + 1.0).to(torch.bfloat16) for i in range(2 * layers)]
    wd = [w.to(DEV) for w in weights]
    proj = torch.empty((layers, wl.total_q, (H + 2 * G) * D), dtype=torch.bfloat16, device=DEV)
    target = torch.from_numpy(argmax.astype(np.int32)).to(DEV)
    qs = torch.empty((layers,) + step.q.shape, dtype=torch.bfloat16, device=DEV)
    outs = torch.empty_like(qs)
    slots = torch.from_numpy(wl.kv_indices.astype(np.int32)).to(DEV)

    def whole_step():
        step.build_tree_visibility()
        for n in range(layers):
            q, k, v = (t.unflatten(1, (-1, D)) for t in proj[n].split([H * D, G * D, G * D], 1))
            outs[n].copy_(step.layer(n, q, k, v, wd[2 * n], wd[2 * n + 1]))
            qs[n].copy_(step.q)
        step.accept(target)
        step.commit()

    def start(seed):
        x = normal(proj.shape, seed, 2.0)
        proj.copy_(x)
        step.kv.copy_(cache)
        step.kv_indices.copy_(slots)
        return x

    def check(x):
        torch.cuda.synchronize()
        step.check_device_errors()
        assert np.array_equal(step.node_token.cpu().numpy(), tok) and np.array_equal(step.parent.cpu().numpy(), par)
        assert np.array_equal(step.depth.cpu().numpy(), dep)
        pos = torch.from_numpy(np.concatenate([p + np.array(d, np.int64) for p, d in zip(batch.P, batch.depth)]))
        new = torch.cat([torch.from_numpy(batch.slots[batch.kv[b + 1] - t: batch.kv[b + 1]].astype(np.int64))
                         for b, (_, t) in enumerate(batch.lens)])
        alen, acc, com, bonus = oracle_mod.accept(tok, par, wl.qo_indptr, argmax, wl.max_depth)
        assert alen.max() > 1
        for got, want in ((step.accept_len, alen), (step.accepted_nodes, acc), (step.commit_tokens, com),
                          (step.bonus, bonus), (step.new_len, wl.prefix_len + alen)):
            assert np.array_equal(got.cpu().numpy(), want)
        come = torch.arange(wl.pool_rows)
        for b, n in enumerate(alen):
            root = int(batch.kv[b + 1] - batch.T[b])
            for k in range(n):
                come[batch.slots[root + k]] = int(batch.slots[root + acc[b][k]])
        for n in range(layers):
            q, k, v = (t.unflatten(1, (-1, D)) for t in x[n].split([H * D, G * D, G * D], 1))
            y, tol = ref.norm_rope(q, weights[2 * n], 1e-6, cs, pos, False)
            rotated = qs[n].cpu()
            assert ((rotated.double() - y).abs() <= tol).all()
            yk, tk = ref.norm_rope(k, weights[2 * n + 1], 1e-6, cs, pos, False)
            # the cache before the commit: the old rows, and the new ones within their roundings.  The
            # attention is then held to its bound on the rows that it read; these are read back through
            # a second append, whose rows are the same, bit for bit.
            kp, vp = cache[2 * n].clone(), cache[2 * n + 1].clone()
            d = batch.device()
            kd, vd, q2 = kp.to(DEV), vp.to(DEV), torch.empty_like(step.q)
            xd = [t.unflatten(1, (-1, D)) for t in x[n].to(DEV).split([H * D, G * D, G * D], 1)]
            lib.ddt_gqa_norm_rope_append(*xd, wd[2 * n], wd[2 * n + 1], 1e-6, step.cos_sin, d["depth"], d["qo_indptr"],
                                         slots, d["kv_indptr"], q2, kd, vd)
            assert torch.equal(q2.cpu(), rotated)
            kp, vp = kd.cpu(), vd.cpu()
            assert ((kp[new].double() - yk).abs() <= tk).all() and torch.equal(vp[new], v)
            o, _, bound, _ = ref.attention(rotated, kp, vp, batch, D ** -0.5)
            assert ((outs[n].double().cpu() - o).abs() <= bound).all()
            assert torch.equal(step.kv[2 * n].cpu(), kp[come]) and torch.equal(step.kv[2 * n + 1].cpu(), vp[come])
        return acc

    x = start(3)
    whole_step()
    check(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole_step()
    for seed in (4, 5):
        x = start(seed)
        graph.replay()
        check(x)

    # a request's row forked to a free one, then everything in use to the front
    before = step.kv.cpu()
    free = next(r for r in range(wl.pool_rows) if r not in set(wl.kv_indices.tolist()))
    a = torch.tensor([int(wl.kv_indices[0])], dtype=torch.int32, device=DEV)
    b = torch.tensor([free], dtype=torch.int32, device=DEV)
    step.copy(a, b)
    step.kv_indices[0] = free
    before[:, free] = before[:, int(a)]
    used = wl.kv_indices.copy()
    used[0] = free
    want_slots, live, come = ref.compact(used.tolist(), wl.pool_rows)
    step.compact()
    torch.cuda.synchronize()
    step.check_device_errors()
    assert step.kv_indices.cpu().tolist() == want_slots and step.live.item() == live
    assert torch.equal(step.kv.cpu(), before[:, torch.tensor(come)])


def test_prefill_chunk_through_the_step(lib):
    # the causal chain in place of the tree: every token sees the prefix and the tokens before it
    from tree_speculative_decoding_gb300.pipeline import GqaVerifyStep
    wl = workload(0x6C1, [40, 7], [20, 9])
    H, G, D = 4, 1, 64
    T = wl.q_len
    par = np.concatenate([np.arange(-1, t - 1) for t in T]).astype(np.int32)
    dep = np.concatenate([np.arange(t) for t in T]).astype(np.int32)
    batch = as_batch(wl, par, dep)
    step = GqaVerifyStep(wl, 1, H, G, D, device=DEV)
    cache = normal(step.kv.shape, 8)
    step.kv.copy_(cache)
    q, k, v = normal((wl.total_q, H, D), 1), normal((wl.total_q, G, D), 2), normal((wl.total_q, G, D), 3)
    step.build_chain_visibility()
    out = step.layer(0, q.to(DEV), k.to(DEV), v.to(DEV))
    torch.cuda.synchronize()
    step.check_device_errors()
    kp, vp = step.kv[0].cpu(), step.kv[1].cpu()
    new = torch.cat([torch.from_numpy(batch.slots[batch.kv[b + 1] - t: batch.kv[b + 1]].astype(np.int64))
                     for b, t in enumerate(T)])
    assert torch.equal(kp[new], k) and torch.equal(vp[new], v)     # no norm and no table: copied
    o, _, bound, _ = ref.attention(q, kp, vp, batch, D ** -0.5)
    assert ((out.double().cpu() - o).abs() <= bound).all()
