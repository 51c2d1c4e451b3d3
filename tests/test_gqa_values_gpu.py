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


@pytest.mark.parametrize("H,T", [(4, 4), (64, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_whose_reference_moves_in_every_block_repeats_itself(ddt, H, T, D):
    # each block's weights are taken twice, and the second ones have to be those that count
    batch = ref.Batch([(3000, T)] * 20, 155, "tree")
    q, k, v, kd, vd = base.attn_inputs(batch, H, 1, D, 156, q_scale=0.01)
    at = torch.from_numpy(batch.slots.astype(np.int64))
    for b in range(batch.B):     # 64 natural units up every 64 columns
        n = int(batch.kv[b + 1] - batch.kv[b])
        k[at[int(batch.kv[b]): int(batch.kv[b + 1])], 0, 0] = (torch.arange(n) // 64 * 2.0).to(torch.bfloat16)
    q[:, :, 0] = 32.0
    kd.copy_(k)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, 1.0)
    clean(ddt)
    o, l, bo, bl = attention_on_device(q, kd, vd, batch, 1.0)
    assert ((out.double() - o).abs() <= bo).all() and ((ls.double() - l).abs() <= bl).all()
    for ctas in (0, 0, 0, 0):
        again, ls2 = base.run_attn(ddt, batch, q, kd, vd, 1.0, ctas)
        assert torch.equal(again, out) and torch.equal(ls2, ls)
    clean(ddt)


# ---------------------------------------------------------------- infinities and NaN
def attention_on_device(q, kd, vd, batch, scale):
    """ref.attention in float64 on the device, request by request and K/V head by K/V head, for long
    requests; infinities and NaN in V reach the rows that see them alone.  The same bounds."""
    T, H, D = q.shape
    G = kd.shape[1]
    u, h8 = 2.0 ** -24, 2.0 ** -8
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -torch.inf, dtype=torch.float64, device=DEV)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(batch.B):
        lo, hi = int(batch.qo[b]), int(batch.qo[b + 1])
        rows = torch.from_numpy(batch.slots[batch.kv[b]: batch.kv[b + 1]].astype(np.int64)).to(DEV)
        vis = torch.from_numpy(batch.vis[b]).to(DEV)
        any_seen, N = vis.any(0), int(vis.sum(1).max()) if vis.numel() else 0
        for g in range(G if hi > lo else 0):
            heads = slice(g * (H // G), (g + 1) * (H // G))
            x = q[lo:hi, heads].to(DEV).double()
            K, V = kd[rows, g].double(), vd[rows, g].double()
            K = torch.where(any_seen[:, None], K, 0.0)
            see = vis[:, None, :].expand(-1, H // G, -1)
            s = (scale * torch.einsum("thd,nd->thn", x, K)).masked_fill(~see, -torch.inf)
            size = (scale * torch.einsum("thd,nd->thn", x.abs(), K.abs())).masked_fill(~see, 0.0).amax(-1)
            ds = (D + 2) * u * size + 4 * u * s.masked_fill(~see, 0.0).abs().amax(-1)
            m = s.amax(-1, keepdim=True).clamp_min(-1e300)
            w = torch.exp(s - m).masked_fill(~see, 0.0)
            total = w.sum(-1)
            p = w / total.clamp_min(1e-300)[..., None]
            fin = torch.where(torch.isfinite(V), V, 0.0)
            o = torch.einsum("thn,nd->thd", p, fin)
            one = see.double()
            plus = torch.einsum("thn,nd->thd", one, ((V == torch.inf) | V.isnan()).double()) > 0
            minus = torch.einsum("thn,nd->thd", one, ((V == -torch.inf) | V.isnan()).double()) > 0
            away = torch.einsum("thn,nd->thd", p, fin.abs())
            b_out[lo:hi, heads] = h8 * o.abs() + away * (h8 * (1 + h8) + 2 * ds[..., None] + (2 * N + 32) * u)
            o = o + torch.where(plus, torch.inf, 0.0) + torch.where(minus, -torch.inf, 0.0)
            l = m[..., 0] + torch.log(total)
            out[lo:hi, heads], lse[lo:hi, heads] = o, l
            b_lse[lo:hi, heads] = (ds + (N + 32) * u + 8 * u * l.abs()).masked_fill(total == 0, 0.0)
    return out, lse, b_out, b_lse


def check_on_device(out, ls, q, kd, vd, batch, scale):
    o, l, bo, bl = attention_on_device(q, kd, vd, batch, scale)
    got, fin = out.double(), torch.isfinite(o)
    assert torch.equal(got.isnan(), o.isnan()) and torch.equal(got == torch.inf, o == torch.inf)
    assert torch.equal(got == -torch.inf, o == -torch.inf)
    err = ((got - o).abs() - bo)[fin]
    assert err.numel() == 0 or float(err.max()) <= 0, f"out over its bound by {float(err.max())}"
    seen = torch.isfinite(l)
    assert torch.equal(torch.isfinite(ls), seen) and ((ls.double() - l).abs() <= bl)[seen].all()


def test_the_form_on_the_device_equals_the_loops(ddt):
    batch = ref.Batch([(90, 9), (0, 3), (33, 40)], 161, "random")
    q, k, v, kd, vd = base.attn_inputs(batch, 12, 4, 64, 162)
    got, want = attention_on_device(q, kd, vd, batch, 0.1), ref.attention(q, k, v, batch, 0.1)
    for x, y in zip(got[:2], want[:2]):
        torch.testing.assert_close(x.cpu(), y, rtol=1e-9, atol=1e-12)
    # the loops count every column of a request among its sums, this form the seen ones
    assert all((x.cpu() <= y * (1 + 1e-9)).all() for x, y in zip(got[2:], want[2:]))


@pytest.mark.parametrize("H,G,D,lens", [
    (8, 2, 64, [(21, 9), (170, 3)]), (64, 2, 128, [(333, 5), (64, 17), (0, 1)]), (12, 1, 64, [(250, 30), (47, 11)]),
    (40, 8, 128, [(127, 33), (3, 17), (250, 1)]), (128, 1, 64, [(511, 3)]), (5, 5, 128, [(700, 1), (2, 1)]),
])
@pytest.mark.parametrize("mask", ["tree", "random"])
@pytest.mark.parametrize("ctas", [0, 1, 3, 29])
def test_attention_of_infinities_and_nan_in_any_place(ddt, H, G, D, lens, mask, ctas):
    # one value in a few hundred, each in the rows that see it alone and with its own sign
    batch = ref.Batch(lens, 163 + H, mask)
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 164, strided=True)
    rng = torch.Generator().manual_seed(165)
    for value in (float("inf"), float("-inf"), float("nan")):
        hit = torch.rand(v.shape, generator=rng) < 3.0 / len(v) / 8
        v[hit] = value
    vd.copy_(v)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5, ctas)
    clean(ddt)
    check_on_device(out, ls, q, kd, vd, batch, D ** -0.5)


LONG = [(20000, 33), (3000, 17), (20000, 9), (700, 33), (9000, 1)]


@pytest.mark.parametrize("H,G,D", [(16, 2, 128), (64, 2, 64)])
@pytest.mark.parametrize("ctas", [0, 5, 64])
@pytest.mark.parametrize("where", ["node", "hidden", "seen", "all"])
def test_attention_of_a_long_request_with_infinities_serves_the_others(ddt, H, G, D, ctas, where):
    """NaN and infinities in one long request's rows: in a node's, in prefix rows that none of its
    nodes sees, in some that all see, in every row.  What it costs is its CTAs' time: the waits of
    other warps do not run out, and the other requests get the bits they get without."""
    batch = ref.Batch(LONG, 171, "tree")
    if where == "hidden":
        batch.vis[0][:, 5:20000:401] = False
        batch.words = np.concatenate([ref.pack_bits(x) for x in batch.vis])
    q, k, v, kd, vd = base.attn_inputs(batch, H, G, D, 172, q_scale=0.5)
    first, first_lse = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5, ctas)
    clean(ddt)
    cols = {"node": [20000 + 7], "hidden": range(5, 20000, 401), "seen": [3, 9000, 9001], "all": range(20033)}[where]
    for n, c in enumerate(cols):
        r = int(batch.slots[c])
        v[r, 0] = (float("nan"), float("inf"), float("-inf"))[n % 3]
        if where == "hidden":
            k[r] = float("nan")
    kd.copy_(k)
    vd.copy_(v)
    out, ls = base.run_attn(ddt, batch, q, kd, vd, D ** -0.5, ctas)
    clean(ddt)
    assert torch.equal(out[33:], first[33:]) and torch.equal(ls, first_lse)
    assert torch.equal(out[:, H // G:], first[:, H // G:])
    check_on_device(out, ls, q, kd, vd, batch, D ** -0.5)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_norms_values_up_to_its_bound(ddt, D, interleaved):
    # every value of a row +-2^60, the largest that the documentation allows: D of their squares sum
    # to 2^127 at most; rows of ordinary size next to them in a warp
    H, G = 8, 2
    batch = ref.Batch([(4, 9)], 181, "tree")
    qkv, w, table = base.append_inputs(batch, H, G, D, 64, True, 182)
    rows = qkv.view(9, H + 2 * G, D)
    for t in range(9):
        big = (torch.arange(H + 2 * G) + t) % 3 > 0
        rows[t, big] = torch.where(rows[t, big] < 0, -1.0, 1.0).to(torch.bfloat16) * 2.0 ** 60
    before = normal((batch.rows, G, D), 1), normal((batch.rows, G, D), 2)
    pools = [t.to(DEV) for t in before]
    q_out = base.run_append(ddt, batch, qkv, w, table, H, G, D, interleaved, True, pools)
    clean(ddt)
    assert torch.isfinite(q_out).all() and (q_out != 0).any(-1).all()
    base.check_append(batch, qkv, w, table, H, G, D, interleaved, True, before, q_out, pools)
