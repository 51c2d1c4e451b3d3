"""Eviction on the GPU, exact against a plain form (tests/_chunk_ref.py)."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_chunk_gpu import DEV, clean, ddt  # noqa: F401  (ddt: the fixture)

pytestmark = pytest.mark.gpu


def weights_of(kind, n, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n, generator=g).mul(2).exp()
    if kind == "ties":       # few values, zeros of both signs among them
        w = torch.randint(-1, 3, (n,), generator=g).float()
        w[::5] = -0.0
    elif kind == "same":
        w = torch.full((n,), 0.25)
    elif kind == "odd":      # infinities, NaN, denormal and negative values
        w = torch.randn(n, generator=g) * 1e-42
        w[::3] = torch.randn(len(w[::3]), generator=g)
        for i, x in enumerate((torch.inf, -torch.inf, torch.nan, -torch.nan)):
            w[i::17] = x
    return w


def run(ddt, w, lens, budget, sinks, recent, seed=1, spare=0, **kw):  # noqa: F811
    total = int(sum(lens))
    slots = np.random.default_rng(seed).permutation(total + 9)[:total].astype(np.int32)
    kept = sum(min(n, max(0, b)) for n, b in zip(lens, budget))
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device=DEV)  # noqa: E731
    new, gone = i32([-7] * (kept + spare)), i32([-7] * (total - kept + spare))
    new_w = torch.full((kept + spare,), -7.0, device=DEV)
    indptr = i32([-7] * (len(lens) + 1))
    ddt.ddt_cache_evict(w.to(DEV), i32(slots), i32(np.concatenate([[0], np.cumsum(lens)])), i32(budget), new, indptr, new_w, gone,
                        sinks=sinks, recent=recent, **kw)
    clean(ddt)
    stay, want_indptr, want_w, go = ref.evict(w, slots, lens, budget, sinks, recent)
    assert indptr.tolist() == want_indptr
    assert new.tolist() == stay + [-7] * spare and gone.tolist() == go + [-7] * spare
    got = new_w[:kept].cpu()
    assert torch.equal(got.view(torch.int32), torch.tensor(want_w, dtype=torch.float32).view(torch.int32)) or \
        torch.equal(torch.nan_to_num(got, 5.5), torch.nan_to_num(torch.tensor(want_w, dtype=torch.float32), 5.5))


CASES = [
    # columns, budgets, sinks, recent
    ([1], [1], 0, 0), ([1], [0], 0, 0), ([0], [5], 2, 2), ([33], [7], 2, 3), ([33], [-4], 2, 3),
    ([100, 0, 7, 31, 32, 1025], [50, 3, 7, 100, 0, 1], 4, 8),
    ([4097], [2048], 4, 256), ([500], [10], 8, 8), ([500], [10], 600, 600), ([500], [499], 0, 1),
    ([8192], [100], 4, 10), ([8193], [4000], 4, 10), ([20000, 5, 16385], [1024, 5, 16384], 4, 100),
    ([70000], [33000], 16, 1024),
]


@pytest.mark.parametrize("lens,budget,sinks,recent", CASES)
@pytest.mark.parametrize("kind", ["spread", "ties", "same", "odd"])
def test_evict(ddt, lens, budget, sinks, recent, kind):  # noqa: F811
    run(ddt, weights_of(kind, sum(lens), 3), lens, budget, sinks, recent, spare=3)


def test_many_requests(ddt):  # noqa: F811
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 40, 1500)]
    run(ddt, weights_of("ties", sum(lens), 4), lens, [int(n) for n in rng.integers(0, 30, 1500)], 2, 3)


@pytest.mark.parametrize("n", [131072, 8 * 45056 + 777])
def test_long_requests(ddt, n):  # noqa: F811
    # the second has more columns than a cluster's shared memory
    run(ddt, weights_of("spread", n + 9, 6), [n, 9], [n // 8, 4], 4, 1000)


def test_columns_ahead_of_the_first_request_and_no_optional_outputs(ddt):  # noqa: F811
    w = weights_of("spread", 60, 2).to(DEV)
    slots = torch.arange(60, dtype=torch.int32, device=DEV)
    new, indptr = torch.full((20,), -7, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    kv = torch.tensor([10, 40, 60], dtype=torch.int32, device=DEV)
    budget = torch.tensor([12, 5], dtype=torch.int32, device=DEV)
    ddt.ddt_cache_evict(w, slots, kv, budget, new, indptr)
    clean(ddt)
    stay, want, _, _ = ref.evict(w[10:].cpu(), np.arange(10, 60), [30, 20], [12, 5], 0, 0)
    assert indptr.tolist() == want and new.tolist() == stay + [-7] * 3


def test_bad_data_is_latched(ddt):  # noqa: F811
    w = torch.ones(50, device=DEV)
    slots = torch.arange(50, dtype=torch.int32, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def go(kv, room=30, max_kv_len=50, go_room=50):
        new, gone, indptr = torch.full((40,), -7, dtype=torch.int32, device=DEV), torch.full((60,), -7, dtype=torch.int32, device=DEV), i32(0, 0, 0, 0)
        ddt.ddt_cache_evict(w, slots, i32(*kv), i32(5, 5, 5), new[:room], indptr, None, gone[:go_room], max_kv_len=max_kv_len)
        torch.cuda.synchronize()
        assert bool((new[room:] == -7).all()) and bool((gone[go_room:] == -7).all())
        return indptr.tolist(), new.tolist(), ddt.ddt_get_error()[1]

    assert go([0, 10, 20, 50]) == ([0, 5, 10, 15], [0, 1, 2, 3, 4, 10, 11, 12, 13, 14, 20, 21, 22, 23, 24] + [-7] * 25, 0)
    for kv, left in (([0, 10, 20, 51], [0, 5, 10, 10]), ([0, 10, 5, 50], [0, 5, 5, 10]), ([-1, 10, 20, 50], [0, 0, 5, 10])):
        indptr, new, bits = go(kv)
        assert bits == 2 and indptr == left
    assert go([0, 10, 20, 50], max_kv_len=20)[0::2] == ([0, 5, 10, 10], 2)
    indptr, new, bits = go([0, 10, 20, 50], room=8)
    assert bits == 2 and new[:8] == [0, 1, 2, 3, 4, 10, 11, 12]
    assert go([0, 10, 20, 50], go_room=7)[2] == 2


def test_graph(ddt):  # noqa: F811
    lens, budget = [9000, 300], [1000, 64]
    w = weights_of("spread", sum(lens), 3)
    slots = torch.randperm(sum(lens), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    new, indptr, kv, bd, wd, sd = i32([0] * 1064), i32([0] * 3), i32([0, 9000, 9300]), i32(budget), w.to(DEV), slots.to(DEV)
    f = lambda: ddt.ddt_cache_evict(wd, sd, kv, bd, new, indptr, max_kv_len=9000, sinks=2, recent=9)  # noqa: E731
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    new.zero_()
    g.replay()
    clean(ddt)
    assert new.tolist() == ref.evict(w, slots.numpy(), lens, budget, 2, 9)[0]
