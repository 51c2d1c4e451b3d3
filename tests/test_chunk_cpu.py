"""Host-side checks of the chunk calls and of the eviction: nothing here reaches a kernel.  And pins of the
plain forms that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref
from tests.test_gqa_cpu import INVALID, UNSUPPORTED, P, call, lib  # noqa: F401  (lib: the fixture)

OUT = ctypes.c_void_p(1 << 20)
ATTN = dict(q=P, k=P, v=P, stride=1024, rows=100, idx=P, kvp=P, qop=P, batch=1, H=64, G=8, D=128, total_q=0, total_kv=40, max_q=9,
            max_kv=40, scale=0.1, cap=0.0, slopes=None, window=0, full=None, ctas=0, out=OUT, lse=None, ws=None, wsb=0, stream=None)
WEIGHTS = dict(q=P, k=P, stride=1024, rows=100, lse=P, idx=P, kvp=P, qop=P, batch=1, H=64, G=8, D=128, total_q=9, total_kv=0, max_q=9,
               max_kv=40, scale=0.1, cap=0.0, slopes=None, window=0, full=None, last=0, prev=None, prevp=None, total_prev=0, decay=1.0,
               ctas=0, w=OUT, ws=None, wsb=0, stream=None)
EVICT = dict(w=P, idx=P, kvp=P, budget=P, batch=0, total_kv=40, max_kv=40, sinks=0, recent=0, new=OUT, total_new=10, newp=P, neww=None,
             gone=None, total_gone=0, stream=None)


@pytest.mark.parametrize("name,good", [("ddt_gqa_chunk_attn", ATTN), ("ddt_gqa_chunk_weights", WEIGHTS)])
def test_chunk_host_checks(lib, name, good):  # noqa: F811
    f = lambda **c: call(lib, name, good, **c)  # noqa: E731
    assert f() == 0 and f(batch=0, total_q=9, total_kv=40) == 0   # nothing to do
    for x in ("q", "k", "kvp", "qop"):
        assert f(**{x: None}) == INVALID, x
    assert f(idx=None, total_kv=40) == INVALID
    for x in ("q", "k"):
        assert f(**{x: ctypes.c_void_p(264)}) == INVALID, x       # not 16-byte aligned
    assert f(ws=ctypes.c_void_p(128)) == INVALID                  # not 256-byte aligned
    for bad in (dict(batch=-1), dict(total_q=-1), dict(total_kv=-1), dict(rows=0), dict(max_kv=8), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1), dict(cap=-1.0), dict(cap=float("nan")),
                dict(cap=float("inf")), dict(window=-1), dict(ctas=-1), dict(H=63), dict(G=0), dict(H=0), dict(G=128),
                dict(stride=1016), dict(stride=1028), dict(max_q=-1)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(D=256, stride=2048), dict(H=136), dict(max_q=2 ** 20 + 1, max_kv=2 ** 21), dict(ctas=513),
                dict(ctas=2, batch=257), dict(rows=2 ** 31), dict(stride=2 ** 39), dict(batch=65536), dict(cap=2.0 ** 21), dict(scale=1e-35),
                dict(scale=1e35), dict(scale=1e-25, cap=2.0 ** 20), dict(scale=1e30, cap=1e-6)):
        assert f(**bad) == UNSUPPORTED, bad
    assert f(max_q=2 ** 20, max_kv=2 ** 31 - 1) == 0


def test_attention_refuses(lib):  # noqa: F811
    f = lambda **c: call(lib, "ddt_gqa_chunk_attn", ATTN, **c)  # noqa: E731
    for x in ("v", "out"):
        assert f(**{x: None}) == INVALID and f(**{x: ctypes.c_void_p(264)}) == INVALID, x
    # an output over the queries, or over the row sums
    n = 9 * 64 * 128 * 2
    at = lambda b: ctypes.c_void_p((1 << 20) + b)  # noqa: E731
    for away in (0, 16, -16, n - 16, 16 - n):
        assert f(total_q=9, q=at(1 << 19), out=at((1 << 19) + away)) == INVALID
    for away in (0, 4, -4, n - 4, 4 - 9 * 64 * 4):
        for over in (1 << 19, 1 << 21):
            assert f(total_q=9, q=at(1 << 19), out=at(1 << 21), lse=at(over + away)) == INVALID


def test_sizing(lib):  # noqa: F811
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    size = lib.ddt_gqa_chunk_attn_workspace_size
    assert size(64, 8, 128, 33, 0) == 0 and size(64, 7, 128, 33, 4) == 0 and size(64, 8, 128, 0, 4) == 0
    for h, g, d, t, c in ((64, 8, 128, 1, 304), (64, 8, 128, 16, 9), (64, 8, 64, 17, 5), (128, 1, 128, 8192, 512)):
        # two parts per CTA of as many rows as an item has, at most 128 or (two tiles) 256; with two tiles also
        # enough for one and twice as many CTAs
        need = lambda rows, c: up(16 * c) + up(2 * c * rows * d * 4) + up(2 * c * rows * 4)  # noqa: B023,E731
        rows = t * (h // g)
        assert size(h, g, d, t, c) == (need(rows, c) if rows <= 128 else max(need(min(rows, 256), c), need(128, 2 * c)))
    ctas = lib.ddt_gqa_chunk_attn_num_ctas
    assert ctas(1, 64, 8, 8192, 8192, 152) == 152 and ctas(64, 64, 8, 1, 16384, 152) == 304 and ctas(257, 64, 8, 1, 16384, 152) == 0
    assert ctas(1, 64, 8, 9, 30, 152) == 0 and ctas(0, 64, 8, 9, 4000, 152) == 0 and ctas(1, 64, 7, 9, 4000, 152) == 0
    assert 0 < ctas(1, 128, 1, 2 ** 20, 2 ** 31 - 1, 1000) <= 512
    assert lib.ddt_gqa_chunk_weights_workspace_size(0) == 0
    assert lib.ddt_gqa_chunk_weights_workspace_size(100) == up(1600) + 200 * 256 * 4
    assert lib.ddt_gqa_chunk_weights_num_ctas(1, 152) == 152 and lib.ddt_gqa_chunk_weights_num_ctas(257, 152) == 0


def test_weights_refuse(lib):  # noqa: F811
    f = lambda **c: call(lib, "ddt_gqa_chunk_weights", WEIGHTS, **c)  # noqa: E731
    at = lambda b: ctypes.c_void_p((1 << 22) + b)  # noqa: E731
    for bad in (dict(lse=None), dict(last=-1), dict(total_prev=-1), dict(prev=P, decay=float("nan")), dict(prev=P, decay=float("inf")),
                dict(prev=P, total_prev=41, total_kv=40), dict(w=None, total_kv=40)):
        assert f(**bad) == INVALID, bad
    for away in (4, -4, 39 * 4, -39 * 4):
        assert f(total_kv=40, w=at(0), prev=at(away), total_prev=40) == INVALID
    assert f(total_kv=40, w=at(0), prev=at(0), prevp=P, total_prev=40) == INVALID   # in place needs sums that stay where they are
    assert f(total_kv=40, w=at(0), lse=at(8)) == INVALID and f(total_kv=40, w=at(0), q=at(32)) == INVALID


def test_evict_host_checks(lib):  # noqa: F811
    f = lambda **c: call(lib, "ddt_cache_evict", EVICT, **c)  # noqa: E731
    assert f() == 0
    for bad in (dict(w=None), dict(idx=None), dict(kvp=None), dict(budget=None), dict(new=None), dict(newp=None), dict(batch=-1),
                dict(total_kv=-1), dict(max_kv=-1), dict(sinks=-1), dict(recent=-1), dict(total_new=-1), dict(total_gone=-1)):
        assert f(**bad) == INVALID, bad
    # outputs over inputs and over each other
    at = {n: ctypes.c_void_p((1 << 20) + (i << 12)) for i, n in enumerate(("w", "idx", "kvp", "budget", "new", "newp", "neww", "gone"))}
    size = dict(w=40, idx=40, kvp=4, budget=3, new=10, newp=4, neww=10, gone=30)
    good = dict(batch=3, total_gone=30, **at)
    for i, o in enumerate(("new", "newp", "neww", "gone")):
        for x in ("w", "idx", "kvp", "budget") + ("new", "newp", "neww", "gone")[:i]:
            for place in (at[x].value, at[x].value + 4 * (size[x] - 1), at[x].value - 4 * (size[o] - 1)):
                assert f(**{**good, o: ctypes.c_void_p(place)}) == INVALID, (o, x)


def test_python_calls_refuse_what_the_library_cannot_see(lib):  # noqa: F811
    from tree_speculative_decoding_gb300 import ddt
    x, i, f = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    with pytest.raises(ValueError, match="CUDA"):
        ddt.ddt_gqa_chunk_attn(x, x, x, i, i, i, 1.0, x)
    with pytest.raises(ValueError, match="CUDA"):
        ddt.ddt_gqa_chunk_weights(x, x, f, i, i, i, 1.0, f)
    with pytest.raises(ValueError, match="CUDA"):
        ddt.ddt_cache_evict(f, i, i, i, i, i)


def test_call_words_of_the_new_calls(lib):  # noqa: F811
    import struct
    for number, count in ((5, 27), (6, 30), (7, 16)):
        assert lib.ddt_call_words(struct.pack("=qq", number, count - 1) + bytes(8 * 40)) == INVALID
        assert lib.ddt_call_words(struct.pack("=qq", number, count) + bytes(8 * 40)) == INVALID   # all pointers null
    assert lib.ddt_call_words(struct.pack("=qq", 8, 0) + bytes(8 * 40)) == INVALID


# ---------------------------------------------------------------- the plain forms
def test_visibility_by_hand():
    c = ref.Chunk([(3, 4)], 1)
    want = {(0, None): ["1111000", "1111100", "1111110", "1111111"],
            (2, None): ["0011000", "0001100", "0000110", "0000011"],
            (2, (1,)): ["1011000", "1001100", "1000110", "1000011"],
            (1, (6,)): ["1111110", "1111110", "1111110", "1111111"]}
    for (window, full), rows in want.items():
        got = ["".join("01"[int(x)] for x in r) for r in ref.visible(c, 0, window, full).tolist()]
        assert got == rows, (window, full)


def test_attention_and_received_agree_with_differences():
    # what a column receives is the derivative of a row's log-sum by its score: of all rows, by a number added
    # to one column's scores
    c = ref.Chunk([(5, 3)], 2)
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(3, 2, 8, generator=g).double(), torch.randn(c.rows, 1, 8, generator=g).double()
    v = torch.zeros(c.rows, 1, 8).double()
    kw = dict(cap=2.0, slopes=torch.tensor([0.3, 0.1]), window=4)
    lse = ref.attention(q, k, v, c, 0.5, **kw)[1]
    w, _ = ref.received(q, k, lse, c, 0.5, **kw)
    assert abs(float(w.sum()) - 6.0) < 1e-6
    p = torch.from_numpy((c.P[0] + np.arange(3)).astype(np.float64))
    seen = ref.visible(c, 0, 4, None)
    for j in range(int(c.N[0])):
        d, up = 1e-6, 0.0
        for h in range(2):
            z, _ = ref.scores(q[:, h], k[torch.from_numpy(c.slots.astype(np.int64)), 0], p, 2.0, float(kw["slopes"][h]), 0.5)
            a, b = z.clone(), z.clone()
            a[:, j] += d
            b[:, j] -= d
            f = lambda x: torch.logsumexp(x.masked_fill(~seen, -torch.inf), 1).sum()  # noqa: E731
            up += float(f(a) - f(b)) / (2 * d)
        assert abs(up - float(w[j])) < 1e-6


def test_eviction_by_hand():
    w = torch.tensor([1.0, float("nan"), 3.0, 3.0, 0.0, -0.0, 2.0])
    assert ref.evict(w, list(range(10, 17)), [7], [3], 0, 0)[0] == [12, 13, 16]
    assert ref.evict(w, list(range(10, 17)), [7], [2], 0, 0)[0] == [12, 13]
    assert ref.evict(w, list(range(10, 17)), [7], [3], 2, 1)[0] == [10, 11, 16]
    assert ref.evict(w, list(range(10, 17)), [7], [6], 0, 0)[3] == [11]
    assert ref.evict(w, list(range(10, 17)), [3, 4], [1, 2], 0, 0) == ([12, 13, 16], [0, 1, 3], [3.0, 3.0, 2.0], [10, 11, 14, 15])
