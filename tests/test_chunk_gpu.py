"""Chunk attention on the GPU, against a plain 64-bit form (tests/_chunk_ref.py,
which also derives the tolerances)."""
import numpy as np
import pytest
import torch

from tests import _chunk_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def ddt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_decoding_gb300 import _build
    _build.build()
    from tree_speculative_decoding_gb300 import ddt as m
    m.ddt_get_error()
    return m


def clean(ddt):
    torch.cuda.synchronize()
    assert ddt.ddt_get_error() == (0, 0)


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def inputs(c, H, G, D, seed, q_scale=1.5):
    return normal((c.total_q, H, D), seed, q_scale), normal((c.rows, G, D), seed + 1), normal((c.rows, G, D), seed + 2)


def slopes_of(H):
    return 2.0 ** (-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H)


def run(ddt, c, q, k, v, scale, cap=0.0, slopes=None, window=0, full=None, lse=True, **kw):
    d = c.device()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV) if lse else None
    ddt.ddt_gqa_chunk_attn(q.to(DEV), k.to(DEV), v.to(DEV), d["kv_indices"], d["kv_indptr"], d["qo_indptr"], scale, out, ls,
                           max_q_len=c.max_q, max_kv_len=c.max_kv, score_cap=cap,
                           slopes=None if slopes is None else slopes.to(DEV), window=window,
                           full_len=None if full is None else torch.tensor(full, dtype=torch.int32, device=DEV), **kw)
    return out, ls


def check(out, ls, want):
    o, l, bo, bl = want
    err = (out.double().cpu() - o).abs() - bo
    assert float(err.max()) <= 0, f"out over its bound by {float(err.max())}"
    if ls is not None:
        err = (ls.double().cpu() - l).abs() - bl
        assert float(err.max()) <= 0, f"lse over its bound by {float(err.max())}"


CASES = [
    # heads, kv heads, dim, (cached, new) per request, cap, slopes, window, full, page
    (8, 2, 64, [(21, 1)], 0.0, False, 0, None, 1),
    (8, 2, 128, [(21, 9)], 0.0, False, 0, None, 1),
    (5, 5, 128, [(0, 1), (1, 1), (63, 1), (64, 1), (127, 1), (200, 1)], 30.0, False, 0, None, 1),
    (16, 16, 64, [(62, 1), (63, 2), (61, 3), (0, 7)], 0.0, True, 0, None, 16),
    (8, 1, 128, [(0, 300)], 0.0, False, 0, None, 64),
    (8, 1, 64, [(0, 300), (5, 0), (130, 65)], 0.0, False, 0, None, 16),
    (16, 2, 128, [(700, 33), (0, 1), (64, 200)], 0.0, False, 100, None, 1),
    (12, 1, 128, [(130, 130), (64, 11)], 20.0, True, 0, None, 64),
    (40, 8, 128, [(500, 150), (3, 17), (250, 1)], 50.0, False, 64, [40, 3, 0], 1),
    (28, 4, 64, [(95, 140), (600, 1), (0, 64)], 0.0, True, 200, [7, 64, 60], 16),
    (4, 2, 128, [(10, 129)], 0.0, False, 1, None, 1),
    (4, 1, 128, [(300, 40), (0, 200)], 0.0, True, 33, [400, 128], 1),
    (64, 1, 64, [(70, 5), (10, 2)], 0.0, False, 0, None, 1),
    (128, 1, 128, [(40, 3)], 15.0, False, 0, None, 64),
    (2, 2, 128, [(0, 513)], 0.0, True, 0, [513], 64),
    (1, 1, 128, [(1500, 1)], 0.0, False, 0, None, 1),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("ctas", [0, 1, 3, 29])
def test_attention(ddt, case, ctas):
    H, G, D, lens, cap, bias, window, full, page = case
    c = ref.Chunk(lens, 11 + H + len(lens), page)
    q, k, v = inputs(c, H, G, D, 5 * H + D, 6.0 if cap else 1.5)
    kw = dict(cap=cap, slopes=slopes_of(H) if bias else None, window=window, full=full)
    out, ls = run(ddt, c, q, k, v, D ** -0.5, num_ctas=ctas, **kw)
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, D ** -0.5, **kw))


@pytest.mark.parametrize("ctas", [2, 5, 7, 16, 64, 128, 512])
@pytest.mark.parametrize("H,T,D", [(8, 1, 128), (16, 70, 128), (16, 33, 64)])
def test_dealt_to_any_number_of_ctas(ddt, ctas, H, T, D):
    # shares that cut the long request many times, and that hold its end, whole requests and a start
    c = ref.Chunk([(1900, T), (40, T), (0, 0), (700, max(1, T // 2))], 3)
    q, k, v = inputs(c, H, 2, D, 9)
    out, ls = run(ddt, c, q, k, v, 0.1, num_ctas=ctas, window=1200, full=[100, 0, 0, 5])
    clean(ddt)
    check(out, ls, ref.attention(q, k, v, c, 0.1, window=1200, full=[100, 0, 0, 5]))
