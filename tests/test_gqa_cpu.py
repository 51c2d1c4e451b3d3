"""Host-side checks of the grouped-query layer and the cache-row calls: nothing
here reaches a kernel.  And pins of the plain forms that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

from tests import _gqa_ref as ref

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_gb300 import _build
    _build.build()
    from tree_speculative_decoding_gb300 import ddt
    return ddt.lib


def call(lib, name, good, **changes):
    """The call with `good` arguments, some of them changed."""
    assert set(changes) <= set(good)
    return getattr(lib, name)(*{**good, **changes}.values())


ATTN = dict(q=P, k=P, v=P, stride=1024, rows=100, idx=P, kvp=P, qop=P, mask=P, mip=P, batch=1, H=64, G=8, D=128,
            total_q=0, total_kv=40, words=18, max_q=9, max_kv=40, scale=0.1, ctas=0, out=P, lse=None, ws=None, wsb=0,
            stream=None)


def test_attention_host_checks(lib):
    f = lambda **c: call(lib, "ddt_gqa_verify_attn", ATTN, **c)  # noqa: E731
    assert f() == 0 and f(batch=0, total_q=9) == 0 and f(max_q=0, total_q=9) == 0   # nothing to do
    for name in ("q", "k", "v", "idx", "kvp", "qop", "mask", "mip", "out"):
        assert f(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "out"):
        assert f(**{name: ctypes.c_void_p(264)}) == INVALID, name    # not 16-byte aligned
    assert f(ws=ctypes.c_void_p(128)) == INVALID                     # not 256-byte aligned
    for bad in (dict(batch=-1), dict(total_q=-1), dict(total_kv=-1), dict(words=-1), dict(rows=0), dict(max_kv=8),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1), dict(ctas=-1), dict(H=63), dict(G=0), dict(H=0),
                dict(G=128), dict(stride=1016), dict(stride=1028), dict(max_q=-1)):
        assert f(**bad) == INVALID, bad
    for bad in (dict(D=96), dict(D=256, stride=2048), dict(H=136), dict(max_q=129, max_kv=129), dict(ctas=513),
                dict(ctas=2, batch=257),
                dict(rows=2 ** 31), dict(batch=65536)):
        assert f(**bad) == UNSUPPORTED, bad


def test_attention_sizing(lib):
    size = lib.ddt_gqa_verify_attn_workspace_size
    assert size(1, 64, 8, 128, 33, 0) == 0 and size(0, 64, 8, 128, 33, 4) == 0 and size(1, 64, 7, 128, 33, 4) == 0
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    # two parts per CTA of as many rows as an item has: q_len x group, at most 128 or 256 (two tiles);
    # with two tiles also enough for one and twice as many CTAs
    def need(b, h, g, d, t, c, tiles):
        rows = min(t * (h // g), 128 * tiles)
        return up(8 * b * g * -(-t * (h // g) // (128 * tiles))) + up(2 * c * rows * d * 4) + up(2 * c * rows * 4)

    for b, h, g, d, t, c in ((1, 64, 8, 128, 1, 304), (3, 64, 8, 128, 16, 9), (2, 64, 8, 64, 17, 5), (256, 128, 1, 128, 128, 512)):
        want = need(b, h, g, d, t, c, 1)
        if t * (h // g) > 128:
            want = max(need(b, h, g, d, t, c, 2), need(b, h, g, d, t, 2 * c, 1))
        assert size(b, h, g, d, t, c) == want
    ctas = lib.ddt_gqa_verify_attn_num_ctas
    for args in ((1, 64, 8, 33, 4129, 152), (64, 64, 8, 1, 16384, 152), (1, 8, 2, 9, 30, 152), (1, 1, 1, 1, 1, 152),
                 (1, 64, 8, 65, 131137, 152), (32, 32, 4, 33, 8225, 1000), (65535, 128, 1, 128, 2 ** 31 - 1, 152)):
        assert 0 <= ctas(*args) <= 512, args
    assert ctas(1, 64, 8, 65, 131137, 152) == 152 and ctas(64, 64, 8, 1, 16384, 152) == 304
    assert ctas(257, 64, 8, 1, 16384, 152) == 0 and ctas(1, 8, 2, 9, 30, 152) == 0
    assert ctas(0, 64, 8, 33, 4129, 152) == 0 and ctas(1, 64, 7, 33, 4129, 152) == 0


APPEND = dict(q=P, qs=1536, k=P, ks=1536, v=P, vs=1536, qw=P, kw=P, eps=1e-6, table=P, max_pos=64, rope=128, il=0,
              depth=P, qop=P, idx=P, kvp=P, batch=1, total_q=0, total_kv=10, H=8, G=2, D=128, q_out=ctypes.c_void_p(512),
              kp=P, vp=P, stride=256, rows=10, stream=None)


def test_append_host_checks(lib):
    f = lambda **c: call(lib, "ddt_gqa_norm_rope_append", APPEND, **c)  # noqa: E731
    assert f() == 0 and f(batch=0, total_q=4) == 0
    assert f(qw=None, kw=None, depth=None) == 0 and f(rope=0, table=None, max_pos=0) == 0
    for name in ("q", "k", "v", "qop", "idx", "kvp", "q_out", "kp", "vp", "table"):
        assert f(**{name: None}) == INVALID, name
    for name in ("q", "k", "v", "qw", "kw", "table", "q_out", "kp", "vp"):
        assert f(**{name: ctypes.c_void_p(264)}) == INVALID, name
    for bad in (dict(qs=1016), dict(ks=248), dict(vs=248), dict(qs=1540), dict(ks=260), dict(vs=260), dict(stride=248),
                dict(stride=260), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rows=0),
                dict(batch=-1), dict(total_q=-1), dict(H=7), dict(G=0), dict(rope=-16), dict(max_pos=-1),
                dict(q_out=P)):   # in place needs rows that stay where they are
        assert f(**bad) == INVALID, bad
    assert f(q_out=P, qs=1024) == 0
    for bad in (dict(rope=24), dict(rope=144), dict(D=96, qs=768), dict(H=256, qs=32768)):
        assert f(**bad) == UNSUPPORTED, bad


COPY = dict(src=P, sgap=2000, srows=10, dst=P, dgap=2000, drows=10, pools=2, row=192, si=P, di=P, n=0, stream=None)
COMMIT = dict(slab=P, gap=1920, rows=10, pools=2, row=192, idx=P, kvp=P, qop=P, alen=P, nodes=P, batch=0, total_kv=10,
              depth=7, new_len=None, stream=None)
COMPACT = dict(slab=P, gap=1920, rows=10, pools=2, row=192, idx=P, total=5, new=P, live=P, ws=P, wsb=0, stream=None)


def test_cache_host_checks(lib):
    for name, good, prefix in (("ddt_cache_copy", COPY, "s"), ("ddt_cache_copy", COPY, "d"), ("ddt_cache_commit", COMMIT, ""),
                               ("ddt_cache_compact", COMPACT, "")):
        f = lambda **c: call(lib, name, good, **c)  # noqa: B023,E731
        assert f() == (WORKSPACE if name == "ddt_cache_compact" else 0)
        base = {"s": "src", "d": "dst", "": "slab"}[prefix]
        for bad in ({base: None}, {base: ctypes.c_void_p(264)}, {prefix + "gap": 1904}, {prefix + "gap": 1928},
                    {prefix + "rows": 0}, {"pools": 0}, {"row": 0}, {"row": 200}, {"row": 8},
                    {prefix + "rows": 2 ** 62}):
            assert f(**bad) == INVALID, (name, bad)
    assert call(lib, "ddt_cache_copy", COPY, n=-1) == INVALID and call(lib, "ddt_cache_copy", COPY, n=1, si=None) == INVALID
    for bad in (dict(idx=None), dict(kvp=None), dict(qop=None), dict(alen=None), dict(nodes=None), dict(batch=-1),
                dict(total_kv=-1)):
        assert call(lib, "ddt_cache_commit", COMMIT, **bad) == INVALID, bad
    for depth in (0, 8):
        assert call(lib, "ddt_cache_commit", COMMIT, depth=depth) == UNSUPPORTED
    for bad in (dict(idx=None), dict(new=None), dict(live=None), dict(total=-1)):
        assert call(lib, "ddt_cache_compact", COMPACT, **bad) == INVALID, bad
    need = lib.ddt_cache_compact_workspace_size(10)
    assert need > 0
    assert call(lib, "ddt_cache_compact", COMPACT, wsb=need - 1) == WORKSPACE
    assert call(lib, "ddt_cache_compact", COMPACT, wsb=need, ws=None) == WORKSPACE
    assert call(lib, "ddt_cache_compact", COMPACT, wsb=need, ws=ctypes.c_void_p(264)) == WORKSPACE
    assert call(lib, "ddt_cache_compact", COMPACT, rows=2 ** 24 + 1, gap=2 ** 33) == UNSUPPORTED
    size = lib.ddt_cache_compact_workspace_size
    assert size(0) == 0 and size(2 ** 24 + 1) == 0
    # two lists of at most half the rows, a bit and a count per 32 rows
    for rows in (1, 31, 4096, 65536, 2 ** 24):
        assert 4 * (rows // 2 + 1) * 2 + rows // 4 <= size(rows) <= 4 * rows + rows // 4 + 2048


def test_python_calls_refuse_what_the_library_cannot_see(lib):
    from tree_speculative_decoding_gb300 import ddt
    x, i = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ddt.ddt_gqa_verify_attn(x, x, x, i, i, i, i, i, 1.0, x)
    with pytest.raises(ValueError, match="CUDA"):
        ddt.ddt_gqa_norm_rope_append(x, x, x, None, None, 0.0, None, None, i, i, i, x, x, x)
    for call_ in (lambda: ddt.ddt_cache_copy(x, x, i, i), lambda: ddt.ddt_cache_commit(x, i, i, i, i, i, 7),
                  lambda: ddt.ddt_cache_compact(x, i, i, i[:1])):
        with pytest.raises(ValueError, match="CUDA"):
            call_()


def test_python_helpers_check_layouts():
    from tree_speculative_decoding_gb300 import ddt
    dev = torch.device("cpu")
    kv = torch.zeros(6, 2, 4, 64, dtype=torch.bfloat16)
    p, stride, n, h, d = ddt._heads(kv[:, 1], dev, "x")
    assert (stride, n, h, d) == (512, 6, 4, 64) and p == kv.data_ptr() + 512
    assert ddt._pools(kv[:, 0], kv[:, 1], dev)[2:] == (512, 6, 4, 64)
    for bad in (kv[..., ::2][:, 0], kv[:, 0].transpose(0, 1), kv[:, 0].float(), kv):
        with pytest.raises(ValueError):
            ddt._heads(bad, dev, "x")
    with pytest.raises(ValueError, match="stride"):
        ddt._pools(kv[:, 0], kv[:, 1].contiguous(), dev)
    with pytest.raises(ValueError):
        ddt._pools(kv[:, 0], kv[:3, 1], dev)
    s = torch.zeros(3, 10, 4, 8)
    assert ddt._slab(s, dev, "x")[1:] == (1280, 10, 3, 128)
    assert ddt._slab(s[::2], dev, "x")[1:] == (2560, 10, 2, 128)
    assert ddt._slab(s[:1], dev, "x")[1:] == (1280, 10, 1, 128)
    for bad in (s[0, 0], s[:, ::2], s.transpose(0, 1), s[:0], s[:, :0]):
        with pytest.raises(ValueError):
            ddt._slab(bad, dev, "x")
    with pytest.raises(ValueError):
        ddt._like(torch.zeros(4, 2)[:, 0], torch.float32, dev, "x")
    with pytest.raises(ValueError):
        ddt._mask_ptr(torch.zeros(3, dtype=torch.int64), dev)


def test_python_calls_refuse_another_device(monkeypatch):
    from tree_speculative_decoding_gb300 import ddt

    class Elsewhere:
        device = torch.device("cuda:1")

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        ddt._on_device(Elsewhere(), "q")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert ddt._on_device(Elsewhere(), "q").index == 1


# ---------------------------------------------------------------- the plain forms
def test_masks_equal_the_oracles(oracle_mod):
    batch = ref.Batch([(21, 9), (64, 33), (0, 1), (31, 128)], 3, "tree")
    par = np.concatenate(batch.parent).astype(np.int32)
    words, start = oracle_mod.compile_visibility(par, batch.qo, batch.P.astype(np.int32))
    assert np.array_equal(words, batch.words) and np.array_equal(start, batch.mask_indptr)


def test_attention_form_equals_the_oracle_where_keys_are_values(oracle_mod):
    # one K/V head whose rows are the latent rows' first 128 values: the latent oracle with the
    # rest of q and of the rows zero
    batch = ref.Batch([(13, 5), (2, 3)], 5, "tree")
    g = torch.Generator().manual_seed(1)
    q = torch.randn(batch.total_q, 4, 128, generator=g).to(torch.bfloat16)
    k = torch.randn(batch.rows, 1, 128, generator=g).to(torch.bfloat16)
    wide = lambda t: torch.cat([t, torch.zeros(*t.shape[:-1], 448, dtype=t.dtype)], -1)  # noqa: E731
    bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    want, want_lse = oracle_mod.verify_attn(bits(wide(q)), bits(wide(k[:, 0])), batch.slots, batch.kv, batch.qo,
                                            batch.words, batch.mask_indptr, 4, 0.1)
    out, lse, bound, _ = ref.attention(q, k, k, batch, 0.1)
    np.testing.assert_allclose(out.reshape(-1, 128).numpy(), np.asarray(want).reshape(-1, 512)[:, :128], rtol=1e-6, atol=1e-7)
    np.testing.assert_allclose(lse.reshape(-1).numpy(), np.asarray(want_lse).reshape(-1), rtol=1e-6)
    assert (bound >= 0).all()


def test_norm_rope_form_keeps_lengths_and_angles():
    # a rotation by a table of cos and sin keeps each pair's length, and position 0 changes nothing
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    ang = np.arange(10)[:, None] * 0.3 * np.arange(1, 17)[None]
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))
    for il in (False, True):
        pos = torch.tensor([0, 1, 2, 3, 9, 4])
        y, _ = ref.norm_rope(x, None, 0.0, table, pos, il)
        assert torch.equal(y[0], x[0].double()) and torch.equal(y[..., 32:], x[..., 32:].double())
        torch.testing.assert_close(y.norm(dim=-1), x.double().norm(dim=-1), rtol=1e-6, atol=0)
    w = torch.full((64,), 2.0, dtype=torch.bfloat16)
    y, _ = ref.norm_rope(x, w, 0.0, None, torch.zeros(6, dtype=torch.int64), False)
    torch.testing.assert_close(y.pow(2).mean(-1), torch.full((6, 2), 4.0, dtype=torch.float64))


def test_compact_form():
    assert ref.compact([5, 1, 5, 7], 8) == ([0, 1, 0, 2], 3, [5, 1, 7, 3, 4, 5, 6, 7])
    assert ref.compact([], 3) == ([], 0, [0, 1, 2])


def test_calls_in_words_answer_as_the_calls_do(lib):
    import struct
    calls = ["ddt_gqa_norm_rope_append", "ddt_gqa_verify_attn", "ddt_cache_copy", "ddt_cache_commit", "ddt_cache_compact"]

    def words(name, args, count=None):
        num = lambda x: 0 if x is None else x.value if isinstance(x, ctypes.c_void_p) else x  # noqa: E731
        w = [struct.pack("=d" if t is ctypes.c_float else "=q", num(x)) for t, x in zip(getattr(lib, name).argtypes, args)]
        return struct.pack("=qq", calls.index(name), len(w) if count is None else count) + b"".join(w)

    for name, good in (("ddt_gqa_norm_rope_append", APPEND), ("ddt_gqa_verify_attn", ATTN)):
        assert len(getattr(lib, name).argtypes) == len(good)
        for changes in ({}, dict(H=63), dict(H=136), dict(D=96), dict(batch=-1), dict(out=None) if "out" in good else {},
                        dict(scale=-1.0) if "scale" in good else dict(eps=-1.0), dict(stride=1028) if "stride" in good else {}):
            args = list({**good, **changes}.values())
            assert lib.ddt_call_words(words(name, args)) == getattr(lib, name)(*args), (name, changes)
        args = list(good.values())
        assert lib.ddt_call_words(words(name, args, len(args) - 1)) == INVALID
        assert lib.ddt_call_words(words(name, list({**good, "H": 64 + 2 ** 32}.values()))) == INVALID   # does not fit
    assert lib.ddt_call_words(struct.pack("=qq", 5, 0)) == INVALID and lib.ddt_call_words(None) == INVALID
    assert lib.ddt_call_words(struct.pack("=qq", -1, 0)) == INVALID
    # a copy of nothing, and one with a bad row width
    args = [P, 1024, 64, P, 1024, 64, 1, 16, None, None, 0, None]
    assert lib.ddt_call_words(words("ddt_cache_copy", args)) == 0
    assert lib.ddt_call_words(words("ddt_cache_copy", args[:7] + [24] + args[8:])) == INVALID


def test_attention_refuses_its_query_as_output(lib):
    assert call(lib, "ddt_gqa_verify_attn", ATTN, total_q=9) == INVALID
