"""Host-side checks of the grouped-query and cache-row calls on empty arrays
and on outputs over inputs: nothing here reaches a kernel."""
import ctypes

import pytest

from tests.test_gqa_cpu import APPEND, ATTN, COMMIT, COMPACT, INVALID, call, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("name,good,array,size", [
    ("ddt_gqa_verify_attn", ATTN, "idx", "total_kv"), ("ddt_gqa_verify_attn", ATTN, "mask", "words"),
    ("ddt_gqa_norm_rope_append", APPEND, "idx", "total_kv"), ("ddt_cache_commit", COMMIT, "idx", "total_kv")])
def test_an_empty_array_may_have_no_address(lib, name, good, array, size):  # noqa: F811
    assert call(lib, name, good, **{array: None, size: 0}) == 0
    assert call(lib, name, good, **{array: None, size: 1}) == INVALID
    assert call(lib, name, good, **{array: None, size: -1}) == INVALID


def at(byte):
    return ctypes.c_void_p(1 << 20 | byte)


@pytest.mark.parametrize("away", [0, 16, -16, 9 * 64 * 128 * 2 - 16, 16 - 9 * 64 * 128 * 2])
def test_attention_refuses_an_output_over_its_query(lib, away):  # noqa: F811
    good = dict(ATTN, total_q=9, q=at(1 << 19), out=at((1 << 19) + away))
    assert call(lib, "ddt_gqa_verify_attn", good) == INVALID


@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("where", ["before", "first", "last"])
def test_append_refuses_an_output_over_its_inputs(lib, name, where):  # noqa: F811
    # three tokens in rows of 1536: the output of 3 x 1024 values reaches into the first row, or
    # starts in the last one
    width = 1024 if name == "q" else 256
    away = {"before": 16 - 3 * 1024 * 2, "first": 32, "last": (2 * 1536 + width) * 2 - 16}[where]
    far = {n: at((3 + i) << 16) for i, n in enumerate(("q", "k", "v"))}
    good = dict(APPEND, total_q=3, **far, q_out=at((far[name].value - (1 << 20)) + away))
    assert call(lib, "ddt_gqa_norm_rope_append", good) == INVALID


def test_compact_refuses_results_over_its_slots(lib):  # noqa: F811
    good = dict(COMPACT, total=5, idx=at(4096), new=at(8192), live=at(12288), ws=at(1 << 17),
                wsb=lib.ddt_cache_compact_workspace_size(10))
    f = lambda **c: call(lib, "ddt_cache_compact", good, **c)  # noqa: E731
    for away in (4, 16, -4, -16):
        assert f(new=at(4096 + away)) == INVALID
    for place in ("idx", "new"):
        for k in range(5):
            assert f(live=ctypes.c_void_p(good[place].value + 4 * k)) == INVALID
