"""Host-side checks of the grouped-query and cache-row calls on empty arrays
and on outputs over inputs: nothing here reaches a kernel."""
import ctypes

import pytest

from tests.test_gqa_cpu import APPEND, ATTN, COMMIT, INVALID, call, lib  # noqa: F401  (lib: the fixture)


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
