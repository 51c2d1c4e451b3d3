"""Host-side checks of the grouped-query and cache-row calls on empty arrays:
nothing here reaches a kernel."""
import pytest

from tests.test_gqa_cpu import APPEND, ATTN, COMMIT, INVALID, call, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("name,good,array,size", [
    ("ddt_gqa_verify_attn", ATTN, "idx", "total_kv"), ("ddt_gqa_verify_attn", ATTN, "mask", "words"),
    ("ddt_gqa_norm_rope_append", APPEND, "idx", "total_kv"), ("ddt_cache_commit", COMMIT, "idx", "total_kv")])
def test_an_empty_array_may_have_no_address(lib, name, good, array, size):  # noqa: F811
    assert call(lib, name, good, **{array: None, size: 0}) == 0
    assert call(lib, name, good, **{array: None, size: 1}) == INVALID
    assert call(lib, name, good, **{array: None, size: -1}) == INVALID
