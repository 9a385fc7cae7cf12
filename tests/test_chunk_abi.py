"""Host-side refusals of the chunk and sequence calls that need no device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pkv():
    from page_wise_rank_gb300 import build
    build.build()
    import page_wise_rank_gb300 as m
    return m


def test_null_store_is_refused(pkv):
    from page_wise_rank_gb300 import _lib
    L = pkv.lib()
    one = (ctypes.c_int32 * 1)(0)
    n = ctypes.c_size_t()
    calls = [
        lambda: L.puzzlekv_chunk_workspace(None, 0, one, one, 1, ctypes.byref(n), None),
        lambda: L.puzzlekv_chunk_attention(None, 0, None, None, None, None, one, one, 1, None, 0, None),
        lambda: L.puzzlekv_append_chunk(None, 0, None, None, one, one, 1, None, 0, None),
        lambda: L.puzzlekv_read_tokens(None, 0, one, one, one, 1, None, None, None),
        lambda: L.puzzlekv_load_factors(None, 0, 0, 0, 1, None, None, None, None, None),
        lambda: L.puzzlekv_copy_sequences(None, one, one, 1, None),
        lambda: L.puzzlekv_truncate_sequences(None, one, one, 1, None),
    ]
    for call in calls:
        assert call() == _lib.ERR_INVALID_ARG
        assert "NULL" in pkv.last_error()


def test_lists_must_match(pkv):
    with pytest.raises(ValueError, match="counts"):
        pkv._ints([1, 2], 1, "counts")
    assert list(pkv._ints([3, 4], 2, "counts")) == [3, 4]
