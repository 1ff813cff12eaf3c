"""PagedKVCache.write_rows where the call that writes refuses its arguments: the sequences are
as long as before, hold the same tokens, and no block is lost."""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa
import paged_kv_cache_345_b200.cache as cm
from paged_kv_cache_345_b200.cache import PagedKVCache
from test_draft_sharing_cpu import BS, D, HKV, plain_copy_blocks, put, rows_held, tables_of


@pytest.fixture
def cache(monkeypatch):
    monkeypatch.setattr(cm, "pa_copy_blocks", plain_copy_blocks)
    monkeypatch.setattr(PagedKVCache, "_to_device", lambda self, a: torch.from_numpy(np.ascontiguousarray(a)))
    return PagedKVCache(24, BS, HKV, D, "f32", "cpu")


def call(cache, seqs, counts, n=None):
    n = sum(counts) if n is None else n
    z = torch.zeros
    return cache.write_rows(z(n, 4, D), z(n, HKV, D), z(n, HKV, D), seqs, counts, z(n, dtype=torch.int32), z(64, D))


@pytest.mark.parametrize("error", [ValueError, TypeError, pa.PagedAttentionError])
def test_a_refused_write_reserves_nothing(cache, monkeypatch, error):
    a, b = cache.add_sequence(), cache.add_sequence()
    put(cache, a, 0, 6)
    put(cache, b, 50, 4)
    child = cache.fork(a)            # (its tail block is shared: the write copies it first)
    free = cache.bm.allocator.num_free()

    def refuse(*args, **kwargs):
        raise error(2, "no") if error is pa.PagedAttentionError else error("no")

    monkeypatch.setattr(cm, "pa_qk_norm_rope_append", refuse)
    with pytest.raises(error):
        call(cache, [b, a], [5, 3])
    assert [cache.context_len(s) for s in (a, b, child)] == [6, 4, 6]
    assert rows_held(cache, a) == rows_held(cache, child) == list(range(6))
    assert rows_held(cache, b) == [50, 51, 52, 53]
    # (the copied tail stays the sequence's own: one block, and nothing besides)
    assert cache.bm.allocator.num_free() == free - 1
    assert len({t[-1] for t in tables_of(cache.bm, [a, b, child])}) == 3
    for s in (a, b, child):
        cache.free(s)
    assert cache.bm.allocator.num_free() == 24


def test_the_binding_itself_refuses(cache):
    s = cache.add_sequence()
    put(cache, s, 0, 5)
    free = cache.bm.allocator.num_free()
    for n in (None, 7):                                  # tensors off the GPU
        with pytest.raises(ValueError):
            call(cache, [s], [9], n)
    with pytest.raises(AttributeError):                  # not a tensor at all
        cache.write_rows(None, None, None, [s], [9], None, None)
    assert cache.context_len(s) == 5 and cache.bm.allocator.num_free() == free


def test_rows_without_a_slot_are_refused(cache):
    """counts that hold no token do not go with rows."""
    s = cache.add_sequence()
    with pytest.raises(ValueError):
        call(cache, [s], [0], 3)
    assert cache.context_len(s) == 0


def test_no_rows_at_all(cache, monkeypatch):
    calls = []
    monkeypatch.setattr(cm, "pa_qk_norm_rope_append", lambda *a, **k: calls.append(a))
    s = cache.add_sequence()
    assert call(cache, [s], [0]).shape == (0, 4, D) and call(cache, [], []).shape == (0, 4, D)
    assert not calls and cache.context_len(s) == 0
