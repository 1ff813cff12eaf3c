"""PagedKVCache.accept with a path length that cannot be: nothing of any sequence changes."""

import pytest
import torch

from test_draft_sharing_cpu import cache, put, rows_held  # noqa: F401  (cache: a fixture)


@pytest.mark.parametrize("lens", [[2, 6], [2, -1], [4, 2]])
def test_a_length_outside_the_rows_changes_no_sequence(cache, lens):  # noqa: F811
    a, b = cache.add_sequence(), cache.add_sequence()
    put(cache, a, 0, 6)
    put(cache, a, 100, 5)
    put(cache, b, 50, 3)
    put(cache, b, 200, 5)
    path = torch.tensor([[0, 3, 4], [0, 2, 4]], dtype=torch.int32)   # (three entries: 4 is too long as well)
    free = cache.bm.allocator.num_free()
    with pytest.raises(ValueError):
        cache.accept([a, b], [5, 5], path, torch.tensor(lens, dtype=torch.int32))
    assert rows_held(cache, a) == [*range(6), *range(100, 105)]
    assert rows_held(cache, b) == [*range(50, 53), *range(200, 205)]
    assert cache.bm.allocator.num_free() == free
    assert cache.accept([a, b], [5, 5], path, torch.tensor([2, 3], dtype=torch.int32)) == [8, 6]
    assert rows_held(cache, a) == [*range(6), 100, 103]
    assert rows_held(cache, b) == [50, 51, 52, 200, 202, 204]
