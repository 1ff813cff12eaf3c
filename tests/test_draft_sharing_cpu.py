"""Forks between the rows of a drafted step and their acceptance: the block manager's
unsharing, and PagedKVCache.accept over it with the kernels' work done by plain torch on
the CPU."""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa
import paged_kv_cache_345_b200.cache as cm
from paged_kv_cache_345_b200.cache import PagedKVCache

BS, HKV, D = 4, 2, 8


def tables_of(bm, seqs):
    return [bm.block_tables([s], max(1, bm.seq_num_blocks(s)))[0][0, :bm.seq_num_blocks(s)].tolist() for s in seqs]


@pytest.mark.parametrize("seed", range(8))
def test_unshare_makes_the_last_tokens_blocks_their_sequences_own(seed):
    rng = np.random.default_rng(seed)
    bm = pa.BlockManager(200, BS)
    seqs = []
    for _ in range(3):
        seqs.append(bm.add_seq())
        bm.append_slots([seqs[-1]], [int(rng.integers(0, 30))])
    for _ in range(5):
        seqs.append(bm.fork(int(rng.choice(seqs))))
        s = int(rng.choice(seqs))
        bm.append_slots([s], [int(rng.integers(0, 6))])
    batch = [int(s) for s in rng.permutation(seqs)[:5]]
    counts = [int(rng.integers(0, bm.seq_len(s) + 1)) for s in batch]
    before = dict(zip(seqs, tables_of(bm, seqs)))
    refs = [bm.allocator.refcount(b) for b in range(200)]
    free = bm.allocator.num_free()
    pairs = bm.unshare(batch, counts)
    after = dict(zip(seqs, tables_of(bm, seqs)))
    came_from = {int(b): int(a) for a, b in pairs}
    assert len(came_from) == len(pairs) == free - bm.allocator.num_free()
    assert all(refs[b] == 0 and refs[a] > 1 for b, a in came_from.items())
    for s in seqs:
        first = (bm.seq_len(s) - counts[batch.index(s)]) // BS if s in batch and counts[batch.index(s)] else len(before[s])
        assert [came_from.get(b, b) for b in after[s]] == before[s]          # the same tokens
        assert after[s][:first] == before[s][:first]
        assert all(bm.allocator.refcount(b) == 1 for b in after[s][first:])
    held = np.bincount(sum(after.values(), []), minlength=200)
    assert [bm.allocator.refcount(b) for b in range(200)] == held.tolist()


@pytest.mark.parametrize("ids,counts", [([0, 0], [1, 1]), ([9], [1]), ([0], [-1]), ([0], [7]), ([0, 1], [6, 6])])
def test_unshare_refuses_and_changes_nothing(ids, counts):
    bm = pa.BlockManager(3, BS)                    # (the last case: two blocks needed, one free)
    s = bm.add_seq()
    bm.append_slots([s], [6])
    c = bm.fork(s)
    c2 = bm.fork(s)
    assert (s, c) == (0, 1)
    before, refs = tables_of(bm, [s, c, c2]), [bm.allocator.refcount(b) for b in range(3)]
    with pytest.raises(pa.PagedAttentionError):
        bm.unshare(ids, counts)
    assert tables_of(bm, [s, c, c2]) == before
    assert [bm.allocator.refcount(b) for b in range(3)] == refs
    with pytest.raises(ValueError):
        bm.unshare([0], [1, 1])


def plain_copy_blocks(kc, vc, pairs, stream=None):
    for a, b in pairs.tolist():
        kc[b], vc[b] = kc[a].clone(), vc[a].clone()


def plain_kv_accept(kc, vc, tables, lens, start, path, path_len, stream=None):
    for c in (kc, vc):
        old = c.clone()
        for s in range(len(lens)):
            base = int(lens[s]) - int(start[s + 1] - start[s])
            slot = lambda t: (int(tables[s, t // BS]), t % BS)  # noqa: E731
            for j in range(int(path_len[s])):
                c[slot(base + j)] = old[slot(base + int(path[s, j]))]


@pytest.fixture
def cache(monkeypatch):
    monkeypatch.setattr(cm, "pa_copy_blocks", plain_copy_blocks)
    monkeypatch.setattr(cm, "pa_kv_accept", plain_kv_accept)
    monkeypatch.setattr(PagedKVCache, "_to_device", lambda self, a: torch.from_numpy(np.ascontiguousarray(a)))
    return PagedKVCache(24, BS, HKV, D, "f32", "cpu")


def rows_held(cache, seq):
    """Each cached token's number (every element of its K row; V's is 1000 more)."""
    n = cache.context_len(seq)
    table = tables_of(cache.bm, [seq])[0]
    k = [cache.k_cache[table[t // BS], t % BS] for t in range(n)]
    v = [cache.v_cache[table[t // BS], t % BS] for t in range(n)]
    assert all((x == x.flatten()[0]).all() and (y == x + 1000).all() for x, y in zip(k, v))
    return [int(x.flatten()[0]) for x in k]


def put(cache, seq, first, n):
    """n tokens numbered from `first` on behind the sequence."""
    slots, cows = cache.bm.append_slots([seq], [n])
    plain_copy_blocks(cache.k_cache, cache.v_cache, torch.from_numpy(cows))
    for i, s in enumerate(slots.tolist()):
        cache.k_cache[s // BS, s % BS] = first + i
        cache.v_cache[s // BS, s % BS] = first + i + 1000


@pytest.mark.parametrize("ctx,n,kept", [(6, 5, [0, 2, 4]), (4, 9, [0, 1, 5, 8]), (7, 1, [0]), (1, 6, [0, 5]), (5, 4, [0, 1, 2])])
def test_a_fork_taken_before_accept_keeps_its_rows(cache, ctx, n, kept):
    seq = cache.add_sequence()
    put(cache, seq, 0, ctx)
    put(cache, seq, 100, n)
    child = cache.fork(seq)
    path = torch.full((1, n), -1, dtype=torch.int32)
    path[0, :len(kept)] = torch.tensor(kept)
    lens = cache.accept([seq], [n], path, torch.tensor([len(kept)], dtype=torch.int32))
    assert lens == [ctx + len(kept)]
    assert rows_held(cache, seq) == [*range(ctx), *(100 + k for k in kept)]
    assert rows_held(cache, child) == [*range(ctx), *range(100, 100 + n)]
    # both go on by themselves, and nothing is lost or left behind
    put(cache, child, 200, 3)
    put(cache, seq, 300, 3)
    assert rows_held(cache, seq) == [*range(ctx), *(100 + k for k in kept), 300, 301, 302]
    assert rows_held(cache, child) == [*range(ctx), *range(100, 100 + n), 200, 201, 202]
    cache.free(seq)
    cache.free(child)
    assert cache.bm.allocator.num_free() == 24


def test_parent_and_fork_accept_different_rows_in_one_call(cache):
    seq = cache.add_sequence()
    put(cache, seq, 0, 6)
    put(cache, seq, 100, 5)
    child = cache.fork(seq)
    path = torch.tensor([[0, 2, 4, -1, -1], [0, 1, 3, 4, -1]], dtype=torch.int32)
    assert cache.accept([seq, child], [5, 5], path, torch.tensor([3, 4], dtype=torch.int32)) == [9, 10]
    assert rows_held(cache, seq) == [0, 1, 2, 3, 4, 5, 100, 102, 104]
    assert rows_held(cache, child) == [0, 1, 2, 3, 4, 5, 100, 101, 103, 104]


def test_accept_without_free_blocks_changes_nothing(cache):
    seq = cache.add_sequence()
    put(cache, seq, 0, 6)
    put(cache, seq, 100, 5)
    child = cache.fork(seq)
    other = cache.add_sequence()
    put(cache, other, 500, 4 * cache.bm.allocator.num_free())
    with pytest.raises(pa.PagedAttentionError, match="PA_ERR_NO_BLOCKS"):
        cache.accept([seq], [5], torch.tensor([[0, 4]], dtype=torch.int32), torch.tensor([2], dtype=torch.int32))
    for s in (seq, child):
        assert rows_held(cache, s) == [0, 1, 2, 3, 4, 5, 100, 101, 102, 103, 104]
