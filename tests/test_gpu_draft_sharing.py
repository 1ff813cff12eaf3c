"""PagedKVCache.accept on the GPU where forks taken since the step's rows were written share
their blocks: every sequence's rows against a list of them."""

import pytest
import torch

import paged_kv_cache_345_b200 as pa
from paged_kv_cache_345_b200.cache import PagedKVCache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8_e4m3"])
@pytest.mark.parametrize("own_stream", [False, True])
def test_forks_keep_the_rows_that_accept_moves(dtype, own_stream):
    side = torch.cuda.Stream() if own_stream else None
    cache = PagedKVCache(64, 8, 2, 64, dtype, DEV, stream=side)
    code = cache.k_cache.dtype

    def held(seq):
        n = cache.context_len(seq)
        tables, _, _ = cache.tables([seq])
        torch.cuda.synchronize()
        t = torch.arange(n, device=DEV)
        slot = tables[0][t // 8].long() * 8 + t % 8
        return [c.view(64 * 8, 2, 64)[slot].clone() for c in (cache.k_cache, cache.v_cache)]

    def rows(n, seed):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn(2, n, 2, 64, generator=gen).to(torch.bfloat16 if dtype == "fp8_e4m3" else code)
        return x[0].to(DEV), x[1].to(DEV)

    a, b = cache.add_sequence(), cache.add_sequence()
    torch.cuda.synchronize()
    cache.write([a, b], [21, 8], *rows(29, 0))
    cache.write([a, b], [13, 5], *rows(18, 1))     # the step's rows
    forks = [cache.fork(a), cache.fork(b)]
    before = {s: held(s) for s in (a, b, *forks)}
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    kept = {a: [0, 3, 4, 12], b: [0, 1], forks[0]: [0, 1, 2, 11, 12]}
    path = i32([k + [-1] * (13 - len(k)) for k in kept.values()])
    lens = i32([len(k) for k in kept.values()])
    torch.cuda.synchronize()
    new = cache.accept(list(kept), [13, 5, 13], path, lens)
    assert pa.pa_device_errors() == 0
    assert new == [25, 10, 26]
    for s in (a, b, *forks):
        base = 21 if s in (a, forks[0]) else 8
        want = list(range(len(before[s][0]))) if s not in kept else [*range(base), *(base + k for k in kept[s])]
        for got, was in zip(held(s), before[s]):
            assert torch.equal(got, was[want])
