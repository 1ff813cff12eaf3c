"""Steps with drafted tokens through PagedKVCache: rows written, attended, verified and
kept, step after step, against a dense float64 model of the same sequences."""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa
from paged_kv_cache_345_b200.cache import PagedKVCache
from test_gpu_tree import tree_parents
from test_gpu_verify import draw_batch, walk

pytestmark = pytest.mark.gpu
DEV = "cuda"


def depths(parents):
    d = np.zeros(len(parents), dtype=np.int64)
    for i, p in enumerate(parents):
        d[i] = d[p] + 1 if p >= 0 else 0
    return d


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
def test_steps(dtype):
    hq, hkv, d, bs, vocab, most = 8, 2, 128, 16, 200, 256
    rng = np.random.default_rng(0)
    scales = dict(k_scale=torch.tensor([0.03, 0.05]), v_scale=torch.tensor([0.04, 0.03])) if dtype == "fp8_e4m3" else {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache = PagedKVCache(96, bs, hkv, d, dtype, DEV, free_order=rng.permutation(96).astype(np.int32), stream=side, **scales)
    ang = np.arange(most)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    cs = torch.from_numpy(table).to(DEV)
    w = torch.ones(d, dtype=torch.bfloat16, device=DEV)

    def rope64(x, pos):
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        c, s = table[pos, :d // 2].astype(np.float64)[:, None], table[pos, d // 2:].astype(np.float64)[:, None]
        a, b = y[..., :d // 2], y[..., d // 2:]
        return np.concatenate([a * c - b * s, b * c + a * s], -1)

    # three prompts; the third sequence is forked from the second and shares its tail block
    seqs, held = [], []          # held: the dense [tokens, Hkv, d] keys and values of each sequence
    for n in (20, 37):
        x = torch.randn(n, (hq + 2 * hkv), d).bfloat16()
        s = cache.add_sequence()
        pos = np.arange(n)
        cache.write_rows(x[:, :hq].to(DEV), x[:, hq:hq + hkv].to(DEV), x[:, hq + hkv:].to(DEV), [s], [n],
                         torch.arange(n, dtype=torch.int32, device=DEV), cs, w, w)
        seqs.append(s)
        held.append((rope64(x[:, hq:hq + hkv].double().numpy(), pos), x[:, hq + hkv:].double().numpy()))
    seqs.append(cache.fork(seqs[1]))
    held.append(held[1])

    for step in range(4):
        counts = [int(c) for c in rng.integers(1, 13, 3)]
        b = draw_batch(50 + step, counts, vocab, "tree", True)
        parents = b["parents"]
        lens = [len(h[0]) for h in held]
        pos = np.concatenate([lens[i] + depths(parents[b["start"][i]:b["start"][i + 1]]) for i in range(3)])
        x = torch.randn(sum(counts), hq + 2 * hkv, d).bfloat16()
        dev = {k: torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for k, v in b.items()}
        packed = x.to(DEV)
        torch.cuda.synchronize()
        q = cache.write_rows(packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:], seqs, counts,
                             torch.from_numpy(pos.astype(np.int32)).to(DEV), cs, w, w)
        torch.cuda.synchronize()
        k64, v64 = rope64(x[:, hq:hq + hkv].double().numpy(), pos), x[:, hq + hkv:].double().numpy()
        if dtype == "bf16":
            out = cache.decode_tree(q, seqs, counts, dev["parents"])
            torch.cuda.synchronize()
            q64 = rope64(x[:, :hq].double().numpy(), pos)
            for i in range(3):
                for r in range(counts[i]):
                    row = b["start"][i] + r
                    own, a = [], r
                    while a >= 0:
                        own.append(b["start"][i] + a)
                        a = parents[b["start"][i] + a]
                    kk, vv = (np.concatenate([h, n[own[::-1]]]) for h, n in zip(held[i], (k64, v64)))
                    for j in range(hq):
                        s = kk[:, j // 4] @ q64[row, j] / np.sqrt(d)
                        p = np.exp(s - s.max())
                        ref = (p / p.sum()) @ vv[:, j // 4]
                        # q and k are rounded to bf16 (2^-8 each): a score is off by up to 2^-7 of
                        # sum |q k|, a weight by twice that; then as in the tree's own tests
                        top = (np.abs(kk[:, j // 4]) @ np.abs(q64[row, j])).max() / np.sqrt(d)
                        mag = (p / p.sum()) @ np.abs(vv[:, j // 4])
                        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -14 + 2 * 2.0 ** -7 * top) * mag
                        assert (np.abs(out[row, j].double().cpu().numpy() - ref) <= tol).all()
        toks = torch.empty(3, max(counts), dtype=torch.int32, device=DEV)
        path, kept = torch.empty_like(toks), torch.empty(3, dtype=torch.int32, device=DEV)
        with torch.cuda.stream(side):
            pa.pa_verify_draft(toks, path, kept, dev["target"], dev["draft"], dev["tokens"], dev["parents"],
                               dev["start"], dev["ua"], dev["us"])
        new = cache.accept(seqs, counts, path, kept)
        torch.cuda.synchronize()
        assert pa.pa_device_errors() == 0
        for i in range(3):
            said, keep = walk(b, i)
            assert toks[i, :len(said)].tolist() == said
            rows = b["start"][i] + np.array(keep)
            held[i] = tuple(np.concatenate([h, n[rows]]) for h, n in zip(held[i], (k64, v64)))
            assert new[i] == len(held[i][0]) == cache.context_len(seqs[i])
            assert cache.bm.seq_num_blocks(seqs[i]) == -(-new[i] // bs)
        # the caches hold every sequence's kept rows, in order
        tables, _, _ = cache.tables(seqs)
        torch.cuda.synchronize()
        for i in range(3):
            t = np.arange(new[i])
            slot = tables[i].cpu().numpy()[t // bs].astype(np.int64) * bs + t % bs
            for c, ref, sc in ((cache.k_cache, held[i][0], scales.get("k_scale")), (cache.v_cache, held[i][1], scales.get("v_scale"))):
                got = c.view(-1, hkv, d)[torch.from_numpy(slot).to(DEV)]
                if dtype == "fp8_e4m3":
                    got, step_, floor = got.view(torch.float8_e4m3fn).double() * sc.double().to(DEV)[:, None], 2.0 ** -4, 2.0 ** -10 * 0.05
                    ref = np.clip(ref, -448 * sc.double().numpy()[:, None], 448 * sc.double().numpy()[:, None])
                else:
                    got, step_, floor = got.double(), 2.0 ** -8, 0.0
                # (2^-18: the float32 norm and rotation, of a pair's larger value)
                err = np.abs(got.cpu().numpy() - ref)
                assert (err <= (step_ + 2.0 ** -18) * np.abs(ref) + floor + 2.0 ** -18 * np.abs(ref).max()).all()
    cache.free(seqs[2])
    cache.free(seqs[1])
    cache.free(seqs[0])
    assert cache.bm.allocator.num_free() == 96


def test_an_e4m3_cache_refuses_tree_attention():
    cache = PagedKVCache(8, 16, 2, 128, "fp8_e4m3", DEV)
    s = cache.add_sequence()
    with pytest.raises(NotImplementedError):
        cache.decode_tree(torch.zeros(1, 8, 128, dtype=torch.bfloat16, device=DEV), [s], [1])
