"""pa_verify_draft against the walk written out in float64 (every token and path equal),
its distribution, and pa_kv_accept against a plain move of rows (bit for bit)."""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa
from test_gpu_tree import tree_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def draw_batch(seed, counts, vocab, kind, sampled, sharp=3.0, noise=1.0):
    rng = np.random.default_rng(seed)
    counts = np.asarray(counts)
    total = int(counts.sum())
    logits = sharp * rng.standard_normal((total, vocab))
    target = softmax(logits)
    draft = softmax(logits + noise * rng.standard_normal((total, vocab)))
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    parents = np.concatenate([tree_parents(rng, n, kind) for n in counts]).astype(np.int32) if total else \
        np.zeros(0, np.int32)
    tokens = np.zeros(total, dtype=np.int32)
    for s, n in enumerate(counts):
        for i in range(1, n):
            row = draft[start[s] + max(0, parents[start[s] + i])].astype(np.float64)
            tokens[start[s] + i] = rng.choice(vocab, p=row / row.sum()) if sampled else \
                np.argsort(-row)[min(vocab - 1, rng.integers(0, 4))]
    return dict(target=target, draft=draft if sampled else None, tokens=tokens, parents=parents, start=start,
                ua=rng.random(total, dtype=np.float32), us=rng.random(len(counts), dtype=np.float32))


def walk(b, s):
    """(tokens, path) of sequence s: children of the last accepted row, in order."""
    a, n = b["start"][s], b["start"][s + 1] - b["start"][s]
    if n == 0:
        return [], []
    clean = lambda p: np.where(p > 0, p, 0).astype(np.float64)  # noqa: E731
    said, path, cur, moved = [], [0], 0, True
    while moved:
        moved = False
        left, z = clean(b["target"][a + cur]), 1.0
        q = clean(b["draft"][a + cur]) if b["draft"] is not None else None
        for i in range(cur + 1, n):
            par = b["parents"][a + i] if b["parents"] is not None else i - 1
            x = b["tokens"][a + i]
            if par != cur or not 0 <= x < len(left):
                continue
            if float(b["ua"][a + i]) * (q[x] if q is not None else 1.0) * z < left[x]:
                said.append(int(x))
                path.append(i)
                cur, moved = i, True
                break
            if q is not None:
                left = np.maximum(left / z - q, 0.0) if z > 0 else np.zeros_like(left)
                z = left.sum()
            else:
                z = max(z - left[x], 0.0)
                left[x] = 0.0
    if left.sum() == 0:
        left = clean(b["target"][a + cur])
    c = np.cumsum(left)
    said.append(int(min((c <= float(b["us"][s]) * c[-1]).sum(), len(c) - 1)))
    return said, path


def run(b, most=None, stream=None, pad=0):
    counts = np.diff(b["start"])
    most = max(1, int(counts.max())) if most is None else most
    s = len(counts)
    t = {k: None if v is None else dev(v) for k, v in b.items()}
    if pad:     # rows of a wider tensor
        for k in ("target", "draft"):
            if t[k] is not None:
                w = torch.full((t[k].shape[0], t[k].shape[1] + pad), 9.0, device=DEV)
                w[:, :-pad] = t[k]
                t[k] = w[:, :-pad]
    out = torch.full((s, most), 77, dtype=torch.int32, device=DEV)
    path, length = torch.full_like(out, 77), torch.full((s,), 77, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    pa.pa_verify_draft(out, path, length, t["target"], t["draft"], t["tokens"], t["parents"], t["start"], t["ua"],
                       t["us"], stream=stream)
    torch.cuda.synchronize()
    return out.cpu().numpy(), path.cpu().numpy(), length.cpu().numpy()


def check(b, got):
    out, path, length = got
    for s in range(len(length)):
        said, kept = walk(b, s)
        assert length[s] == len(said)
        assert out[s, :len(said)].tolist() == said and (out[s, len(said):] == -1).all()
        assert path[s, :len(kept)].tolist() == kept and (path[s, len(kept):] == -1).all()


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("counts,vocab,kind", [
    ([1], 17, "chain"),                         # nothing drafted: a plain draw
    ([5], 32000, "chain"),
    ([4, 1, 0, 9], 1000, "tree"),
    ([16] * 6, 257, "star"),                    # many children of one row, tokens among them twice
    ([33, 2, 64], 4099, "forest"),
    ([3] * 40, 1, "tree"),                      # one token
    ([7, 8], 50257, "tree"),
    ([300], 100, "tree"),
    ([6] * 700, 33, "tree"),                    # one CTA a sequence
])
def test_verify_matches_the_walk(counts, vocab, kind, sampled):
    for seed in range(3):
        b = draw_batch(1000 * seed + vocab, counts, vocab, kind, sampled, sharp=[3.0, 1.0, 6.0][seed])
        got = run(b)
        assert pa.pa_device_errors() == 0
        check(b, got)
        if kind == "chain":
            again = run({**b, "parents": None})
            assert all(np.array_equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("vocab,pad", [(128256, 0), (130001, 3), (99001, 1)])
def test_rows_summed_again_after_many_rejections(vocab, pad):
    # more values than a cluster keeps on chip; (130001, 3): 16-byte-aligned rows with an odd end
    b = draw_batch(vocab, [9, 12, 1, 10], vocab, "star", True, sharp=1.5, noise=0.7)
    start = b["start"]
    b["ua"][:] = 0.99999994
    for s in (0, 1):                       # the least likely tokens: rejected
        rows = slice(start[s] + 1, start[s + 1])
        b["tokens"][rows] = np.argsort(b["target"][start[s]])[:start[s + 1] - start[s] - 1]
    # the second one's sixth child is accepted, and its own children rejected again
    six = start[1] + 6
    b["tokens"][six], b["ua"][six] = int(b["target"][start[1]].argmax()), 0.0
    b["parents"][six + 1:start[2]] = 6
    b["tokens"][six + 1:start[2]] = np.argsort(b["target"][six])[:start[2] - six - 1]
    check(b, run(b, pad=pad))
    assert pa.pa_device_errors() == 0


def test_rows_of_a_wider_tensor_and_wider_outputs():
    b = draw_batch(5, [6, 3], 1001, "tree", True)
    for pad in (1, 3, 23):
        check(b, run(b, most=11, pad=pad))


def test_numbers_at_the_ends():
    b = draw_batch(6, [4, 4, 4], 500, "tree", True)
    b["target"][0, :10] = 0.0
    b["us"][:] = [0.0, 1.0 - 2.0 ** -24, 0.5]
    b["ua"][:] = 0.0                            # always accepted where the target may say it
    check(b, run(b))
    b["ua"][:] = 1.0 - 2.0 ** -24
    check(b, run(b))


def test_equal_distributions_are_always_accepted():
    b = draw_batch(7, [9] * 8, 300, "chain", True, noise=0.0)
    b["draft"] = b["target"].copy()
    out, path, length = run(b)
    assert (length == 9).all()
    check(b, (out, path, length))


def test_no_mass_left_and_values_that_count_as_zero():
    b = draw_batch(8, [3], 64, "star", True)
    b["target"][0] = 0.0
    b["target"][0, 5] = 0.4                     # below the draft's everywhere: nothing is left
    b["draft"][0] = 1.0 / 64
    b["draft"][0, 5] = 0.9
    b["tokens"][1:] = [5, 5]
    b["ua"][:] = 0.99
    b["target"][0, 7] = -1.0
    b["target"][0, 8] = np.nan
    got = run(b)
    assert pa.pa_device_errors() == 0
    assert got[0][0, 0] == 5 and got[2][0] == 1
    check(b, got)


def test_bad_rows_are_flagged():
    b = draw_batch(9, [4, 4], 100, "tree", True)
    b["tokens"][1] = 100
    got = run(b)
    assert pa.pa_device_errors() == pa.PA_DEVERR_DRAFT
    check(b, got)                               # never tried
    b = draw_batch(9, [4, 4], 100, "tree", True)
    b["parents"][2] = 3
    run(b)
    assert pa.pa_device_errors() == pa.PA_DEVERR_DRAFT
    b = draw_batch(9, [1, 4], 100, "tree", True)
    b["target"][0] = 0.0                        # a last row without mass
    out, _, length = run(b)
    assert pa.pa_device_errors() == pa.PA_DEVERR_DRAFT
    assert out[0, 0] == -1 and length[0] == 1
    b = draw_batch(9, [4, 4], 100, "tree", True)
    out, path, length = run(b, most=3)          # more rows than the caller says
    assert pa.pa_device_errors() == pa.PA_DEVERR_CONTEXT
    assert (length == 0).all() and (out == -1).all() and (path == -1).all()


def test_distribution_is_the_targets():
    """The first token over many draws, against the target's probabilities: a count of n
    draws at probability p is within 6 standard deviations, sqrt(n p (1 - p)), in all but
    one of 10^8 cases per value."""
    vocab, n = 6, 20000
    rng = np.random.default_rng(3)
    p, q = softmax(rng.standard_normal(vocab)), softmax(rng.standard_normal(vocab))
    for sampled in (True, False):
        kids = 3
        rows = 1 + kids
        target = np.tile(p, (n * rows, 1))
        tokens = np.zeros((n, rows), dtype=np.int32)
        tokens[:, 1:] = rng.choice(vocab, size=(n, kids), p=q / q.astype(np.float64).sum()) if sampled else \
            np.argsort(-q)[:kids]
        b = dict(target=target, draft=np.tile(q, (n * rows, 1)) if sampled else None, tokens=tokens.reshape(-1),
                 parents=np.tile(np.array([-1, 0, 0, 0], np.int32), n), start=np.arange(0, n * rows + 1, rows, dtype=np.int32),
                 ua=rng.random(n * rows, dtype=np.float32), us=rng.random(n, dtype=np.float32))
        out, _, _ = run(b)
        got = np.bincount(out[:, 0], minlength=vocab)
        pd = p.astype(np.float64) / p.astype(np.float64).sum()
        assert (np.abs(got - n * pd) <= 6 * np.sqrt(n * pd * (1 - pd))).all(), (got, n * pd)


def test_captured_and_on_another_stream():
    b = draw_batch(11, [8, 8], 3000, "tree", True)
    want = run(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert all(np.array_equal(x, y) for x, y in zip(run(b, stream=side), want))
    t = {k: dev(v) for k, v in b.items()}
    out = torch.zeros(2, 8, dtype=torch.int32, device=DEV)
    path, length = torch.zeros_like(out), torch.zeros(2, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_verify_draft(out, path, length, t["target"], t["draft"], t["tokens"], t["parents"], t["start"], t["ua"], t["us"])
    for seed in (11, 12):
        b = draw_batch(seed, [8, 8], 3000, "tree", True)
        for k, v in b.items():
            t[k].copy_(dev(v))
        g.replay()
        torch.cuda.synchronize()
        check(b, (out.cpu().numpy(), path.cpu().numpy(), length.cpu().numpy()))


def test_verify_binding_refuses():
    b = draw_batch(12, [3], 50, "tree", True)
    t = {k: dev(v) for k, v in b.items()}
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    a = dict(out_tokens=z(1, 3), out_path=z(1, 3), out_len=z(1), target_probs=t["target"], draft_probs=t["draft"],
             draft_tokens=t["tokens"], parents=t["parents"], query_start=t["start"], u_accept=t["ua"], u_sample=t["us"])
    for over, err in [(dict(target_probs=t["target"].bfloat16()), TypeError), (dict(draft_probs=t["draft"][:2]), ValueError),
                      (dict(out_path=z(1, 2)), ValueError), (dict(draft_tokens=t["tokens"].long()), TypeError),
                      (dict(u_sample=t["us"][:0]), ValueError), (dict(u_accept=t["ua"].cpu()), ValueError),
                      (dict(target_probs=t["target"].t().contiguous().t()), ValueError)]:
        with pytest.raises(err):
            pa.pa_verify_draft(**{**a, **over})


# --------------------------------------------------------------- pa_kv_accept

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


def accept_case(ctx, counts, paths, hkv, d, bs, kind, seed=0):
    rng = np.random.default_rng(seed)
    lens = np.asarray(ctx) + np.asarray(counts)
    need = -(-np.maximum(lens, 1) // bs)
    pool = int(need.sum()) + 2
    ids = rng.permutation(pool)
    tables = np.zeros((len(lens), int(need.max())), dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        tables[s, :k] = ids[at:at + k]
        at += k
    raw = torch.from_numpy(rng.integers(0, 256, (2, pool * bs, hkv * d * DT[kind].itemsize), dtype=np.uint8))
    most = max(1, max(len(p) for p in paths))
    path = np.full((len(paths), most), -1, dtype=np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    want = raw.clone()
    for s, p in enumerate(paths):
        base = lens[s] - counts[s]
        slot = lambda t: tables[s, t // bs] * bs + t % bs  # noqa: B023,E731
        for j, i in enumerate(p):
            want[:, slot(base + j)] = raw[:, slot(base + i)]
    caches = [raw[i].to(DEV).view(DT[kind]).view(pool, bs, hkv, d) for i in (0, 1)]
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    args = [*caches, dev(tables), dev(lens.astype(np.int32)), dev(start), dev(path),
            dev(np.array([len(p) for p in paths], dtype=np.int32))]
    return args, want


def same_bits(args, want):
    return all(torch.equal(c.reshape(want.shape[1], -1).view(torch.uint8).cpu(), want[i]) for i, c in enumerate(args[:2]))


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("ctx,counts,paths,hkv,d,bs", [
    ([0], [1], [[0]], 2, 64, 1),
    ([10, 0, 7], [4, 3, 0], [[0, 2], [0, 1, 2], []], 8, 128, 16),
    ([63, 64, 5], [9, 12, 6], [[0, 1, 3, 8], [0, 11], [0, 1, 2, 5]], 1, 64, 4),
    ([30], [200], [[0] + list(range(2, 200, 2))], 4, 128, 64),      # a path of several batches
    ([5], [40], [list(range(1, 40))], 2, 128, 16),                  # every row moves by one
    ([100] * 70, [8] * 70, [[0, 3, 7]] * 70, 8, 64, 256),
])
def test_accept_moves_rows(ctx, counts, paths, hkv, d, bs, kind):
    args, want = accept_case(ctx, counts, paths, hkv, d, bs, kind, seed=len(ctx) + bs)
    pa.pa_kv_accept(*args)
    assert pa.pa_device_errors() == 0
    assert same_bits(args, want)


@pytest.mark.parametrize("paths,flag", [
    ([[0, 2, 1], [0, 1]], "PA_DEVERR_DRAFT"),       # not increasing
    ([[0, 9], [0, 1]], "PA_DEVERR_DRAFT"),          # past its rows
    ([[0, 0], [0, 1]], "PA_DEVERR_DRAFT"),          # twice the same row
])
def test_bad_paths_are_flagged_and_skipped(paths, flag):
    args, want = accept_case([10, 10], [4, 4], [[0], paths[1]], 2, 64, 16, "bf16", seed=1)
    args[5] = dev(np.array([(p + [-1] * 4)[:4] for p in paths], dtype=np.int32))
    args[6] = dev(np.array([len(p) for p in paths], dtype=np.int32))
    pa.pa_kv_accept(*args)
    assert pa.pa_device_errors() == getattr(pa, flag)
    assert same_bits(args, want)


def test_bad_lengths_and_tables_are_flagged_and_skipped():
    for what, flag in (("len", pa.PA_DEVERR_DRAFT), ("ctx", pa.PA_DEVERR_CONTEXT), ("table", pa.PA_DEVERR_BLOCK_ID)):
        args, _ = accept_case([16, 16], [4, 4], [[0, 2], [0, 3]], 2, 64, 4, "bf16", seed=2)
        _, want = accept_case([16, 16], [4, 4], [[0], [0, 3]], 2, 64, 4, "bf16", seed=2)
        if what == "len":
            args[6][0] = 5
        elif what == "ctx":
            args[3][0] = 3
        else:
            args[2][0, 4] = 10 ** 6
        pa.pa_kv_accept(*args)
        assert pa.pa_device_errors() == flag
        assert same_bits(args, want)
