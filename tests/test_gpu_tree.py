"""pa_decode_tree against float64 attention over each row's own keys.

Tolerance, from the arithmetic: each softmax weight is rounded to bf16 (relative
2^-8 at most) in the numerator and, the same way, in the row sum, so an output is
off by at most 2 * 2^-8 * sum_t p_t |v_t|; exponentials and sums in float32 add
less than 2^-14 of that sum. A score sums products in at most 16 float32 steps,
off by 2^-20 of X = scale * sum |q k|, which moves a weight by that much of
itself, twice over (numerator and sum). The output's own rounding is 2^-8 of its
value.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa
from gpu_harness import poison

pytestmark = pytest.mark.gpu
DEV = "cuda"


def tree_parents(rng, n, kind):
    """Parents of n rows: 'chain', 'star' (all follow row 0), 'tree' or 'forest' (some follow
    the context alone)."""
    i = np.arange(n)
    if kind == "chain":
        p = i - 1
    elif kind == "star":
        p = np.where(i == 0, -1, 0)
    else:
        p = np.minimum(i - 1, (rng.random(n) * i).astype(int))
        if kind == "forest":
            p[rng.random(n) < 0.3] = -1
        p[:1] = -1
    return p.astype(np.int32)


class Batch:
    """Paged caches whose every unwritten row is NaN, with the step's rows in place."""

    def __init__(self, ctx, counts, hq, hkv, d, bs, kind="tree", seed=0, spare_rows=0, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        self.counts = np.asarray(counts)
        self.lens = np.asarray(ctx) + self.counts
        need = -(-np.maximum(self.lens, 1) // bs)
        pool = int(need.sum()) + 2
        ids = rng.permutation(pool)
        self.tables = np.full((len(need), int(need.max())), 10 ** 9, dtype=np.int32)  # unused entries: never read
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = ids[at:at + k]
            at += k
        gen = torch.Generator().manual_seed(seed)
        self.kc = torch.zeros(pool, bs, hkv, d, dtype=torch.bfloat16)
        self.vc = torch.zeros_like(self.kc)
        poison(self.kc)
        poison(self.vc)
        for s, L in enumerate(self.lens):
            t = np.arange(L)
            slot = torch.from_numpy(self.tables[s, t // bs].astype(np.int64) * bs + t % bs)
            for c in (self.kc, self.vc):
                c.view(-1, hkv, d)[slot] = torch.randn(len(t), hkv, d, generator=gen).bfloat16()
        total = int(self.counts.sum())
        self.q = (qscale * torch.randn(total + spare_rows, hq, d, generator=gen)).bfloat16()
        self.start = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)
        self.parents = np.concatenate([tree_parents(rng, n, kind) for n in self.counts] +
                                      [np.full(spare_rows, -1, dtype=np.int32)])
        self.chain = kind == "chain"
        self.scale = 1.0 / np.sqrt(d)

    def run(self, parents="given", out=None, workspace=None, stream=None):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        q = self.q.to(DEV)
        out = torch.full_like(q, float("nan")) if out is None else out
        most = max(1, int(self.counts.max()))
        if workspace is None:
            workspace = torch.empty(pa.pa_decode_tree_workspace_bytes(self.hq, self.hkv, self.d, most),
                                    dtype=torch.uint8, device=DEV)
            workspace.random_(0, 256)       # its contents on entry mean nothing
        par = dev(self.parents.astype(np.int32)) if parents == "given" else None
        pa.pa_decode_tree(out, q, self.kc.to(DEV), self.vc.to(DEV), dev(self.tables),
                          dev(self.lens.astype(np.int32)), dev(self.start), par, most, self.scale,
                          workspace, stream=stream)
        torch.cuda.synchronize()
        return out

    def expected(self):
        """(reference, tolerance) in float64, row by row from the definition."""
        n_all = int(self.counts.sum())
        ref = np.zeros((n_all, self.hq, self.d))
        tol = np.zeros_like(ref)
        group = self.hq // self.hkv
        kf, vf = (c.view(-1, self.hkv, self.d).double().numpy() for c in (self.kc, self.vc))
        q = self.q.double().numpy()
        for s, L in enumerate(self.lens):
            t = np.arange(L)
            slot = self.tables[s, t // self.bs].astype(np.int64) * self.bs + t % self.bs
            k, v = kf[slot], vf[slot]
            n = self.counts[s]
            for i in range(n):
                keys = list(range(L - n))
                own, a = [], i
                while a >= 0:
                    own.append(L - n + a)
                    a = self.parents[self.start[s] + a]
                keys = np.array(keys + own[::-1])
                row = self.start[s] + i
                for h in range(self.hkv):
                    x = q[row, h * group:(h + 1) * group] @ k[keys, h].T * self.scale
                    w = np.exp(x - x.max(-1, keepdims=True))
                    w /= w.sum(-1, keepdims=True)
                    ref[row, h * group:(h + 1) * group] = w @ v[keys, h]
                    mag = w @ np.abs(v[keys, h])
                    top = (np.abs(q[row, h * group:(h + 1) * group]) @ np.abs(k[keys, h]).T).max() * self.scale
                    tol[row, h * group:(h + 1) * group] = (2.0 ** -7 + 2.0 ** -14 + 2.0 ** -19 * top) * mag
        return ref, tol + 2.0 ** -8 * np.abs(ref)


def check(batch, out, what=""):
    assert pa.pa_device_errors() == 0
    ref, tol = batch.expected()
    got = out[:len(ref)].double().cpu().numpy()
    assert np.isfinite(got).all(), what
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"{what}: off by up to {(err / tol).max():.2f} of the tolerance"


@pytest.mark.parametrize("ctx,counts,hq,hkv,d,bs,kind", [
    ([0], [1], 4, 2, 64, 8, "chain"),                       # one token, nothing before it
    ([5], [1], 8, 8, 128, 16, "chain"),                     # a plain decode
    ([300], [8], 32, 8, 128, 16, "tree"),
    ([0, 0, 1], [3, 70, 64], 8, 2, 64, 16, "tree"),         # no context: whole tiles a row sees nothing of
    ([63, 64, 65, 127, 128], [1, 2, 3, 1, 65], 8, 2, 128, 32, "forest"),   # tile edges
    ([1000, 0, 17, 4096], [16, 0, 5, 9], 16, 2, 128, 64, "tree"),          # a sequence without rows
    ([200, 33], [100, 128], 4, 4, 128, 256, "star"),
    ([90], [300], 8, 1, 128, 16, "tree"),                   # several items of rows
    ([2500, 10], [17, 33], 4, 1, 64, 128, "chain"),
    ([700] * 5, [12, 1, 31, 4, 20], 8, 8, 64, 8, "forest"),
    ([3000], [2], 64, 8, 128, 16, "chain"),                 # one sequence cut into many parts
])
def test_tree_matches_float64(ctx, counts, hq, hkv, d, bs, kind):
    b = Batch(ctx, counts, hq, hkv, d, bs, kind, seed=len(ctx) + d)
    check(b, b.run())
    if kind == "chain":                                     # without parents: chains, bit for bit
        assert torch.equal(b.run(parents=None), b.run())


@pytest.mark.parametrize("seed", range(8))
def test_tree_matches_float64_on_drawn_batches(seed):
    rng = np.random.default_rng(100 + seed)
    s = int(rng.integers(1, 12))
    hkv, group = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 4, 8]))
    b = Batch(rng.integers(0, 900, s), rng.integers(0, 40, s) + (np.arange(s) == 0), hkv * group, hkv,
              int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 256])),
              ["tree", "forest", "chain", "star"][seed % 4], seed=seed, qscale=[1.0, 4.0][seed % 2])
    check(b, b.run(), f"seed {seed}")


@pytest.mark.parametrize("length", [383, 384, 385, 448, 449])
@pytest.mark.parametrize("rows", [9, 70])
def test_tables_around_the_shortest_that_may_be_cut(length, rows):
    # (six tiles are not cut and need no merge; two sequences, so that a cut could fall inside)
    for bs in (16, 64):
        b = Batch([length - rows, 0], [rows, 1], 32, 8, 128, bs, "tree", seed=length + rows)
        check(b, b.run(), f"block size {bs}")


def test_more_sequences_than_threads():
    rng = np.random.default_rng(3)
    s = 700
    b = Batch(rng.integers(0, 40, s), rng.integers(0, 4, s), 2, 1, 64, 8, "tree", seed=9)
    check(b, b.run())


def test_large_scores_and_a_moving_reference():
    # scores of up to some hundreds: the reference maximum moves, weights underflow
    b = Batch([900], [9], 8, 2, 128, 16, "tree", seed=2, qscale=30.0)
    check(b, b.run())


def test_rows_past_the_last_sequence_stay():
    b = Batch([50, 70], [5, 3], 8, 2, 128, 16, "tree", seed=4, spare_rows=6)
    out = torch.full((14, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    b.run(out=out)
    check(b, out)
    assert (out[8:] == 7.0).all()


def test_same_result_on_any_block_size_placement_and_call():
    outs, parents = [], None
    for bs in (8, 16, 64, 256):
        b = Batch([333, 1200, 64], [9, 20, 1], 8, 2, 128, bs, "tree", seed=5)
        # (the trees are drawn after the placement, whose draws go by the pool's size)
        parents = b.parents if parents is None else parents
        b.parents = parents
        ws = torch.empty(pa.pa_decode_tree_workspace_bytes(8, 2, 128, 64), dtype=torch.uint8, device=DEV)
        outs.append(b.run(workspace=ws))        # a workspace for more rows serves fewer
        assert torch.equal(outs[-1], b.run())
    # (the rows of a sequence are drawn in token order: the same for every block size)
    assert all(torch.equal(outs[0], o) for o in outs[1:])


def test_a_key_that_a_row_does_not_see_may_be_nan():
    b = Batch([100], [6], 8, 2, 128, 16, "star", seed=6)
    L = int(b.lens[0])
    t = L - 1                                   # the last row: nobody's ancestor
    slot = int(b.tables[0, t // 16]) * 16 + t % 16
    clean = b.run()
    b.kc.view(-1, 2, 128)[slot] = float("nan")
    out = b.run()
    assert torch.equal(out[:5], clean[:5])
    assert torch.isnan(out[5]).all()


@pytest.mark.parametrize("what", ["context", "range", "parent", "table"])
def test_bad_indices_are_flagged_and_skipped(what):
    b = Batch([40, 60], [4, 4], 8, 2, 128, 16, "tree", seed=7)
    good = b.run()
    flag = pa.PA_DEVERR_CONTEXT
    if what == "context":
        b.lens[0] = 3                           # fewer tokens than rows
    elif what == "range":
        b.start = np.array([0, 9, 8], dtype=np.int32)   # past the batch, then backwards
    elif what == "parent":
        b.parents[2] = 2                        # its own parent
        flag = pa.PA_DEVERR_DRAFT
    else:
        b.tables[0, 1] = 10 ** 6
        flag = pa.PA_DEVERR_BLOCK_ID
    out = torch.full_like(b.q, 5.0, device=DEV)
    b.run(out=out)
    assert pa.pa_device_errors() == flag
    if what in ("context", "range"):
        assert (out[:4] == 5.0).all()
    if what != "range":
        # (cut differently where a sequence fell out: the same to rounding)
        assert torch.allclose(out[4:].float(), good[4:].float(), atol=2e-2)


def test_two_captured_graphs_share_a_workspace_and_follow_the_lengths():
    b = Batch([500, 900], [8, 8], 32, 8, 128, 16, "tree", seed=8)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    ws = torch.empty(pa.pa_decode_tree_workspace_bytes(32, 8, 128, 8), dtype=torch.uint8, device=DEV)
    q, kc, vc = b.q.to(DEV), b.kc.to(DEV), b.vc.to(DEV)
    tables, start, par = dev(b.tables), dev(b.start), dev(b.parents)
    lens = dev(b.lens.astype(np.int32))
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for o in outs:
            pa.pa_decode_tree(o, q, kc, vc, tables, lens, start, par, 8, b.scale, ws)
    torch.cuda.synchronize()
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pa.pa_decode_tree(o, q, kc, vc, tables, lens, start, par, 8, b.scale, ws)
        graphs.append(g)
    for new in (b.lens, b.lens - np.array([200, 31])):
        b.lens = np.asarray(new)
        lens.copy_(dev(b.lens.astype(np.int32)))
        for o, g in zip(outs, graphs):
            o.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            check(b, o)


def test_on_another_stream():
    b = Batch([500], [8], 8, 2, 128, 16, "tree", seed=10)
    want = b.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(b.run(stream=side), want)


def test_binding_refuses():
    b = Batch([40], [4], 8, 2, 128, 16, "tree", seed=11)
    q = b.q.to(DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    args = dict(out=torch.empty_like(q), q=q, k_cache=b.kc.to(DEV), v_cache=b.vc.to(DEV),
                block_tables=torch.from_numpy(b.tables).to(DEV), context_lens=i32(44), query_start=i32(0, 4),
                parents=i32(-1, 0, 0, 1), max_query_len=4, scale=0.1, workspace=ws)
    for over, err in [(dict(parents=i32(-1, 0)), ValueError), (dict(query_start=i32(0)), ValueError),
                      (dict(workspace=None), ValueError), (dict(workspace=ws[:16]), pa.PagedAttentionError),
                      (dict(parents=torch.zeros(4, dtype=torch.int64, device=DEV)), TypeError),
                      (dict(q=q.float()), TypeError), (dict(q=q.cpu()), ValueError),
                      (dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError)]:
        with pytest.raises(err):
            pa.pa_decode_tree(**{**args, **over})
