"""The operators of a drafted decoding step over the paged cache, in plain torch and through the package.

A step that verifies drafted tokens runs, per layer, the rows operator (norms of
the query and key heads, the position rotation, the write into the cache) and
the attention of every drafted token over the cache and its own ancestors; after
the last layer it verifies the drafted tokens against the target's
probabilities, and moves the cache rows of the accepted ones into place.

`listed()` and `draw(rng)` give the cases, `prepare(case, seed)` a program's
data, `run(state)` one pass, `work(case)` what a pass cannot do without, and
`exact(case, seed)` the definition in 64 bits. `own` chooses between the plain
forms (elementary torch operations) and the package's calls.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}   # of the rows
# the eight request lengths of the Llama-3-8B batch in workloads/synth.py
BATCH_LENGTHS = (128, 700, 1500, 300, 2900, 50, 4100, 900)


def listed():
    return [
        # two sequences of 7 and 33 tokens written at once, float32, head_dim 64: the smallest call
        {"name": "rows_small_f32", "op": "rows", "tokens": 40, "hq": 4, "hkv": 2, "d": 64, "bs": 4, "kind": "f32", "rot": 64,
         "interleaved": False, "norm": True},
        # the next token of each of eight requests: what latency is worth
        {"name": "rows_step", "op": "rows", "tokens": 8, "hq": 32, "hkv": 8, "d": 128, "bs": 16, "kind": "bf16", "rot": 128,
         "interleaved": False, "norm": True},
        # sixteen drafted tokens for each of 256 requests into an E4M3 cache, half of each head rotated, in pairs
        {"name": "rows_drafts_e4m3", "op": "rows", "tokens": 4096, "hq": 32, "hkv": 8, "d": 128, "bs": 16, "kind": "e4m3", "rot": 64,
         "interleaved": True, "norm": True},
        # the eight whole prompts of the Llama-3-8B batch: the largest
        {"name": "rows_prompts", "op": "rows", "tokens": 10578, "hq": 32, "hkv": 8, "d": 128, "bs": 16, "kind": "bf16", "rot": 128,
         "interleaved": False, "norm": True},
        # one request, eight drafted tokens on a short context: latency
        {"name": "tree_single", "op": "tree", "seqs": 1, "nodes": 8, "ragged": False, "ctx": "flat", "len": 300, "hq": 32, "hkv": 8,
         "d": 128, "bs": 16, "tree": True},
        # the Llama-3-8B batch with a tree of sixteen tokens each
        {"name": "tree_batch8", "op": "tree", "seqs": 8, "nodes": 16, "ragged": False, "ctx": "batch", "len": 4100, "hq": 32, "hkv": 8,
         "d": 128, "bs": 16, "tree": True},
        # 256 requests of lognormal lengths, one to sixteen drafted tokens each
        {"name": "tree_batch256", "op": "tree", "seqs": 256, "nodes": 16, "ragged": True, "ctx": "lognormal", "len": 4096, "hq": 32,
         "hkv": 8, "d": 128, "bs": 16, "tree": True},
        # long contexts and wide trees
        {"name": "tree_long", "op": "tree", "seqs": 4, "nodes": 64, "ragged": False, "ctx": "flat", "len": 32768, "hq": 32, "hkv": 8,
         "d": 128, "bs": 16, "tree": True},
        # a chain of four drafted tokens of one request, a small vocabulary
        {"name": "verify_chain", "op": "verify", "seqs": 1, "nodes": 5, "ragged": False, "vocab": 32000, "tree": False, "sampled": True},
        # a tree of sixteen for each of 64 requests, a large vocabulary
        {"name": "verify_trees", "op": "verify", "seqs": 64, "nodes": 16, "ragged": True, "vocab": 128256, "tree": True, "sampled": True},
        # the drafted rows of the Llama-3-8B batch, written and then moved into place
        {"name": "accept_batch8", "op": "accept", "seqs": 8, "nodes": 16, "ctx": "batch", "len": 4100, "hkv": 8, "d": 128, "bs": 16,
         "kind": "bf16"},
        # the same for 256 requests over an E4M3 cache
        {"name": "accept_256_e4m3", "op": "accept", "seqs": 256, "nodes": 32, "ctx": "flat", "len": 500, "hkv": 8, "d": 128, "bs": 16,
         "kind": "e4m3"},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rows", "tree", "tree", "verify", "accept"))
    hkv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8))
    if op == "rows":
        d, kind = rng.choice((64, 128)), rng.choice(("f32", "bf16", "bf16", "e4m3"))
        tokens = _between(rng, 1, 8192)
        if kind == "f32" and tokens * hkv * (group + 2) * d > 20_000_000:
            tokens = max(1, 20_000_000 // (hkv * (group + 2) * d))
        return {"op": "rows", "tokens": tokens, "hq": hkv * group, "hkv": hkv, "d": d, "bs": rng.choice((1, 4, 16, 64, 256)), "kind": kind,
                "rot": rng.choice((d, d // 2, 16)), "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.8}
    if op == "tree":
        seqs, nodes = _between(rng, 1, 96), _between(rng, 1, 64)
        length = _between(rng, 1, max(64, min(16384, 400_000 // (seqs * max(1, nodes * group // 64)))))
        return {"op": "tree", "seqs": seqs, "nodes": nodes, "ragged": rng.random() < 0.6, "ctx": rng.choice(("flat", "uniform")),
                "len": length, "hq": hkv * group, "hkv": hkv, "d": rng.choice((64, 128, 128)), "bs": rng.choice((8, 16, 16, 32, 64, 256)),
                "tree": rng.random() < 0.7}
    if op == "verify":
        vocab = _between(rng, 97, 152_001)
        seqs = _between(rng, 1, 96)
        nodes = _between(rng, 1, max(1, min(24, 100_000_000 // (vocab * seqs))))
        return {"op": "verify", "seqs": seqs, "nodes": nodes, "ragged": rng.random() < 0.5, "vocab": vocab, "tree": rng.random() < 0.6,
                "sampled": rng.random() < 0.7}
    return {"op": "accept", "seqs": _between(rng, 1, 200), "nodes": _between(rng, 1, 48), "ctx": rng.choice(("flat", "uniform")),
            "len": _between(rng, 1, 700), "hkv": hkv, "d": rng.choice((64, 128)), "bs": rng.choice((1, 4, 16, 64, 256)),
            "kind": rng.choice(("f32", "bf16", "e4m3"))}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Host lengths of a case, the same for every seed: tokens cached before the step (None for verification) and rows of the step."""
    rng = np.random.default_rng([case["seqs"], case["nodes"], 77])
    counts = _counts(case, rng)
    return (_context(case, rng) if "ctx" in case else None), counts


def _context(case, rng):
    """Tokens cached before the step, for each sequence."""
    n, most = case["seqs"], case["len"]
    if case["ctx"] == "batch":
        return np.asarray(BATCH_LENGTHS[:n], dtype=np.int64)
    if case["ctx"] == "lognormal":      # mean 600, sigma 0.75, 16 .. 4096, as workloads/configs.py has it
        x = rng.lognormal(math.log(600.0) - 0.5 * 0.75 ** 2, 0.75, n)
        return np.clip(np.rint(x), 16, most).astype(np.int64)
    if case["ctx"] == "uniform":
        return rng.integers(0, most + 1, n)
    return np.full(n, most, dtype=np.int64)


def _counts(case, rng):
    """Rows of this step, for each sequence: its last token and what was drafted after it."""
    n = np.full(case["seqs"], case["nodes"], dtype=np.int64)
    if case.get("ragged") and case["nodes"] > 1:
        n = rng.integers(1, case["nodes"] + 1, case["seqs"])
        n[0] = case["nodes"]
    return n


def _parents(counts, tree, rng):
    """The row that each row follows, within its sequence; -1 for the first. Trees branch near their roots."""
    out = []
    for n in counts:
        i = np.arange(n)
        p = i - 1
        if tree:
            p = np.minimum(p, (rng.random(n) ** 1.5 * i).astype(np.int64))
            p[0] = -1
        out.append(p)
    return np.concatenate(out)


def _tables(lens, bs, rng, spare=3):
    """Block tables over a shuffled pool, and its size."""
    need = -(-np.maximum(lens, 1) // bs)
    pool = int(need.sum()) + spare
    ids = rng.permutation(pool)
    tables = np.zeros((len(lens), int(need.max())), dtype=np.int32)
    at = 0
    for s, k in enumerate(need):
        tables[s, :k] = ids[at:at + k]
        at += k
    return tables, pool


def _slots(tables, bs, first, counts):
    """Flat slots of counts[s] rows from position first[s] on."""
    return np.concatenate([tables[s, np.arange(a, a + n) // bs].astype(np.int64) * bs + np.arange(a, a + n) % bs
                           for s, (a, n) in enumerate(zip(first, counts))])


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _rand(gen, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 77])
    gen = torch.Generator(DEV)
    gen.manual_seed(int(seed) * 31 + 5)
    s = dict(case)
    if case["op"] == "rows":
        n, hq, hkv, d, bs = (case[k] for k in ("tokens", "hq", "hkv", "d", "bs"))
        dt = TYPES[case["kind"]]
        # one packed row of projections a token: q, k and v are views of it
        packed = _rand(gen, n, (hq + 2 * hkv) * d, dtype=dt)
        s["q"] = packed[:, :hq * d].view(n, hq, d)
        s["k"] = packed[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        s["v"] = packed[:, (hq + hkv) * d:].view(n, hkv, d)
        pool = -(-n // bs) + 3
        slots = rng.permutation(pool * bs)[:n]
        slots[rng.random(n) < 0.03] = -1        # padding rows of a captured batch
        s["slots"] = _dev(slots.astype(np.int64))
        most = 8192
        s["positions"] = _dev(rng.integers(0, most, n).astype(np.int32))
        rot = case["rot"]
        angle = np.arange(most)[:, None] * 500000.0 ** (-np.arange(0, rot, 2) / rot)
        s["cos_sin"] = _dev(np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32))
        s["qw"] = (1.0 + 0.2 * _rand(gen, d)).to(dt) if case["norm"] else None
        s["kw"] = (1.0 + 0.2 * _rand(gen, d)).to(dt) if case["norm"] else None
        s["eps"] = 1e-6
        cache = torch.uint8 if case["kind"] == "e4m3" else dt
        s["kc"] = torch.zeros(pool, bs, hkv, d, dtype=cache, device=DEV)
        s["vc"] = torch.zeros(pool, bs, hkv, d, dtype=cache, device=DEV)
        s["ks"] = _dev(((1.0 + 0.37 * np.arange(hkv)) / 32.0).astype(np.float32)) if case["kind"] == "e4m3" else None
        s["vs"] = _dev(((1.3 + 0.29 * np.arange(hkv)) / 32.0).astype(np.float32)) if case["kind"] == "e4m3" else None
        s["out"] = torch.empty(n, hq, d, dtype=dt, device=DEV)
        return s
    if case["op"] == "tree":
        hq, hkv, d, bs = (case[k] for k in ("hq", "hkv", "d", "bs"))
        ctx, counts = _lengths(case)
        lens = ctx + counts
        tables, pool = _tables(lens, bs, rng)
        total = int(counts.sum())
        s["q"] = _rand(gen, total, hq, d, dtype=torch.bfloat16)
        s["kc"] = _rand(gen, pool, bs, hkv, d, dtype=torch.bfloat16)
        s["vc"] = _rand(gen, pool, bs, hkv, d, dtype=torch.bfloat16)
        s["tables"], s["lens"] = _dev(tables), _dev(lens.astype(np.int32))
        s["start"] = _dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        s["parents"] = _dev(_parents(counts, True, rng).astype(np.int32)) if case["tree"] else None
        s["most"] = int(counts.max())
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty_like(s["q"])
        return s
    if case["op"] == "verify":
        vocab = case["vocab"]
        counts = _lengths(case)[1]
        total = int(counts.sum())
        start = np.concatenate([[0], np.cumsum(counts)])
        parents = _parents(counts, case["tree"], rng)
        # a draft that resembles the target: logits that share most of their variance
        logits = 3.0 * _rand(gen, total, vocab)
        s["target"] = torch.softmax(logits, dim=1)
        logits += 1.0 * _rand(gen, total, vocab)
        draft = torch.softmax(logits, dim=1)
        parent_row = _dev(np.where(parents < 0, 0, parents) + np.repeat(start[:-1], counts))
        pick = torch.multinomial(draft[parent_row], 1, generator=gen) if case["sampled"] else \
            draft[parent_row].topk(min(4, vocab), dim=1).indices.gather(1, _dev(rng.integers(0, min(4, vocab), (total, 1))))
        s["draft"] = draft if case["sampled"] else None     # None: drafts picked, not sampled
        s["tokens"] = pick[:, 0].to(torch.int32)
        s["parents"] = _dev(parents.astype(np.int32)) if case["tree"] else None
        s["start"] = _dev(start.astype(np.int32))
        s["ua"] = torch.rand(total, generator=gen, device=DEV)
        s["us"] = torch.rand(case["seqs"], generator=gen, device=DEV)
        s["most"] = int(counts.max())
        for name in ("out", "path"):
            s[name] = torch.empty(case["seqs"], s["most"], dtype=torch.int32, device=DEV)
        s["len"] = torch.empty(case["seqs"], dtype=torch.int32, device=DEV)
        return s
    # accept: the step's rows at the end of each context, and the path that verification kept
    hkv, d, bs = (case[k] for k in ("hkv", "d", "bs"))
    dt = TYPES[case["kind"]]
    n, seqs = case["nodes"], case["seqs"]
    ctx, counts = _lengths(case)
    lens = ctx + counts
    tables, pool = _tables(lens, bs, rng)
    path, plen = np.full((seqs, n), -1, dtype=np.int32), np.zeros(seqs, dtype=np.int32)
    for i in range(seqs):
        keep = np.sort(rng.permutation(n - 1)[:rng.integers(0, min(n, 9))]) + 1 if n > 1 else np.zeros(0, dtype=np.int64)
        path[i, :1 + len(keep)] = np.concatenate([[0], keep])
        plen[i] = 1 + len(keep)
    s["k"], s["v"] = _rand(gen, seqs * n, hkv, d, dtype=dt), _rand(gen, seqs * n, hkv, d, dtype=dt)
    cache = torch.uint8 if case["kind"] == "e4m3" else dt
    s["kc"] = torch.zeros(pool, bs, hkv, d, dtype=cache, device=DEV)
    s["vc"] = torch.zeros(pool, bs, hkv, d, dtype=cache, device=DEV)
    s["ks"] = _dev(((1.0 + 0.37 * np.arange(hkv)) / 32.0).astype(np.float32)) if case["kind"] == "e4m3" else None
    s["vs"] = _dev(((1.3 + 0.29 * np.arange(hkv)) / 32.0).astype(np.float32)) if case["kind"] == "e4m3" else None
    s["slots"] = _dev(_slots(tables, bs, ctx, counts))
    s["tables"], s["lens"] = _dev(tables), _dev(lens.astype(np.int32))
    s["start"] = _dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    s["path"], s["plen"] = _dev(path), _dev(plen)
    return s


# ------------------------------------------------------------ the plain forms

def _norm(x, w, eps):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    rot, rest = x[..., :r], x[..., r:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = rot[..., :r // 2], rot[..., r // 2:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([rot, rest], dim=-1)


def _store(cache, slots, rows, scale):
    """Rows (float32) into the cache at their slots; a negative slot is skipped."""
    keep = slots >= 0
    if scale is not None:
        codes = (rows / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        codes = rows.to(cache.dtype)
    cache.view(-1, *cache.shape[2:])[slots[keep]] = codes[keep]


def _rows(s):
    half = s["cos_sin"].shape[1] // 2
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    s["out"].copy_(_rotate(_norm(s["q"], s["qw"], s["eps"]), cos, sin, s["interleaved"]))
    _store(s["kc"], s["slots"], _rotate(_norm(s["k"], s["kw"], s["eps"]), cos, sin, s["interleaved"]), s["ks"])
    _store(s["vc"], s["slots"], s["v"].float(), s["vs"])


def _values(cache):
    return cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache


def _ancestors(parents, counts, nodes):
    """[S, nodes, nodes] truth values: row i follows row j (or is it); rows past a sequence's own follow nothing else."""
    seqs = counts.shape[0]
    i = torch.arange(nodes, device=DEV)
    link = (parents[:, :, None] == i) & (i < counts[:, None])[:, :, None]
    reach = (link | torch.eye(nodes, dtype=torch.bool, device=DEV)).float()
    steps = 1
    while steps < nodes:        # paths of up to 2, 4, 8 ... links
        reach = (reach @ reach).clamp(max=1.0)
        steps *= 2
    return reach.view(seqs, nodes, nodes) > 0


def _padded(x, start, counts, nodes, fill):
    """Ragged rows [total, ...] as [S, nodes, ...]."""
    i = torch.arange(nodes, device=DEV)
    at = (start[:-1, None] + i).clamp(max=x.shape[0] - 1)
    live = i < counts[:, None]
    return torch.where(live.view(*live.shape, *(1,) * (x.dim() - 1)), x[at.long()], torch.full((), fill, dtype=x.dtype, device=DEV)), live


def _tree(s):
    kc, lens, start, nodes = s["kc"], s["lens"].long(), s["start"].long(), s["most"]
    bs, hkv, d = kc.shape[1:]
    group = s["hq"] // hkv
    counts = start[1:] - start[:-1]
    most = s["tables"].shape[1] * bs
    t = torch.arange(most, device=DEV)
    slot = s["tables"].long()[:, t // bs] * bs + t % bs                       # [S, T]
    keys = kc.view(-1, hkv, d)[slot].float().permute(0, 2, 3, 1)              # [S, Hkv, d, T]
    values = s["vc"].view(-1, hkv, d)[slot].float().permute(0, 2, 1, 3)
    q, live = _padded(s["q"], start, counts, nodes, 0.0)
    q = q.float().view(-1, nodes, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(-1, hkv, nodes * group, d)
    parents = _padded(s["parents"].long(), start, counts, nodes, -1)[0] if s["parents"] is not None else \
        (torch.arange(nodes, device=DEV) - 1).expand(len(counts), nodes)
    rel = t - (lens - counts)[:, None]                                        # the row that a key belongs to, below 0: before the step
    inside = _ancestors(parents, counts, nodes).gather(2, rel.clamp(0, nodes - 1)[:, None].expand(-1, nodes, -1))
    seen = ((rel < 0)[:, None] | (inside & (rel >= 0)[:, None])) & (t < lens[:, None])[:, None]
    seen = seen[:, :, None].expand(-1, -1, group, -1).reshape(len(counts), 1, nodes * group, most)
    x = torch.matmul(q, keys) * s["scale"]
    x = torch.where(seen, x, torch.full((), -math.inf, device=DEV))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, values) / p.sum(-1, keepdim=True)
    o = o.view(-1, hkv, nodes, group, d).permute(0, 2, 1, 3, 4).reshape(-1, nodes, hkv * group, d)
    s["out"].copy_(o[live])


def _verify(s):
    """The rows in order: a row is tried where it follows the last accepted one. Residuals and sums in 64 bits."""
    start, nodes, vocab = s["start"].long(), s["most"], s["target"].shape[1]
    counts = start[1:] - start[:-1]
    seqs = len(counts)
    each = torch.arange(seqs, device=DEV)
    parents = _padded(s["parents"].long(), start, counts, nodes, -2)[0] if s["parents"] is not None else \
        torch.arange(-1, nodes - 1, device=DEV).expand(seqs, nodes)
    cur = torch.zeros(seqs, dtype=torch.long, device=DEV)
    left = s["target"][start[:-1]].double()         # what is left of the target's distribution
    total = torch.ones(seqs, dtype=torch.float64, device=DEV)
    s["out"].fill_(-1)
    s["path"].fill_(-1)
    s["path"][:, 0] = 0
    length = torch.ones(seqs, dtype=torch.long, device=DEV)
    for i in range(1, nodes):
        row = (start[:-1] + i).clamp(max=s["tokens"].shape[0] - 1)
        tried = (parents[:, i] == cur) & (i < counts)
        token = s["tokens"][row].long()
        here = start[:-1] + cur
        q = s["draft"][here].double() if s["draft"] is not None else torch.zeros(seqs, vocab, dtype=torch.float64, device=DEV).scatter_(1, token[:, None], 1.0)
        taken = tried & (s["ua"][row].double() * q[each, token] * total < left[each, token])
        no = tried & ~taken
        if s["draft"] is not None:
            rest = torch.where(total[:, None] > 0, (left / total[:, None] - q).clamp(min=0.0), 0.0)
            mass = rest.sum(1)
        else:
            rest = left.scatter(1, token[:, None], 0.0)
            mass = (total - left[each, token]).clamp(min=0.0)
        left = torch.where(no[:, None], rest, left)
        total = torch.where(no, mass, total)
        s["out"][each[taken], length[taken] - 1] = token[taken].int()
        s["path"][each[taken], length[taken]] = i
        length = length + taken
        cur = torch.where(taken, torch.full_like(cur, i), cur)
        left = torch.where(taken[:, None], s["target"][row].double(), left)
        total = torch.where(taken, torch.ones_like(total), total)
    # where nothing is left: the target's own row
    sums = torch.where(left.sum(1, keepdim=True) > 0, left, s["target"][start[:-1] + cur].double()).cumsum(1)
    last = torch.searchsorted(sums, (s["us"].double() * sums[:, -1])[:, None], right=True)[:, 0].clamp(max=vocab - 1)
    s["out"][each, length - 1] = last.int()
    s["len"].copy_(length)


def _accept(s):
    _store(s["kc"], s["slots"], s["k"].float(), s["ks"])
    _store(s["vc"], s["slots"], s["v"].float(), s["vs"])
    bs = s["kc"].shape[1]
    first = s["lens"].long() - (s["start"][1:] - s["start"][:-1]).long()
    j = torch.arange(s["path"].shape[1], device=DEV)
    live = j < s["plen"][:, None]
    slot = lambda pos: s["tables"].long().gather(1, pos // bs) * bs + pos % bs     # noqa: E731
    source = slot(first[:, None] + s["path"].long().clamp(min=0))[live]
    target = slot(first[:, None] + j.expand(len(first), -1))[live]
    for cache in (s["kc"], s["vc"]):
        flat = cache.view(-1, *cache.shape[2:])
        flat[target] = flat[source]


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_345_b200 as pa
        if op == "rows":
            pa.pa_qk_norm_rope_append(s["out"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["kc"], s["vc"], s["cos_sin"],
                                      q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], interleaved=s["interleaved"],
                                      k_scale=s["ks"], v_scale=s["vs"])
        elif op == "tree":
            if "ws" not in s:       # a program keeps its workspace
                s["ws"] = torch.empty(pa.pa_decode_tree_workspace_bytes(s["hq"], s["hkv"], s["d"], s["most"]), dtype=torch.uint8, device=DEV)
            pa.pa_decode_tree(s["out"], s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["start"], s["parents"], s["most"], s["scale"],
                              s["ws"])
        elif op == "verify":
            pa.pa_verify_draft(s["out"], s["path"], s["len"], s["target"], s["draft"], s["tokens"], s["parents"], s["start"], s["ua"],
                               s["us"])
        else:
            if s["ks"] is None:
                pa.pa_kv_append(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
            else:
                pa.pa_kv_append_fp8(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
            pa.pa_kv_accept(s["kc"], s["vc"], s["tables"], s["lens"], s["start"], s["path"], s["plen"])
    else:
        {"rows": _rows, "tree": _tree, "verify": _verify, "accept": _accept}[op](s)
    if op == "rows":
        return {"q": s["out"], "k": _values(s["kc"]), "v": _values(s["vc"])}
    if op == "tree":
        return s["out"]
    if op == "verify":
        return {"tokens": s["out"], "path": s["path"], "len": s["len"]}
    return {"k": _values(s["kc"]), "v": _values(s["vc"])}


# ------------------------------------------------------------ what a pass needs

def work(case):
    if case["op"] == "rows":
        n, hq, hkv, d = (case[k] for k in ("tokens", "hq", "hkv", "d"))
        e = 4 if case["kind"] == "f32" else 2
        c = 1 if case["kind"] == "e4m3" else e
        # q read and written, k and v read and written, a table row, a position and a slot each
        return {"bytes": n * (2 * hq * d * e + 2 * hkv * d * (e + c) + case["rot"] * 4 + 12), "flops": n * (hq + hkv) * d * 7}
    if case["op"] == "tree":
        ctx, counts = _lengths(case)
        hq, hkv, d = (case[k] for k in ("hq", "hkv", "d"))
        keys, total = int((ctx + counts).sum()), int(counts.sum())
        # every cached row once, the queries and the outputs
        return {"bytes": keys * hkv * d * 4 + total * hq * d * 4, "flops": 4 * hq * d * int(((ctx + counts) * counts).sum())}
    if case["op"] == "verify":
        # the row that the last token is sampled from, of the target and (where drafts were sampled) of the draft
        rows = 2 if case["sampled"] else 1
        return {"bytes": case["seqs"] * (case["vocab"] * 4 * rows + 4 + 8) + case["seqs"] * case["nodes"] * 16, "flops": case["seqs"] * case["vocab"] * 4}
    e = 4 if case["kind"] == "f32" else 2
    c = 1 if case["kind"] == "e4m3" else e
    row = 2 * case["hkv"] * case["d"]
    moved = 1 + (min(case["nodes"], 9) - 1) / 2         # rows of a path, on average
    return {"bytes": case["seqs"] * row * (case["nodes"] * (e + c) + 2 * moved * c), "flops": 0}


# ------------------------------------------------------ the definitions, in 64 bits

def _exact_rows(s):
    n, half = s["tokens"], s["rot"] // 2
    place = s["positions"].long()
    cos, sin = s["cos_sin"][place, :half].double(), s["cos_sin"][place, half:].double()

    def turned(x, w):
        y = x.double().clone()
        if w is not None:
            y /= torch.sqrt((y * y).sum(-1, keepdim=True) / s["d"] + s["eps"])
            y *= w.double()
        z = y.clone()
        for i in range(half):       # pair i: the angle's complex rotation
            a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
            z[:, :, a] = y[:, :, a] * cos[:, i, None] - y[:, :, b] * sin[:, i, None]
            z[:, :, b] = y[:, :, a] * sin[:, i, None] + y[:, :, b] * cos[:, i, None]
        return z

    def cache(rows, scale, like):
        out = torch.zeros(like.shape[0] * like.shape[1], s["hkv"], s["d"], dtype=torch.float64, device=DEV)
        if scale is not None:
            rows = (rows / scale.double()[None, :, None]).clamp(-448, 448)
        for_ = (s["slots"] >= 0).nonzero()[:, 0]
        out[s["slots"][for_]] = rows[for_]
        return out.view(like.shape)

    assert n == len(place)
    return {"q": turned(s["q"], s["qw"]), "k": cache(turned(s["k"], s["kw"]), s["ks"], s["kc"]), "v": cache(s["v"].double(), s["vs"], s["vc"])}


def _exact_tree(s):
    bs, hkv, d = s["kc"].shape[1:]
    group = s["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    tables, lens, start = s["tables"].cpu().numpy(), s["lens"].tolist(), s["start"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else None
    for i, length in enumerate(lens):
        a, b = start[i], start[i + 1]
        n = b - a
        blocks = torch.from_numpy(tables[i, :-(-length // bs)].astype(np.int64)).to(DEV)
        keys = s["kc"][blocks].reshape(-1, hkv, d)[:length].double()
        values = s["vc"][blocks].reshape(-1, hkv, d)[:length].double()
        seen = np.zeros((n, length), dtype=bool)
        seen[:, :length - n] = True
        for r in range(n):
            at = r
            while at >= 0:
                seen[r, length - n + at] = True
                at = parents[a + at] if parents is not None else at - 1
        hidden = torch.from_numpy(~seen).to(DEV)
        for h in range(hkv):
            q = s["q"][a:b, h * group:(h + 1) * group].double()
            x = torch.einsum("rgd,td->grt", q, keys[:, h]) * s["scale"]
            x[hidden.expand(group, -1, -1)] = -math.inf
            w = torch.softmax(x, dim=-1)
            out[a:b, h * group:(h + 1) * group] = torch.einsum("grt,td->rgd", w, values[:, h])
    return out


def _exact_verify(s):
    """Each sequence's walk from its definition: the children of the last accepted row, in order."""
    start, tokens, ua, us = s["start"].tolist(), s["tokens"].tolist(), s["ua"].tolist(), s["us"].tolist()
    parents = s["parents"].tolist() if s["parents"] is not None else None
    out = torch.full(s["out"].shape, -1, dtype=torch.int32)
    path = torch.full(s["path"].shape, -1, dtype=torch.int32)
    length = torch.zeros(len(us), dtype=torch.int32)
    for i in range(len(us)):
        a, n = start[i], start[i + 1] - start[i]
        kids = {}
        for r in range(1, n):
            kids.setdefault(parents[a + r] if parents is not None else r - 1, []).append(r)
        said, kept, at, more = [], [0], 0, True
        while more:
            more = False
            p, mass = s["target"][a + at].double(), 1.0
            q = s["draft"][a + at].double() if s["draft"] is not None else None
            for r in kids.get(at, ()):
                x = tokens[a + r]
                if ua[a + r] * (float(q[x]) if q is not None else 1.0) * mass < float(p[x]):
                    said.append(x)
                    kept.append(r)
                    at, more = r, True
                    break
                if q is not None:
                    p = torch.clamp(p / mass - q, min=0) if mass > 0 else torch.zeros_like(p)
                    mass = float(p.sum())
                else:
                    mass = max(0.0, mass - float(p[x]))
                    p = p.clone()
                    p[x] = 0
        if float(p.sum()) == 0:     # nothing left
            p = s["target"][a + at].double()
        c = torch.cumsum(p, 0)
        said.append(min(int((c <= us[i] * float(c[-1])).sum()), len(c) - 1))
        out[i, :len(said)] = torch.tensor(said, dtype=torch.int32)
        path[i, :len(kept)] = torch.tensor(kept, dtype=torch.int32)
        length[i] = len(said)
    return {"tokens": out, "path": path, "len": length}


def _exact_accept(s):
    bs, n = s["kc"].shape[1], s["nodes"]
    tables, lens, path, plen = s["tables"].tolist(), s["lens"].tolist(), s["path"].tolist(), s["plen"].tolist()
    spot = lambda i, pos: tables[i][pos // bs] * bs + pos % bs      # noqa: E731
    # each slot's row of the step: its own, or the accepted one that moved there
    at, row = [], []
    for i, length in enumerate(lens):
        base = length - n
        for j in range(n):
            at.append(spot(i, base + j))
            row.append(i * n + (path[i][j] if j < plen[i] else j))
    got = {}
    for name, rows, scale in (("k", s["k"], s["ks"]), ("v", s["v"], s["vs"])):
        x = rows.double()
        if scale is not None:
            x = (x / scale.double()[None, :, None]).clamp(-448, 448)
        like = s[name + "c"]
        out = torch.zeros(like.shape[0] * bs, *like.shape[2:], dtype=torch.float64, device=DEV)
        out[torch.tensor(at, device=DEV)] = x[torch.tensor(row, device=DEV)]
        got[name] = out.view(like.shape)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"rows": _exact_rows, "tree": _exact_tree, "verify": _exact_verify, "accept": _exact_accept}[case["op"]](s)
