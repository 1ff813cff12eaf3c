"""The calls for drafted tokens on the CPU: what the host refuses, workspace sizes, and
the block manager's truncation against the oracle's blocks. No kernel launch."""

import ctypes

import numpy as np
import pytest

import paged_kv_cache_345_b200 as pa
from oracle import blocks as oblk

FAKE = ctypes.c_void_p(0x10000)   # never dereferenced: every call fails before a CUDA call
ODD = ctypes.c_void_p(0x10004)


def _rows(**over):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, so=4096, sq=6144, sk=6144, sv=6144, pos=FAKE,
             slots=FAKE, n=4, cs=FAKE, maxpos=8192, rot=128, il=0, qw=FAKE, kw=FAKE, eps=1e-6,
             kc=FAKE, vc=FAKE, ks=None, vs=None, nb=64, bs=16, Hq=32, Hkv=8, D=128, dt=pa.PA_BF16)
    a.update(over)
    st = pa._lib.pa_qk_norm_rope_append(
        a["out"], a["q"], a["k"], a["v"], a["so"], a["sq"], a["sk"], a["sv"], a["pos"], a["slots"],
        a["n"], a["cs"], a["maxpos"], a["rot"], a["il"], a["qw"], a["kw"], a["eps"], a["kc"],
        a["vc"], a["ks"], a["vs"], a["nb"], a["bs"], a["Hq"], a["Hkv"], a["D"], a["dt"], None)
    return st, pa._lib.pa_last_error().decode()


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), pa.PA_ERR_INVALID),
    (dict(q=None), pa.PA_ERR_INVALID),
    (dict(cs=None), pa.PA_ERR_INVALID),
    (dict(D=96), pa.PA_ERR_UNSUPPORTED),
    (dict(dt=9), pa.PA_ERR_UNSUPPORTED),
    (dict(rot=0), pa.PA_ERR_INVALID),
    (dict(rot=24), pa.PA_ERR_INVALID),                    # half of it is not whole 16-byte pieces
    (dict(rot=144), pa.PA_ERR_INVALID),
    (dict(maxpos=0), pa.PA_ERR_INVALID),
    (dict(eps=float("nan")), pa.PA_ERR_INVALID),
    (dict(eps=-1e-6), pa.PA_ERR_INVALID),
    (dict(sq=4088), pa.PA_ERR_INVALID),                   # shorter than a row of q
    (dict(sk=1020), pa.PA_ERR_INVALID),
    (dict(sv=6148), pa.PA_ERR_INVALID),                   # not a multiple of 16 bytes
    (dict(k=ODD), pa.PA_ERR_INVALID),
    (dict(cs=ODD), pa.PA_ERR_INVALID),
    (dict(kw=ODD), pa.PA_ERR_INVALID),
    (dict(ks=FAKE, vs=FAKE), pa.PA_ERR_INVALID),          # scales without an E4M3 cache
    (dict(dt=pa.PA_FP8_E4M3), pa.PA_ERR_INVALID),         # an E4M3 cache without scales
    (dict(dt=pa.PA_FP8_E4M3, ks=FAKE), pa.PA_ERR_INVALID),
    (dict(nb=0), pa.PA_ERR_INVALID),
    (dict(Hkv=0), pa.PA_ERR_INVALID),
])
def test_rows_rejects_on_host(over, status):
    st, msg = _rows(**over)
    assert st == status, msg
    assert msg


def test_rows_of_no_tokens_is_a_no_op():
    assert _rows(n=0)[0] == pa.PA_OK


def _tree(**over):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, qs=FAKE, par=FAKE, S=2, tq=32, Hq=32,
             Hkv=8, D=128, bs=16, nb=64, mbps=8, most=16, scale=0.1, ws=FAKE, wsb=1 << 30,
             dt=pa.PA_BF16)
    a.update(over)
    st = pa._lib.pa_decode_tree(a["out"], a["q"], a["k"], a["v"], a["bt"], a["cl"], a["qs"], a["par"],
                                a["S"], a["tq"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["nb"],
                                a["mbps"], a["most"], a["scale"], a["ws"], a["wsb"], a["dt"], None)
    return st, pa._lib.pa_last_error().decode()


@pytest.mark.parametrize("over,status", [
    (dict(S=-1), pa.PA_ERR_INVALID),
    (dict(tq=-1), pa.PA_ERR_INVALID),
    (dict(out=None), pa.PA_ERR_INVALID),
    (dict(qs=None), pa.PA_ERR_INVALID),
    (dict(dt=pa.PA_F32), pa.PA_ERR_UNSUPPORTED),
    (dict(dt=pa.PA_FP8_E4M3), pa.PA_ERR_UNSUPPORTED),
    (dict(D=96), pa.PA_ERR_UNSUPPORTED),
    (dict(Hq=30), pa.PA_ERR_INVALID),
    (dict(Hq=24), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=4), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=24), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=512), pa.PA_ERR_UNSUPPORTED),
    (dict(most=33), pa.PA_ERR_INVALID),                   # more than total_q
    (dict(scale=0.0), pa.PA_ERR_INVALID),
    (dict(scale=float("inf")), pa.PA_ERR_INVALID),
    (dict(q=ctypes.c_void_p(0x10008)), pa.PA_ERR_INVALID),
    (dict(par=ctypes.c_void_p(0x10002)), pa.PA_ERR_INVALID),
    (dict(ws=None), pa.PA_ERR_INVALID),
    (dict(wsb=1000), pa.PA_ERR_INVALID),
    (dict(nb=0), pa.PA_ERR_INVALID),
])
def test_tree_rejects_on_host(over, status):
    st, msg = _tree(**over)
    assert st == status, msg
    assert msg


def test_tree_without_work_is_a_no_op():
    assert _tree(S=0)[0] == pa.PA_OK
    assert _tree(tq=0)[0] == pa.PA_OK


def test_tree_workspace_grows_with_the_rows_and_is_bounded():
    sizes = [pa.pa_decode_tree_workspace_bytes(32, 8, 128, n) for n in (1, 8, 16, 32, 64, 1000)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] > 0
    assert sizes[-1] == sizes[-2] < 64 << 20
    assert pa.pa_decode_tree_workspace_bytes(32, 8, 128, 0) == 0
    assert pa.pa_decode_tree_workspace_bytes(30, 8, 128, 4) == 0


def _verify(**over):
    a = dict(ot=FAKE, op=FAKE, ol=FAKE, tp=FAKE, ts=1000, dp=FAKE, ds=1000, tok=FAKE, par=FAKE, qs=FAKE,
             ua=FAKE, us=FAKE, S=2, tq=8, V=1000, most=4)
    a.update(over)
    st = pa._lib.pa_verify_draft(a["ot"], a["op"], a["ol"], a["tp"], a["ts"], a["dp"], a["ds"], a["tok"],
                                 a["par"], a["qs"], a["ua"], a["us"], a["S"], a["tq"], a["V"],
                                 a["most"], None)
    return st, pa._lib.pa_last_error().decode()


@pytest.mark.parametrize("over,status", [
    (dict(S=-1), pa.PA_ERR_INVALID),
    (dict(most=0), pa.PA_ERR_INVALID),
    (dict(tq=0), pa.PA_ERR_INVALID),
    (dict(V=0), pa.PA_ERR_INVALID),
    (dict(ts=999), pa.PA_ERR_INVALID),
    (dict(ds=999), pa.PA_ERR_INVALID),
    (dict(most=1025), pa.PA_ERR_UNSUPPORTED),
    (dict(tp=None), pa.PA_ERR_INVALID),
    (dict(us=None), pa.PA_ERR_INVALID),
    (dict(tok=ctypes.c_void_p(0x10002)), pa.PA_ERR_INVALID),
])
def test_verify_rejects_on_host(over, status):
    st, msg = _verify(**over)
    assert st == status, msg
    assert msg


def test_verify_of_no_sequences_is_a_no_op():
    assert _verify(S=0)[0] == pa.PA_OK


def _accept(**over):
    a = dict(k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, qs=FAKE, p=FAKE, pl=FAKE, S=2, most=4, nb=64, bs=16, mbps=8,
             Hkv=8, D=128, dt=pa.PA_BF16)
    a.update(over)
    st = pa._lib.pa_kv_accept(a["k"], a["v"], a["bt"], a["cl"], a["qs"], a["p"], a["pl"], a["S"], a["most"],
                              a["nb"], a["bs"], a["mbps"], a["Hkv"], a["D"], a["dt"], None)
    return st, pa._lib.pa_last_error().decode()


@pytest.mark.parametrize("over,status", [
    (dict(S=-1), pa.PA_ERR_INVALID),
    (dict(most=-1), pa.PA_ERR_INVALID),
    (dict(bs=24), pa.PA_ERR_INVALID),
    (dict(dt=5), pa.PA_ERR_UNSUPPORTED),
    (dict(Hkv=1, D=4), pa.PA_ERR_UNSUPPORTED),            # rows of 8 bytes
    (dict(p=None), pa.PA_ERR_INVALID),
    (dict(v=ODD), pa.PA_ERR_INVALID),
    (dict(mbps=0), pa.PA_ERR_INVALID),
])
def test_accept_rejects_on_host(over, status):
    st, msg = _accept(**over)
    assert st == status, msg
    assert msg


def test_accept_without_work_is_a_no_op():
    assert _accept(S=0)[0] == pa.PA_OK
    assert _accept(most=0)[0] == pa.PA_OK


# ------------------------------------------------------------- truncation

def _truncate(m: oblk.BlockManager, seq: int, new_len: int) -> None:
    """The oracle's blocks, rolled back: whole blocks past the last token leave, last first."""
    keep = oblk.blocks_for(new_len, m.block_size)
    while len(m.tables[seq]) > keep:
        m.decref(m.tables[seq].pop())
    m.lengths[seq] = new_len


@pytest.mark.parametrize("seed", range(6))
def test_truncate_matches_the_oracle(seed):
    rng = np.random.default_rng(seed)
    bs, nb = int(rng.choice([1, 4, 16])), 60
    bm, om = pa.BlockManager(nb, bs), oblk.BlockManager(nb, bs)
    seqs = [(bm.add_seq(), om.new_sequence()) for _ in range(3)]
    for _ in range(120):
        i = int(rng.integers(len(seqs)))
        a, o = seqs[i]
        op = rng.random()
        if op < 0.5:
            n = int(rng.integers(1, 9))
            if om.blocks_needed(o, n) <= om.num_free():
                slots, cows = bm.append_slots([a], [n])
                oslots, ocows = om.add_tokens(o, n)
                assert slots.tolist() == oslots and [tuple(c) for c in cows.tolist()] == ocows
        elif op < 0.85:
            n = int(rng.integers(0, om.lengths[o] + 1))
            bm.truncate(a, n)
            _truncate(om, o, n)
        elif len(seqs) < 6:
            seqs.append((bm.fork(a), om.fork(o)))
        assert bm.seq_len(a) == om.lengths[o] and bm.allocator.num_free() == om.num_free()
        assert [bm.allocator.refcount(b) for b in range(nb)] == om.refcount
        if om.tables[o]:
            tables, _ = bm.block_tables([a], len(om.tables[o]))
            assert tables[0].tolist() == om.tables[o]


@pytest.mark.parametrize("new_len", [-1, 6])
def test_truncate_refuses_and_changes_nothing(new_len):
    bm = pa.BlockManager(8, 4)
    s = bm.add_seq()
    bm.append_slots([s], [5])
    with pytest.raises(pa.PagedAttentionError):
        bm.truncate(s, new_len)
    with pytest.raises(pa.PagedAttentionError):
        bm.truncate(s + 1, 0)
    assert bm.seq_len(s) == 5 and bm.seq_num_blocks(s) == 2


@pytest.mark.parametrize("call,args", [
    (pa.pa_kv_accept, 7), (pa.pa_verify_draft, 10), (pa.pa_decode_tree, 11), (pa.pa_qk_norm_rope_append, 9),
])
def test_tensors_off_the_gpu_and_other_objects_are_refused(call, args):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        call(*[torch.zeros(2, 8, 1, 64)] * args)
    with pytest.raises(TypeError, match="must be a tensor"):
        call(*[3] * args)
