"""E4M3 caches whose K holds its codes as uint8 and V as float8_e4m3fn, or the other way
round: the bytes are the same, and so is every call's result."""

import pytest
import torch

import paged_kv_cache_345_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
U8, F8 = torch.uint8, torch.float8_e4m3fn
NB, BS, HKV, D = 8, 4, 2, 64


def caches(kt, vt):
    gen = torch.Generator().manual_seed(3)
    both = torch.randint(0, 0x78, (2, NB, BS, HKV, D), generator=gen, dtype=U8).to(DEV)
    return both[0].view(kt), both[1].view(vt)


def as_bytes(kc, vc):
    return kc.view(U8).cpu(), vc.view(U8).cpu()


def rows(n, heads):
    gen = torch.Generator().manual_seed(n + heads)
    return torch.randn(n, heads, D, generator=gen).bfloat16().to(DEV)


SLOTS = torch.tensor([3, 17, 30, -1, 9], device=DEV) if torch.cuda.is_available() else None


def append(kc, vc):
    sc = torch.tensor([0.02, 0.05], device=DEV)
    pa.pa_kv_append_fp8(rows(5, HKV), rows(5, HKV), SLOTS, kc, vc, sc, 2 * sc)


def write_rows(kc, vc):
    sc = torch.tensor([0.02, 0.05], device=DEV)
    ang = torch.arange(8)[:, None] * torch.logspace(0, -3, 32)[None]
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
    q = rows(5, 4)
    pa.pa_qk_norm_rope_append(torch.empty_like(q), q, rows(5, HKV), rows(5, HKV),
                              torch.arange(5, dtype=torch.int32, device=DEV), SLOTS, kc, vc, cs,
                              k_scale=sc, v_scale=sc)


def accept(kc, vc):
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pa.pa_kv_accept(kc, vc, i32(5, 2, 7)[None], i32(10), i32(0, 6), i32(0, 2, 5)[None], i32(3))


@pytest.mark.parametrize("kt,vt", [(U8, F8), (F8, U8), (F8, F8)])
@pytest.mark.parametrize("call", [append, write_rows, accept])
def test_either_type_of_codes(call, kt, vt):
    want = caches(U8, U8)
    before = as_bytes(*want)
    call(*want)
    got = caches(kt, vt)
    call(*got)
    assert pa.pa_device_errors() == 0
    for w, g, b in zip(as_bytes(*want), as_bytes(*got), before):
        assert torch.equal(w, g) and not torch.equal(w, b)


def test_other_pairs_of_types_are_refused():
    kc, vc = caches(U8, U8)
    bf = torch.zeros(kc.shape, dtype=torch.bfloat16, device=DEV)
    sc = torch.ones(HKV, device=DEV)
    for k, v in ((kc, bf), (bf, vc), (bf, bf)):
        with pytest.raises(TypeError):
            pa.pa_kv_append_fp8(rows(5, HKV), rows(5, HKV), SLOTS, k, v, sc, sc)
    with pytest.raises(TypeError):
        pa.pa_kv_append(rows(5, HKV), rows(5, HKV), SLOTS, bf, vc)
    with pytest.raises(TypeError):
        pa.pa_kv_append(rows(5, HKV).float(), rows(5, HKV).float(), SLOTS, bf.float(), bf)
    with pytest.raises(TypeError):
        pa.pa_kv_append(kc.view(-1, HKV, D)[:5], kc.view(-1, HKV, D)[:5], SLOTS, kc, vc.view(F8))
