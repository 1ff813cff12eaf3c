"""pa_qk_norm_rope_append against the formula in float64.

Tolerances, from the arithmetic: in float32 a normed value carries the errors of
the mean (at most 12 additions), the reciprocal root (2 ulp), and two products,
and a rotated one two products and a sum more: less than 16 half steps (2^-24
each) of |y_a| + |y_b| for its pair, 2^-20 (|y_a| + |y_b|). What is stored in fewer bits is
rounded once more: bf16 2^-8 of the value, E4M3 2^-4 of it or half its smallest
step (2^-10) in units of the scale; the division by the scale adds 2^-24.
"""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


class Rows:
    def __init__(self, n, hq, hkv, d, kind, rot, interleaved, norm, bs=16, seed=0, most=512, packed=True):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.kind, self.rot, self.interleaved, self.hkv, self.d = kind, rot, interleaved, hkv, d
        dt = F32 if kind == "f32" else BF16
        x = torch.randn(n, (hq + 2 * hkv) * d, generator=g) * torch.from_numpy(10.0 ** rng.uniform(-2, 1, (n, 1))).float()
        x = x.to(dt).to(DEV)
        if packed:
            self.q = x[:, :hq * d].view(n, hq, d)
            self.k = x[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
            self.v = x[:, (hq + hkv) * d:].view(n, hkv, d)
        else:
            self.q, self.k, self.v = (t.reshape(n, -1, d).contiguous() for t in
                                      (x[:, :hq * d], x[:, hq * d:(hq + hkv) * d], x[:, (hq + hkv) * d:]))
        nb = -(-n // bs) + 2
        slots = rng.permutation(nb * bs)[:n].astype(np.int64)
        if n > 4:
            slots[rng.permutation(n)[:n // 5]] = -1
        pos = rng.integers(0, most, n).astype(np.int32)
        pos[0] = most - 1
        if n > 4:
            pos[n // 2] = -1                    # a padding row
        self.slots, self.pos = torch.from_numpy(slots).to(DEV), torch.from_numpy(pos).to(DEV)
        ang = np.arange(most)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        self.cs = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(DEV)
        self.qw = (1 + 0.3 * torch.randn(d, generator=g)).to(dt).to(DEV) if norm in ("both", "q") else None
        self.kw = (1 + 0.3 * torch.randn(d, generator=g)).to(dt).to(DEV) if norm in ("both", "k") else None
        ct = torch.uint8 if kind == "e4m3" else dt
        self.kc = torch.zeros(nb, bs, hkv, d, dtype=ct, device=DEV)
        self.vc = torch.zeros_like(self.kc)
        sc = lambda a, b: (a + b * torch.arange(hkv)).float().div(32).to(DEV)  # noqa: E731
        self.ks, self.vs = (sc(1.0, 0.37), sc(1.3, 0.29)) if kind == "e4m3" else (None, None)
        self.out = torch.full((n, hq, d), 3.0, dtype=dt, device=DEV)
        self.eps = 1e-5

    def run(self, out=None, stream=None):
        out = self.out if out is None else out
        pa.pa_qk_norm_rope_append(out, self.q, self.k, self.v, self.pos, self.slots, self.kc, self.vc, self.cs,
                                  self.qw, self.kw, self.eps, self.interleaved, self.ks, self.vs, stream=stream)
        torch.cuda.synchronize()
        return out

    def formula(self, x, w):
        """(value, |y_a| + |y_b| of its pair) in float64."""
        y = x.double().cpu()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + self.eps) * w.double().cpu()
        half = self.rot // 2
        p = self.pos.cpu().long().clamp(min=0)
        c, s = self.cs.cpu().double()[p, :half][:, None], self.cs.cpu().double()[p, half:][:, None]
        z, mag = y.clone(), y.abs()
        ia = torch.arange(0, self.rot, 2) if self.interleaved else torch.arange(half)
        ib = ia + (1 if self.interleaved else half)
        a, b = y[..., ia], y[..., ib]
        z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
        return z, mag


def near(got, ref, mag, step, floor=0.0):
    tol = step * ref.abs() + 2.0 ** -20 * mag + floor
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), f"off by up to {(err / tol.clamp(min=1e-300)).max():.2f} of the tolerance"


def check(r):
    assert pa.pa_device_errors() == 0
    live = (r.pos >= 0).cpu()
    step = 2.0 ** -24 if r.kind == "f32" else 2.0 ** -8
    ref, mag = r.formula(r.q, r.qw)
    near(r.out[live.to(DEV)], ref[live], mag[live], step)
    assert (r.out[~live.to(DEV)] == 3.0).all()              # padding rows stay
    kref, kmag = r.formula(r.k, r.kw)
    keep = live & (r.slots.cpu() >= 0)
    at = r.slots.cpu()[keep]
    kc, vc = (c.view(-1, r.hkv, r.d).cpu() for c in (r.kc, r.vc))
    if r.kind == "e4m3":
        ks, vs = r.ks.cpu().double()[:, None], r.vs.cpu().double()[:, None]
        kv, vv = kc.view(torch.float8_e4m3fn).double(), vc.view(torch.float8_e4m3fn).double()
        near(kv[at], (kref[keep] / ks).clamp(-448, 448), kmag[keep] / ks, 2.0 ** -4 + 2.0 ** -20, 2.0 ** -10)
        near(vv[at], (r.v.cpu().double()[keep] / vs).clamp(-448, 448), torch.zeros(1).double(), 2.0 ** -4 + 2.0 ** -20,
             2.0 ** -10)
    else:
        near(kc[at], kref[keep], kmag[keep], step)
        assert torch.equal(vc[at], r.v.cpu()[keep])         # bit for bit
    rest = torch.ones(len(kc), dtype=torch.bool)
    rest[at] = False
    assert (kc[rest].float() == 0).all() and (vc[rest].float() == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n,hq,hkv,d,rot,interleaved,norm", [
    (1, 4, 2, 64, 64, False, "both"),
    (8, 32, 8, 128, 128, False, "both"),
    (9, 32, 8, 128, 64, True, "both"),
    (33, 1, 1, 128, 16, False, "both"),         # one q head: its row shares an instruction with k and v
    (7, 3, 1, 64, 32, True, "q"),
    (5, 7, 7, 64, 16, False, "k"),
    (40, 8, 2, 128, 96, False, None),
    (301, 16, 4, 128, 128, True, None),
    (700, 64, 8, 64, 48, False, "both"),
])
def test_rows_match_the_formula(n, hq, hkv, d, rot, interleaved, norm, kind):
    r = Rows(n, hq, hkv, d, kind, rot, interleaved, norm, seed=n + d, packed=n != 9)
    r.run()
    check(r)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    r = Rows(21, 8, 2, 128, "bf16", 128, interleaved, "both", seed=1, packed=False)
    want = r.run().clone()
    live = r.pos >= 0
    assert torch.equal(r.run(out=r.q)[live], want[live])


def test_rows_of_zeros_and_of_huge_values():
    r = Rows(6, 4, 2, 128, "bf16", 128, False, "both", seed=2, packed=False)
    r.q[0] = 0.0
    r.k[1] = 0.0
    r.q[2] = 1e15                               # squares up to 1e30: their mean is finite
    r.run()
    check(r)


def test_values_past_the_rotated_part_may_be_infinite():
    r = Rows(3, 4, 2, 128, "bf16", 64, False, None, seed=3, packed=False)
    r.q[0, 0, 100] = float("inf")
    r.run()
    assert torch.isinf(r.out[0, 0, 100]) and torch.isfinite(r.out[0, 0, :100]).all()


def test_e4m3_rows_saturate_and_round_once():
    r = Rows(4, 2, 1, 64, "e4m3", 64, False, None, seed=4, packed=False)
    r.v[0] = 1000.0
    r.k[1] = -1000.0
    r.run()
    vc = r.vc.view(-1, 1, 64).view(torch.float8_e4m3fn).float()
    if int(r.slots[0]) >= 0:
        assert (vc[r.slots[0]] == 448.0).all()
    check(r)


def test_equal_to_append_without_norm_and_at_position_zero():
    # angle 0 and no norm: the rows as they are, where pa_kv_append puts them
    r = Rows(50, 4, 2, 128, "bf16", 128, False, None, seed=5, packed=False)
    r.pos.zero_()
    r.run()
    kc, vc = torch.zeros_like(r.kc), torch.zeros_like(r.vc)
    pa.pa_kv_append(r.k, r.v, r.slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(r.out, r.q) and torch.equal(r.kc, kc) and torch.equal(r.vc, vc)


def test_bad_positions_and_slots_are_flagged_and_skipped():
    r = Rows(4, 4, 2, 128, "bf16", 128, False, "both", seed=6)
    r.pos[1] = 512
    r.run()
    assert pa.pa_device_errors() == pa.PA_DEVERR_POSITION
    assert (r.out[1] == 3.0).all() and not (r.out[0] == 3.0).all()
    r = Rows(4, 4, 2, 128, "bf16", 128, False, "both", seed=6)
    want = r.run().clone()
    r.kc.zero_()
    r.slots[2] = 10 ** 12
    r.run()
    assert pa.pa_device_errors() == pa.PA_DEVERR_SLOT
    assert torch.equal(r.out, want)             # the query is still made


def test_captured_and_on_another_stream():
    r = Rows(16, 8, 2, 128, "bf16", 128, False, "both", seed=7)
    want = r.run().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r.out.fill_(3.0)
    torch.cuda.synchronize()
    assert torch.equal(r.run(stream=side), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_qk_norm_rope_append(r.out, r.q, r.k, r.v, r.pos, r.slots, r.kc, r.vc, r.cs, r.qw, r.kw, r.eps)
    r.out.fill_(3.0)
    r.kc.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.out, want)
    check(r)


def test_no_tokens():
    r = Rows(1, 4, 2, 64, "bf16", 64, False, "both")
    e = lambda t: t[:0]  # noqa: E731
    pa.pa_qk_norm_rope_append(e(r.out), e(r.q), e(r.k), e(r.v), e(r.pos), e(r.slots), r.kc, r.vc, r.cs, r.qw, r.kw)
    assert pa.pa_device_errors() == 0


def test_binding_refuses():
    r = Rows(4, 4, 2, 64, "bf16", 64, False, "both", packed=False)
    a = dict(q_out=r.out, q=r.q, k=r.k, v=r.v, positions=r.pos, slot_mapping=r.slots, k_cache=r.kc, v_cache=r.vc,
             cos_sin=r.cs, q_weight=r.qw, k_weight=r.kw)
    wide = torch.zeros(4, 4, 128, dtype=BF16, device=DEV)
    for over, err in [(dict(q=r.q.float()), TypeError), (dict(positions=r.pos.long()), TypeError),
                      (dict(q=wide[:, :, ::2]), ValueError), (dict(k=wide[:, :2, :64]), ValueError),
                      (dict(k_scale=torch.ones(2, device=DEV), v_scale=torch.ones(2, device=DEV)), ValueError),
                      (dict(q_weight=r.qw[:32]), ValueError), (dict(v=r.v[:3]), ValueError),
                      (dict(cos_sin=r.cs[:, :24].contiguous()), pa.PagedAttentionError),
                      (dict(cos_sin=r.cs.double()), TypeError), (dict(q=r.q.cpu()), ValueError)]:
        with pytest.raises(err):
            pa.pa_qk_norm_rope_append(**{**a, **over})
