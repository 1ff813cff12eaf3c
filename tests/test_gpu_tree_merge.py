"""pa_decode_tree where a row's item is cut and one part holds nothing but NaN scores for it:
the row is NaN, as in an item that is not cut. (The maximum that a part reports ignores NaN;
the part's sum does not.)"""

import numpy as np
import pytest
import torch

import paged_kv_cache_345_b200 as pa
from test_gpu_tree import Batch, check

pytestmark = pytest.mark.gpu


def nan_keys(b, seq, positions):
    for t in positions:
        b.kc[b.tables[seq, t // b.bs], t % b.bs] = float("nan")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n,ctx", [
    (8, 8, 1, 4096),     # the last tile is the row's own key alone, a part of its own for some heads
    (32, 8, 1, 8192),
    (16, 2, 3, 4096),
    (8, 1, 40, 12800),   # 320 rows: two query tiles
])
def test_rows_whose_own_keys_are_nan_are_nan_wherever_the_cuts_lie(hq, hkv, n, ctx, d):
    b = Batch([ctx], [n], hq, hkv, d, 16, "star", seed=31)
    nan_keys(b, 0, range(ctx, ctx + n))
    out = b.run()
    assert pa.pa_device_errors() == 0
    assert torch.isnan(out).all()


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (32, 8, 64)])
def test_a_row_that_does_not_see_the_nan_key_is_right_beside_one_that_does(hq, hkv, d):
    """Row 0 and 64 rows that follow it: the last one's key opens a tile of its own."""
    n = 65
    b = Batch([4096], [n], hq, hkv, d, 16, "star", seed=32)
    clean = b.kc.clone()
    nan_keys(b, 0, [4096 + n - 1])
    out = b.run()
    assert torch.isnan(out[n - 1]).all()
    b.kc = clean         # (the oracle: no other row sees that key)
    got = out.clone()
    got[n - 1] = torch.from_numpy(b.expected()[0][n - 1]).to(out)
    check(b, got)


def test_a_part_of_unseen_keys_adds_nothing():
    """Rows of a star that see one key of the step's five tiles each: their other parts hold
    no key for them, and are left out."""
    n = 300
    b = Batch([600], [n], 4, 4, 128, 16, "star", seed=33)
    check(b, b.run())
    assert np.asarray(b.lens)[0] == 900
