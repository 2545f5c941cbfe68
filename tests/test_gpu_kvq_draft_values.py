"""GPU tests of drafts over the 8-bit cache whose later tokens hold NaN, infinities or the type's largest values: a row's
output depends on the slots up to its own only."""
import math

import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import RING, check_attend, normal
from test_gpu_kvq_attend import filled, run
from test_gpu_kvq_cache import i32, make, same_bits

pytestmark = pytest.mark.gpu
BF, F, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def clean_status():
    ua.get_device_status()


# n slots, Tq drafts of G rows a KV head, the bad slot: the last draft's or one in the middle; drafts inside 16 slots, over
# the borders of 16 slots and of a block, in front of the first slot, in several row tiles, rows that see no slot of the 16
DRAFTS = [(5, 4, 1, 4), (68, 4, 4, 67), (68, 4, 4, 65), (81, 4, 2, 80), (97, 8, 3, 96), (130, 4, 4, 129), (2, 4, 2, 1),
          (191, 5, 8, 190), (120, 40, 1, 100), (127, 20, 2, 127 - 10)]


@pytest.mark.parametrize("n,Tq,G,slot", DRAFTS)
@pytest.mark.parametrize("dt,fmt,d", [(BF, E4, 64), (BF, I8, 128), (F, I8, 64), (F, E4, 128)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, "largest"])
def test_a_later_drafts_value_does_not_reach_earlier_rows(n, Tq, G, slot, dt, fmt, d, value):
    value = torch.finfo(dt).max if value == "largest" else value
    B, Hkv = 2, 2
    c = filled(B, Hkv, d, [n, n], fmt, dt, seed=61)
    q, g = normal((B, Tq, Hkv * G, d), 62, dt), normal((B, Tq, Hkv * G, d), 63, dt)
    want, wl = run(c, q, g=g)
    check_attend(c, q, [n, n], want, wl, g=g)
    own = n - Tq + torch.arange(Tq)                  # the rows' slots
    early, late = own < slot, own >= slot
    assert late.any()
    c.v_ring[0, 1, slot % RING, 5] = value           # sequence 0, KV head 1, one element
    o, lse = run(c, q, g=g)
    assert same_bits(lse, wl) and same_bits(o[1], want[1]) and same_bits(o[0, :, :G], want[0, :, :G])
    assert same_bits(o[0, early, G:], want[0, early, G:])
    rest = [i for i in range(d) if i != 5]
    assert same_bits(o[0, late, G:][..., rest], want[0, late, G:][..., rest])
    if not math.isfinite(value):
        assert not torch.isfinite(o[0, late, G:, 5]).any()
    # a key: the rows that see it may be anything, NaN where it is NaN
    c.v_ring[0, 1, slot % RING, 5] = 0.0
    want, wl = run(c, q, g=g)
    c.k_ring[0, 1, slot % RING, 7] = value
    o, lse = run(c, q, g=g)
    assert same_bits(o[1], want[1]) and same_bits(o[0, :, :G], want[0, :, :G]) and same_bits(lse[1], wl[1])
    assert same_bits(o[0, early, G:], want[0, early, G:]) and same_bits(lse[0, G:, early], wl[0, G:, early])
    if value != value:
        assert torch.isnan(o[0, late, G:]).all() and torch.isnan(lse[0, G:, late]).all()
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("dt", [BF, F])
def test_several_such_values_and_hidden_slots(dt):
    """All later drafts' values are bad, some of them hidden by the bias, fewer queries than drafts in one sequence."""
    n, Tq, H, d = [70, 100], 6, 6, 64
    c = filled(2, 2, d, n, E4, dt, seed=64)
    q = normal((2, Tq, H, d), 65, dt)
    bias = normal((2, 2, c.capacity), 66, F)
    bias[:, :, 66] = -math.inf
    kw = dict(bias=bias, n_q=i32([6, 3]))
    bad = {0: (66, 67, 68, 69), 1: (98, 99)}
    out = [torch.zeros_like(q), torch.zeros_like(q)]
    for i in range(2):
        ua.kvq_attend(c, q, out=out[i], **kw)
        for b, slots in bad.items():
            for j, s in enumerate(slots):
                c.v_ring[b, :, s % RING, j:] = (math.nan, math.inf, -math.inf, math.inf)[j]
    want, o = out
    # sequence 0: queries in slots 64 .. 69; 66 is hidden; sequence 1: queries in slots 97, 98, 99
    assert same_bits(o[0, :3], want[0, :3]) and same_bits(o[1, :1], want[1, :1])
    for row, first in ((o[0, 3], 1), (o[0, 4], 1), (o[0, 5], 1), (o[1, 1], 0), (o[1, 2], 0)):
        assert not torch.isfinite(row[:, first:]).any()
    assert same_bits(o[0, 3:, :, 0], want[0, 3:, :, 0])
    assert torch.isnan(o[0, 4][:, 2:]).all()         # +inf and -inf
    assert (o[1, 3:] == 0).all() and ua.get_device_status() == 0


@pytest.mark.parametrize("dt,fmt", [(BF, I8), (F, E4)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_rows_before_a_finished_block_that_is_not_finite(dt, fmt, which):
    """80 drafts, one of them bad and in a finished block: the rows in front of that block are as without it, all rows
    from the block's first slot on that see a slot of it are NaN."""
    T, Tq, d = 200, 80, 64
    k, v = normal((1, T, 1, d), 67, dt), normal((1, T, 1, d), 68, dt)
    q = normal((1, Tq, 2, d), 69, dt)
    outs = []
    for bad in (False, True):
        if bad:
            (k if which == "k" else v)[0, 190, 0, 3] = math.nan
        c = make(1, 1, d, 256, fmt, dt)
        ua.kvq_append(c, k, v, theta=0.0)
        outs.append(run(c, q))
    (want, wl), (o, lse) = outs
    assert same_bits(o[0, :8], want[0, :8]) and same_bits(lse[0, :, :8], wl[0, :, :8])       # slots 120 .. 127
    assert torch.isnan(o[0, 8:]).all()
    if which == "v":
        assert same_bits(lse, wl)
