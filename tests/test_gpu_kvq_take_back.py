"""GPU tests of the 8-bit cache's append with tokens taken back: which starts it accepts, and that every start
it accepts leaves the cache that never saw the tokens taken back."""
import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import BLOCK, RING, normal
from test_gpu_kvq_cache import check, i32, make, same_bits

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
STATE = ("k", "v", "k_scale", "v_scale", "k_ring", "v_ring", "n_kept", "ring_state")


@pytest.fixture(autouse=True)
def clean_status():
    ua.get_device_status()                           # (reading clears it)


def rows(n, seed, B=1, Hkv=1, d=64):
    return normal((B, n, Hkv, d), seed, BF), normal((B, n, Hkv, d), seed + 1, BF)


def put(c, k, v, lo, hi, **kw):
    """Tokens lo .. hi - 1 of k and v, appended in one call."""
    ua.kvq_append(c, k[:, lo:hi].contiguous(), v[:, lo:hi].contiguous(), theta=0.0, **kw)


# a call keeps the rows of the block its end lies in and of the one before: at a border the former has none yet
@pytest.mark.parametrize("end,start", [(128, 10), (128, 63), (192, 69), (256, 129), (256, 186), (320, 191), (4096, 3970)])
@pytest.mark.parametrize("n_new", [0, 1, 80])
def test_a_start_whose_rows_one_call_did_not_keep_is_refused(end, start, n_new):
    c = make(1, 1, 64, end + 128, E4, BF)
    k, v = rows(end + 80, 1)
    put(c, k, v, 0, end)
    old = {x: getattr(c, x).clone() for x in STATE}
    put(c, k, v, end, end + 80, start=i32([start]), n_new=i32([n_new]))
    assert ua.get_device_status() == 1
    for x in STATE:
        assert same_bits(getattr(c, x), old[x]), x


def test_a_start_behind_rows_that_were_overwritten_is_refused():
    """190 slots, taken back to a border and filled again in one call up to a border: the first block of that call was
    never in the ring, which still holds the rejected rows."""
    c = make(1, 1, 64, 384, E4, BF)
    k, v = rows(400, 3)
    put(c, k, v, 0, 190)
    put(c, k, v, 200, 328, start=i32([64]))
    assert c.n_kept.tolist() == [192] and ua.get_device_status() == 0
    old = {x: getattr(c, x).clone() for x in STATE}
    put(c, k, v, 0, 1, start=i32([100]))
    assert ua.get_device_status() == 1
    for x in STATE:
        assert same_bits(getattr(c, x), old[x]), x


@pytest.mark.parametrize("end", [64, 128, 192, 256, 257, 319])
@pytest.mark.parametrize("back", [1, 63, 64])
def test_up_to_a_block_of_tokens_may_always_be_taken_back(end, back):
    c = make(1, 1, 64, 448, E4, BF)
    k, v = rows(400, 5)
    put(c, k, v, 0, end)
    put(c, k, v, 320, 400, start=i32([end - back]))
    assert ua.get_device_status() == 0
    K, V = (torch.cat([x[:, :end - back], x[:, 320:400]], 1) for x in (k, v))
    check(c, K, V, [end - back + 80], True)


@pytest.mark.parametrize("single", [False, True])
def test_every_start_after_every_end(single):
    """Sequence e holds e slots, 0 .. 400, from one call or from single tokens.  Whatever start is accepted has its
    block's earlier rows in the ring; a start on a border, and one up to 64 slots back, is accepted; a refused one
    leaves the count."""
    N, B = 400, 401
    c = make(B, 1, 64, 448, E4, BF)
    k, v = rows(N + 1, 7, B)
    end = torch.arange(B, device="cuda")
    if single:
        for t in range(N):
            put(c, k, v, t, t + 1, n_new=(end > t).int())
    else:
        put(c, k, v, 0, N, n_new=end.int())
    assert torch.equal(c.n_kept, end.int()) and ua.get_device_status() == 0
    old = {x: getattr(c, x).clone() for x in STATE}
    for s in range(N + 1):
        for x in STATE:
            getattr(c, x).view(torch.uint8).copy_(old[x].view(torch.uint8))
        here = end == s                              # there one token is appended, elsewhere none
        put(c, k, v, s, s + 1, start=torch.full((B,), s, dtype=torch.int32, device="cuda"), n_new=here.int())
        taken = c.n_kept == s + here.int()
        assert (taken | (c.n_kept == end)).all()
        must = (end >= s) & ((end - s <= BLOCK) | (s % BLOCK == 0))
        assert taken[must].all() and not taken[end < s].any(), s
        at = torch.arange(s // BLOCK * BLOCK, s, device="cuda")
        for x, ring in ((k, c.k_ring), (v, c.v_ring)):
            right = (ring[:, 0, at % RING] == x[:, at, 0]).flatten(1).all(1)
            assert right[taken].all(), (s, end[taken & ~right].tolist())
        assert ua.get_device_status() == (0 if taken.all() else 1)
