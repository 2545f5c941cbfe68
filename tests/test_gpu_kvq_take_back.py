"""GPU tests of the 8-bit cache's append with tokens taken back: which starts it accepts, and that every start
it accepts leaves the cache that never saw the tokens taken back."""
import random

import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import BLOCK, RING, d64, encode, normal, rows_of
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


def check_read(c, K, V, n):
    """What the attention reads of n[b] slots, one KV head: the finished blocks' codes and the unfinished block's rows.  (The
    block before has its rows in the ring only where the sequence was not taken back behind it.)"""
    assert c.n_kept.tolist() == n and int(c.ring_state[-1]) == 0
    for b in range(c.B):
        for name, X in (("k", K), ("v", V)):
            got, done = rows_of(c, name, b, 0, n[b]), n[b] // BLOCK * BLOCK
            for j in range(0, done, BLOCK):
                codes, s = encode(X[b, j:j + BLOCK, 0], c.k.dtype)
                assert torch.equal(got[j:j + BLOCK], d64(codes.view(c.k.dtype)) * d64(s)), (name, b, j)
            assert torch.equal(got[done:], d64(X[b, done:n[b], 0])), (name, b)


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


@pytest.mark.parametrize("n", [300, 320, 1000])
@pytest.mark.parametrize("start", [64, 128, 192])
@pytest.mark.parametrize("m", [0, 1, 10, 64, 100])
def test_a_sequence_goes_on_after_a_border_far_back(n, start, m):
    """A prefix of whole blocks kept, a few tokens appended, then one token at a time past two borders: the cache that
    never held what was taken back.  The block before the prefix's end has left the ring and is refused."""
    c = make(1, 1, 64, 1024, E4, BF)
    k, v = rows(n, 11)
    k2, v2 = rows(300, 13)
    put(c, k, v, 0, n)
    put(c, k2, v2, 0, max(m, 1), start=i32([start]), n_new=i32([m]))
    for t in range(m, m + 130):
        put(c, k2, v2, t, t + 1)
        if t == m:
            put(c, k2, v2, 0, 1, start=i32([start - 10]))
            assert ua.get_device_status() == 1
    assert ua.get_device_status() == 0
    check(c, *(torch.cat([x[:, :start], y[:, :m + 130]], 1) for x, y in ((k, k2), (v, v2))), [start + m + 130], True)


def test_random_walks_of_appends_and_starts():
    """32 sequences append 0 to 150 tokens at a time, going on, back a little, back to borders and to anywhere.  A model
    keeps what each row of the ring was last given: an accepted start finds its block's rows there; going on, a border, and
    up to 64 slots back (not behind the place of the last way back) are never refused; the cache at the end holds the tokens
    that were kept."""
    B, T, cap, steps = 32, 150, 704, 60
    rng = random.Random(5)
    c = make(B, 1, 64, cap, E4, BF, page=128)
    K, V = rows(steps * T, 17, B)
    held = [[] for _ in range(B)]                    # the token in each slot
    ring = [[None] * RING for _ in range(B)]         # (slot, token)
    back = [0] * B
    refused = 0
    for step in range(steps):
        start, new = [], []
        for b in range(B):
            n = len(held[b])
            at = rng.choice([n, n, n, max(0, n - rng.randint(1, 64)), BLOCK * rng.randint(0, n // BLOCK), rng.randint(0, n)])
            m = rng.choice([0, 1, 1, 4, 63, 64, 128, rng.randint(0, T)])
            m = min(m, T, cap - at)
            if at + m == n and m:                    # (a refusal leaves n slots too)
                m -= 1
            start.append(at)
            new.append(m)
        lo = step * T
        put(c, K, V, lo, lo + T, start=i32(start), n_new=i32(new))
        got = c.n_kept.tolist()
        for b, (at, m) in enumerate(zip(start, new)):
            n, block = len(held[b]), at // BLOCK * BLOCK
            intact = all(ring[b][j % RING] == (j, held[b][j]) for j in range(block, at))
            must = at == n or at % BLOCK == 0 or at >= max(n - BLOCK, back[b])
            assert intact or not must                # (the model itself)
            if got[b] != at + m:
                assert got[b] == n and not must, (step, b, n, at, m)
                refused += 1
                continue
            assert intact, (step, b, n, at, m)
            if at < n:
                back[b] = at
            held[b] = held[b][:at] + list(range(lo, lo + m))
            for j in range(max(at, ((at + m) // BLOCK - 1) * BLOCK), at + m):
                ring[b][j % RING] = (j, held[b][j])
        assert ua.get_device_status() in (0, 1)
    assert 0 < refused < B * steps // 4
    n = [len(x) for x in held]
    idx = torch.tensor([x + [0] * (cap - len(x)) for x in held], device="cuda")
    pick = torch.arange(B, device="cuda")[:, None]
    check_read(c, K[pick, idx], V[pick, idx], n)


@pytest.mark.parametrize("m", [1, 10, 64, 70])
def test_a_prefix_without_rows_is_not_taken_for_one(m):
    """A slot count set by hand on a block's border (codes from elsewhere, nothing in the ring): the sequence goes on from
    it, and a start inside the prefix's last block stays refused however it goes on."""
    c = make(1, 1, 64, 512, E4, BF)
    k, v = rows(400, 21)
    c.n_kept.fill_(128)
    put(c, k, v, 0, m)
    assert c.n_kept.tolist() == [128 + m] and ua.get_device_status() == 0
    for n_new in (0, 1):
        put(c, k, v, 0, 1, start=i32([100]), n_new=i32([n_new]))
        assert ua.get_device_status() == 1 and c.n_kept.tolist() == [128 + m]
    put(c, k, v, m, m + 1)
    put(c, k, v, m, m + 1, start=i32([128 + m]))     # one token back
    put(c, k, v, m + 1, m + 100)
    assert ua.get_device_status() == 0
    n, lead = 128 + m + 100, torch.zeros_like(k[:, :128])
    check_read(c, torch.cat([lead, k], 1), torch.cat([lead, v], 1), [n])
