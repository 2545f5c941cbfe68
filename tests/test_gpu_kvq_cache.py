"""GPU tests of the 8-bit cache's append: ring rows, codes and scales against their definition, the
same cache however the tokens are split into calls, ragged batches, tokens taken back, refusals."""
import math

import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import BLOCK, RING, THETA, d64, encode, norm_rope, normal, rows_of, within

pytestmark = pytest.mark.gpu
BF, F, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(B, Hkv, d, cap, fmt, dt, page=0, seed=0):
    if not page:
        return ua.KVQCache.empty(B, Hkv, d, cap, fmt, dt)
    per = -(-cap // page)
    c = ua.KVQCache.paged(B, Hkv, d, page, per, B * per + 3, fmt, dt)
    perm = torch.randperm(B * per + 3, generator=torch.Generator().manual_seed(seed))[:B * per]
    c.page_table.copy_(perm.reshape(B, per).to(torch.int32))
    return c


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def check(cache, K, V, n, exact_keys, kbound=None):
    """Everything an append up to n[b] slots of rows K, V [B, N, Hkv, d] leaves (K in the activation type where
    exact_keys, else in 64 bits with kbound)."""
    assert cache.n_kept.tolist() == n
    assert int(cache.ring_state[-1]) == 0
    for b in range(cache.B):
        for h in range(cache.Hkv):
            for blk in range(n[b] // BLOCK):
                pg = b if cache.page_table is None else int(cache.page_table[b, blk * BLOCK // cache.page_size])
                at = blk * BLOCK % cache.page_size
                rows = slice(blk * BLOCK, (blk + 1) * BLOCK)
                for X, codes, sc in ((V, cache.v, cache.v_scale), (K, cache.k, cache.k_scale)):
                    got, s = codes[pg, h, at:at + BLOCK], sc[pg, h, at // BLOCK].cpu()
                    if X is V or exact_keys:
                        want, ws = encode(X[b, rows, h], codes.dtype)
                        assert torch.equal(s.nan_to_num(-1), ws.nan_to_num(-1)), (b, h, blk, s, ws)
                        assert torch.equal(got.view(torch.uint8).cpu(), want), (b, h, blk)
                    else:
                        # the row rounded to the activation type, then half a step of the code
                        x = X[b, rows, h]
                        off = (d64(got) * d64(s) - x).abs()
                        act = kbound[b, rows, h] + 2.0 ** -8 * (x.abs() + kbound[b, rows, h]) if cache.dtype == BF else 1e-5 * (1 + x.abs())
                        step = d64(s) / 2 if codes.dtype == I8 else torch.maximum(2.0 ** -4 * (x.abs() + act), d64(s) * 2.0 ** -10)
                        assert (off <= act + step * 1.0001).all(), (b, h, blk, float((off - act - step).max()))
            late = range(max(0, (n[b] // BLOCK - 1) * BLOCK), n[b])
            if len(late):
                at = [j % RING for j in late]
                assert same_bits(cache.v_ring[b, h][at], V[b, late.start:late.stop, h])
                if exact_keys:
                    assert same_bits(cache.k_ring[b, h][at], K[b, late.start:late.stop, h])
                else:
                    within("ring", cache.k_ring[b, h][at], K[b, late.start:late.stop, h], kbound[b, late.start:late.stop, h], cache.dtype)


CASES = [(1, 1, 1, 64, 0), (2, 63, 2, 64, 0), (2, 64, 3, 128, 0), (1, 65, 8, 64, 128), (3, 200, 2, 128, 128),
         (2, 449, 1, 64, 256), (5, 128, 6, 64, 0)]


@pytest.mark.parametrize("B,T,Hkv,d,page", CASES)
@pytest.mark.parametrize("fmt", [I8, E4])
@pytest.mark.parametrize("dt", [BF, F])
def test_stores_and_encodes_as_defined(B, T, Hkv, d, page, fmt, dt):
    c = make(B, Hkv, d, T + 70, fmt, dt, page)
    k, v = normal((B, T, Hkv, d), 1, dt), normal((B, T, Hkv, d), 2, dt, scale=5.0)
    ua.kvq_append(c, k, v, theta=0.0)               # neither norm nor rotation: keys are stored as they are
    check(c, k, v, [T] * B, True)
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("B,T,Hkv,d,page", CASES)
@pytest.mark.parametrize("dt,fmt", [(BF, E4), (BF, I8), (F, E4)])
def test_norm_and_rotation_on_the_way(B, T, Hkv, d, page, dt, fmt):
    c = make(B, Hkv, d, T + 70, fmt, dt, page)
    G = 3
    q, k, v = normal((B, T, Hkv * G, d), 3, dt), normal((B, T, Hkv, d), 4, dt), normal((B, T, Hkv, d), 5, dt)
    wq, wk = 1 + 0.3 * normal((d,), 6, F), 1 + 0.3 * normal((d,), 7, F)
    pos = (torch.arange(T, dtype=torch.int32) * 3 + 100000).repeat(B, 1).cuda()
    qo = ua.kvq_append(c, k, v, q, wq=wq, wk=wk, pos=pos)
    K, kb = norm_rope(k, wk, pos, 1e-6, THETA)
    check(c, K, v, [T] * B, False, kb)
    Q, qb = norm_rope(q, wq, pos, 1e-6, THETA)
    within("q", qo, Q, qb, dt)
    # positions default to the slots' numbers
    c2 = make(B, Hkv, d, T + 70, fmt, dt, page)
    q2 = ua.kvq_append(c2, k, v, q)
    slots = torch.arange(T, dtype=torch.int32).repeat(B, 1)
    K, kb = norm_rope(k, None, slots, 1e-6, THETA)
    check(c2, K, v, [T] * B, False, kb)
    Q, qb = norm_rope(q, None, slots, 1e-6, THETA)
    within("q", q2, Q, qb, dt)
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("dt,fmt,d,page", [(BF, E4, 64, 0), (BF, I8, 128, 128), (F, I8, 64, 128)])
def test_same_cache_however_the_tokens_come(dt, fmt, d, page):
    """One call, single tokens, and uneven chunks give the same bits."""
    B, T, Hkv = 2, 330, 2
    k, v = normal((B, T, Hkv, d), 11, dt), normal((B, T, Hkv, d), 12, dt)
    wk = 1 + 0.3 * normal((d,), 13, F)
    runs = []
    for cuts in ([T], [1] * T, [50, 14, 1, 129, 3, 64, 69], [130, 200]):
        c = make(B, Hkv, d, T, fmt, dt, page, seed=4)
        at = 0
        for m in cuts:
            ua.kvq_append(c, k[:, at:at + m].contiguous(), v[:, at:at + m].contiguous(), wk=wk)
            at += m
        assert c.n_kept.tolist() == [T] * B
        runs.append([torch.stack([rows_of(c, x, b, h, T) for b in range(B) for h in range(Hkv)]) for x in "kv"]
                    + [c.k_ring.clone(), c.v_ring.clone()])
    kept = [j % RING for j in range((T // BLOCK - 1) * BLOCK, T)]
    for other in runs[1:]:
        assert torch.equal(runs[0][0], other[0]) and torch.equal(runs[0][1], other[1])
        for i in (2, 3):
            assert torch.equal(runs[0][i][:, :, kept], other[i][:, :, kept])
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("fmt", [I8, E4])
def test_ragged_batch_leaves_everything_else(fmt):
    B, T, Hkv, d = 5, 150, 2, 64
    c = make(B, Hkv, d, 320, fmt, BF, 128)
    k0, v0 = normal((B, 90, Hkv, d), 21, BF), normal((B, 90, Hkv, d), 22, BF)
    n0 = [0, 1, 64, 90, 77]
    ua.kvq_append(c, k0, v0, n_new=i32(n0), theta=0.0)
    before = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale, c.k_ring, c.v_ring)]
    k, v = normal((B, T, Hkv, d), 23, BF), normal((B, T, Hkv, d), 24, BF)
    k[4, 3:], v[4, 3:] = math.nan, math.inf          # rows behind a sequence's last token may hold anything
    new = [150, 63, 0, 100, 3]
    ua.kvq_append(c, k, v, n_new=i32(new), theta=0.0)
    K = torch.zeros(B, 320, Hkv, d, dtype=BF, device="cuda")
    V = torch.zeros_like(K)
    for b in range(B):
        for X, a, z in ((K, k0, k), (V, v0, v)):
            X[b, :n0[b]] = a[b, :n0[b]]
            X[b, n0[b]:n0[b] + new[b]] = z[b, :new[b]]
    check(c, K, V, [a + z for a, z in zip(n0, new)], True)
    # sequence 2 appended nothing, and pages of no finished block are as they were
    assert torch.equal(c.k_ring[2], before[4][2]) and torch.equal(c.v_ring[2], before[5][2])
    used = set()
    for b in range(B):
        used |= {(int(c.page_table[b, j * BLOCK // 128]), j % 2) for j in range((n0[b] + new[b]) // BLOCK)}
    for pg in range(c.pool_pages):
        for half in range(2):
            if (pg, half) not in used:
                rows = slice(half * 64, half * 64 + 64)
                assert torch.equal(c.k.view(torch.uint8)[pg, :, rows], before[0][pg, :, rows])
                assert torch.equal(c.v_scale[pg, :, half], before[3][pg, :, half])
    assert ua.get_device_status() == 0


def test_tokens_taken_back():
    """Drafts rejected, another continuation appended: the cache is the one that never saw them."""
    B, Hkv, d = 3, 2, 64
    k, v = normal((B, 200, Hkv, d), 31, BF), normal((B, 200, Hkv, d), 32, BF)
    c = make(B, Hkv, d, 256, E4, BF)
    ua.kvq_append(c, k[:, :126].contiguous(), v[:, :126].contiguous(), theta=0.0)
    wrong = normal((B, 8, Hkv, d), 33, BF)
    ua.kvq_append(c, wrong, wrong, theta=0.0)        # 126 .. 133: block 1 is encoded with wrong rows
    assert c.n_kept.tolist() == [134] * B
    start = i32([126, 128, 134])
    ua.kvq_append(c, k[:, 126:146].contiguous(), v[:, 126:146].contiguous(), start=start, theta=0.0)
    K, V = k.clone(), v.clone()
    for b, s in ((1, 128), (2, 134)):
        for X, x in ((K, k), (V, v)):
            X[b, 126:s] = wrong[b, :s - 126]
            X[b, s:s + 20] = x[b, 126:146]
    check(c, K, V, [146, 148, 154], True)
    assert ua.get_device_status() == 0
    # begun anew
    ua.kvq_append(c, k[:, :70].contiguous(), v[:, :70].contiguous(), start=i32([0, 0, 0]), theta=0.0)
    check(c, k, v, [70] * B, True)
    # nothing appended, two tokens taken back
    ua.kvq_append(c, wrong, wrong, start=i32([68, 70, 64]), n_new=i32([0, 0, 0]), theta=0.0)
    check(c, k, v, [68, 70, 64], True)
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("what,start,n_new,code", [
    ("capacity", None, [5, 4, 0], 5), ("above", [101, 100, 100], None, 1), ("negative", [100, -1, 100], None, 1),
    ("too many", None, [1, 9, 1], 1), ("fewer than none", None, [1, -1, 1], 1), ("ring", [20, 100, 100], None, 1)])
def test_refused_sequences_stay_as_they_were(what, start, n_new, code):
    B, Hkv, d, T = 3, 2, 64, 8
    cap = 128 if what == "capacity" else 256
    c = make(B, Hkv, d, cap, I8, BF)
    n = [124, 124, 128] if what == "capacity" else [100] * 3
    if what == "ring":                               # 190 slots were filled: block 0 has left the ring, block 1 has not
        ua.kvq_append(c, normal((B, 190, Hkv, d), 40, BF), normal((B, 190, Hkv, d), 40, BF), theta=0.0)
        ua.kvq_append(c, normal((B, 1, Hkv, d), 40, BF), normal((B, 1, Hkv, d), 40, BF), start=i32([100] * 3), n_new=i32([0] * 3), theta=0.0)
        assert c.n_kept.tolist() == [100] * 3 and ua.get_device_status() == 0
    else:
        ua.kvq_append(c, normal((B, 128, Hkv, d), 41, BF), normal((B, 128, Hkv, d), 42, BF), n_new=i32(n), theta=0.0)
    old = [t.clone() for t in (c.k, c.v, c.k_scale, c.k_ring, c.v_ring, c.n_kept)]
    k, v = normal((B, T, Hkv, d), 43, BF), normal((B, T, Hkv, d), 44, BF)
    ua.kvq_append(c, k, v, start=None if start is None else i32(start), n_new=None if n_new is None else i32(n_new), theta=0.0)
    assert ua.get_device_status() == code
    bad = {"capacity": [0], "above": [0], "negative": [1], "too many": [1], "fewer than none": [1], "ring": [0]}[what]
    for b in range(B):
        st = n[b] if start is None else start[b]
        m = T if n_new is None else n_new[b]
        if b in bad:
            assert int(c.n_kept[b]) == n[b]
            for t, o in zip((c.k, c.v, c.k_scale, c.k_ring, c.v_ring), old):
                assert torch.equal(t[b].view(torch.uint8), o[b].view(torch.uint8))
        else:
            assert int(c.n_kept[b]) == st + m
            at = [j % RING for j in range(st, st + m)]
            assert torch.equal(c.k_ring[b][:, at], k[b, :m].transpose(0, 1))
    assert int(c.ring_state[-1]) == 0


def test_rows_that_were_never_there_are_refused():
    """A slot count set by hand inside a block has no rows in the ring to encode it from; on a block's border none are
    needed."""
    c = make(2, 1, 64, 256, E4, BF)
    k = normal((2, 70, 1, 64), 45, BF)
    c.n_kept.copy_(i32([70, 64]))
    ua.kvq_append(c, k, k, theta=0.0)
    assert ua.get_device_status() == 1
    assert c.n_kept.tolist() == [70, 134]
    want, s = encode(k[1, :64, 0], E4)
    assert torch.equal(c.k[1, 0, 64:128].view(torch.uint8).cpu(), want)


@pytest.mark.parametrize("pos_given", [True, False])
@pytest.mark.parametrize("start_given", [True, False])
def test_long_prompts_queries(pos_given, start_given):
    """So many tokens that the queries take their own kernel (or, with positions that are the slot counts this
    call changes, not): queries, counts and cache as for a short call, and right before the next kernel."""
    B, T, H, Hkv, d = 2, 1500, 4, 2, 64
    c = make(B, Hkv, d, 1600, E4, BF)
    k0 = normal((B, 64, Hkv, d), 46, BF)
    ua.kvq_append(c, k0, k0, theta=0.0)
    q, k, v = normal((B, T, H, d), 47, BF), normal((B, T, Hkv, d), 48, BF), normal((B, T, Hkv, d), 49, BF)
    pos = (64 + torch.arange(T, dtype=torch.int32)).repeat(B, 1)
    qo = ua.kvq_append(c, k, v, q, pos=pos.cuda() if pos_given else None, start=i32([64, 64]) if start_given else None)
    total = qo.float().sum() + c.n_kept.sum()            # (a kernel that does not start early)
    Q, qb = norm_rope(q, None, pos, 1e-6, THETA)
    within("q", qo, Q, qb, BF)
    K, kb = norm_rope(k, None, pos, 1e-6, THETA)
    check(c, torch.cat([d64(k0), K], 1), torch.cat([k0, v], 1), [T + 64] * B, False, torch.cat([torch.zeros(B, 64, Hkv, d), kb], 1))
    assert torch.isfinite(total)
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("B,T,what", [(2, 3000, "start"), (3, 1, "pos"), (2600, 1, "pos"), (2600, 1, "start")])
def test_slot_counts_themselves_as_positions(B, T, what):
    """n_kept given as start or as a token's position: what the call found there, though it changes it."""
    H, Hkv, d = 4, 2, 64
    a, e = make(B, Hkv, d, T + 128, E4, BF), make(B, Hkv, d, T + 128, E4, BF)
    k0, n0 = normal((B, 70, Hkv, d), 91, BF), i32([i % 71 for i in range(B)])
    q, k, v = normal((B, T, H, d), 92, BF), normal((B, T, Hkv, d), 93, BF), normal((B, T, Hkv, d), 94, BF)
    for c in (a, e):
        ua.kvq_append(c, k0, k0, n_new=n0, theta=0.0)
    of = lambda x: x if what == "start" else x[:, None]  # noqa: E731
    got = ua.kvq_append(a, k, v, q, **{what: of(a.n_kept)})
    want = ua.kvq_append(e, k, v, q, **{what: of(n0)})
    assert torch.equal(got, want)
    for name in ("k", "v", "k_scale", "v_scale", "k_ring", "v_ring", "ring_state", "n_kept"):
        assert same_bits(getattr(a, name), getattr(e, name)), name
    assert ua.get_device_status() == 0


def test_bad_page_is_skipped_and_reported():
    B, Hkv, d = 2, 2, 64
    c = make(B, Hkv, d, 256, E4, BF, 128)
    c.page_table[0, 1] = c.pool_pages                # outside the pool
    c.page_table[1, 0] = -1
    k, v = normal((B, 200, Hkv, d), 51, BF), normal((B, 200, Hkv, d), 52, BF)
    ua.kvq_append(c, k, v, theta=0.0)
    assert ua.get_device_status() == 1
    assert c.n_kept.tolist() == [200, 200]
    pg = int(c.page_table[1, 1])
    want, s = encode(v[1, 128:192, 1], E4)
    assert torch.equal(c.v[pg, 1, :64].view(torch.uint8).cpu(), want) and float(c.v_scale[pg, 1, 0]) == float(s)


@pytest.mark.parametrize("fmt", [I8, E4])
def test_extreme_blocks(fmt):
    """Zeros, the smallest and largest magnitudes, one element far above the rest, values that are not finite."""
    d = 64
    k = torch.zeros(1, 64 * 7, 1, d, dtype=F, device="cuda")
    k[0, 64:128] = normal((64, 1, d), 61, F, scale=1e-36)        # below 2^-100
    k[0, 128:192] = normal((64, 1, d), 62, F, scale=1e-28)
    k[0, 192:256] = normal((64, 1, d), 63, F, scale=1e36)
    k[0, 256:320] = normal((64, 1, d), 64, F)
    k[0, 300, 0, 5] = 448.0 * 2 ** 20                            # exactly at a power of two's border
    k[0, 320:384] = normal((64, 1, d), 65, F)
    k[0, 350, 0, 7] = math.inf
    k[0, 384:448] = normal((64, 1, d), 66, F)
    k[0, 400, 0, 63] = math.nan
    c = make(1, 1, d, 448, fmt, F)
    ua.kvq_append(c, k, -k, theta=0.0)
    check(c, k, -k, [448], True)


def test_slices_and_graph_replays():
    """q, k and v as slices of one projection; a captured step appends one token at each replay."""
    B, H, Hkv, d = 2, 4, 2, 64
    T = 70
    qkv = normal((T, B, 1, (H + 2 * Hkv) * d), 71, BF)
    x = qkv[0].clone()
    wq, wk = 1 + 0.2 * normal((d,), 72, F), 1 + 0.2 * normal((d,), 73, F)

    def views(x):
        q, k, v = x.split([H * d, Hkv * d, Hkv * d], -1)
        return k.unflatten(-1, (Hkv, d)), v.unflatten(-1, (Hkv, d)), q.unflatten(-1, (H, d))

    a, e = make(B, Hkv, d, 128, E4, BF), make(B, Hkv, d, 128, E4, BF)
    qo = torch.empty(B, 1, H, d, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ua.kvq_append(a, *views(x), wq=wq, wk=wk, q_out=qo)
    for t in range(T):
        x.copy_(qkv[t])
        graph.replay()
        k, v, q = (y.contiguous() for y in views(qkv[t]))
        want = ua.kvq_append(e, k, v, q, wq=wq, wk=wk)
        assert torch.equal(qo, want)
    assert a.n_kept.tolist() == e.n_kept.tolist() == [T] * B
    for name in ("k", "v", "k_scale", "v_scale", "k_ring", "v_ring", "ring_state"):
        assert torch.equal(getattr(a, name).view(torch.uint8), getattr(e, name).view(torch.uint8)), name


def test_page_pool_hands_out_pages():
    c = ua.KVQCache.paged(2, 2, 64, 128, 3, 8)
    pool = ua.PagePool(c)
    pool.ensure([130, 256])
    assert pool.pages_in_use() == 4
    k, v = normal((2, 256, 2, 64), 81, BF), normal((2, 256, 2, 64), 82, BF)
    ua.kvq_append(c, k, v, n_new=i32([130, 256]), theta=0.0)
    check(c, k, v, [130, 256], True)
    pool.release()
    assert pool.pages_in_use() == 4
    assert ua.get_device_status() == 0
