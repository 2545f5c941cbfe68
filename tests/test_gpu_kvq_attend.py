"""GPU tests of attention over the 8-bit cache against a 64-bit plain form of what the cache holds, with
the error bounds derived in softmax_layers.py."""
import math

import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import THETA, check_attend, d64, fill_random, norm_rope, normal, rows_of
from test_gpu_kvq_cache import i32, make

pytestmark = pytest.mark.gpu
BF, F, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
PARTS = 148 * 2 * 16 * 130 * 4                       # bytes of the workspace before its counters


def filled(B, Hkv, d, n, fmt, dt, page=0, seed=0, cap=None):
    c = make(B, Hkv, d, cap or max(max(n), 1), fmt, dt, page, seed)
    fill_random(c, seed)
    c.n_kept.copy_(i32(n))
    return c


def run(c, q, **kw):
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), 7.0, device="cuda")
    o = ua.kvq_attend(c, q, lse=lse, **kw)
    return o, lse


LENGTHS = [[1], [0], [63], [64], [65], [128, 0, 1], [333, 64, 20], [1000], [129, 640, 77, 500, 3]]


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("fmt", [I8, E4])
@pytest.mark.parametrize("dt,d,G", [(BF, 64, 4), (BF, 128, 3), (F, 64, 1), (F, 128, 8)])
def test_single_tokens(n, fmt, dt, d, G):
    B, Hkv = len(n), 2
    c = filled(B, Hkv, d, n, fmt, dt, seed=3)
    q = normal((B, 1, Hkv * G, d), 4, dt)
    o, lse = run(c, q)
    check_attend(c, q, n, o, lse)
    assert ua.get_device_status() == 0


@pytest.mark.parametrize("Tq,G,n", [(2, 4, [70, 2, 1]), (3, 3, [200, 64, 131]), (4, 4, [300]), (5, 8, [65, 400]), (16, 1, [16, 90]),
                                    (33, 2, [129, 40]), (7, 1, [6, 64])])
@pytest.mark.parametrize("fmt,dt,d", [(E4, BF, 64), (I8, BF, 128), (I8, F, 64), (E4, F, 128)])
def test_drafts_see_the_slots_up_to_their_own(Tq, G, n, fmt, dt, d):
    B, Hkv = len(n), 2
    c = filled(B, Hkv, d, n, fmt, dt, page=128, seed=5)
    q = normal((B, Tq, Hkv * G, d), 6, dt)
    o, lse = run(c, q)                               # (queries in front of the first slot see nothing)
    check_attend(c, q, n, o, lse)


@pytest.mark.parametrize("dt", [BF, F])
def test_ragged_queries_leave_the_other_rows(dt):
    n, nq, Tq, H = [100, 64, 9, 300], [0, 1, 5, 3], 5, 6
    c = filled(4, 2, 64, n, E4, dt, seed=7)
    q = normal((4, Tq, H, 64), 8, dt)
    out = torch.full_like(q, 3.0)
    lse = torch.full((4, H, Tq), 7.0, device="cuda")
    got = ua.kvq_attend(c, q, n_q=i32(nq), out=out, lse=lse)
    assert got is out
    check_attend(c, q, n, out, lse, n_q=nq)
    for b in range(4):
        assert (out[b, nq[b]:] == 3.0).all() and (lse[b, :, nq[b]:] == 7.0).all()
        assert not (lse[b, :, :nq[b]] == 7.0).any()


@pytest.mark.parametrize("fmt,dt,d", [(E4, BF, 64), (I8, F, 128)])
def test_bias_and_gate(fmt, dt, d):
    n, B, Hkv, H, Tq = [333, 70, 5], 3, 2, 6, 2
    c = filled(B, Hkv, d, n, fmt, dt, seed=9)
    q, g = normal((B, Tq, H, d), 10, dt), normal((B, Tq, H, d), 11, dt, scale=3.0)
    bias = normal((B, Hkv, c.capacity), 12, F, scale=2.0)
    bias[torch.rand(bias.shape, generator=torch.Generator().manual_seed(1)).cuda() < 0.3] = -math.inf
    bias[0, 0, 64:128] = -math.inf                   # a whole block
    bias[1, 1] = -math.inf                           # a whole row: its outputs are 0
    bias[2, :, :] = torch.finfo(F).min               # the lowest finite value only weighs: all slots alike
    bias[:, :, max(n):] = math.nan                   # behind the last slot: never read
    o, lse = run(c, q, bias=bias, g=g)
    check_attend(c, q, n, o, lse, bias=bias, g=g)
    assert (o[1, :, 3:] == 0).all() and (lse[1, 3:] == -math.inf).all()


def test_lowest_bias_equals_uniform_weights():
    c = filled(1, 1, 64, [130], I8, F, seed=13)
    q = normal((1, 1, 2, 64), 14, F)
    bias = torch.full((1, 1, c.capacity), torch.finfo(F).min, device="cuda")
    o, _ = run(c, q, bias=bias)
    v = rows_of(c, "v", 0, 0, 130).mean(0)
    # every logit rounds to the same value: weights are equal; 130 additions in fp32, probabilities in two f16 parts
    assert (d64(o[0, 0]) - v).abs().max() <= 300 * 2.0 ** -24 * float(rows_of(c, "v", 0, 0, 130).abs().max())


def test_masked_slots_may_hold_anything():
    """NaN and infinities: in an unfinished block under a -inf bias; in a block whose slots are all hidden; behind the
    last slot; not read at all."""
    n = [64 * 3 + 20]
    for dt in (BF, F):
        c = filled(1, 1, 64, n, E4, dt, seed=15)
        q = normal((1, 2, 4, 64), 16, dt)
        bias = torch.zeros(1, 1, c.capacity, device="cuda")
        bias[0, 0, 64:128] = -math.inf
        bias[0, 0, 195] = -math.inf
        want, wl = run(c, q, bias=bias)
        c.k_scale[0, 0, 1] = math.nan                # what an append leaves for a block with a value that is not finite
        c.v_scale[0, 0, 1] = math.nan
        for r in (c.k_ring, c.v_ring):
            r[0, 0, 195 % 128] = math.nan
            r[0, 0, [(192 + j) % 128 for j in range(20, 64)]] = math.inf
            r[0, 0, [(128 + j) % 128 for j in range(64)]] = math.nan      # the finished block's copy
        o, l2 = run(c, q, bias=bias)
        assert torch.equal(o, want) and torch.equal(l2, wl)
        # seen, it spoils the rows that see it, and no others
        bias[0, 0, 64] = 0.0
        o, _ = run(c, q, bias=bias)
        assert torch.isnan(o).all()


def test_values_not_finite_spoil_only_rows_that_see_them():
    B, Hkv, d = 2, 2, 64
    k, v = normal((B, 130, Hkv, d), 17, BF), normal((B, 130, Hkv, d), 18, BF)
    k[0, 10, 1, 3] = math.nan
    v[1, 129, 0, 0] = math.inf
    c = make(B, Hkv, d, 192, I8, BF)
    ua.kvq_append(c, k, v, theta=0.0)
    o, _ = run(c, normal((B, 1, 4, d), 19, BF))
    assert torch.isnan(o[0, 0, 2:]).all() and torch.isfinite(o[0, 0, :2]).all()
    assert not torch.isfinite(o[1, 0, :2]).all() and torch.isfinite(o[1, 0, 2:]).all()


@pytest.mark.parametrize("dt", [BF, F])
def test_large_logits_and_uneven_scales(dt):
    """One slot takes nearly all weight; blocks' value scales far apart; queries far from 1."""
    n = [64 * 5 + 7]
    for mul, vmul in ((1e4, 1.0), (1e-6, 1.0), (1.0, 2.0 ** 40)):
        c = filled(1, 2, 128, n, I8, dt, seed=21)
        c.v_scale[:, :, 2] *= vmul
        q = normal((1, 1, 4, 128), 22, dt, scale=mul)
        o, lse = run(c, q)
        check_attend(c, q, n, o, lse)


def test_many_small_weights_are_not_lost():
    """One slot far above 4000 others that together still weigh as much: they are below f16's range
    against the maximum, and must count."""
    N, d = 4097, 64
    c = make(1, 1, d, 4160, E4, BF)
    k = torch.zeros(1, N, 1, d, dtype=BF, device="cuda")
    k[0, 0, 0, 0] = 8.0
    v = normal((1, N, 1, d), 23, BF)
    v[0, 1:] = v[0, 1:].abs()
    ua.kvq_append(c, k, v, theta=0.0)
    bias = torch.full((1, 1, c.capacity), -18.0, device="cuda")   # e^-18 = 1.5e-8
    bias[0, 0, 0] = 0.0
    q = torch.zeros(1, 1, 1, d, dtype=BF, device="cuda")
    o, lse = run(c, q, bias=bias)
    check_attend(c, q, [N], o, lse, bias=bias)
    q[0, 0, 0, 0] = -1.0
    for sh in (-12.0, -16.0):
        bias[0, 0, 1:] = sh
        o, lse = run(c, q, bias=bias)
        check_attend(c, q, [N], o, lse, bias=bias)


@pytest.mark.parametrize("n,H,Hkv,page", [([20000], 8, 2, 0), ([5000, 1, 17000, 300, 64], 8, 2, 1024), ([40] * 300, 4, 1, 0),
                                          ([0] * 150 + [9000] + [2] * 150, 2, 1, 128)])
def test_work_split_over_the_gpu(n, H, Hkv, page):
    """Long sequences in many parts, ragged batches, many short sequences (more than one scan of lengths)."""
    c = filled(len(n), Hkv, 64, n, E4, BF, page=page, seed=25)
    q = normal((len(n), 1, H, 64), 26, BF)
    ws = ua.alloc_workspace(ua.kvq_attend_workspace_size(c, H, 1), "cuda")
    o, lse = run(c, q, ws=ws)
    check_attend(c, q, n, o, lse)
    again, l2 = run(c, q, ws=ws)                     # the workspace serves the next call, the order is fixed
    assert torch.equal(o, again) and torch.equal(lse, l2)
    assert (ws[PARTS:] == 0).all()
    assert ua.get_device_status() == 0


def test_one_workspace_for_calls_of_different_shapes():
    a, b = filled(1, 2, 128, [9000], E4, BF, seed=27), filled(7, 2, 128, [700, 3, 64, 2000, 1, 0, 90], I8, BF, seed=28)
    qa, qb = normal((1, 1, 16, 128), 29, BF), normal((7, 4, 4, 128), 30, BF)
    size = max(ua.kvq_attend_workspace_size(a, 16, 1), ua.kvq_attend_workspace_size(b, 4, 4))
    ws = ua.alloc_workspace(size, "cuda")
    want = [run(a, qa)[0], run(b, qb)[0]]
    for _ in range(2):
        assert torch.equal(run(a, qa, ws=ws)[0], want[0])
        assert torch.equal(run(b, qb, ws=ws)[0], want[1])
    assert (ws[PARTS:] == 0).all()


def test_bad_counts_and_pages_are_reported():
    c = filled(3, 1, 64, [100, 200, 50], E4, BF, page=128, seed=31)
    q = normal((3, 1, 2, 64), 32, BF)
    want, _ = run(c, q)
    for bad in (-1, 257):
        c.n_kept[1] = bad
        o, lse = run(c, q)
        assert ua.get_device_status() == 1
        assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2]) and (o[1] == 0).all()
    c.n_kept[1] = 200
    o = ua.kvq_attend(c, q, n_q=i32([1, 2, 1]))
    assert ua.get_device_status() == 1
    c.page_table[1, 0] = c.pool_pages
    o, _ = run(c, q)
    assert ua.get_device_status() == 1
    assert torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


def test_stale_workspace_is_reported():
    c = filled(1, 1, 64, [5000], E4, BF, seed=33)
    q = normal((1, 1, 4, 64), 34, BF)
    ws = ua.alloc_workspace(ua.kvq_attend_workspace_size(c, 4, 1), "cuda")
    ws[PARTS:PARTS + 4] = 0x7f
    run(c, q, ws=ws)
    assert ua.get_device_status() == 1


@pytest.mark.parametrize("dt,fmt", [(BF, E4), (F, I8)])
def test_a_layers_steps_together(dt, fmt):
    """Prompt, single tokens, drafts of which some are taken back, through append and attention, captured
    replays among them: the outputs are those of the operators' definitions on the tokens' own keys."""
    B, H, Hkv, d = 2, 4, 2, 64
    T0, steps = 100, 70
    c = make(B, Hkv, d, 256, fmt, dt, page=128, seed=1)
    wq, wk = 1 + 0.2 * normal((d,), 41, F), 1 + 0.2 * normal((d,), 42, F)
    new = lambda T, s: (normal((B, T, Hkv, d), s, dt), normal((B, T, Hkv, d), s + 1, dt), normal((B, T, H, d), s + 2, dt))  # noqa: E731
    K, V = [], []

    def held(n):
        """64-bit keys and values as the definition stores them, from the inputs alone."""
        k, _ = norm_rope(torch.cat(K, 1)[:, :n], wk, torch.arange(n, dtype=torch.int32).repeat(B, 1), 1e-6, THETA)
        return k, d64(torch.cat(V, 1)[:, :n])

    k, v, q = new(T0, 50)
    n_new = i32([T0, T0 - 40])
    ua.kvq_append(c, k, v, q, wq=wq, wk=wk, n_new=n_new)
    ua.kvq_append(c, k[:, T0 - 40:].contiguous(), v[:, T0 - 40:].contiguous(), wk=wk, n_new=i32([0, 40]))
    K.append(k)
    V.append(v)
    n = T0
    ks, vs, qs = (x.clone() for x in new(1, 60))
    qo, out = torch.empty_like(qs), torch.empty_like(qs)
    ws = ua.alloc_workspace(ua.kvq_attend_workspace_size(c, H, 1), "cuda")
    ua.kvq_append(c, ks, vs, qs, wq=wq, wk=wk, q_out=qo, start=i32([n, n]), n_new=i32([0, 0]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ua.kvq_append(c, ks, vs, qs, wq=wq, wk=wk, q_out=qo)
        ua.kvq_attend(c, qo, out=out, ws=ws)
    for s in range(steps):
        k, v, q = new(1, 100 + 3 * s)
        ks.copy_(k), vs.copy_(v), qs.copy_(q)
        graph.replay()
        K.append(k)
        V.append(v)
        n += 1
    check_attend(c, qo, [n] * B, out, None)          # the last step, against what the cache holds
    # the cache holds the inputs' keys to half a step of the codes and of the activation type
    kk, vv = held(n)
    for b in range(B):
        for h in range(Hkv):
            for x, y in ((kk, "k"), (vv, "v")):
                got = rows_of(c, y, b, h, n)
                amax = x[b, :, h].abs().max()
                step = amax / 254 if fmt == I8 else 2.0 ** -4 * amax
                assert (got - x[b, :n, h]).abs().max() <= step + 2.0 ** -7 * amax
    # four drafts, two of them rejected, then four others
    k, v, q = new(4, 900)
    qd = ua.kvq_append(c, k, v, q, wq=wq, wk=wk)
    check_attend(c, qd, [n + 4] * B, ua.kvq_attend(c, qd), None)
    k, v, q = new(4, 910)
    qd = ua.kvq_append(c, k, v, q, wq=wq, wk=wk, start=i32([n + 2, n + 2]))
    check_attend(c, qd, [n + 6] * B, ua.kvq_attend(c, qd), None)
    assert c.n_kept.tolist() == [n + 6] * B
    assert ua.get_device_status() == 0


def test_on_another_stream_and_as_three_dimensional_queries():
    c = filled(2, 2, 64, [300, 70], E4, BF, seed=51)
    q = normal((2, 8, 64), 52, BF)
    want = ua.kvq_attend(c, q[:, None].contiguous())[:, 0]
    ws = ua.alloc_workspace(ua.kvq_attend_workspace_size(c, 8), "cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = ua.kvq_attend(c, q, stream=s, ws=ws)
    s.synchronize()
    assert o.shape == q.shape and torch.equal(o, want)


def test_a_layer_on_a_stream_of_its_own():
    """Every call with stream=, outputs and scratch made by the wrappers, while the current stream is busy (and its
    free memory is full of ones): nothing of the calls is queued there."""
    B, T, H, Hkv, d = 2, 900, 8, 2, 64
    q, k, v = normal((B, T, H, d), 41, BF), normal((B, T, Hkv, d), 42, BF), normal((B, T, Hkv, d), 43, BF)
    wq, wk = 1 + 0.2 * normal((d,), 44, F), 1 + 0.2 * normal((d,), 45, F)
    last = q[:, -1:].contiguous()

    def layer(c, **kw):
        qo = ua.kvq_append(c, k, v, q, wq=wq, wk=wk, **kw)
        o = ua.kvq_attend(c, last, **kw)
        f = ua.qk_norm_rope_fwd(q, k, wq, wk, **kw)
        g = ua.qk_norm_rope_bwd(q, k, wq, wk, q, k, **kw)
        return [qo, o, *f.values(), *g.values()]

    a, b = make(B, Hkv, d, 1024, E4, BF), make(B, Hkv, d, 1024, E4, BF)
    want = layer(a)
    s = torch.cuda.Stream()
    junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 20, 3 << 20, 1 << 22)]
    torch.cuda.synchronize()
    del junk
    torch.cuda._sleep(100_000_000)
    got = layer(b, stream=s)
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert ua.get_device_status() == 0
