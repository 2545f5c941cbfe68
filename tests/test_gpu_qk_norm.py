"""GPU tests of the per-head norm with position rotation and of its gradients against 64-bit plain
forms, with the error bounds derived in softmax_layers.py, and against finite differences."""
import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import THETA, norm_rope, norm_rope_bwd, normal, within

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
EPS = 1e-6

SHAPES = [(1, 1, 1, 1, 64), (1, 1, 32, 8, 128), (2, 17, 6, 2, 64), (3, 50, 5, 3, 128), (1, 333, 8, 1, 64), (40, 1, 24, 8, 128)]


def inputs(B, T, H, Hkv, d, dt, seed):
    q, k = normal((B, T, H, d), seed, dt), normal((B, T, Hkv, d), seed + 1, dt, scale=3.0)
    wq, wk = 1 + 0.3 * normal((d,), seed + 2, F), 1 + 0.3 * normal((d,), seed + 3, F)
    pos = torch.randint(0, 300000, (B, T), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
    return q, k, wq, wk, pos


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("gains,rope", [(True, True), (True, False), (False, True)])
def test_forward(shape, dt, gains, rope):
    q, k, wq, wk, pos = inputs(*shape, dt, 11)
    theta = THETA if rope else 0.0
    r = ua.qk_norm_rope_fwd(q, k, wq if gains else None, wk if gains else None, pos=pos, eps=EPS, theta=theta)
    for got, x, w in ((r["q"], q, wq), (r["k"], k, wk)):
        ref, bound = norm_rope(x, w if gains else None, pos, EPS, theta)
        within("y", got, ref, bound, dt)


def test_positions_default_to_the_index_and_may_be_negative():
    q, k, wq, wk, _ = inputs(2, 9, 2, 2, 64, F, 5)
    pos = torch.arange(9, dtype=torch.int32).repeat(2, 1)
    a = ua.qk_norm_rope_fwd(q, k, wq, wk)
    b = ua.qk_norm_rope_fwd(q, k, wq, wk, pos=pos.cuda())
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["k"], b["k"])
    c = ua.qk_norm_rope_fwd(q, None, wq, pos=-pos.cuda())
    assert c["k"] is None
    ref, bound = norm_rope(q, wq, -pos, EPS, THETA)
    within("y", c["q"], ref, bound, F)


def test_one_side_only_keys():
    q, k, wq, wk, pos = inputs(2, 21, 4, 2, 128, BF, 6)
    r = ua.qk_norm_rope_fwd(None, k, None, wk, pos=pos)
    ref, bound = norm_rope(k, wk, pos, EPS, THETA)
    within("k", r["k"], ref, bound, BF)
    g = ua.qk_norm_rope_bwd(None, k, None, wk, None, k, pos=pos)
    assert g["dq"] is None and g["dwq"] is None
    dx, b, dw, bw = norm_rope_bwd(k, wk, k, pos, EPS, THETA)
    within("dk", g["dk"], dx, b, BF)
    within("dwk", g["dwk"], dw, bw, F)


@pytest.mark.parametrize("dt", [BF, F])
def test_slices_of_a_fused_projection(dt):
    B, T, H, Hkv, d = 2, 19, 4, 2, 64
    qkv = normal((B, T, (H + 2 * Hkv) * d), 21, dt)
    q, k = qkv[..., :H * d].unflatten(-1, (H, d)), qkv[..., H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
    w = 1 + 0.1 * normal((d,), 22, F)
    a = ua.qk_norm_rope_fwd(q, k, w, w)
    b = ua.qk_norm_rope_fwd(q.contiguous(), k.contiguous(), w, w)
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["k"], b["k"])
    dq, dk = normal(q.shape, 23, dt), normal(k.shape, 24, dt)
    ga, gb = ua.qk_norm_rope_bwd(q, k, w, w, dq, dk), ua.qk_norm_rope_bwd(q.contiguous(), k.contiguous(), w, w, dq, dk)
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("shape", SHAPES + [(2, 5000, 2, 1, 64)])
@pytest.mark.parametrize("gains,rope", [(True, True), (True, False), (False, True)])
def test_backward(shape, dt, gains, rope):
    q, k, wq, wk, pos = inputs(*shape, dt, 31)
    dq, dk = normal(q.shape, 32, dt), normal(k.shape, 33, dt)
    theta = THETA if rope else 0.0
    g = ua.qk_norm_rope_bwd(q, k, wq if gains else None, wk if gains else None, dq, dk, pos=pos, eps=EPS, theta=theta)
    for x, w, dy, dx, dw in ((q, wq, dq, "dq", "dwq"), (k, wk, dk, "dk", "dwk")):
        ref, bound, refw, boundw = norm_rope_bwd(x, w if gains else None, dy, pos, EPS, theta)
        within(dx, g[dx], ref, bound, dt)
        if gains:
            within(dw, g[dw], refw, boundw, F)
        else:
            assert g[dw] is None
    again = ua.qk_norm_rope_bwd(q, k, wq if gains else None, wk if gains else None, dq, dk, pos=pos, eps=EPS, theta=theta)
    for n, t in g.items():
        assert t is None or torch.equal(t, again[n]), n


def test_plain_gradients_against_differences():
    """The 64-bit gradient the kernels are held to, against central differences of the 64-bit forward."""
    B, T, H, d = 1, 2, 2, 64
    x, w = normal((B, T, H, d), 41, F, "cpu").double(), 1 + 0.3 * normal((d,), 42, F, "cpu").double()
    dy = normal((B, T, H, d), 43, F, "cpu").double()
    pos = torch.tensor([[3, 70000]], dtype=torch.int32)
    dx, _, dw, _ = norm_rope_bwd(x, w, dy, pos, EPS, THETA)
    f = lambda x, w: float((norm_rope(x, w, pos, EPS, THETA)[0] * dy).sum())  # noqa: E731
    h = 1e-6                                        # differences: h^2 of the third derivative, 1e-16 / h of the value
    for at in [(0, 0, 0, 0), (0, 0, 1, 33), (0, 1, 0, 63), (0, 1, 1, 31)]:
        e = torch.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx[at])) < 1e-7
    for i in (0, 40):
        e = torch.zeros_like(w)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[i])) < 1e-7


def test_zero_and_tiny_heads():
    d = 64
    x = normal((1, 20, 3, d), 51, F)
    x[0, 3] = 0.0
    x[0, 7, 1] *= 1e-18                              # its mean square is far below eps
    w = torch.ones(d, device="cuda")
    r = ua.qk_norm_rope_fwd(x, None, w)
    ref, bound = norm_rope(x, w, torch.arange(20, dtype=torch.int32)[None], EPS, THETA)
    within("y", r["q"], ref, bound, F)
    assert (r["q"][0, 3] == 0).all()


def test_captured_in_a_graph_on_another_stream():
    q, k, wq, wk, pos = inputs(2, 37, 4, 2, 128, BF, 61)
    dq, dk = normal(q.shape, 62, BF), normal(k.shape, 63, BF)
    want, wantg = ua.qk_norm_rope_fwd(q, k, wq, wk, pos=pos), ua.qk_norm_rope_bwd(q, k, wq, wk, dq, dk, pos=pos)
    shape = ua.ua_qk_shape(2, 37, 4, 2, 128, 0, 0, 0, EPS, THETA, ua.UA_BF16)
    ws = torch.empty(ua.qk_norm_rope_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        r = ua.qk_norm_rope_fwd(q, k, wq, wk, pos=pos)
        g = ua.qk_norm_rope_bwd(q, k, wq, wk, dq, dk, pos=pos, ws=ws)
    for _ in range(2):
        for t in (*r.values(), *g.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(r[n], want[n])
        for n in wantg:
            assert torch.equal(g[n], wantg[n])


def test_in_front_of_universal_attention():
    """Learned gains around a Universal Attention layer, rotation off (the layer rotates by itself): unit
    gains give the layer's own query norm, and the chain's gain gradient matches differences of the chain."""
    B, T, H, Hkv, d = 1, 96, 4, 2, 64
    q, k = normal((B, T, H, d), 71, F), normal((B, T, Hkv, d), 72, F)
    v, gt = normal((B, T, Hkv, d), 73, F), normal((B, T, H, d), 74, F)
    aq, ak = normal((B, T, Hkv), 75, F) - 2, normal((B, T, Hkv), 76, F) - 2
    alpha, beta = torch.full((Hkv,), 3.0, device="cuda"), torch.full((Hkv,), -2.0, device="cuda")
    one = torch.ones(d, device="cuda")
    n = ua.qk_norm_rope_fwd(q, None, one, theta=0.0)["q"]
    a = ua.prefill_fwd(n, k, v, gt, aq, ak, alpha, beta)
    b = ua.prefill_fwd(q, k, v, gt, aq, ak, alpha, beta, variant=ua.VAR_QUERY_NORM)
    torch.testing.assert_close(a["o"], b["o"], rtol=1e-4, atol=1e-5)
    w = 1 + 0.3 * normal((d,), 77, F)
    do = normal((B, T, H, d), 78, F)

    def loss(w):
        n = ua.qk_norm_rope_fwd(q, None, w, theta=0.0)["q"]
        r = ua.prefill_fwd(n, k, v, gt, aq, ak, alpha, beta)
        return n, r, float((r["o"].double() * do.double()).sum())

    n, r, _ = loss(w)
    gr = ua.prefill_bwd(n, k, v, gt, aq, ak, alpha, beta, r["o"], r["lse"], r["b_final"], do)
    dw = ua.qk_norm_rope_bwd(q, None, w, None, gr["dq"], None, theta=0.0)["dwq"]
    u = normal((d,), 79, F)
    h = 2.0 ** -7                                    # fp32 chain: the loss is a sum of 24576 terms each off by ~2^-22
    diff = (loss(w + h * u)[2] - loss(w - h * u)[2]) / (2 * h)
    want = float((dw.double() * u.double()).sum())
    # h^2 of the third derivative (the logits' scale is 1/8: below 1e-2 of the slope) and 2^-22 sqrt(24576) / h = 5e-3
    assert abs(diff - want) <= 2e-2 * (1 + abs(want)) * 2, (diff, want)
    assert ua.get_device_status() == 0
