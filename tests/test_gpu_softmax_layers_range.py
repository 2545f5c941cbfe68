"""GPU tests of the softmax-layer operators at the ends of the magnitudes that the header states."""
import pytest
import torch

from kv_cache_compression_ua_b200 import ua
from softmax_layers import THETA, check_attend, norm_rope, norm_rope_bwd, normal, within
from test_gpu_kvq_attend import filled, run
from test_gpu_kvq_cache import make

pytestmark = pytest.mark.gpu
BF, F, I8, E4 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
EPS = 1e-6


def up_to(x, e):
    """x scaled so that its largest magnitude is 2^e."""
    return (x.float() * (2.0 ** e / float(x.float().abs().max()))).to(x.dtype)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("d", [64, 128])
def test_heads_up_to_2_to_the_60(dt, d):
    x, dy, w = up_to(normal((2, 30, 3, d), 1, dt), 60), normal((2, 30, 3, d), 2, dt), 1 + 0.3 * normal((d,), 3, F)
    x[0, 0] = 2.0 ** 60                              # every element: the largest sum of squares
    pos = torch.arange(30, dtype=torch.int32).repeat(2, 1)
    ref, bound = norm_rope(x, w, pos, EPS, THETA)
    within("y", ua.qk_norm_rope_fwd(x, None, w, eps=EPS)["q"], ref, bound, dt)
    dx, b, dw, bw = norm_rope_bwd(x, w, dy, pos, EPS, THETA)
    g = ua.qk_norm_rope_bwd(x, None, w, None, dy, None, eps=EPS)
    within("dx", g["dq"], dx, b, dt)
    within("dw", g["dwq"], dw, bw, F)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("fmt", [I8, E4])
@pytest.mark.parametrize("e", [80, -80])
def test_values_up_to_2_to_the_80(dt, fmt, e):
    """5000 slots and an unfinished block of values of that size, weighed alike: the sums are the largest there are."""
    N, d = 5000, 64
    k, v = normal((1, N, 2, d), 4, dt), up_to(normal((1, N, 2, d), 5, dt).abs(), e)
    q = normal((1, 2, 4, d), 6, dt, scale=0.01)
    c = make(1, 2, d, 5056, fmt, dt)
    ua.kvq_append(c, k, v, theta=0.0)
    o, lse = run(c, q)
    check_attend(c, q, [N], o, lse)
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("dt", [BF, F])
def test_queries_and_keys_far_from_one(dt):
    """Queries of 2^40 against keys of 2^-40 and the other way round: the logits are ordinary."""
    n = [200, 70]
    for e in (40, -40):
        c = filled(2, 2, 64, n, E4, dt, seed=7)
        c.k_scale.mul_(2.0 ** -e)
        c.k_ring.mul_(2.0 ** -e)
        q = normal((2, 3, 8, 64), 8, dt, scale=2.0 ** e)
        o, lse = run(c, q)
        check_attend(c, q, n, o, lse)
