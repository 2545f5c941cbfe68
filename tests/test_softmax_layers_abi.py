"""CPU checks of the softmax-layer entry points: sizes, and refusals on the host before any launch
(the pointers are never followed), and the 64-bit plain forms the GPU tests compare with."""
import ctypes

import pytest
import torch

from kv_cache_compression_ua_b200 import build as ua_build
from kv_cache_compression_ua_b200 import ua
from softmax_layers import encode, norm_rope

FAKE = 0x7f0000000000
P, S, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    ua_build.build()
    return ua.load_library()


def qk(**kw):
    s = dict(B=2, T=5, H=4, Hkv=2, d=64, q_ld=0, k_ld=0, v_ld=0, eps=1e-6, rope_theta=5e5, dtype=ua.UA_BF16)
    return ua.ua_qk_shape(**(s | kw))


def kvq(**kw):
    s = dict(B=2, Hkv=2, d=64, capacity=256, dtype=ua.UA_BF16, format=ua.UA_KVQ_E4M3, page_size=0, max_pages=0,
             pool_pages=0, page_table=None)
    s |= {n: FAKE for n in ("k", "v", "k_scale", "v_scale", "k_ring", "v_ring", "n_kept", "ring_state")}
    return ua.ua_kvq(**(s | kw))


PAGED = dict(page_size=128, max_pages=2, pool_pages=5, page_table=FAKE)


def fwd(lib, s, **kw):
    a = dict(q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, pos=FAKE, q_out=FAKE, k_out=FAKE) | kw
    return lib.ua_qk_norm_rope_fwd(ctypes.byref(s), *[P(x) for x in a.values()], None)


def bwd(lib, s, nbytes=1 << 30, **kw):
    a = dict(q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, pos=FAKE, dq_out=FAKE, dk_out=FAKE, dq=FAKE, dk=FAKE, dwq=FAKE, dwk=FAKE,
             ws=FAKE) | kw
    return lib.ua_qk_norm_rope_bwd(ctypes.byref(s), *[P(x) for x in a.values()], S(nbytes), None)


def append(lib, c, s, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, wq=FAKE, wk=FAKE, pos=FAKE, n_new=FAKE, start=FAKE, q_out=FAKE) | kw
    return lib.ua_kvq_append(ctypes.byref(c), ctypes.byref(s), *[P(x) for x in a.values()], None)


def attend(lib, c, H=4, Tq=1, scale=0.125, nbytes=1 << 30, **kw):
    a = dict(q=FAKE, g=FAKE, bias=FAKE, n_q=FAKE, o=FAKE, lse=FAKE, ws=FAKE) | kw
    v = [P(x) for x in a.values()]
    return lib.ua_kvq_attend(ctypes.byref(c), H, Tq, *v[:4], F(scale), *v[4:], S(nbytes), None)


BAD_SHAPES = [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=-1), INVALID),
              (dict(rope_theta=-1.0), INVALID), (dict(rope_theta=float("nan")), INVALID), (dict(rope_theta=float("inf")), INVALID),
              (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(d=96), UNSUPPORTED),
              (dict(dtype=7), UNSUPPORTED), (dict(q_ld=255), INVALID), (dict(k_ld=100), INVALID), (dict(v_ld=-128), INVALID),
              (dict(q_ld=257), ALIGN), (dict(k_ld=132), ALIGN), (dict(v_ld=129), ALIGN),
              (dict(H=1 << 26), UNSUPPORTED), (dict(B=1 << 20, T=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_shapes_refused(lib, kw, code):
    s = qk(**kw)
    n = S(0)
    assert fwd(lib, s) == code and bwd(lib, s) == code and append(lib, kvq(), s) == code
    assert lib.ua_qk_norm_rope_bwd_workspace_size(ctypes.byref(s), ctypes.byref(n)) == code


def test_norm_pointers_refused(lib):
    s = qk()
    assert lib.ua_qk_norm_rope_fwd(None, *[P(FAKE)] * 7, None) == INVALID
    assert fwd(lib, s, q=None, k=None, q_out=None, k_out=None) == INVALID
    for kw in (dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None)):
        assert fwd(lib, s, **kw) == INVALID
    for n in ("q", "k", "q_out", "k_out"):
        assert fwd(lib, s, **{n: FAKE + 8}) == ALIGN
    for n in ("wq", "wk", "pos"):
        assert fwd(lib, s, **{n: FAKE + 2}) == ALIGN
    for kw in (dict(q=None), dict(dq_out=None), dict(dk=None), dict(dwq=None), dict(dwk=None), dict(ws=None),
               dict(q=None, k=None)):
        assert bwd(lib, s, **kw) == INVALID
    for n in ("dq_out", "dk", "ws"):
        assert bwd(lib, s, **{n: FAKE + 8}) == ALIGN
    n = S(0)
    assert lib.ua_qk_norm_rope_bwd_workspace_size(ctypes.byref(s), ctypes.byref(n)) == OK and n.value > 0
    assert bwd(lib, s, nbytes=n.value - 1) == WORKSPACE
    assert lib.ua_qk_norm_rope_bwd_workspace_size(ctypes.byref(s), None) == INVALID


BAD_CACHES = [(dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(capacity=0), INVALID), (dict(capacity=1 << 30), INVALID),
              (dict(capacity=100), INVALID), (dict(d=80), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
              (dict(format=2), UNSUPPORTED), (dict(k=None), INVALID), (dict(ring_state=None), INVALID),
              (dict(v_ring=FAKE + 8), ALIGN), (dict(n_kept=FAKE + 4), ALIGN),
              (PAGED | dict(page_size=64, max_pages=4), INVALID), (PAGED | dict(page_size=192), INVALID),
              (PAGED | dict(max_pages=3), INVALID), (PAGED | dict(pool_pages=0), INVALID),
              (PAGED | dict(page_table=FAKE + 2), ALIGN), (PAGED | dict(page_size=1 << 21), INVALID)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_caches_refused(lib, kw, code):
    c = kvq(**kw)
    n = S(0)
    assert append(lib, c, qk()) == code and attend(lib, c) == code
    assert lib.ua_kvq_attend_workspace_size(ctypes.byref(c), 4, 1, ctypes.byref(n)) == code


def test_append_refused(lib):
    for kw in (dict(B=3), dict(Hkv=4), dict(d=128), dict(dtype=ua.UA_F32)):
        assert append(lib, kvq(), qk(**kw)) == INVALID
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(q_out=None)):
        assert append(lib, kvq(), qk(), **kw) == INVALID
    for n in ("q", "k", "v", "q_out"):
        assert append(lib, kvq(), qk(), **{n: FAKE + 4}) == ALIGN
    for n in ("wk", "pos", "n_new", "start"):
        assert append(lib, kvq(), qk(), **{n: FAKE + 1}) == ALIGN


def test_attend_refused(lib):
    c = kvq()
    for H, Tq in ((0, 1), (3, 1), (4, 0), (-4, 1), (4, -1)):
        assert attend(lib, c, H=H, Tq=Tq) == INVALID
    assert attend(lib, c, H=1 << 26) == UNSUPPORTED and attend(lib, c, Tq=1 << 30) == UNSUPPORTED
    for kw in (dict(q=None), dict(o=None), dict(ws=None), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert attend(lib, c, **kw) == INVALID
    for n in ("q", "g", "bias", "o", "ws"):
        assert attend(lib, c, **{n: FAKE + 8}) == ALIGN
    for n in ("n_q", "lse"):
        assert attend(lib, c, **{n: FAKE + 2}) == ALIGN
    n = S(0)
    assert lib.ua_kvq_attend_workspace_size(ctypes.byref(c), 4, 3, ctypes.byref(n)) == OK
    assert attend(lib, c, Tq=3, nbytes=n.value - 1) == WORKSPACE


def test_binding_refuses_before_the_library_sees_anything():
    z = torch.zeros
    with pytest.raises(ValueError):
        ua.KVQCache.empty(1, 1, 64, 128, device="cpu")           # not on a GPU
    with pytest.raises(ValueError):
        ua.KVQCache.empty(1, 1, 64, 128, fmt=torch.uint8, device="cpu")
    with pytest.raises(ValueError):
        ua.qk_norm_rope_fwd(None, None)
    with pytest.raises(ValueError):
        ua.qk_norm_rope_fwd(z(1, 2, 2, 64), None)                # not on a GPU
    with pytest.raises(ValueError):
        ua.qk_norm_rope_fwd(z(2, 2, 64), None)


def test_encoding_of_the_plain_form():
    """A worked block of each format: the scale, ties to even, the border between powers of two."""
    x = torch.zeros(64, 64)
    x[0, :6] = torch.tensor([127.0, -127.0, 2.5, 3.5, -0.5, 0.49])
    codes, s = encode(x, torch.int8)
    assert float(s) == 1.0 and codes.view(torch.int8)[0, :6].tolist() == [127, -127, 2, 4, 0, 0]
    for amax, want in ((448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (0.875, 2.0 ** -9), (1.0, 2.0 ** -8)):
        x[0, 0] = amax
        x[0, 1:] = 0
        codes, s = encode(x, torch.float8_e4m3fn)
        assert float(s) == want, (amax, s)
        # half a step at amax: codes of 257..448 are 32 apart
        assert abs(float(codes.view(torch.float8_e4m3fn)[0, 0].float() * s) - amax) <= 16 * want
    x[0, 0] = float("nan")
    assert torch.isnan(encode(x, torch.int8)[1])


def test_plain_rotation_by_hand():
    x = torch.zeros(1, 1, 1, 64)
    x[..., 0], x[..., 32] = 3.0, 4.0
    y, _ = norm_rope(x, None, torch.tensor([[1]]), 0.0, 5e5)     # frequency 1 for the first pair
    c, s = 0.5403023058681398, 0.8414709848078965
    assert abs(float(y[0, 0, 0, 0]) - (3 * c - 4 * s)) < 1e-12 and abs(float(y[0, 0, 0, 32]) - (4 * c + 3 * s)) < 1e-12
    w = torch.full((64,), 2.0)
    y, _ = norm_rope(x, w, torch.tensor([[0]]), 0.0, 0.0)        # mean square 25 / 64
    assert abs(float(y[0, 0, 0, 0]) - 2 * 3 * 8 / 5) < 1e-12
