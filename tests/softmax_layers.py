"""Plain 64-bit forms of the softmax-layer operators on the CPU, and their error bounds (shared by
the tests; nothing here uses the library's arithmetic)."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24                                    # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BLOCK, RING = 64, 128
THETA = 500000.0


def d64(t):
    return t.detach().cpu().to(torch.float32).double() if t.dtype != torch.float64 else t.detach().cpu()


def angles(pos, d, theta):
    f = theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)
    return d64(pos)[..., None, None] * f            # [B, T, 1, d/2]


def rotate(x, a, back=False):
    h = x.shape[-1] // 2
    c, s = torch.cos(a), torch.sin(a) * (-1 if back else 1)
    return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)


def pair_size(y):
    """|(y_m, y_{m+d/2})| for each element: what a rotation's rounding errors are relative to."""
    h = y.shape[-1] // 2
    m = torch.hypot(y[..., :h], y[..., h:])
    return torch.cat([m, m], -1)


def norm_rope(x, w, pos, eps, theta):
    """(result, absolute error bound before the final rounding).  Bound: the mean square's sum (19
    additions, halved by the root), rsqrtf (2 ulp), two products, the angle (1.6), sincospif (2 ulp) and the
    rotation (3 roundings) come to 22 half steps of the pair's size; 32 are allowed."""
    y = d64(x)
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * d64(w)
    if theta:
        y = rotate(y, angles(pos, y.shape[-1], theta))
    return y, 32 * U32 * pair_size(y)


def norm_rope_bwd(x, w, dy, pos, eps, theta):
    """dx, its bound, dw, its bound.  dx: 64 half steps of the terms' sizes (the row sums' 20 additions
    twice, the products and the rotation).  dw: each term as above, and the additions: at most 8 of a
    lane's terms in a row of 64, 64 rows, then 37 + 16 partial sums -- the sizes here -- below 400."""
    g = d64(dy)
    if theta:
        g = rotate(g, angles(pos, g.shape[-1], theta), back=True)
    if w is None:
        return g, 32 * U32 * pair_size(g), None, None
    x, w = d64(x), d64(w)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh, n = x * r, g * w
    dx = r * (n - xh * (n * xh).mean(-1, keepdim=True))
    size = r * (pair_size(g) * w.abs() + xh.abs() * (pair_size(g) * w.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, 64 * U32 * size, (g * xh).sum((0, 1, 2)), 400 * U32 * (pair_size(g) * xh.abs()).sum((0, 1, 2))


def within(name, got, ref, bound, dtype):
    """|got - ref| <= bound + half a step of the output's type (relative to the value; below the normal
    numbers absolute)."""
    got = d64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{name}: NaN in other places"
    ok = (got - ref).abs() <= bound + HALF[dtype] * (ref.abs() + bound) + 2.0 ** -126
    ok |= torch.isnan(ref) | (got == ref)
    bad = (~ok).nonzero()
    assert not len(bad), f"{name}: {len(bad)} of {ok.numel()} off, first at {bad[0].tolist()}: " \
        f"{got[tuple(bad[0])]} against {ref[tuple(bad[0])]}, bound {bound.expand_as(ref)[tuple(bad[0])]}"


def encode(rows, fmt):
    """A block [64, d] in the activation type -> (codes, scale), as the header defines them (in fp32)."""
    x = rows.detach().cpu().float()
    amax = x.abs().max()
    if not torch.isfinite(x).all():
        return torch.zeros(x.shape, dtype=torch.uint8), torch.tensor(math.nan)
    if amax < 2.0 ** -100:
        return torch.zeros(x.shape, dtype=torch.uint8), torch.tensor(0.0)
    if fmt == torch.int8:
        s = amax / 127.0
        return torch.round(x * torch.div(torch.tensor(127.0), amax)).to(torch.int8).view(torch.uint8), s
    e = -200
    while float(amax) / 2.0 ** e > 448.0:
        e += 1
    s = torch.tensor(2.0 ** e)
    return (x / s).to(torch.float8_e4m3fn).view(torch.uint8), s


def fill_random(cache, seed, scale=1.0):
    """Random codes, scales and ring rows in an existing cache, as an append would leave them: finite
    codes, positive scales (power-of-two ones for e4m3)."""
    g = torch.Generator(device=cache.k.device)
    g.manual_seed(seed)
    for codes, sc, ring in ((cache.k, cache.k_scale, cache.k_ring), (cache.v, cache.v_scale, cache.v_ring)):
        x = torch.randn(codes.shape, generator=g, device=codes.device)
        if codes.dtype == torch.int8:
            codes.copy_(torch.round(x * 40).clamp(-127, 127).to(torch.int8))
            sc.copy_(scale * (0.5 + torch.rand(sc.shape, generator=g, device=codes.device)) / 40)
        else:
            codes.view(torch.uint8).copy_((x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            sc.copy_(scale * 2.0 ** torch.randint(-8, -5, sc.shape, generator=g, device=codes.device).float())
        ring.copy_((scale * torch.randn(ring.shape, generator=g, device=codes.device)).to(ring.dtype))


def rows_of(cache, which, b, h, n):
    """The first n slots of sequence b, head h, in 64 bits."""
    codes, sc, ring = ((cache.k, cache.k_scale, cache.k_ring) if which == "k" else (cache.v, cache.v_scale, cache.v_ring))
    ps, out = cache.page_size, []
    for blk in range(n // BLOCK):
        pg = b if cache.page_table is None else int(cache.page_table[b, blk * BLOCK // ps])
        at = blk * BLOCK % ps
        out.append(d64(codes[pg, h, at:at + BLOCK]) * d64(sc[pg, h, at // BLOCK]))
    left = [j % RING for j in range(n // BLOCK * BLOCK, n)]
    out.append(d64(ring[b, h][left]))
    return torch.cat(out)


def offsets_of(cache, which, b, h, n):
    """[n, 1]: 128 scales of an int8 slot of a bf16 cache: its products are formed with code + 128, so the rounding of
    their sums is relative to |value| + 128 scales.  0 for e4m3, for fp32 and for rows in the ring."""
    out = torch.zeros(n, 1, dtype=torch.float64)
    if cache.k.dtype == torch.int8 and cache.dtype == torch.bfloat16:
        sc = cache.k_scale if which == "k" else cache.v_scale
        for blk in range(n // BLOCK):
            pg = b if cache.page_table is None else int(cache.page_table[b, blk * BLOCK // cache.page_size])
            out[blk * BLOCK:(blk + 1) * BLOCK] = 128 * d64(sc[pg, h, blk * BLOCK % cache.page_size // BLOCK])
    return out


def attend(cache, q, n, *, g=None, bias=None, n_q=None, scale=None):
    """o [B,Tq,H,d], its bound, lse [B,H,Tq], its bound, and the rows that are written [B,Tq].

    Bounds: a logit's products are exact, their fp32 sum and the scaling lose (d + 8) half steps of
    sum |q||k| (fp32 queries and keys of three bf16 parts: 2^-22 of it more), the bias 4 of its size and the
    logit's.  A logit off by e moves every probability by a factor within e; probabilities are f16 (2^-11) or,
    for fp32, two f16 parts (2^-22), exp2 is off by 2^-22 and its argument's rounding by 2^-23 |x - m|,
    the sums by the number of their terms in a lane: 64 half steps + 20 for each merge.  The weighted values'
    sums round 4 times a block and once for the offset, by up to a whole step of |value| + offset: 24 half steps
    (the offset: see offsets_of)."""
    B, Tq, H, d = q.shape
    Hkv = cache.Hkv
    G = H // Hkv
    f32 = q.dtype == torch.float32
    scale = d ** -0.5 if scale is None else scale
    o, ob = torch.zeros(B, Tq, H, d, dtype=torch.float64), torch.zeros(B, Tq, H, d, dtype=torch.float64)
    lse, lb = torch.full((B, H, Tq), -math.inf, dtype=torch.float64), torch.zeros(B, H, Tq, dtype=torch.float64)
    written = torch.zeros(B, Tq, dtype=torch.bool)
    for b in range(B):
        nb, nq = int(n[b]), Tq if n_q is None else int(n_q[b])
        written[b, :nq] = True
        for h in range(Hkv):
            k, v = rows_of(cache, "k", b, h, nb), rows_of(cache, "v", b, h, nb)
            ka, va = k.abs() + offsets_of(cache, "k", b, h, nb), v.abs() + offsets_of(cache, "v", b, h, nb)
            bs = d64(bias[b, h, :nb]) if bias is not None else torch.zeros(nb, dtype=torch.float64)
            for i in range(nq):
                see = max(0, nb - nq + i + 1)
                keep = (torch.arange(nb) < see) & (bs != -math.inf)
                if not keep.any():
                    continue
                kk, vv, bb = k[keep], v[keep], bs[keep]
                ka_, va_ = ka[keep], va[keep]
                x0 = scale * d64(q[b, i, h * G:(h + 1) * G]) @ kk.T
                x = x0 + bb
                mag = abs(scale) * d64(q[b, i, h * G:(h + 1) * G]).abs() @ ka_.T
                ex = (d + 8) * U32 * mag + (2.0 ** -21 * mag if f32 else 0) + 4 * U32 * (bb.abs() + x.abs())
                m = x.max(-1, keepdim=True).values
                p = torch.exp(x - m)
                z = p.sum(-1, keepdim=True)
                p = p / z
                each = ex + 2.0 ** -22 + 2.0 ** -23 * (m - x) * 1.5 + 160 * U32
                zerr = (p * each).sum(-1, keepdim=True)
                perr = each + (2.0 ** -21 if f32 else 2.0 ** -11)
                hs = slice(h * G, (h + 1) * G)
                o[b, i, hs] = p @ vv
                ob[b, i, hs] = (p * perr) @ vv.abs() + zerr * (p @ vv.abs()) + 24 * U32 * (p @ va_)
                lse[b, hs, i] = (m + torch.log(z))[:, 0]
                lb[b, hs, i] = zerr[:, 0] + 8 * U32 * (1 + m[:, 0].abs() + torch.log(z)[:, 0].abs())
    if g is not None:
        s = torch.sigmoid(d64(g))
        o, ob = o * s, ob * s + 16 * U32 * (o * s).abs()
    return o, ob, lse, lb, written


def check_attend(cache, q, n, got, got_lse, **kw):
    o, ob, lse, lb, written = attend(cache, q, n, **kw)
    w = written[:, :, None, None].expand_as(o)
    within("o", torch.where(w, d64(got), 0.0), torch.where(w, o, 0.0), torch.where(w, ob, 0.0), q.dtype)
    if got_lse is not None:
        wl = written[:, None, :].expand_as(lse)
        a, r = torch.where(wl, d64(got_lse), 0.0), torch.where(wl, lse, 0.0)
        assert torch.equal(torch.isinf(a), torch.isinf(r)), "lse: infinities in other places"
        fin = torch.isfinite(r)
        assert ((a - r).abs()[fin] <= lb[fin]).all(), float(((a - r).abs()[fin] / lb[fin].clamp(min=1e-30)).max())


def normal(shape, seed, dtype, device="cuda", scale=1.0):
    g = np.random.default_rng(seed)
    return (torch.from_numpy(g.standard_normal(shape)) * scale).to(torch.float32).to(dtype).to(device)
