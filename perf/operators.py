"""Measured cases of the softmax-layer operators: the per-head norm of queries and keys with the
position rotation (forward, backward), the append to the 8-bit cache, and attention over that cache.

`run` computes them in elementary torch operations, or, where `own` is true, through the calls of
`kv_cache_compression_ua_b200.ua`.
"""
import math

import torch

own = False

BLOCK = 64          # slots that share one scale
RING = 128          # rows a sequence and head keep in the activation type
EPS = 1e-6
THETA = 500000.0
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
ACT_BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------- cases
def _norm(name, op, B, T, H, Hkv, d, dt, rope, packed):
    c = {"op": op, "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "dt": dt, "rope": rope, "packed": packed}
    return {"name": name, **c} if name else c


def _append(name, B, T, H, Hkv, d, dt, fmt, page, cap, fill, short):
    c = {"op": "append", "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "dt": dt, "fmt": fmt, "page": page,
         "cap": cap, "fill": fill, "short": short}
    return {"name": name, **c} if name else c


def _attend(name, B, T, H, Hkv, d, dt, fmt, page, n, ragged, bias, gate):
    c = {"op": "attend", "B": B, "T": T, "H": H, "Hkv": Hkv, "d": d, "dt": dt, "fmt": fmt, "page": page,
         "n": n, "ragged": ragged, "bias": bias, "gate": gate}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the 3B layer's training shape: every layer's queries and keys, once forward and once backward
        _norm("norm_rope_fwd_3b", "fwd", 4, 8192, 24, 8, 128, "bf16", True, False),
        _norm("norm_rope_bwd_3b", "bwd", 4, 8192, 24, 8, 128, "bf16", True, False),
        # a short odd batch in fp32, queries and keys still inside the fused projection's output
        _norm("norm_rope_fwd_f32_packed", "fwd", 3, 517, 6, 2, 64, "f32", True, True),
        # in front of a Universal Attention layer of the 1B shape, which rotates by itself
        _norm("norm_bwd_f32_1b", "bwd", 2, 2047, 32, 8, 64, "f32", False, False),
        # one decode step of the 1B shape: a token for each of 32 sequences, pages of 128 slots
        _append("append_token_1b", 32, 1, 32, 8, 64, "bf16", "e4m3", 128, 16512, 16000, False),
        # the prompts of a 1B batch, ragged, into empty caches
        _append("append_prompt_1b", 8, 4096, 32, 8, 64, "bf16", "e4m3", 0, 4160, 0, True),
        # the next chunk of long prompts of the 3B shape, padded to the longest, paged
        _append("append_chunk_3b", 4, 1003, 24, 8, 128, "bf16", "e4m3", 256, 9216, 6400, True),
        # one short conversation: latency
        _attend("attend_token_short", 1, 1, 32, 8, 64, "bf16", "e4m3", 0, 333, False, False, False),
        # the decode workload of the 1B shape: 32 ragged sequences of about 16k tokens
        _attend("attend_token_1b_16k", 32, 1, 32, 8, 64, "bf16", "int8", 0, 16384, True, False, False),
        # the 3B shape at its training length, with a forget-gate bias for each slot and the output gate
        _attend("attend_token_3b_bias", 4, 1, 24, 8, 128, "bf16", "e4m3", 128, 8192, True, True, True),
        # one very long document, pages of 256 slots
        _attend("attend_token_long", 1, 1, 32, 8, 128, "bf16", "e4m3", 256, 262144, False, False, False),
        # drafts of four tokens to verify, in fp32
        _attend("attend_draft_f32", 5, 4, 24, 8, 64, "f32", "int8", 0, 3001, True, False, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "append", "attend", "attend"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    dt = rng.choice(["bf16", "bf16", "f32"])
    B = _log(rng, 1, 32)
    most = 4 * 8192 * 32 * 128                      # elements of the largest listed norm
    if op in ("fwd", "bwd"):
        T = _log(rng, 1, max(1, min(16384, most // (2 * B * (H + Hkv) * d))))
        return _norm(None, op, B, T, H, Hkv, d, dt, rng.random() < 0.75, rng.random() < 0.3)
    page = rng.choice([0, 128, 256, 1024])
    if op == "append":
        # a step of a few tokens at any place, or a chunk that starts on a block's border
        few = rng.random() < 0.5
        T = rng.randint(1, 16) if few else _log(rng, 64, max(64, min(8192, most // (4 * B * (H + 2 * Hkv) * d))))
        fill = rng.randint(0, 4000) if few else 64 * rng.randint(0, 60)
        cap = 1024 * -(-(fill + T) // 1024)
        return _append(None, B, T, H, Hkv, d, "bf16", "e4m3", page, cap, fill, rng.random() < 0.5)
    T = rng.choice([1, 1, 1, 2, 3, 5, 8])
    n = _log(rng, 1, max(64, min(262144, 32 * 16384 * 8 * 64 // (2 * B * Hkv * d))))
    n = max(n, T)
    return _attend(None, B, T, H, Hkv, d, dt, rng.choice(["int8", "e4m3"]), page, n, rng.random() < 0.7,
                   rng.random() < 0.3, rng.random() < 0.3)


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * (seed + 1))
    return g


def _normal(g, shape, dt):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)


def _ints(g, lo, hi, n):
    """n whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda").to(torch.int32)


def _pages(g, B, page, cap):
    """Pages of the pool in a shuffled order: [B, cap / page], with a few pages to spare."""
    per = -(-cap // page)
    order = torch.randperm(B * per + 3, generator=g, device="cuda")
    return order[:B * per].to(torch.int32).reshape(B, per), B * per + 3


def _store(g, c, cap):
    """An empty cache's tensors: pages [P, Hkv, page, d] and what belongs to them."""
    B, Hkv, d, act = c["B"], c["Hkv"], c["d"], DT[c["dt"]]
    if c["page"]:
        table, pool = _pages(g, B, c["page"], cap)
        page = c["page"]
    else:
        table, pool, page = None, B, cap
    kw = dict(device="cuda")
    s = {"page": page, "table": table, "pool": pool, "cap": table.shape[1] * page if table is not None else cap}
    for x in ("k", "v"):
        s[x + "c"] = torch.zeros(pool, Hkv, page, d, dtype=torch.uint8, **kw).view(CODE[c["fmt"]])
        s[x + "s"] = torch.zeros(pool, Hkv, page // BLOCK, dtype=torch.float32, **kw)
        s[x + "t"] = torch.zeros(B, Hkv, RING, d, dtype=act, **kw)
    return s


def _encode(x, fmt):
    """Blocks [..., 64, d] -> codes and one scale a block."""
    amax = x.float().abs().amax((-2, -1))
    if fmt == "int8":
        s = amax / 127.0
        y = x.float() / torch.where(s > 0, s, 1.0)[..., None, None]
        return torch.round(y).clamp(-127, 127).to(torch.int8), s
    m, e = torch.frexp(amax)                        # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
    s = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(torch.int32)), 0.0)
    y = x.float() / torch.where(s > 0, s, 1.0)[..., None, None]
    return y.to(torch.float8_e4m3fn), s


def _put(pool, at, x):
    """pool.view(bytes)[at] = x for 8-bit tensors."""
    pool.view(torch.uint8)[at] = x.view(torch.uint8)


def prepare(case, seed):
    c, g = case, _gen(seed)
    B, T, H, Hkv, d, act = c["B"], c["T"], c["H"], c["Hkv"], c["d"], DT[c["dt"]]
    st = {"case": dict(c)}
    if c["op"] in ("fwd", "bwd", "append"):
        if c.get("packed"):                          # slices of the fused projection's output
            qkv = _normal(g, (B, T, (H + 2 * Hkv) * d), act)
            st["q"] = qkv[..., :H * d].unflatten(-1, (H, d))
            st["k"] = qkv[..., H * d:(H + Hkv) * d].unflatten(-1, (Hkv, d))
        else:
            st["q"], st["k"] = _normal(g, (B, T, H, d), act), _normal(g, (B, T, Hkv, d), act)
        st["wq"] = 1 + 0.2 * _normal(g, (d,), torch.float32)
        st["wk"] = 1 + 0.2 * _normal(g, (d,), torch.float32)
    if c["op"] in ("fwd", "bwd"):
        # several documents packed into a row: positions start anew
        first = _ints(g, 0, max(0, T - 1), B)[:, None]
        t = torch.arange(T, device="cuda", dtype=torch.int32)[None]
        st["pos"] = torch.where(t < first, t, t - first).to(torch.int32).contiguous()
        if c["op"] == "bwd":
            st["dq"], st["dk"] = _normal(g, (B, T, H, d), act), _normal(g, (B, T, Hkv, d), act)
        return st
    if c["op"] == "append":
        st["v"] = _normal(g, (B, T, Hkv, d), act)
        st |= _store(g, c, c["cap"])
        few = T < BLOCK
        if few:                                      # a step at any place of the sequence
            start = torch.clamp(c["fill"] - _ints(g, 0, min(c["fill"], 500), B), min=0)
        else:                                        # a chunk on a block's border
            start = torch.clamp(c["fill"] - BLOCK * _ints(g, 0, 8, B), min=0)
        st["start"] = start.to(torch.int32)
        st["n_new"] = _ints(g, max(1, T // 2), T, B) if c["short"] else torch.full((B,), T, dtype=torch.int32, device="cuda")
        st["kt"].copy_(_normal(g, st["kt"].shape, act))
        st["vt"].copy_(_normal(g, st["vt"].shape, act))
        st["pos"] = (st["start"][:, None] + torch.arange(T, device="cuda", dtype=torch.int32)[None]).to(torch.int32).contiguous()
        st["n"] = st["start"].clone()
        n_own = st["start"].clone()
    else:
        n_own = _attend_inputs(st, c, g)
    if own:
        from kv_cache_compression_ua_b200 import ua
        st["cache"] = ua.KVQCache(B, Hkv, d, st["cap"], act, st["kc"], st["vc"], st["ks"], st["vs"], st["kt"], st["vt"],
                                  n_own, page_table=st["table"])
        if c["op"] == "attend":
            st["ws"] = ua.alloc_workspace(ua.kvq_attend_workspace_size(st["cache"], H, T), "cuda")
    return st


def _attend_inputs(st, c, g):
    B, T, H, Hkv, d, act = c["B"], c["T"], c["H"], c["Hkv"], c["d"], DT[c["dt"]]
    unit = max(BLOCK, c["page"])
    st |= _store(g, c, unit * -(-c["n"] // unit))
    n = torch.full((B,), c["n"], dtype=torch.int32, device="cuda")
    if c["ragged"]:
        n = torch.clamp(n - _ints(g, 0, c["n"] // 3, B), min=T).to(torch.int32)
        n[0] = c["n"]
    st["n"] = n
    st["q"] = _normal(g, (B, T, H, d), act)
    for x in ("k", "v"):                             # keys and values of each page, a page's heads at their own size
        size = 0.5 + torch.rand(Hkv, generator=g, device="cuda")
        for i in range(0, st["pool"], max(1, (1 << 26) // (Hkv * st["page"] * d))):
            part = st[x + "c"][i:i + max(1, (1 << 26) // (Hkv * st["page"] * d))]
            y = torch.randn(part.shape, generator=g, device="cuda") * size[:, None, None]
            code, s = _encode(y.unflatten(2, (-1, BLOCK)), c["fmt"])
            _put(part, slice(None), code.flatten(2, 3))
            st[x + "s"][i:i + part.shape[0]] = s
        st[x + "t"].copy_(torch.randn(st[x + "t"].shape, generator=g, device="cuda") * size[:, None, None])
    st["bias"] = None
    if c["bias"]:                                    # log of a forget gate, summed from the end; some slots masked out
        f = -0.01 * torch.rand(B, Hkv, st["cap"], generator=g, device="cuda")
        b = f.flip(-1).cumsum(-1).flip(-1)
        b[torch.rand(b.shape, generator=g, device="cuda") < 0.05] = -math.inf
        st["bias"] = b.contiguous()
    st["gate"] = _normal(g, (B, T, H, d), act) if c["gate"] else None
    return n


# --------------------------------------------------------------------------------- plain forms
def _rotation(pos, d):
    f = THETA ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    a = pos.double()[..., None] * f                  # angles of far positions: 64 bits
    return a.cos().float()[..., None, :], a.sin().float()[..., None, :]


def _rot(x, cs, back=False):
    (c, s), (a, b) = cs, x.chunk(2, -1)
    s = -s if back else s
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _norm_rope(x, w, cs):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return y if cs is None else _rot(y, cs)


def _norm_rope_bwd(x, w, dy, cs):
    x, dy = x.float(), dy.float()
    g = dy if cs is None else _rot(dy, cs, back=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dn = g * w
    return r * (dn - xh * (dn * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1, 2), dtype=torch.float64).float()


def _run_append(st):
    c = st["case"]
    B, T, act, dev = c["B"], c["T"], DT[c["dt"]], "cuda"
    cs = _rotation(st["pos"], c["d"])
    q = _norm_rope(st["q"], st["wq"], cs).to(act)
    new = {"k": _norm_rope(st["k"], st["wk"], cs).to(act), "v": st["v"]}
    start, end = st["start"].long(), (st["start"] + st["n_new"]).long()
    j0 = start // BLOCK
    nb = (T + 2 * BLOCK - 2) // BLOCK                # blocks a call can touch
    r = torch.arange(nb * BLOCK, device=dev)[None]   # rows of the window that starts at block j0
    t = r - (start % BLOCK)[:, None]
    is_new = (t >= 0) & (t < st["n_new"][:, None])
    bi = torch.arange(B, device=dev)[:, None]
    slot = j0[:, None] * BLOCK + r
    done = (j0[:, None] + torch.arange(nb, device=dev)[None] + 1) * BLOCK <= end[:, None]
    b, j = done.nonzero(as_tuple=True)
    blk = j0[b] + j
    per = st["page"] // BLOCK
    page = st["table"][b, blk // per].long() if st["table"] is not None else b
    tb, tt = (((torch.arange(T, device=dev)[None] < st["n_new"][:, None])
               & ((start[:, None] + torch.arange(T, device=dev)[None]) // BLOCK >= (end // BLOCK - 1)[:, None]))
              .nonzero(as_tuple=True))
    ring = (start[tb] + tt) % RING
    for x in ("k", "v"):
        win = torch.where(is_new[..., None, None], new[x][bi, t.clamp(0, T - 1)], st[x + "t"].transpose(1, 2)[bi, slot % RING])
        code, s = _encode(win.unflatten(1, (nb, BLOCK))[b, j].transpose(1, 2), c["fmt"])
        _put(st[x + "c"].unflatten(2, (per, BLOCK)), (page, slice(None), blk % per), code)
        st[x + "s"][page, :, blk % per] = s
        st[x + "t"][tb, :, ring] = new[x][tb, tt]
    st["n"].copy_(end)
    return {"q": q, "k": st["kc"], "v": st["vc"], "kscale": st["ks"], "vscale": st["vs"], "ktail": st["kt"],
            "vtail": st["vt"], "n": st["n"]}


def _slots(st, x, N):
    """The first N slots of every sequence in 32 bits, [B, Hkv, N, d]."""
    c = st["case"]
    pool = st[x + "c"].float() * st[x + "s"].repeat_interleave(BLOCK, -1)[..., None]
    if st["table"] is not None:
        pool = pool[st["table"].long()].transpose(1, 2).flatten(2, 3)
    y = pool[:, :, :N]
    j = torch.arange(N, device="cuda")
    tail = st[x + "t"].float()[:, :, j % RING]
    late = j[None] >= (st["n"].long() // BLOCK * BLOCK)[:, None]
    return torch.where(late[:, None, :, None], tail, y) if c["n"] % BLOCK or c["ragged"] else y


def _run_attend(st):
    c = st["case"]
    B, T, H, Hkv, d, N = c["B"], c["T"], c["H"], c["Hkv"], c["d"], c["n"]
    G = H // Hkv
    q = st["q"].float().view(B, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, d)
    x = q @ _slots(st, "k", N).transpose(-1, -2) * d ** -0.5
    if st["bias"] is not None:
        x = x + st["bias"][:, :, None, :N]
    j = torch.arange(N, device="cuda")
    last = st["n"].long()[:, None] - T + torch.arange(T, device="cuda")[None]       # [B, T]
    x = x.view(B, Hkv, G, T, N).masked_fill(j > last[:, None, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, G * T, N) @ _slots(st, "v", N)
    o = o.view(B, Hkv, G, T, d) / torch.where(z > 0, z, 1.0)
    lse = (m + torch.log(z))[..., 0].reshape(B, H, T)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, H, d)
    if st["gate"] is not None:
        o = o * torch.sigmoid(st["gate"].float())
    return {"o": o.to(DT[c["dt"]]), "lse": lse}


def run(st):
    c = st["case"]
    op, act = c["op"], DT[c["dt"]]
    if own:
        from kv_cache_compression_ua_b200 import ua
        theta = THETA if c.get("rope", True) else 0.0
        if op == "fwd":
            return ua.qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], pos=st["pos"], eps=EPS, theta=theta)
        if op == "bwd":
            return ua.qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["dq"], st["dk"], pos=st["pos"], eps=EPS,
                                       theta=theta)
        if op == "append":
            q = ua.kvq_append(st["cache"], st["k"], st["v"], st["q"], wq=st["wq"], wk=st["wk"], pos=st["pos"],
                              n_new=st["n_new"], start=st["start"], eps=EPS, theta=THETA)
            return {"q": q, "k": st["kc"], "v": st["vc"], "kscale": st["ks"], "vscale": st["vs"], "ktail": st["kt"],
                    "vtail": st["vt"], "n": st["cache"].n_kept}
        lse = torch.empty(c["B"], c["H"], c["T"], dtype=torch.float32, device="cuda")
        o = ua.kvq_attend(st["cache"], st["q"], g=st["gate"], bias=st["bias"], lse=lse, ws=st["ws"])
        return {"o": o, "lse": lse}
    if op == "append":
        return _run_append(st)
    if op == "attend":
        return _run_attend(st)
    cs = _rotation(st["pos"], c["d"]) if c["rope"] else None
    if op == "fwd":
        return {"q": _norm_rope(st["q"], st["wq"], cs).to(act), "k": _norm_rope(st["k"], st["wk"], cs).to(act)}
    dq, dwq = _norm_rope_bwd(st["q"], st["wq"], st["dq"], cs)
    dk, dwk = _norm_rope_bwd(st["k"], st["wk"], st["dk"], cs)
    return {"dq": dq.to(act), "dk": dk.to(act), "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------------------------------- work
def work(case):
    c = case
    B, T, H, Hkv, d, e = c["B"], c["T"], c["H"], c["Hkv"], c["d"], ACT_BYTES[c["dt"]]
    rows = B * T
    if c["op"] in ("fwd", "bwd"):
        x = rows * (H + Hkv) * d
        return {"bytes": x * e * (2 if c["op"] == "fwd" else 3) + rows * 4 + 2 * d * 4, "flops": x * (7 if c["op"] == "fwd" else 16)}
    if c["op"] == "append":
        rows = rows * (0.75 if c["short"] else 1.0)
        held = 1 if T >= BLOCK else e                # a chunk's blocks end up in codes, a step's rows in the ring
        # queries are rotated for padded rows too
        return {"bytes": B * T * H * d * e * 2 + rows * Hkv * d * 2 * (e + held), "flops": (B * T * H + 2 * rows * Hkv) * d * 7}
    n = B * c["n"] * (5 / 6 if c["ragged"] else 1.0)
    byte = n * Hkv * (2 * d + 8 / BLOCK + (4 if c["bias"] else 0)) + B * T * H * d * e * (3 if c["gate"] else 2)
    return {"bytes": byte, "flops": 4 * n * T * H * d}


# --------------------------------------------------------------------------------------- exact
def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    d, half = c["d"], c["d"] // 2
    if c["op"] in ("fwd", "bwd"):
        # the rotation as a product of complex numbers: component m is the real part, m + d/2 the imaginary one
        turn = None
        if c["rope"]:
            f = torch.exp(torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 * math.log(THETA) / d))
            a = st["pos"].to(torch.float64)[:, :, None, None] * f
            turn = torch.polar(torch.ones_like(a), a)

        def turned(y, by):
            z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * by
            return torch.cat([z.real, z.imag], -1)

        res = {}
        for x, w in (("q", "wq"), ("k", "wk")):
            v, gain = st[x].double(), st[w].double()
            size = (v.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            if c["op"] == "fwd":
                y = v / size * gain
                res[x] = y if turn is None else turned(y, turn)
                continue
            dy = st["d" + x].double()
            dy = dy if turn is None else turned(dy, turn.conj())
            res["dw" + x] = (dy * (v / size)).flatten(0, 2).sum(0)
            h = dy * gain
            res["d" + x] = h / size - v * (h * v).sum(-1, keepdim=True) / (d * size.pow(3))
        return res
    if c["op"] == "append":
        # what is encoded has no exact value of its own: the rotated queries do
        f = torch.exp(torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 * math.log(THETA) / d))
        a = st["pos"].to(torch.float64)[:, :, None, None] * f
        v = st["q"].double()
        y = v / (v.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * st["wq"].double()
        z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * torch.polar(torch.ones_like(a), a)
        return {"q": torch.cat([z.real, z.imag], -1), "k": None, "v": None, "kscale": None, "vscale": None, "ktail": None,
                "vtail": None, "n": None}
    B, T, H, Hkv = c["B"], c["T"], c["H"], c["Hkv"]
    G, per = H // Hkv, st["page"]
    o = torch.zeros(B, T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["n"].tolist()):
        full = n - n % BLOCK
        pages = range(b, b + 1) if st["table"] is None else st["table"][b].tolist()
        for h in range(Hkv):
            kv = []
            for x in ("k", "v"):
                rows = [(st[x + "c"][pg, h].to(torch.float32).double().view(-1, BLOCK, d) * st[x + "s"][pg, h].double()[:, None, None])
                        .reshape(-1, d) for pg in list(pages)[:-(-full // per)]]
                rows = torch.cat(rows)[:full] if rows else torch.zeros(0, d, dtype=torch.float64, device="cuda")
                at = [s % RING for s in range(full, n)]
                kv.append(torch.cat([rows, st[x + "t"][b, h, at].double()]) if at else rows)
            for i in range(T):
                see = n - T + i + 1
                x = (st["q"][b, i, h * G:(h + 1) * G].double() @ kv[0][:see].T) / math.sqrt(d)
                if st["bias"] is not None:
                    x = x + st["bias"][b, h, :see].double()
                lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, -1)
                w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
                o[b, i, h * G:(h + 1) * G] = w @ kv[1][:see]
    if st["gate"] is not None:
        o = o / (1 + torch.exp(-st["gate"].double()))
    return {"o": o, "lse": lse}
