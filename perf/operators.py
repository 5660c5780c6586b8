"""Cases of the prefix-cache operators: per-head norm and rotation of queries and
keys, the paged key-value cache (written, also in 8 bits, and read back for the
denoising loop) and attention of one new token over it.

``own`` chooses between the library's calls and the same operators written in plain
torch.  A case is a dict of plain values; its ``op`` is one of

* ``rotate``: per-head RMSNorm and rotate-half rotation of q and k;
* ``store``:  a layer's new keys and values into their pages (q, k normed and rotated
  in the same pass where ``base`` is above 0); 8-bit pages are read back, since codes
  mean nothing without their scales;
* ``read``:   the pages of every layer as the contiguous prefix K/V of the sampler;
* ``attend``: attention of one new token a sample over the pages.
"""
import math

import torch

own = False

DEV = "cuda"
POOL = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _rotate(name, b, t, heads, kv, dim, dtype, norm, far, sliced):
    return {"name": name, "op": "rotate", "b": b, "t": t, "heads": heads, "kv": kv, "dim": dim, "dtype": dtype,
            "norm": norm, "base": 10000.0, "far": far, "sliced": sliced}


def _store(name, b, t, heads, kv, dim, dtype, pool, page, base, norm, ragged):
    return {"name": name, "op": "store", "b": b, "t": t, "heads": heads, "kv": kv, "dim": dim, "dtype": dtype,
            "pool": pool, "page": page, "base": base, "norm": norm, "ragged": ragged}


def _read(name, layers, b, p, kv, dim, pool, page, low, holes, dtype):
    return {"name": name, "op": "read", "layers": layers, "b": b, "p": p, "kv": kv, "dim": dim, "pool": pool,
            "page": page, "low": low, "holes": holes, "dtype": dtype}


def _attend(name, b, heads, kv, dim, pool, page, low, high, holes):
    return {"name": name, "op": "attend", "b": b, "heads": heads, "kv": kv, "dim": dim, "pool": pool, "page": page,
            "low": low, "high": high, "holes": holes}


def listed():
    return [
        # one text token of one robot: nothing but latency
        _rotate("rotate one token", 1, 1, 8, 1, 256, "bf16", True, 816, False),
        # the prefix (3 cameras x 256 + 48 text tokens) of 32 robots
        _rotate("rotate 32 prefixes", 32, 816, 8, 1, 256, "bf16", True, 0, False),
        # odd lengths in fp32, sliced from a fused projection, far along a long context, no norms
        _rotate("rotate far f32", 5, 77, 28, 4, 128, "f32", False, 200000, True),
        # a decoding step of 8 robots: q and k normed and rotated, k and v into bf16 pages
        _store("store 8 tokens", 8, 1, 8, 1, 256, "bf16", "bf16", 16, 10000.0, True, False),
        # padded prefixes of 64 robots rotated and quantised to e4m3 pages, and read back
        _store("store 64 prefixes e4m3", 64, 816, 0, 1, 256, "bf16", "e4m3", 64, 10000.0, False, True),
        # fp32 rows that are rotated already, 4 kv heads, odd pages of int8
        _store("store f32 rows int8", 3, 301, 0, 4, 128, "f32", "int8", 20, 0.0, False, True),
        # what the 18-layer sampler needs before the loop: one robot, 10 padded tokens, e4m3 pages
        _read("read 18 layers e4m3", 18, 1, 816, 1, 256, "e4m3", 16, 806, True, "bf16"),
        # the same for 16 robots with two cameras each, bf16 pages
        _read("read 18 layers 16 robots", 18, 16, 560, 1, 256, "bf16", 64, 500, False, "bf16"),
        # one robot's next token over its prefix
        _attend("attend one robot", 1, 8, 1, 256, "bf16", 16, 806, 806, True),
        # 128 robots with ragged prefixes
        _attend("attend 128 robots", 128, 8, 1, 256, "bf16", 64, 600, 816, False),
        # two very long histories in e4m3: all the work lies along the keys
        _attend("attend long e4m3", 2, 8, 1, 256, "e4m3", 64, 100001, 262144, False),
        # 28 heads on 4, int8 in odd pages, empty to long samples, holes
        _attend("attend ragged int8", 24, 28, 4, 128, "int8", 20, 0, 16001, True),
    ]


HEADS = ((8, 1), (28, 4), (16, 2), (4, 4), (16, 1), (9, 3), (1, 1), (20, 2))
PAGES = (1, 7, 16, 20, 32, 64, 128)


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def _one(rng):
    op = rng.choice(("rotate", "store", "store", "read", "attend", "attend", "attend"))
    heads, kv = rng.choice(HEADS)
    dim = rng.choice((64, 128, 256, 256))
    pool = rng.choice(("bf16", "e4m3", "int8"))
    page = rng.choice(PAGES)
    if op == "rotate":
        c = _rotate("", _spread(rng, 1, 64), _spread(rng, 1, 2048), heads, kv, dim, rng.choice(("bf16", "f32")),
                    rng.random() < 0.6, rng.choice((0, 1000, 500000)), rng.random() < 0.5)
    elif op == "store":
        base = rng.choice((0.0, 10000.0, 500000.0))
        c = _store("", _spread(rng, 1, 64), _spread(rng, 1, 1500), heads if base and pool == "bf16" else 0, kv, dim,
                   rng.choice(("bf16", "f32")), pool, page, base, bool(base) and rng.random() < 0.5,
                   rng.random() < 0.5)
    elif op == "read":
        p = _spread(rng, 1, 2000)
        c = _read("", rng.choice((1, 2, 18)), _spread(rng, 1, 32), p, kv, dim, pool, page, rng.randint(0, p),
                  rng.random() < 0.5, rng.choice(("bf16", "f32")))
    else:
        high = _spread(rng, 1, 100000)
        c = _attend("", _spread(rng, 1, 128), heads, kv, dim, pool, page, rng.randint(0, high), high,
                    rng.random() < 0.4)
    del c["name"]
    return c


def draw(rng):
    top = max(work(c)["bytes"] for c in listed())
    while True:
        c = _one(rng)
        slots = c["b"] * c.get("high", c.get("p", c.get("t", 1))) * c["kv"] * c["dim"]
        if work(c)["bytes"] <= top and slots <= 2 ** 27:
            return c


def _counts(n, low, high):
    """n lengths from `low` to `high` of a case, out of order, both ends among them."""
    if n == 1:
        return [high]
    steps = [low + (high - low) * i // (n - 1) for i in range(n)]
    return [steps[(i * 7919 + 3) % n] for i in range(n)] if math.gcd(7919, n) == 1 else steps[::-1]


def _lens(c):
    if c["op"] == "store":
        return _counts(c["b"], 0 if c["ragged"] else c["t"], c["t"])
    return _counts(c["b"], c["low"], c.get("high", c.get("p")))


def _size(name):
    return {"bf16": 2, "f32": 4, "e4m3": 1, "int8": 1}[name]


def work(case):
    c, d, op = case, case["dim"], case["op"]
    if op == "rotate":
        rows = c["b"] * c["t"] * (c["heads"] + c["kv"])
        return {"bytes": 2 * rows * d * _size(c["dtype"]) + 4 * c["b"], "flops": rows * d * (7 if c["norm"] else 3)}
    rows = sum(_lens(c)) * c["kv"]
    cell = d * _size(c["pool"]) + (4 if c["pool"] != "bf16" else 0)
    if op == "store":
        q = c["b"] * c["t"] * c["heads"]
        moved = 2 * rows * (d * _size(c["dtype"]) + cell) + 2 * q * d * _size(c["dtype"])
        if c["pool"] != "bf16":
            moved += 2 * rows * cell + 2 * c["b"] * c["t"] * c["kv"] * d * 2
        return {"bytes": moved + 8 * c["b"], "flops": 8 * (2 * rows + q) * d}
    if op == "read":
        out = c["layers"] * c["b"] * c["kv"] * c["p"]
        return {"bytes": 2 * (c["layers"] * rows * cell + out * d * _size(c["dtype"])) + 2 * c["b"] * c["p"],
                "flops": 2 * out * d}
    return {"bytes": 2 * rows * cell + 4 * c["b"] * c["heads"] * (d + 1),
            "flops": 4 * sum(_lens(c)) * c["heads"] * d}


# ---- what a program has in hand ------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(g, b, tokens, page):
    """Every sample's pages, scattered over a pool with a few pages to spare."""
    per = -(-tokens // page)
    pages = b * per + 3
    return torch.randperm(pages, device=DEV, generator=g)[:b * per].to(torch.int32).view(b, per), pages


def _pools(c, g, layers, pages, seen):
    """Pools whose rows hold keys and values, 8-bit ones with the scales of such rows; the
    rows that no sample sees (`seen` says which are) hold what an earlier owner left: NaN."""
    s, none = {}, ~seen.view(pages, c["page"])
    for name in ("k", "v"):
        shape = (layers, pages, c["page"], c["kv"], c["dim"])
        if c["pool"] == "bf16":
            s[name] = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
            s[name].masked_fill_(none[None, :, :, None, None], math.nan)
        else:
            top = TOP[c["pool"]]
            x = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16).mul_(0.27 * top).clamp_(-top, top)
            s[name] = x.round_().to(torch.int8) if c["pool"] == "int8" else x.to(torch.float8_e4m3fn)
            if c["pool"] == "int8":
                scale = (torch.rand(shape[:-1], device=DEV, generator=g) + 0.5) * (3.7 / top)
            else:
                scale = torch.exp2(torch.randint(-8, -5, shape[:-1], device=DEV, generator=g).float())
            s[name + "_scale"] = scale
            s[name + "_scale"].masked_fill_(none[None, :, :, None], math.nan)
    return s


def prepare(case, seed):
    c, g = case, _generator(seed)
    b, d, op = c["b"], c["dim"], c["op"]
    s = {"case": c}
    if op in ("rotate", "store"):
        dt, hq, kv = TYPE[c["dtype"]], c["heads"], c["kv"]
        if op == "rotate" and c["sliced"]:
            whole = _normal(g, b, c["t"], hq + 2 * kv, d, dtype=dt)
            s["q"], s["k"] = whole[:, :, :hq], whole[:, :, hq:hq + kv]
        else:
            s["q"] = _normal(g, b, c["t"], hq, d, dtype=dt) if hq else None
            s["k"] = _normal(g, b, c["t"], kv, d, dtype=dt)
            s["v"] = _normal(g, b, c["t"], kv, d, dtype=dt)
        s["q_gain"] = 0.1 * _normal(g, d) if c["norm"] and hq else None
        s["k_gain"] = 0.1 * _normal(g, d) if c["norm"] else None
    if op == "rotate":
        s["start"] = _ints([c["far"] + 3 * i for i in range(b)])
        return s
    if op == "store":
        # ahead of the new tokens lie those of a prefix that ends inside a page
        first = [(5 * i) % 40 for i in range(b)]
        s["table"], pages = _table(g, b, c["t"] + 40, c["page"])
        s["start"], s["count"] = _ints(first), _ints(_lens(c))
        s["lens"] = s["start"] + s["count"]
        shape = (1, pages, c["page"], c["kv"], d)
        for name in ("k", "v"):
            s["pool_" + name] = torch.zeros(shape, device=DEV, dtype=POOL[c["pool"]])
            s["scale_" + name] = torch.zeros(shape[:-1], device=DEV) if c["pool"] != "bf16" else None
        if own:
            from vla_flow_matching_b200 import pi0x
            s["cache"] = pi0x.KVCache(s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"])
        return s
    lens = _lens(c)
    tokens = max(1, c.get("high", c.get("p")))
    s["table"], pages = _table(g, b, tokens, c["page"])
    s["lens"] = _ints(lens)
    s["mask"] = (torch.rand(b, tokens, device=DEV, generator=g) < 0.95).to(torch.uint8) if c["holes"] else None
    seen = torch.zeros(pages * c["page"], dtype=torch.bool, device=DEV)
    seen[_rows(s["table"], tokens, c["page"])] = _valid(s, tokens)
    pools = _pools(c, g, c.get("layers", 1), pages, seen)
    for name in ("k", "v"):
        s["pool_" + name], s["scale_" + name] = pools[name], pools.get(name + "_scale")
    if op == "attend":
        s["q"] = _normal(g, b, c["heads"], d, dtype=torch.bfloat16)
    if own:
        from vla_flow_matching_b200 import pi0x
        s["cache"] = pi0x.KVCache(s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"])
    return s


# ---- the library's calls ---------------------------------------------------------


def _run_own(s):
    from vla_flow_matching_b200 import pi0x
    c = s["case"]
    if c["op"] == "rotate":
        return pi0x.qk_norm_rope(s["q"], s["k"], s["start"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                                 rope_base=c["base"], eps=EPS)
    cache = s["cache"]
    if c["op"] == "store":
        q = cache.write(0, s["k"], s["v"], s["table"], s["start"], s["count"], q=s["q"], q_gain=s["q_gain"],
                        k_gain=s["k_gain"], rope_base=c["base"] or None, eps=EPS)
        if c["pool"] == "bf16":
            return {"q": q, "k": s["pool_k"], "v": s["pool_v"]}
        k, v, _ = cache.read(s["table"], s["lens"], c["t"] + 40)
        return {"q": q, "k": k, "v": v}
    if c["op"] == "read":
        k, v, mask = cache.read(s["table"], s["lens"], c["p"], mask=s["mask"], dtype=TYPE[c["dtype"]])
        return {"k": k, "v": v, "mask": mask}
    out, lse = cache.attend(0, s["q"], s["table"], s["lens"], mask=s["mask"])
    return {"out": out, "lse": lse}


# ---- plain torch -----------------------------------------------------------------


def _norm_rotate(x, gain, pos, base):
    """x (B,T,H,D), pos (B,T): RMSNorm of every head with gain 1 + g, then rotate-half."""
    y = x.float()
    if gain is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * (1.0 + gain)
    half = y.shape[-1] // 2
    freq = base ** (-torch.arange(half, device=y.device, dtype=torch.float64) / half)
    angle = pos.double()[..., None] * freq
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    a, b = y[..., :half], y[..., half:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _rows(table, p, page):
    """Pool rows (as page * page_size + offset) of positions 0..p-1 of every sample."""
    at = torch.arange(p, device=table.device)
    return table[:, at // page].long() * page + at % page


def _codes(x, pool):
    """x in the pool's type, and the scale of each row: the largest value's share of 127 in
    int8, the least power of two that brings the row within 448 in e4m3."""
    if pool == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1)
    if pool == "int8":
        scale = (top / TOP[pool]).clamp_min(2.0 ** -126)
        return (x / scale[..., None]).round().to(torch.int8), scale
    part, power = torch.frexp(top)
    scale = torch.exp2((power - 8 - (part <= 0.875).to(torch.int32)).clamp_min(-126).float())
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _fetch(pool, scale, rows):
    """Rows of (layers, pages, page, heads, dim) pools in fp32: (layers, B, P, heads, dim)."""
    x = pool.flatten(1, 2)
    if x.dtype == torch.float8_e4m3fn:
        x = x.view(torch.uint8)[:, rows].view(torch.float8_e4m3fn).float()
    else:
        x = x[:, rows].float()
    return x if scale is None else x * scale.flatten(1, 2)[:, rows][..., None]


def _valid(s, p):
    ok = torch.arange(p, device=DEV)[None] < s["lens"][:, None]
    return ok if s.get("mask") is None else ok & (s["mask"][:, :p] != 0)


def _read_plain(s, p, dtype):
    ok = _valid(s, p)
    rows = _rows(s["table"], p, s["case"]["page"])
    got = [torch.where(ok[None, :, :, None, None], _fetch(s["pool_" + n], s["scale_" + n], rows), 0.0)
           .transpose(2, 3).contiguous().to(dtype) for n in ("k", "v")]
    return got[0], got[1], ok.to(torch.uint8)


def _put(pool, where, new, rows):
    """rows (B,T,...) to their slots `where` (B,T); slots that get no new row keep theirs."""
    if pool.dtype == torch.float8_e4m3fn:
        pool, rows = pool.view(torch.uint8), rows.view(torch.uint8)
    pool = pool.flatten(0, 2)
    pool[where] = torch.where(new.view(new.shape + (1,) * (rows.dim() - 2)), rows, pool[where])


def _store_plain(s):
    c, b, t = s["case"], s["case"]["b"], s["case"]["t"]
    k, v, q = s["k"].float(), s["v"].float(), s["q"]
    step = torch.arange(t, device=DEV)[None]
    pos = s["start"][:, None].long() + step
    if c["base"]:
        k = _norm_rotate(k, s["k_gain"], pos, c["base"])
        q = None if q is None else _norm_rotate(q, s["q_gain"], pos, c["base"]).to(q.dtype)
    new = (step < s["count"][:, None]).expand(b, t)
    where = torch.gather(s["table"].long(), 1, pos // c["page"]) * c["page"] + pos % c["page"]
    for name, x in (("k", k), ("v", v)):
        codes, scale = _codes(x, c["pool"])
        _put(s["pool_" + name], where, new, codes)
        if scale is not None:
            _put(s["scale_" + name], where, new, scale)
    if c["pool"] == "bf16":
        return {"q": q, "k": s["pool_k"], "v": s["pool_v"]}
    k, v, _ = _read_plain(s, t + 40, torch.bfloat16)
    return {"q": q, "k": k, "v": v}


def _attend_plain(s):
    c = s["case"]
    p = s["table"].shape[1] * c["page"] if s["mask"] is None else s["mask"].shape[1]
    ok = _valid(s, p)[:, None, None]
    rows = _rows(s["table"], p, c["page"])
    k = _fetch(s["pool_k"], s["scale_k"], rows)[0].transpose(1, 2)
    v = _fetch(s["pool_v"], s["scale_v"], rows)[0].transpose(1, 2)
    v = torch.where(ok.transpose(2, 3), v, 0.0)
    q = s["q"].float().unflatten(1, (c["kv"], -1))
    x = torch.where(ok, (q @ k.transpose(2, 3)) * c["dim"] ** -0.5, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    out = torch.where(total > 0, (e @ v) / total, 0.0)
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": (m + torch.log(total)).squeeze(-1).flatten(1)}


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "rotate":
        pos = state["start"][:, None] + torch.arange(c["t"], device=DEV)[None]
        return tuple(_norm_rotate(state[n], state[n + "_gain"], pos, c["base"]).to(state[n].dtype) for n in ("q", "k"))
    if c["op"] == "store":
        return _store_plain(state)
    if c["op"] == "read":
        k, v, mask = _read_plain(state, c["p"], TYPE[c["dtype"]])
        return {"k": k, "v": v, "mask": mask}
    return _attend_plain(state)


# ---- the definitions in 64 bits ----------------------------------------------------


def _turned(x, gain, first, base):
    """Rows x (T,H,D) in 64 bits at positions first, first + 1, ...: normed and turned pair by pair."""
    x = x.double()
    t, _, d = x.shape
    if gain is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        x = x + x * gain.double()
    turn = torch.arange(first, first + t, device=DEV, dtype=torch.float64)[:, None] / torch.pow(
        torch.full((), base, device=DEV, dtype=torch.float64), 2.0 * torch.arange(d // 2, device=DEV).double() / d)
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * torch.polar(torch.ones_like(turn), turn)[:, None]
    return torch.cat((z.real, z.imag), -1)


def _held(x, pool):
    """What a row of x (64 bits) stands for once it is held in a page."""
    if pool == "bf16":
        return x.to(torch.bfloat16).double()
    scale = x.abs().max(-1, keepdim=True).values / TOP[pool]
    scale = torch.maximum(scale, torch.full_like(scale, 2.0 ** -126))
    if pool == "e4m3":
        scale = torch.pow(2.0, torch.ceil(torch.log2(scale)))
    y = x / scale
    if pool == "int8":
        return torch.round(y) * scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)  # e4m3: 3 bits, lowest exponent -6
    return torch.clamp(torch.round(y / step) * step, -448.0, 448.0) * scale


def _keys(s, name, layer, b, n):
    """Rows 0..n-1 of sample b in 64 bits, with their slots taken page by page."""
    page = s["case"]["page"]
    pages = s["table"][b, :-(-n // page)].long()
    codes = s["pool_" + name][layer]
    if codes.dtype == torch.float8_e4m3fn:
        x = codes.view(torch.uint8).index_select(0, pages).view(torch.float8_e4m3fn).double()
    else:
        x = codes.index_select(0, pages).double()
    if s["scale_" + name] is not None:
        x = x * s["scale_" + name][layer].index_select(0, pages).double()[..., None]
    return x.flatten(0, 1)[:n]


def _seen(s, b, n):
    return torch.ones(n, dtype=torch.bool, device=DEV) if s.get("mask") is None else s["mask"][b, :n] != 0


def exact(case, seed):
    c, s = case, prepare(case, seed)
    b, d = c["b"], c["dim"]
    if c["op"] == "rotate":
        first = s["start"].tolist()
        return tuple(torch.stack([_turned(s[n][i], s[n + "_gain"], first[i], c["base"]) for i in range(b)])
                     for n in ("q", "k"))
    if c["op"] == "store":
        first, count, p = s["start"].tolist(), s["count"].tolist(), c["t"] + 40
        q = None if s["q"] is None else torch.stack(
            [_turned(s["q"][i], s["q_gain"], first[i], c["base"]) for i in range(b)])
        whole = []
        for name in ("k", "v"):
            pool = torch.zeros(s["pool_k"].shape[1:], device=DEV, dtype=torch.float64).flatten(0, 1)
            span = torch.zeros(b, c["kv"], p, d, device=DEV, dtype=torch.float64)
            for i in range(b):
                x = s[name][i, :count[i]]
                x = _turned(x, s["k_gain"], first[i], c["base"]) if name == "k" and c["base"] else x.double()
                x = x if c["pool"] == "bf16" else _held(x, c["pool"])
                span[i, :, first[i]:first[i] + count[i]] = x.transpose(0, 1)
                at = torch.arange(first[i], first[i] + count[i], device=DEV)
                pool[s["table"][i].long()[at // c["page"]] * c["page"] + at % c["page"]] = x
            whole.append(pool.view(s["pool_k"].shape) if c["pool"] == "bf16" else span[None])
        return {"q": q, "k": whole[0], "v": whole[1]}
    lens = s["lens"].tolist()
    if c["op"] == "read":
        out = {n: torch.zeros(c["layers"], b, c["kv"], c["p"], d, device=DEV, dtype=torch.float64) for n in ("k", "v")}
        mask = torch.zeros(b, c["p"], device=DEV, dtype=torch.uint8)
        for i in range(b):
            ok = _seen(s, i, lens[i])
            mask[i, :lens[i]] = ok.to(torch.uint8)
            for n in ("k", "v"):
                for layer in range(c["layers"]):
                    x = _keys(s, n, layer, i, lens[i])
                    x[~ok] = 0.0
                    out[n][layer, i, :, :lens[i]] = x.transpose(0, 1)
        return {"k": out["k"], "v": out["v"], "mask": mask}
    out = torch.zeros(b, c["heads"], d, device=DEV, dtype=torch.float64)
    lse = torch.full((b, c["heads"]), -math.inf, device=DEV, dtype=torch.float64)
    for i in range(b):
        ok = _seen(s, i, lens[i])
        if not bool(ok.any()):
            continue
        k, v = _keys(s, "k", 0, i, lens[i])[ok], _keys(s, "v", 0, i, lens[i])[ok]
        q = s["q"][i].double().view(c["kv"], -1, d)
        x = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(d)
        z = torch.logsumexp(x, -1)
        out[i] = torch.einsum("hgn,nhd->hgd", torch.exp(x - z[..., None]), v).flatten(0, 1)
        lse[i] = z.flatten()
    return {"out": out, "lse": lse}
