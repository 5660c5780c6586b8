"""The paged prefix cache on the GPU: per-head norm and rotation, page writes and reads,
attention of one new token, and the sampler on a cache, each against its formula in 64 bits.

Tolerances count roundings.  An output of type t is off by at most half a step,
``finfo(t).eps / 2`` of its value; what is computed in fp32 before that adds its share,
given at each check.
"""
import concurrent.futures
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from vla_flow_matching_b200 import build, pi0x

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- formulas in 64 bits ---------------------------------------------------------


def rotated(x, gain, pos, base, eps=1e-6):
    """x (B,T,H,D) at positions (B,T)."""
    y = x.double()
    D = y.shape[-1]
    if gain is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * (1.0 + gain.double())
    if base:
        i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
        a = pos.double()[..., None, None] * base ** (-2.0 * i / D)
        lo, hi = y[..., :D // 2], y[..., D // 2:]
        y = torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)
    return y


def rotated_slack(y):
    """fp32 work before the last rounding: D squares and their sum, rsqrt and two products
    (D/2 + 8 roundings at most in a norm's mean as halves), the angle and two products and a
    sum, all relative to a pair's length."""
    D = y.shape[-1]
    pair = torch.hypot(y[..., :D // 2], y[..., D // 2:])
    return torch.cat([pair, pair], -1) * (D / 2 + 24) * U32


def check_rotated(got, x, gain, pos, base):
    y = rotated(x, gain, pos, base)
    tol = half_step(got.dtype) * y.abs() * (1 + 2 ** -7) + rotated_slack(y) + 1e-40
    assert bool(((got.double() - y).abs() <= tol).all()), float(((got.double() - y).abs() - tol).max())


def values(pool, scale):
    """What pool rows stand for, in 64 bits (float8 has no indexing of its own: cast first)."""
    x = pool.float().double()
    return x if scale is None else x * scale.double()[..., None]


def slots(cache, layer, name, table, b, n):
    """(n, kv, D) values of slots 0..n-1 of sample b and whether each has a page."""
    ps = cache.page_size
    pages = table[b].tolist()
    v = values(getattr(cache, name)[layer], getattr(cache, name + "_scale")[layer] if cache.k_scale is not None else None)
    at = [pages[p // ps] for p in range(n)]
    ok = torch.tensor([0 <= x < cache.num_pages for x in at], device="cuda", dtype=torch.bool)
    rows = torch.tensor([x if 0 <= x < cache.num_pages else 0 for x in at], device="cuda", dtype=torch.long)
    return v[rows, torch.arange(n, device="cuda") % ps], ok


def make_cache(dtype, layers, pages, ps, kv, D, seed):
    """Pools as a prefix leaves them: N(0,1) rows."""
    c = pi0x.KVCache.empty(layers, pages, ps, kv, D, dtype)
    g = rng(seed)
    for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        if dtype == "bf16":
            pool.copy_(randn(g, *pool.shape))
        elif dtype == "int8":
            pool.copy_(torch.randint(-127, 128, pool.shape, device="cuda", generator=g).to(torch.int8))
            scale.copy_((torch.rand(scale.shape, device="cuda", generator=g) + 0.5) / 64)
        else:
            pool.copy_((randn(g, *pool.shape) * 64).clamp(-448, 448).to(torch.float8_e4m3fn))
            scale.copy_(torch.exp2(torch.randint(-8, -5, scale.shape, device="cuda", generator=g).float()))
    return c


def scattered(g, B, per, pages):
    return torch.randperm(pages, device="cuda", generator=g)[:B * per].to(torch.int32).view(B, per)


# ---- norm and rotation -----------------------------------------------------------


@pytest.mark.parametrize("B,T,hq,hk,D,dtype,norm,base,first", [
    (1, 1, 8, 1, 256, BF16, True, 10000.0, 0),
    (1, 1, 1, 0, 64, F32, True, 10000.0, 5),
    (3, 7, 28, 4, 128, BF16, True, 1000000.0, 100000),
    (2, 33, 9, 3, 64, F32, False, 10000.0, 2 ** 31 - 200),
    (2, 5, 8, 1, 256, F32, True, None, -40),
    (5, 301, 8, 1, 256, BF16, False, 10000.0, -40),
    (1, 2000, 16, 2, 128, F32, True, 500000.0, 0),
])
def test_qk_norm_rope_matches_the_formula(B, T, hq, hk, D, dtype, norm, base, first):
    g = rng(B * T + D)
    q, k = randn(g, B, T, hq, D, dtype=dtype), randn(g, B, T, hk, D, dtype=dtype) if hk else None
    gains = [0.2 * randn(g, D) if norm else None for _ in range(2)]
    start = ints([first + 11 * b for b in range(B)])
    qo, ko = pi0x.qk_norm_rope(q, k, start, q_gain=gains[0], k_gain=gains[1] if hk else None, rope_base=base)
    pos = start.long()[:, None] + torch.arange(T, device="cuda")
    check_rotated(qo, q, gains[0], pos, base)
    if hk:
        check_rotated(ko, k, gains[1], pos, base)


def test_qk_norm_rope_of_slices_one_gain_given_positions_and_in_place():
    g = rng(1)
    B, T, hq, hk, D = 2, 9, 6, 2, 128
    fused = randn(g, B, T, hq + 2 * hk, D, dtype=BF16)
    q, k = fused[:, :, :hq], fused[:, :, hq:hq + hk]
    pos = torch.randint(-1000, 100000, (B, T), device="cuda", generator=g).int()
    gain = 0.1 * randn(g, D)
    qo, ko = pi0x.qk_norm_rope(q, k, positions=pos, k_gain=gain)
    check_rotated(qo, q, None, pos, 10000.0)
    check_rotated(ko, k, gain, pos, 10000.0)
    v = fused[:, :, hq + hk:].clone()
    qi, ki = pi0x.qk_norm_rope(q, k, positions=pos, k_gain=gain, q_out=q, k_out=k)
    assert qi.data_ptr() == q.data_ptr() and torch.equal(qi, qo) and torch.equal(ki, ko)
    assert torch.equal(fused[:, :, hq + hk:], v)
    # transposed storage: (B, heads, T, D) seen as (B, T, heads, D)
    t = randn(g, B, hq, T, D, dtype=F32).transpose(1, 2)
    check_rotated(pi0x.qk_norm_rope(t, positions=pos)[0], t, None, pos, 10000.0)


def test_qk_norm_rope_edge_values():
    q = torch.zeros(1, 4, 1, 64, device="cuda")
    q[0, 1], q[0, 2, 0, 3], q[0, 3] = 1e18, float("nan"), 1e-18
    gain = torch.zeros(64, device="cuda")
    out = pi0x.qk_norm_rope(q, q_gain=gain, rope_base=None)[0]
    assert torch.equal(out[0, 0], torch.zeros_like(out[0, 0]))            # a zero row stays zero
    assert bool(((out[0, 1] - 1).abs() < 1e-5).all())                     # 1e36 squares still fit fp32
    assert bool(out[0, 2].isnan().all())
    assert bool(((out[0, 3] - 1e-15).abs() < 1e-20).all())                # eps 1e-6 holds the gain at 1e3
    inf = torch.full((1, 1, 1, 64), float("inf"), device="cuda")
    assert bool(pi0x.qk_norm_rope(inf, rope_base=None)[0].isinf().all())  # nothing to do: bits pass through


def test_empty_batches_return_empty():
    q = torch.zeros(0, 3, 8, 64, device="cuda", dtype=BF16)
    assert pi0x.qk_norm_rope(q, q)[0].shape == q.shape
    c = pi0x.KVCache.empty(1, 2, 4, 1, 64)
    table = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    k = torch.zeros(0, 3, 1, 64, device="cuda", dtype=BF16)
    assert c.write(0, k, k, table, none) is None
    assert c.attend(0, torch.zeros(0, 8, 64, device="cuda", dtype=BF16), table, none)[0].shape == (0, 8, 64)
    assert c.read(table, none, 5)[0].shape == (1, 0, 1, 5, 64)


def test_python_refusals_on_the_gpu():
    g = rng(3)
    c = pi0x.KVCache.empty(2, 8, 4, 2, 64, "bf16")
    q, k = randn(g, 2, 3, 4, 64, dtype=BF16), randn(g, 2, 3, 2, 64, dtype=BF16)
    table, lens = ints([[0, 1], [2, 3]]), ints([1, 2])
    bad = [
        (ValueError, lambda: pi0x.qk_norm_rope(q, k.float(), lens)),
        (ValueError, lambda: pi0x.qk_norm_rope(q.half())),
        (ValueError, lambda: pi0x.qk_norm_rope(q[0])),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k[:, :2])),
        (ValueError, lambda: pi0x.qk_norm_rope(q.transpose(2, 3))),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k, lens.long())),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k, ints([1, 2, 3]))),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k, positions=lens)),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k, q_gain=torch.zeros(32, device="cuda"))),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k, q_out=torch.empty_like(k))),
        (ValueError, lambda: pi0x.qk_norm_rope(q, k.cpu(), lens)),
        (pi0x.Pi0xError, lambda: pi0x.qk_norm_rope(q[..., :32].contiguous())),
        (pi0x.Pi0xError, lambda: pi0x.qk_norm_rope(q, rope_base=0.25)),
        (pi0x.Pi0xError, lambda: pi0x.qk_norm_rope(randn(g, 2, 3, 4, 65, dtype=BF16)[..., :64])),
        (ValueError, lambda: c.write(0, q, q, table, lens)),
        (ValueError, lambda: c.write(0, k, k[:, :1], table, lens)),
        (ValueError, lambda: c.write(0, k, k, table[:1], lens)),
        (ValueError, lambda: c.write(0, k, k, table.T, lens)),
        (ValueError, lambda: c.write(0, k, k, table, None)),
        (ValueError, lambda: c.write(0, k, k, table, lens, q=q.float())),
        (pi0x.Pi0xError, lambda: c.write(2, k, k, table, lens)),
        (pi0x.Pi0xError, lambda: c.write(-1, k, k, table, lens)),
        (ValueError, lambda: c.read(table, ints([1]), 3)),
        (ValueError, lambda: c.read(table, lens, 3, mask=torch.ones(2, 4, device="cuda", dtype=torch.uint8))),
        (ValueError, lambda: c.read(table, lens, 3, dtype=torch.float16)),
        (ValueError, lambda: c.read(table, lens, -3)),
        (ValueError, lambda: c.read(table, lens, 3, k_out=torch.empty(2, 2, 3, 2, 64, device="cuda", dtype=BF16))),
        (pi0x.Pi0xError, lambda: c.read(table, lens, 3, layer0=1, layers=2)),
        (ValueError, lambda: c.attend(0, q, table, lens)),
        (ValueError, lambda: c.attend(0, q[:, 0].float(), table, lens)),
        (ValueError, lambda: c.attend(0, q[:, 0], table, None)),
        (ValueError, lambda: c.attend(0, q[:, 0], table, lens, mask=torch.ones(2, 0, device="cuda", dtype=torch.uint8))),
        (ValueError, lambda: c.attend(0, q[:, 0], table, lens, lse=torch.empty(2, 3, device="cuda"))),
        (pi0x.Pi0xError, lambda: c.attend(0, q[:, 0, :3], table, lens)),
        (pi0x.Pi0xError, lambda: c.attend(5, q[:, 0], table, lens)),
        (pi0x.Pi0xError, lambda: c.attend(0, q[:, 0], table, lens, scale=float("nan"))),
        (OverflowError, lambda: c.attend(2 ** 40, q[:, 0], table, lens)),
        (AttributeError, lambda: c.attend(0, [1.0], table, lens)),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()


# ---- writing and reading pages -----------------------------------------------------


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,T,kv,D,ps,dtype", [
    (1, 1, 1, 256, 16, BF16), (3, 13, 4, 64, 5, F32), (2, 100, 1, 256, 1, BF16), (4, 37, 2, 128, 64, F32)])
def test_cache_write_holds_the_rows(pool, B, T, kv, D, ps, dtype):
    g = rng(T + D + ps)
    per = -(-(T + 21) // ps)
    c = pi0x.KVCache.empty(2, B * per + 2, ps, kv, D, pool)
    table = scattered(g, B, per, c.num_pages)
    k, v = randn(g, B, T, kv, D, dtype=dtype), randn(g, B, T, kv, D, dtype=dtype)
    k[0, 0, 0] = 0                       # a zero row
    v[0, 0, 0] *= 1e-30                  # below the least scale's codes in part
    start = ints([(7 * b) % 21 for b in range(B)])
    count = ints([max(0, T - 5 * b) for b in range(B)])
    assert c.write(1, k, v, table, start, count) is None
    for name, x in (("k", k), ("v", v)):
        pools, scales = getattr(c, name), getattr(c, name + "_scale")
        want = torch.zeros_like(pools, dtype=F32)
        wscale = None if scales is None else torch.zeros_like(scales)
        for b in range(B):
            for t in range(int(count[b])):
                pos = int(start[b]) + t
                page, off = int(table[b, pos // ps]), pos % ps
                row = x[b, t].float()
                if pool == "bf16":
                    want[1, page, off] = row.to(BF16).float()
                    continue
                top = row.abs().amax(-1)
                if pool == "int8":
                    # by a tensor: torch divides a CUDA tensor by a number as a product with 1/number
                    sc = (top / torch.full_like(top, 127.0)).clamp_min(2.0 ** -126)
                    want[1, page, off] = (row / sc[:, None]).round()
                else:
                    part, power = torch.frexp(top.double() / 448)  # exact at 448 * 2^n, unlike a logarithm
                    power = (power - (part == 0.5).int()).clamp_min(-126)
                    sc = torch.ldexp(torch.ones_like(top), torch.where(top == 0, -126, power))
                    want[1, page, off] = (row / sc[:, None]).to(torch.float8_e4m3fn).float()
                wscale[1, page, off] = sc
        assert torch.equal(pools.float(), want), name      # layer 0 and the slots without a token stay zero
        if scales is not None:
            assert torch.equal(scales, wscale), (name, scales[scales != wscale], wscale[scales != wscale])


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
def test_cache_write_rotates_and_norms_in_the_same_pass(pool):
    g = rng(9)
    B, T, hq, kv, D, ps = 3, 11, 8, 2, 128, 4
    c = pi0x.KVCache.empty(1, 3 * 8, ps, kv, D, pool)
    table = scattered(g, B, 8, c.num_pages)
    q, k, v = (randn(g, B, T, h, D, dtype=BF16) for h in (hq, kv, kv))
    gq, gk = 0.2 * randn(g, D), 0.2 * randn(g, D)
    start, count = ints([0, 13, 21]), ints([11, 0, 7])
    qo = c.write(0, k, v, table, start, count, q=q, q_gain=gq, k_gain=gk, rope_base=10000.0)
    pos = start.long()[:, None] + torch.arange(T, device="cuda")
    check_rotated(qo, q, gq, pos, 10000.0)               # every row of q, whatever count says
    y = rotated(k, gk, pos, 10000.0)
    for b in range(B):
        n = int(count[b])
        got, _ = slots(c, 0, "k", table, b, int(start[b]) + n)
        want = y[b, :n]
        got = got[int(start[b]):]
        top = want.abs().amax(-1, keepdim=True)
        # half a step: of the value (bf16, e4m3) or of the scale (int8); e4m3's least step is
        # 2^-9 of a scale that is at most top / 224
        step = {"bf16": half_step(BF16) * want.abs(), "int8": top / 254 * (1 + 2 ** -10),
                "e4m3": 2.0 ** -4 * want.abs() + top / 224 * 2.0 ** -10}[pool]
        tol = step * (1 + 2 ** -7) + 2 * rotated_slack(want)
        assert bool(((got - want).abs() <= tol).all())
        gv, _ = slots(c, 0, "v", table, b, int(start[b]) + n)
        vt = v[b, :n].double()
        assert bool(((gv[int(start[b]):] - vt).abs() <= {
            "bf16": 0.0 * vt, "int8": vt.abs().amax(-1, keepdim=True) / 254 * (1 + 2 ** -10),
            "e4m3": 2.0 ** -4 * vt.abs() + vt.abs().amax(-1, keepdim=True) / 224 * 2.0 ** -10}[pool]).all())


def test_cache_write_leaves_out_what_has_no_page():
    g = rng(2)
    c = pi0x.KVCache.empty(1, 4, 4, 1, 64, "bf16")
    c.k.fill_(7.0)
    c.v.fill_(7.0)
    big = 2 ** 31 - 1
    table = ints([[0, -1, 4], [big, 2, -big - 1]])
    k = randn(g, 2, 14, 1, 64, dtype=BF16)
    c.write(0, k, k, table, ints([-2, 0]))                # sample 0: slots -2..11, sample 1: slots 0..13
    want = torch.full_like(c.k, 7.0)
    want[0, 0, :, 0] = k[0, 2:6, 0]
    want[0, 2, :, 0] = k[1, 4:8, 0]
    assert torch.equal(c.k, want) and torch.equal(c.v, want)
    c.write(0, k, k, table, ints([big, big]), ints([-3, big]))
    assert torch.equal(c.k, want)


@pytest.mark.parametrize("pool", ["e4m3", "int8"])
def test_rows_that_are_not_finite_stand_for_nan(pool):
    c = pi0x.KVCache.empty(1, 1, 4, 1, 64, pool)
    k = torch.ones(1, 4, 1, 64, device="cuda")
    k[0, 1, 0, 5], k[0, 2, 0, 63], k[0, 3] = float("nan"), float("-inf"), 3e38
    c.write(0, k, k, ints([[0]]), ints([0]))
    got = c.read(ints([[0]]), ints([4]), 4, dtype=F32)[0][0, 0, 0]
    assert bool(got[1:3].isnan().all()) and bool(got[0].isfinite().all())
    assert bool(((got[3] / 3e38 - 1).abs() < 2.0 ** -4).all())


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("layers,B,P,kv,D,ps,out", [
    (3, 2, 50, 1, 256, 16, BF16), (1, 1, 1, 1, 64, 1, F32), (2, 5, 77, 4, 128, 7, BF16), (2, 3, 65, 2, 64, 64, F32)])
def test_cache_read_gives_the_rows_and_zeros(pool, layers, B, P, kv, D, ps, out):
    g = rng(P)
    per = -(-P // ps) + 1
    c = make_cache(pool, layers + 1, B * per, ps, kv, D, P)
    table = scattered(g, B, per, c.num_pages)
    if B > 1:
        table[1, 0], table[1, 1] = -1, c.num_pages
    lens = ints([[P, P // 2, 0, -3, 10 ** 9][b % 5] for b in range(B)])
    mask = torch.rand(B, P, device="cuda", generator=g) < 0.8
    for m in (None, mask):
        k, v, seen = c.read(table, lens, P, mask=m, layer0=1, dtype=out)
        for b in range(B):
            at = torch.arange(P, device="cuda")
            _, page_ok = slots(c, 0, "k", table, b, P)
            ok = (at < int(lens[b])) & page_ok & (True if m is None else m[b])
            assert torch.equal(seen[b].bool(), ok)
            for name, got in (("k", k), ("v", v)):
                for layer in range(layers):
                    x, _ = slots(c, layer + 1, name, table, b, P)
                    want = torch.where(ok[:, None, None], x, 0.0).transpose(0, 1)
                    # code * scale is rounded to fp32, then to the output's type
                    assert torch.equal(got[layer, b], want.float().to(out)), (name, b, layer)


def test_masked_slots_are_not_read():
    c = pi0x.KVCache.empty(1, 2, 8, 1, 64, "bf16")
    c.k.fill_(float("nan"))
    c.v.fill_(float("inf"))
    c.k[0, 1, :4], c.v[0, 1, :4] = 1.0, 2.0
    table, mask = ints([[1, 0]]), torch.zeros(1, 16, dtype=torch.uint8, device="cuda")
    mask[0, :3] = 5
    k, v, seen = c.read(table, ints([16]), 16, mask=mask)
    assert float(k.float().sum()) == 3 * 64 and float(v.float().sum()) == 6 * 64 and int(seen.sum()) == 3
    out, lse = c.attend(0, torch.ones(1, 3, 64, device="cuda", dtype=BF16), table, ints([16]), mask=mask)
    assert torch.equal(out, torch.full_like(out, 2.0))
    assert bool(((lse - (8.0 + math.log(3))).abs() < 1e-5).all())


# ---- attention of one new token ----------------------------------------------------


def check_attend(c, layer, q, table, lens, mask, scale, out, lse):
    B, H, D = q.shape
    G = H // c.kv_heads
    cap = table.shape[1] * c.page_size
    scale = D ** -0.5 if scale is None else scale
    for b in range(B):
        n = max(0, min(int(lens[b]), cap))
        n = n if mask is None else min(n, mask.shape[1])
        k, ok = slots(c, layer, "k", table, b, n)
        v, _ = slots(c, layer, "v", table, b, n)
        if mask is not None:
            ok = ok & mask[b, :n].bool()
        k, v = k[ok], v[ok]
        if k.shape[0] == 0:
            assert torch.equal(out[b], torch.zeros_like(out[b])) and bool((lse[b] == -math.inf).all()), b
            continue
        x = q[b].double().view(c.kv_heads, G, D)
        s = torch.einsum("hgd,nhd->hgn", x, k) * scale
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[..., None])
        o = torch.einsum("hgn,nhd->hgd", p, v)
        mass = torch.einsum("hgn,nhd->hgd", p, v.abs())
        # scores: D fp32 products and sums, the scales, log2(e) and the exponential (2^-22 of it
        # and one rounding of a difference of scores); sums of p over the keys
        size = torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()).amax(-1) * abs(scale)
        delta = (D + 16) * U32 * (size + 1) + k.shape[0] * U32 + 2.0 ** -21
        # probabilities in the type of the matrix product, bf16 at the coarsest
        tol = half_step(BF16) * o.abs() + (half_step(BF16) + 2 * delta[..., None]) * mass * 1.01 + 1e-30
        err = (out[b].double().view_as(o) - o).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()))
        zerr = (lse[b].double().view_as(z) - z).abs()
        assert bool((zerr <= delta + 4 * U32 * z.abs()).all()), (b, float(zerr.max()))


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,H,kv,D,ps,lens", [
    (1, 8, 1, 256, 16, [816]),
    (1, 1, 1, 64, 1, [1]),
    (4, 8, 1, 256, 64, [0, 1, 63, 65]),
    (3, 28, 4, 128, 20, [300, 0, 1023]),
    (2, 9, 3, 64, 7, [129, 500]),
    (2, 4, 4, 128, 16, [17, 2000]),
    (5, 20, 2, 256, 128, [15, 16, 17, -5, 10 ** 6]),
    (1, 33, 1, 128, 32, [700]),
    (130, 8, 1, 64, 16, [i * 5 % 97 for i in range(130)]),
    (1, 8, 1, 256, 64, [20000]),
    (400, 8, 1, 256, 16, [i * 37 % 701 for i in range(400)]),        # more units than CTAs, evenly split and joined
    (6, 12, 2, 128, 64, [9000, 0, 1, 30000, 17000, 64]),            # a few long ones: units over many CTAs
    (33, 3, 3, 256, 32, [i * 53 % 2000 for i in range(33)]),
    (3, 20, 2, 256, 16, [6000, 77, 9001]),                          # more than 8 query heads a kv head
    (2, 48, 2, 128, 64, [15000, 3]),
    (90, 16, 1, 64, 8, [i * 31 % 400 for i in range(90)]),
])
def test_attend_matches_the_formula(pool, B, H, kv, D, ps, lens):
    g = rng(sum(lens) % 1000 + D)
    cap = max(1, max(n for n in lens if n < 10 ** 6))
    per = -(-cap // ps)
    c = make_cache(pool, 2, B * per + 1, ps, kv, D, H + D)
    table, lens = scattered(g, B, per, c.num_pages), ints(lens)
    q = randn(g, B, H, D, dtype=BF16)
    out, lse = c.attend(1, q, table, lens)
    check_attend(c, 1, q, table, lens, None, None, out, lse)
    mask = (torch.rand(B, max(1, cap - 3), device="cuda", generator=g) < 0.7).to(torch.uint8)
    mask[-1] = 0                                           # a sample whose mask leaves nothing
    table[0, 0] = -1
    table[-1, -1] = c.num_pages
    out, lse = c.attend(1, q, table, lens, mask=mask, scale=0.3)
    check_attend(c, 1, q, table, lens, mask, 0.3, out, lse)


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("lens", [[5, 0, 70], [0, 0, 0], [1, 130, 2000]])
def test_attend_of_short_samples_in_a_long_table(pool, lens):
    g = rng(21)
    c = make_cache(pool, 1, 40, 64, 2, 128, 22)
    table = torch.full((3, 4096), -1, device="cuda", dtype=torch.int32)
    table[:, :32] = torch.randint(0, 40, (3, 32), device="cuda", generator=g, dtype=torch.int32)
    q, lens = randn(g, 3, 8, 128, dtype=BF16), ints(lens)
    out, lse = c.attend(0, q, table, lens)
    check_attend(c, 0, q, table, lens, None, None, out, lse)


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
def test_attend_extremes(pool):
    g = rng(4)
    c = make_cache(pool, 1, 40, 16, 1, 128, 3)
    table, lens = torch.arange(40, device="cuda", dtype=torch.int32)[None], ints([640])
    q = randn(g, 1, 8, 128, dtype=BF16)
    for scale in (0.0, -0.2, 8.0):                         # equal weights, the far end, nearly one key
        out, lse = c.attend(0, q, table, lens, scale=scale)
        check_attend(c, 0, q, table, lens, None, scale, out, lse)
    big = q * 2.0 ** 60                                    # scores near 2^66: one key takes all
    out, lse = c.attend(0, big, table, lens)
    check_attend(c, 0, big, table, lens, None, None, out, lse)
    tiny = q * 2.0 ** -100
    out, lse = c.attend(0, tiny, table, lens)
    check_attend(c, 0, tiny, table, lens, None, None, out, lse)
    zero = torch.zeros_like(q)
    out, lse = c.attend(0, zero, table, lens)
    check_attend(c, 0, zero, table, lens, None, None, out, lse)
    if pool != "bf16":                                     # value scales far apart
        c.v_scale[0, ::3] = 2.0 ** 40
        c.v_scale[0, 1::3] = 2.0 ** -100
        out, lse = c.attend(0, q, table, lens)
        check_attend(c, 0, q, table, lens, None, None, out, lse)
    # a visible row that is not finite shows
    if pool == "bf16":
        c.v[0, 7, 3, 0, 11] = float("nan")
        out, _ = c.attend(0, q, table, lens)
        assert bool(out[0, :, 11].isnan().all()) and int(out.isnan().sum()) == 8
    else:
        c.k_scale[0, 7, 3] = float("nan")
        assert bool(c.attend(0, q, table, lens)[0].isnan().all())


def test_attend_takes_slices_and_gives_the_same_bits_every_time():
    g = rng(6)
    c = make_cache("bf16", 1, 300, 16, 2, 128, 5)
    table, lens = scattered(g, 3, 90, 300), ints([1300, 40, 777])
    fused = randn(g, 3, 1, 12, 128, dtype=BF16)
    q = fused[:, 0, 2:10]
    out, lse = c.attend(0, q, table, lens)
    check_attend(c, 0, q, table, lens, None, None, out, lse)
    for _ in range(5):
        again = c.attend(0, q, table, lens)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    # rows of a batch do not depend on the others
    o1, l1 = c.attend(0, q[1:2], table[1:2].contiguous(), lens[1:2])
    check_attend(c, 0, q[1:2], table[1:2], lens[1:2], None, None, o1, l1)
    given = torch.empty_like(out), torch.empty_like(lse)
    assert c.attend(0, q, table, lens, out=given[0], lse=given[1])[0] is given[0]
    assert torch.equal(given[0], out) and torch.equal(given[1], lse)


def test_offsets_beyond_32_bits():
    """A pool of 2.6e9 codes: the last pages lie past 2^31 elements."""
    D, ps = 256, 64
    pages = 160000
    c = pi0x.KVCache.empty(1, pages, ps, 1, D, "e4m3")
    assert c.k.numel() > 2 ** 31
    g = rng(8)
    table = ints([[pages - 1, 0, pages - 2, pages // 2 + 7]])
    k, v = randn(g, 1, 250, 1, D, dtype=BF16), randn(g, 1, 250, 1, D, dtype=BF16)
    c.write(0, k, v, table, ints([0]))
    got = c.read(table, ints([250]), 250, dtype=F32)
    for x, y in zip(got[:2], (k, v)):
        y = y[0, :, 0].float()
        top = y.abs().amax(-1, keepdim=True)
        assert bool(((x[0, 0, 0] - y).abs() <= 2.0 ** -4 * y.abs() + top / 224 * 2.0 ** -10).all())
    q = randn(g, 1, 8, D, dtype=BF16)
    out, lse = c.attend(0, q, table, ints([250]))
    kk, vv = got[0][0, 0, 0].double(), got[1][0, 0, 0].double()
    p = torch.softmax(q[0].double() @ kk.T / 16, -1)
    tol = half_step(BF16) * (p @ vv).abs() + (half_step(BF16) + 1e-4) * (p @ vv.abs())
    assert bool(((out[0].double() - p @ vv).abs() <= tol).all())


# ---- streams, graphs, runs together --------------------------------------------------


def test_calls_on_two_streams_at_once():
    g = rng(10)
    c = make_cache("bf16", 1, 400, 16, 1, 256, 5)
    tables = [scattered(g, 2, 60, 400) for _ in range(2)]
    qs = [randn(g, 2, 8, 256, dtype=BF16) for _ in range(2)]
    lens = ints([900, 333])
    want = [c.attend(0, q, t, lens) for q, t in zip(qs, tables)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(c.attend(0, qs[i % 2], tables[i % 2], lens))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_calls_from_several_threads():
    g = rng(12)
    caches = [make_cache("int8", 1, 200, 16, 1, 256, 30 + i) for i in range(4)]
    table, lens = scattered(g, 2, 60, 200), ints([900, 333])
    q, k, v = (randn(g, 2, 1, h, 256, dtype=BF16) for h in (8, 1, 1))
    bases = [1e4, 5e5, 1e2, 1e6]

    def step(i):
        qo = caches[i].write(0, k, v, table, lens - 1, q=q, rope_base=bases[i])
        return (qo,) + caches[i].attend(0, qo[:, 0], table, lens)

    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()

    def many(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [step(i) for _ in range(20)]
            torch.cuda.current_stream().synchronize()
        return got

    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        for i, got in enumerate(pool.map(many, range(4))):
            for one in got:
                assert all(torch.equal(x, y) for x, y in zip(one, want[i])), i


FIRST_CALLS = """
import torch
from vla_flow_matching_b200 import pi0x
c = pi0x.KVCache.empty(2, 1800, 16, 1, 256, "e4m3")
q, k, v = (torch.randn(2, 1, h, 256, device="cuda", dtype=torch.bfloat16) for h in (8, 1, 1))
table = torch.arange(1800, device="cuda", dtype=torch.int32).view(2, 900)
start = torch.tensor([1900, 3], device="cuda", dtype=torch.int32)
lens = start + 1
def step():
    a, b = pi0x.qk_norm_rope(q, k, start)
    c.write(0, b, v, table, start)
    c.write(1, k, v, table, start, q=q, rope_base=10000.0)
    return (a,) + c.attend(0, a[:, 0], table, lens) + c.attend(0, a[:, 0], table[:, :4].contiguous(), lens) + \
        c.read(table, lens, 1901)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, step()))
print("same")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_the_pools_of_a_cache_stay_its_own():
    c = pi0x.KVCache.empty(1, 2, 16, 1, 64)
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(c, name, c.k)


def test_captured_step_follows_its_inputs():
    """Write and attend captured once; each replay writes the next token and sees it.  A
    second graph of the same calls keeps its own workspace."""
    g = rng(11)
    B, H, kv, D, ps = 2, 8, 1, 256, 16
    c = make_cache("e4m3", 1, 200, ps, kv, D, 5)
    d = make_cache("e4m3", 1, 200, ps, kv, D, 5)
    table, start = scattered(g, B, 80, 200), ints([1000, 30])
    lens = start + 1
    q, k, v = (randn(g, B, 1, h, D, dtype=BF16) for h in (H, kv, kv))

    def step(cache):
        qo = cache.write(0, k, v, table, start, q=q, rope_base=10000.0)
        return (qo,) + cache.attend(0, qo[:, 0], table, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c)
        step(d)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step(c)))
    for i in range(4):
        for x in (q, k, v):
            x.copy_(randn(g, *x.shape))
        start.add_(1)
        lens.add_(1)
        graph, got = graphs[i % 2]
        graph.replay()
        want = step(d)
        for x, y in zip(got, want):
            assert torch.equal(x, y), i
    torch.cuda.synchronize()
    assert torch.equal(c.k.view(torch.uint8), d.k.view(torch.uint8)) and torch.equal(c.k_scale, d.k_scale)


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
def test_prefix_then_tokens_together(pool):
    """A padded prefix written at once, then four tokens one by one, each attended over all
    that is there: against the 64-bit formula over what the pages hold."""
    g = rng(12)
    B, H, kv, D, ps, P = 3, 14, 2, 128, 12, 100
    per = -(-(P + 4) // ps)
    c = pi0x.KVCache.empty(2, B * per, ps, kv, D, pool)
    table, lens = scattered(g, B, per, c.num_pages), ints([100, 0, 61])
    gain = 0.1 * randn(g, D)
    for layer in range(2):
        k, v = randn(g, B, P, kv, D, dtype=BF16), randn(g, B, P, kv, D, dtype=BF16)
        c.write(layer, k, v, table, torch.zeros_like(lens), lens, k_gain=gain, rope_base=10000.0)
    for _ in range(4):
        for layer in range(2):
            q, k, v = (randn(g, B, 1, h, D, dtype=BF16) for h in (H, kv, kv))
            qo = c.write(layer, k, v, table, lens, q=q, q_gain=gain, k_gain=gain, rope_base=10000.0)
            check_rotated(qo, q, gain, lens.long()[:, None], 10000.0)
            out, lse = c.attend(layer, qo[:, 0], table, lens + 1)
            check_attend(c, layer, qo[:, 0], table, lens + 1, None, None, out, lse)
        lens = lens + 1
    assert bool((c.read(table, lens, P + 4)[2].sum(1) == lens).all())


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B", [1, 4], ids=["loop", "multi"])
def test_sampler_on_a_cache_matches_contiguous_prefixes(pool, B):
    """pi0x_sample_cache gives, bit for bit, what pi0x_sample gives on the K/V the pages hold."""
    from vla_flow_matching_b200 import synth
    import dataclasses
    wl = synth.WORKLOADS["tiny"]
    inp = synth.make_inputs(wl)
    dims = wl.dims
    sampler = pi0x.Sampler(dims, inp.weights, pi0x.PI0X_BF16)
    g = rng(13)
    P, ps = 90, 16
    c = pi0x.KVCache.empty(dims.depth, 40, ps, 1, 256, pool)
    table = scattered(g, B, -(-P // ps), 40)
    lens = ints([[90, 33, 0, 64][b] for b in range(B)])
    start = torch.zeros_like(lens)
    for layer in range(dims.depth):
        k, v = randn(g, B, P, 1, 256, dtype=BF16), randn(g, B, P, 1, 256, dtype=BF16)
        c.write(layer, k, v, table, start, lens, rope_base=10000.0)
    mask = (torch.rand(B, P, device="cuda", generator=g) < 0.9).to(torch.uint8)
    state, x1 = randn(g, B, dims.state_dim), randn(g, B, dims.horizon, dims.action_dim)
    k, v, seen = c.read(table, lens, P, mask=mask)
    want = sampler.sample([k[l, :, 0].contiguous() for l in range(dims.depth)],
                          [v[l, :, 0].contiguous() for l in range(dims.depth)], seen, state, x1, wl.num_steps)
    sampler.sync()
    got = sampler.sample_cache(c, table, lens, P, state, x1, wl.num_steps, mask=mask)
    sampler.sync()
    assert torch.equal(got, want) and bool(got.isfinite().all())
    host = sampler.sample_cache(c, table, lens, P, state.cpu(), x1.cpu(), wl.num_steps, mask=mask)
    sampler.sync()
    assert torch.equal(host, want.cpu())
    with pytest.raises(pi0x.Pi0xError) as e:
        sampler.sample_cache(pi0x.KVCache.empty(dims.depth + 1, 40, ps), table, lens, P, state, x1, wl.num_steps)
    assert e.value.status == pi0x.PI0X_EINVAL
    sampler.close()
