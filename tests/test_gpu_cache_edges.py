"""Edges of the paged prefix cache on the GPU: how exact what the calls return is, and inputs
that the contract allows but that are rare.  Tolerances count roundings, as in
test_gpu_cache.py.
"""
import dataclasses
import math

import pytest
import torch

from vla_flow_matching_b200 import build, pi0x, synth

from .test_gpu_cache import (BF16, F32, U32, check_attend, check_rotated, half_step, ints, make_cache, randn, rng, rotated,
                             rotated_slack, scattered, slots)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


# ---- attention -----------------------------------------------------------------------


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("B,H,kv,D,n", [(1, 8, 1, 256, 2), (3, 4, 2, 64, 300), (2, 20, 1, 128, 77), (1, 8, 1, 256, 6000)])
def test_attention_weights_keep_their_bits(pool, B, H, kv, D, n):
    """Values of +1 and -1 whose weights are nearly equal: outputs far below the weights, which show
    what a weight's rounding costs.  Only one element of a query and of a key is not zero, so a
    score is one product."""
    g = rng(n + D)
    ps = 16
    per = -(-n // ps)
    c = pi0x.KVCache.empty(1, B * per, ps, kv, D, pool)
    table = torch.arange(B * per, device="cuda", dtype=torch.int32).view(B, per)
    code = torch.randint(-7, 8, (B * per, ps, kv), device="cuda", generator=g).float()  # exact in every type
    c.k[0, ..., 3] = code.to(c.k.dtype)
    sign = 1.0 - 2.0 * (torch.arange(B * per * ps, device="cuda").view(-1, ps, 1) % 2)
    c.v[0] = sign[..., None].expand(-1, -1, kv, D).to(c.v.dtype)
    if pool != "bf16":
        c.k_scale.fill_(1.0)
        c.v_scale.fill_(1.0)
    q = torch.zeros(B, H, D, device="cuda", dtype=BF16)
    q[..., 3] = 1.0 + torch.arange(H, device="cuda").to(BF16) / 64
    scale = 0.0013
    out, lse = c.attend(0, q, table, ints([n] * B), scale=scale)
    k = code.view(B, per * ps, kv)[:, :n].double()
    s = torch.einsum("bhg,bnh->bhgn", q[..., 3].double().view(B, kv, -1), k).flatten(1, 2) * scale
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    o = (p * sign.view(B, -1)[:, None, :n].double()).sum(-1)
    # a product and the scale's, the exponential, and the sums of n weights in fp32
    delta = 8 * U32 * (s.abs().amax(-1) + 1) + n * U32 + 2.0 ** -21
    weight = 2.0 ** -15 if pool == "bf16" else half_step(torch.float16)
    tol = half_step(BF16) * o.abs() * (1 + 2 ** -6) + (weight + 2 * delta) * 1.01
    err = (out.double() - o[..., None]).abs().amax(-1)
    assert bool((err <= tol).all()), float((err - tol).max())
    assert bool(((lse.double() - z).abs() <= delta + 4 * U32 * z.abs()).all())


@pytest.mark.parametrize("D,H", [(256, 8), (64, 20)])
@pytest.mark.parametrize("far", [0.0, 30.0])
def test_infinite_values_stay_infinite(D, H, far):
    c = pi0x.KVCache.empty(1, 4, 16, 1, D, "bf16")
    c.v.fill_(1.0)
    c.v[0, 1, 3, 0, 5], c.v[0, 2, 7, 0, 9] = math.inf, -math.inf
    c.k[0, 1, 3, 0, 0] = -1.0                                # the infinite value's weight is e^-far
    q = torch.zeros(1, H, D, device="cuda", dtype=BF16)
    q[..., 0] = 1.0
    out, lse = c.attend(0, q, ints([[0, 1, 2, 3]]), ints([64]), scale=far)
    want = torch.ones_like(out)
    want[..., 5], want[..., 9] = math.inf, -math.inf
    assert torch.equal(out, want) and bool(lse.isfinite().all())


@pytest.mark.parametrize("pool", ["e4m3", "int8"])
@pytest.mark.parametrize("B,H,kv,D,n", [(2, 8, 1, 256, 500), (3, 20, 1, 64, 99), (1, 8, 2, 128, 9000)])
def test_scales_of_either_sign_and_zero(pool, B, H, kv, D, n):
    """A row stands for code * scale, whatever the scale's sign."""
    g = rng(n)
    per = -(-n // 16)
    c = make_cache(pool, 1, B * per, 16, kv, D, n)
    table, lens = scattered(g, B, per, B * per), ints([n - 7 * b for b in range(B)])
    for s in (c.k_scale, c.v_scale):
        s.mul_(torch.randint(-1, 2, s.shape, device="cuda", generator=g))
    q = randn(g, B, H, D, dtype=BF16)
    out, lse = c.attend(0, q, table, lens)
    check_attend(c, 0, q, table, lens, None, None, out, lse)
    c.v_scale.fill_(-0.5)
    out, lse = c.attend(0, q, table, lens)
    check_attend(c, 0, q, table, lens, None, None, out, lse)
    c.v_scale.fill_(0.0)
    assert not bool(c.attend(0, q, table, lens)[0].any())


# ---- codes -------------------------------------------------------------------------------


def e4m3_of(y):
    """Values that rows of y (64 bits) stand for in e4m3 pages, and their scales, in 64 bits throughout."""
    part, power = torch.frexp(y.abs().amax(-1) / 448)  # exact at 448 * 2^n
    scale = torch.ldexp(torch.ones_like(part), torch.clamp(power - (part == 0.5).int(), min=-126))
    scale = torch.where(y.abs().amax(-1) == 0, 2.0 ** -126, scale)
    x = y / scale[..., None]
    step = torch.ldexp(torch.ones_like(x), torch.frexp(x.abs().clamp_min(2.0 ** -6))[1] - 4)
    return (x / step).round() * step, scale


@pytest.mark.parametrize("D,dtype,size,rounds,most", [
    (256, BF16, 1.0, 32, 6),              # 67 million values
    (128, F32, 1.0, 2, 2), (64, F32, 1.0, 2, 2),
    (256, F32, 2.0 ** -136, 1, 2), (64, BF16, 2.0 ** -131, 1, 2)])  # codes below 2^-126, where fp32 holds fewer bits
def test_e4m3_codes_are_those_of_the_formula(D, dtype, size, rounds, most):
    """Keys normed and rotated on their way into e4m3 pages have the 64-bit formula's codes.  Sines and
    cosines are exact to 2^-32, so a code may differ where a value lies that near to the border of two:
    about 2^-31 * 11 borders a value * 4 (pairs longer than their halves), 1 in 50 million.  In fp32 it
    is 1 in 2.5 million."""
    g = rng(D)
    B, T = 16, 2 ** 17 // D
    ps = 64
    c = pi0x.KVCache.empty(1, B * T // ps, ps, 1, D, "e4m3")
    table = torch.arange(B * T // ps, device="cuda", dtype=torch.int32).view(B, -1)
    zero = ints([0] * B)
    wrong = 0
    for i in range(rounds):
        k = (randn(g, B, T, 1, D) * size).to(dtype)
        gain, first = 0.2 * randn(g, D), torch.randint(0, 3000, (B, T), device="cuda", generator=g, dtype=torch.int32)
        c.write(0, k, k, table, zero, positions=first, k_gain=gain, rope_base=1e4)
        y = rotated(k, gain, first, 1e4, eps=float(torch.tensor(1e-6)))
        want, scale = e4m3_of(y)
        assert torch.equal(c.k_scale.view(B, T, 1).double(), scale)
        wrong += int((c.k.float().view(B, T, 1, D).double() != want).sum())
        want, scale = e4m3_of(k.double())  # values as they are: every code
        assert torch.equal(c.v_scale.view(B, T, 1).double(), scale)
        assert torch.equal(c.v.float().view(B, T, 1, D).double(), want)
    assert wrong <= most, wrong


@pytest.mark.parametrize("pool", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,hq,kv,norm,base", [
    (64, 6, 2, True, 1e4), (128, 3, 1, False, 1e2), (256, 8, 1, True, 5e5), (256, 0, 3, True, None), (64, 1, 1, False, 1.0)])
def test_rows_are_turned_at_their_positions_on_the_way_in(pool, dtype, D, hq, kv, norm, base):
    """Positions other than the slots; rows of both types and every head dim into pages of every type."""
    g = rng(D + kv)
    B, T, ps = 3, 23, 8
    c = pi0x.KVCache.empty(1, 3 * 6, ps, kv, D, pool)
    table, start, count = scattered(g, B, 6, c.num_pages), ints([0, 17, 4]), ints([23, 9, 0])
    pos = torch.randint(-1000, 200000, (B, T), device="cuda", generator=g, dtype=torch.int32)
    q = randn(g, B, T, hq, D, dtype=dtype) if hq else None
    k, v = randn(g, B, T, kv, D, dtype=dtype), randn(g, B, T, kv, D, dtype=dtype)
    gq, gk = (0.2 * randn(g, D) if norm else None for _ in range(2))
    qo = c.write(0, k, v, table, start, count, q=q, positions=pos, q_gain=gq if hq else None, k_gain=gk, rope_base=base)
    if hq:
        check_rotated(qo, q, gq, pos, base)
    y = rotated(k, gk, pos, base)
    for b in range(B):
        first, n = int(start[b]), int(count[b])
        for name, want in (("k", y[b, :n]), ("v", v[b, :n].double())):
            got, _ = slots(c, 0, name, table, b, first + n)
            top = want.abs().amax(-1, keepdim=True)
            # half a step: of the value (bf16, e4m3) or of the scale (int8); e4m3's least step is 2^-9 of
            # a scale that is at most top / 224
            step = {"bf16": half_step(BF16) * want.abs(), "int8": top / 254 * (1 + 2 ** -10),
                    "e4m3": 2.0 ** -4 * want.abs() + top / 224 * 2.0 ** -10}[pool]
            slack = 2 * rotated_slack(want) if name == "k" else 0.0
            assert bool(((got[first:] - want).abs() <= step * (1 + 2 ** -7) + slack).all()), (b, name)
        before, _ = slots(c, 0, "k", table, b, first)
        assert not bool(before.any())


# ---- layouts ---------------------------------------------------------------------------


def test_strides_of_dimensions_of_one_do_not_count():
    """torch leaves the stride of a dimension of size 1 at any value."""
    g = rng(14)
    D = 64
    q = randn(g, 3, 4, D, dtype=BF16)
    odd = torch.as_strided(q, (3, 1, 4, D), (4 * D, 3, D, 1))
    start = ints([5, 0, 700])
    want = pi0x.qk_norm_rope(q[:, None], q[:, None, :1], start)
    got = pi0x.qk_norm_rope(odd, torch.as_strided(q, (3, 1, 1, D), (4 * D, 1, 7, 1)), start)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c, d = (pi0x.KVCache.empty(1, 3, 4, 1, D) for _ in range(2))
    table, slot = ints([[0], [1], [2]]), ints([0, 3, 2])
    c.write(0, q[:, None, :1], q[:, None, 1:2], table, slot, rope_base=1e4)
    d.write(0, torch.as_strided(q, (3, 1, 1, D), (4 * D, 1, 7, 1)),
            torch.as_strided(q, (3, 1, 1, D), (4 * D, 5, 1, 1), D), table, slot, rope_base=1e4)
    assert torch.equal(c.k, d.k) and torch.equal(c.v, d.v)
    one = torch.as_strided(q, (1, 4, D), (3, D, 1))
    assert torch.equal(c.attend(0, one, table[:1], slot[:1] + 1)[0], c.attend(0, q[:1], table[:1], slot[:1] + 1)[0])


def test_inputs_that_require_gradients_are_plain_data():
    g = rng(19)
    q, k = (torch.nn.Parameter(randn(g, 2, 3, h, 64, dtype=BF16)) for h in (4, 2))
    gain = torch.nn.Parameter(0.1 * randn(g, 64))
    c, d = (pi0x.KVCache.empty(1, 2, 4, 2, 64) for _ in range(2))
    table, zero = ints([[0], [1]]), ints([0, 0])
    got = c.write(0, k, k * 2, table, zero, q=q, q_gain=gain, rope_base=1e4)
    want = d.write(0, k.detach(), k.detach() * 2, table, zero, q=q.detach(), q_gain=gain.detach(), rope_base=1e4)
    assert torch.equal(got, want) and torch.equal(c.k, d.k) and torch.equal(c.v, d.v)
    out, lse = c.attend(0, q[:, 0], table, zero + 3)
    assert not (got.requires_grad or out.requires_grad or lse.requires_grad)
    assert torch.equal(out, d.attend(0, q[:, 0].detach(), table, zero + 3)[0])


def test_reads_of_no_slots_take_their_mask():
    c = pi0x.KVCache.empty(2, 3, 4, 1, 64)
    table, lens = ints([[0, 1], [2, -1]]), ints([5, 0])
    for mask in (None, torch.zeros(2, 0, dtype=torch.uint8, device="cuda"), torch.zeros(2, 0, dtype=bool, device="cuda")):
        k, v, seen = c.read(table, lens, 0, mask=mask)
        assert k.shape == v.shape == (2, 2, 1, 0, 64) and seen.shape == (2, 0) and seen.dtype == torch.uint8
    with pytest.raises(ValueError):
        c.read(table, lens, 3, mask=torch.zeros(2, 0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        c.read(table, lens, 0, mask=torch.zeros(2, 1, dtype=torch.uint8, device="cuda"))


# ---- the sampler on a cache ------------------------------------------------------------


def test_sampler_buffers_settle_when_shapes_alternate():
    """After one round of two shapes, neither of which covers the other, calls allocate nothing."""
    dims = synth.WORKLOADS["tiny"].dims
    sampler = pi0x.Sampler(dims, synth.make_weights(dims, 0), pi0x.PI0X_BF16)
    g = rng(15)
    c = make_cache("bf16", dims.depth, 64, 64, 1, 256, 16)
    calls, free = [], []
    for B, P in ((48, 128), (1, 3000)):
        table = torch.randint(0, 64, (B, -(-P // 64)), device="cuda", generator=g, dtype=torch.int32)
        calls.append((table, ints([P - b for b in range(B)]), P, randn(g, B, dims.state_dim),
                      randn(g, B, dims.horizon, dims.action_dim)))
    first = []
    for i in range(6):
        table, lens, P, state, x1 = calls[i % 2]
        got = sampler.sample_cache(c, table, lens, P, state, x1, 2)
        sampler.sync()
        if i < 2:
            first.append(got)
        else:
            assert torch.equal(got, first[i % 2])
        free.append(torch.cuda.mem_get_info()[0])
    assert len(set(free[1:])) == 1, free
    sampler.close()


def test_sampler_on_a_cache_refuses_wrong_states_and_noise():
    dims = synth.WORKLOADS["tiny"].dims
    sampler = pi0x.Sampler(dims, synth.make_weights(dims, 0), pi0x.PI0X_BF16)
    c = pi0x.KVCache.empty(dims.depth, 4, 16)
    table, lens = ints([[0], [1]]), ints([16, 3])
    state, x1 = (torch.zeros(2, *shape, device="cuda") for shape in ((dims.state_dim,), (dims.horizon, dims.action_dim)))
    for bad in (dict(state=state[:1]), dict(x1=x1[:1]), dict(state=state.double()), dict(x1=x1.to(BF16)),
                dict(x1=x1.transpose(1, 2)), dict(state=state[:, ::2]), dict(x0=x1[:1]), dict(x0=x1.double()),
                dict(state=state.cpu().numpy()[:1]), dict(state=None), dict(x1=[0.0])):
        kw = dict(state=state, x1=x1)
        kw.update(bad)
        with pytest.raises((ValueError, pi0x.Pi0xError)):
            sampler.sample_cache(c, table, lens, 16, num_steps=1, **kw)
    got = sampler.sample_cache(c, table, lens, 16, state, x1, 1)
    sampler.sync()
    host = sampler.sample_cache(c, table, lens, 16, state.cpu().numpy(), x1.cpu().numpy(), 1)
    sampler.sync()
    assert torch.equal(got.cpu(), torch.from_numpy(host))
    sampler.close()


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_fp32_sampler_on_a_cache_matches_contiguous_prefixes(pool):
    dims = synth.WORKLOADS["tiny"].dims
    sampler = pi0x.Sampler(dims, synth.make_weights(dims, 0), pi0x.PI0X_FP32)
    g = rng(17)
    B, P = 2, 70
    c = make_cache(pool, dims.depth, 12, 16, 1, 256, 18)
    table, lens = scattered(g, B, 5, 12), ints([70, 31])
    mask = (torch.rand(B, P, device="cuda", generator=g) < 0.9).to(torch.uint8)
    state, x1 = randn(g, B, dims.state_dim), randn(g, B, dims.horizon, dims.action_dim)
    k, v, seen = c.read(table, lens, P, mask=mask)
    want = sampler.sample([x.contiguous() for x in k[:, :, 0]], [x.contiguous() for x in v[:, :, 0]], seen, state, x1, 2)
    sampler.sync()
    got = sampler.sample_cache(c, table, lens, P, state, x1, 2, mask=mask)
    sampler.sync()
    assert torch.equal(got, want) and bool(got.isfinite().all())
    sampler.close()
