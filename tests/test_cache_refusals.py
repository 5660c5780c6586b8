"""Refusals of the paged prefix cache calls: seen from the host, before any launch (CPU only)."""
import ctypes

import pytest
import torch

from vla_flow_matching_b200 import build as B
from vla_flow_matching_b200 import pi0x
from vla_flow_matching_b200.pi0x import Cache, Rotation, Rows

EINVAL, EUNSUP = pi0x.PI0X_EINVAL, pi0x.PI0X_EUNSUPPORTED
PTR = 1 << 20  # stands for an aligned device address; nothing reads it
F32, BF16, E4M3, INT8 = pi0x.PI0X_DTYPE_F32, pi0x.PI0X_DTYPE_BF16, pi0x.PI0X_DTYPE_E4M3, pi0x.PI0X_DTYPE_INT8


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pi0x.load()


def cache(**kw):
    d = dict(k=PTR, v=PTR, k_scale=0, v_scale=0, layers=2, num_pages=4, page_size=16, kv_heads=2, head_dim=128,
             dtype=BF16)
    d.update(kw)
    return Cache(*[d[n] for n, _ in Cache._fields_])


def rows(data=PTR, b=1024, t=256, h=128):
    return Rows(data, b, t, h)


BAD_CACHES = [
    (dict(k=0), EINVAL), (dict(v=0), EINVAL), (dict(k=PTR + 8), EINVAL), (dict(layers=0), EINVAL),
    (dict(num_pages=0), EINVAL), (dict(page_size=0), EINVAL), (dict(kv_heads=0), EINVAL), (dict(kv_heads=65536), EINVAL),
    (dict(head_dim=96), EUNSUP), (dict(head_dim=512), EUNSUP), (dict(dtype=F32), EUNSUP), (dict(dtype=7), EUNSUP),
    (dict(dtype=E4M3), EINVAL), (dict(dtype=INT8, k_scale=PTR), EINVAL), (dict(dtype=INT8, k_scale=PTR, v_scale=PTR + 2), EINVAL),
    (dict(num_pages=1 << 27), EINVAL),  # 2 layers x 2^27 pages x 16 rows: 2^32 rows
]


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=[str(k) for k, _ in BAD_CACHES])
def test_bad_caches_are_refused_by_every_call(lib, kw, status):
    c, r = cache(**kw), rows()
    assert lib.pi0x_cache_write(c, 0, BF16, 1, 1, r, r, PTR, 4, PTR, None, None, 0, None, None, None) == status
    assert lib.pi0x_cache_read(c, 0, 1, 1, 8, PTR, 4, PTR, None, BF16, PTR, PTR, None, None) == status
    assert lib.pi0x_cache_attention(c, 0, 1, 8, r, PTR, 4, PTR, None, 0, 1.0, PTR, None, PTR, 1 << 40, None) == status
    assert lib.pi0x_cache_attention_workspace(c, 1, 8, 4) == 0
    assert lib.pi0x_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), EINVAL), (dict(layer=-1), EINVAL), (dict(dtype=E4M3), EUNSUP), (dict(B=0), EINVAL),
    (dict(T=0), EINVAL), (dict(k=None), EINVAL), (dict(k=rows(PTR + 4)), EINVAL), (dict(v=rows(t=252)), EINVAL),
    (dict(v=rows(h=100)), EINVAL), (dict(v=rows(b=4)), EINVAL), (dict(table=None), EINVAL), (dict(pages=0), EINVAL),
    (dict(pages=1 << 27), EINVAL), (dict(start=None), EINVAL), (dict(heads=8), EINVAL),
    (dict(heads=8, rot=Rotation(0, 0, 0, 1e-6, 1e4)), EINVAL), (dict(heads=-1), EINVAL),
    (dict(rot=Rotation(0, PTR, 0, 0.0, 1e4)), EINVAL), (dict(rot=Rotation(0, 0, 0, 1e-6, 0.5)), EINVAL),
    (dict(rot=Rotation(0, 0, 0, 1e-6, float("nan"))), EINVAL), (dict(rot=Rotation(0, PTR + 2, 0, 1e-6, 1e4)), EINVAL),
    (dict(rot=Rotation(0, 0, PTR + 1, 1e-6, 1e4)), EINVAL), (dict(start=PTR + 2), EINVAL), (dict(table=PTR + 2), EINVAL),
    (dict(B=1 << 16, T=1 << 14), EINVAL),
], ids=str)
def test_cache_write_refuses(lib, kw, status):
    d = dict(layer=0, dtype=BF16, B=1, T=1, k=rows(), v=rows(), table=PTR, pages=4, start=PTR, rot=None, heads=0)
    d.update(kw)
    assert lib.pi0x_cache_write(cache(), d["layer"], d["dtype"], d["B"], d["T"], d["k"], d["v"], d["table"], d["pages"],
                                d["start"], None, d["rot"], d["heads"], None, None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(layer0=1, layers=2), EINVAL), (dict(layers=0), EINVAL), (dict(P=0), EINVAL), (dict(lens=None), EINVAL),
    (dict(lens=PTR + 3), EINVAL), (dict(k=None), EINVAL), (dict(k=PTR + 8), EINVAL), (dict(dtype=INT8), EUNSUP), (dict(B=1 << 16, P=1 << 15), EINVAL),
], ids=str)
def test_cache_read_refuses(lib, kw, status):
    d = dict(layer0=0, layers=1, B=1, P=8, lens=PTR, dtype=BF16, k=PTR)
    d.update(kw)
    assert lib.pi0x_cache_read(cache(), d["layer0"], d["layers"], d["B"], d["P"], PTR, 4, d["lens"], None, d["dtype"],
                               d["k"], PTR, None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), EINVAL), (dict(heads=0), EINVAL), (dict(heads=7), EINVAL), (dict(lens=None), EINVAL),
    (dict(out=None), EINVAL), (dict(out=PTR + 2), EINVAL), (dict(q=None), EINVAL), (dict(q=rows(PTR + 2)), EINVAL),
    (dict(mask=PTR, mask_len=0), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(B=65536), EINVAL), (dict(heads=65536), EINVAL), (dict(B=60000, heads=60000), EINVAL),
    (dict(scale=3e38), EINVAL), (dict(lens=PTR + 1), EINVAL),
], ids=str)
def test_cache_attention_refuses(lib, kw, status):
    d = dict(layer=0, B=1, heads=8, q=rows(), lens=PTR, mask=None, mask_len=0, scale=0.1, out=PTR)
    d.update(kw)
    assert lib.pi0x_cache_attention(cache(), d["layer"], d["B"], d["heads"], d["q"], PTR, 4, d["lens"], d["mask"],
                                    d["mask_len"], d["scale"], d["out"], None, PTR, 1 << 40, None) == status


def test_cache_attention_refuses_a_short_workspace(lib):
    need = lib.pi0x_cache_attention_workspace(cache(), 1, 8, 64)
    if need:
        for work, size in ((None, need), (PTR + 4, need), (PTR, need - 1)):
            assert lib.pi0x_cache_attention(cache(), 0, 1, 8, rows(), PTR, 64, PTR, None, 0, 1.0, PTR, None, work, size,
                                            None) == EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(rot=None), EINVAL), (dict(dtype=INT8), EUNSUP), (dict(dim=32), EUNSUP), (dict(heads=0, kv=0), EINVAL),
    (dict(heads=-1), EINVAL), (dict(B=0), EINVAL), (dict(q=None), EINVAL), (dict(k_out=None), EINVAL),
    (dict(k_out=rows(PTR + 8)), EINVAL), (dict(rot=Rotation(PTR, 0, 0, -1.0, 1e4)), EINVAL),
    (dict(rot=Rotation(0, 0, 0, 1e-6, -1.0)), EINVAL), (dict(dtype=F32, q=rows(t=2)), EINVAL),
    (dict(B=1 << 20, T=1 << 10), EINVAL),
], ids=str)
def test_qk_norm_rope_refuses(lib, kw, status):
    d = dict(dtype=BF16, B=1, T=1, heads=8, kv=1, dim=128, q=rows(), k=rows(), rot=Rotation(0, 0, 0, 1e-6, 1e4),
             k_out=rows())
    d.update(kw)
    assert lib.pi0x_qk_norm_rope(d["dtype"], d["B"], d["T"], d["heads"], d["kv"], d["dim"], d["q"], d["k"], None,
                                 d["rot"], rows(), d["k_out"], None) == status


@pytest.mark.parametrize("b,t,h", [(0, 256, 128), (1024, 0, 128), (1024, 256, 0), (1024, 256, 64), (1024, -64, 128)])
def test_outputs_whose_rows_overlap_are_refused(lib, b, t, h):
    bad, rot = rows(PTR, b, t, h), Rotation(0, 0, 0, 1e-6, 1e4)
    assert lib.pi0x_qk_norm_rope(BF16, 2, 2, 2, 0, 128, rows(), None, None, rot, bad, None, None) == EINVAL
    assert lib.pi0x_qk_norm_rope(BF16, 2, 2, 0, 2, 128, None, rows(), None, rot, None, bad, None) == EINVAL
    assert lib.pi0x_cache_write(cache(), 0, BF16, 2, 2, rows(), rows(), PTR, 4, PTR, None, rot, 2, rows(), bad,
                                None) == EINVAL
    assert b"overlap" in lib.pi0x_last_error()


def test_sample_cache_refuses_null_arguments(lib):
    assert lib.pi0x_sample_cache(None, cache(), 1, 8, PTR, 4, PTR, None, PTR, PTR, 1, PTR, None) == EINVAL
    assert lib.pi0x_sample_cache(None, None, 1, 8, None, 0, None, None, None, None, 1, None, None) == EINVAL


def test_python_binding_refuses_host_tensors_and_wrong_layouts():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pi0x.qk_norm_rope(q, q)
    pool = torch.zeros(1, 4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pi0x.KVCache(pool, pool)
    with pytest.raises(ValueError, match="contiguous"):
        pi0x.KVCache(pool.transpose(2, 3), pool.transpose(2, 3))
    with pytest.raises(ValueError, match="one type"):
        pi0x.KVCache(pool.half(), pool.half())
    with pytest.raises(ValueError, match="k_scale"):
        pi0x.KVCache(pool.to(torch.int8), pool.to(torch.int8))
    with pytest.raises(ValueError, match="take none"):
        pi0x.KVCache(pool, pool, torch.zeros(1, 4, 16, 2), torch.zeros(1, 4, 16, 2))
    with pytest.raises(ValueError, match="scales"):
        pi0x.KVCache(pool.to(torch.int8), pool.to(torch.int8), torch.zeros(1, 4, 16), torch.zeros(1, 4, 16))
    with pytest.raises(ValueError, match="dtype"):
        pi0x.KVCache.empty(1, 1, 1, dtype="fp4")
