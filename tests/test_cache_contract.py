"""What the paged prefix cache's calls take and refuse, seen from the host before any launch (CPU
only; a call that is taken ends at its launch where there is no device)."""
import os
import subprocess
import sys

import pytest
import torch

from vla_flow_matching_b200 import build as B
from vla_flow_matching_b200 import pi0x
from vla_flow_matching_b200.pi0x import Rotation

from .test_cache_refusals import BF16, E4M3, EINVAL, F32, INT8, PTR, cache, rows

# the calls below that are taken get addresses that nothing may read: never where they could be launched
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")
ROT = Rotation(0, 0, 0, 1e-6, 1e4)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return pi0x.load()


def rope_into(lib, out, shape, dtype=BF16):
    b, t, h = shape
    return lib.pi0x_qk_norm_rope(dtype, b, t, h, 0, 128, rows(), None, None, ROT, out, None, None)


# (batch, tokens, heads), strides: rows of different indices share memory although every stride alone is 128 or more
SHARED = [((2, 2, 2), (128, 128, 128)), ((2, 2, 2), (256, 256, 128)), ((2, 2, 2), (256, 128, 128)),
          ((2, 3, 4), (1024, 384, 128)), ((2, 3, 1), (256, 128, 128)), ((3, 1, 4), (-384, 0, 128)),
          ((2, 2, 2), (-2 ** 63, 0, 128))]


@no_gpu
@pytest.mark.parametrize("shape,strides", SHARED, ids=str)
def test_outputs_that_share_memory_across_dimensions_are_refused(lib, shape, strides):
    assert rope_into(lib, rows(PTR, *strides), shape) == EINVAL
    assert b"overlap" in lib.pi0x_last_error()
    b, t, h = shape
    assert lib.pi0x_cache_write(cache(), 0, BF16, b, t, rows(), rows(), PTR, 4, PTR, None, ROT, h, rows(),
                                rows(PTR, *strides), None) == EINVAL
    assert b"overlap" in lib.pi0x_last_error()


@no_gpu
@pytest.mark.parametrize("shape,strides", [
    ((2, 3, 4), (1536, 512, 128)), ((2, 3, 4), (128, 256, 768)), ((2, 3, 4), (-4096, 1024, -256)),
    ((1, 1, 1), (0, 0, 0)), ((1, 3, 1), (0, 128, 0)), ((2, 1, 1), (2 ** 62, 0, 0)), ((2, 2, 2), (192, 1024, 2048))],
    ids=str)
def test_outputs_whose_rows_lie_apart_are_taken(lib, shape, strides):
    assert rope_into(lib, rows(PTR, *strides), shape) != EINVAL
    assert rope_into(lib, rows(PTR, *strides), shape, F32) != EINVAL


# ---- attention's workspace and sizes -------------------------------------------------------

EVEN = [dict(), dict(dtype=E4M3, k_scale=PTR, v_scale=PTR), dict(dtype=INT8, k_scale=PTR, v_scale=PTR, head_dim=256)]


@no_gpu
@pytest.mark.parametrize("kw", EVEN, ids=str)
@pytest.mark.parametrize("heads", [8, 40])
def test_attention_refuses_a_missing_or_short_workspace(lib, kw, heads):
    """A table of 65536 slots is shared out evenly, with parts in the workspace."""
    c, pages = cache(**kw), 4096
    need = lib.pi0x_cache_attention_workspace(c, 1, heads, pages)
    assert need > 0

    def call(work, size):
        return lib.pi0x_cache_attention(c, 0, 1, heads, rows(), PTR, pages, PTR, None, 0, 1.0, PTR, None, work, size, None)

    for work, size in ((None, need), (PTR + 4, need), (PTR, need - 1), (PTR, 0)):
        assert call(work, size) == EINVAL and b"workspace" in lib.pi0x_last_error()
    assert call(PTR, need) != EINVAL


@pytest.mark.parametrize("B,heads,pages", [(65536, 8, 4096), (1, 131072, 4096), (60000, 60000, 64), (65535, 8, 1 << 23)])
def test_sizes_that_attention_refuses_need_no_workspace(lib, B, heads, pages):
    c = cache()
    assert lib.pi0x_cache_attention(c, 0, B, heads, rows(), PTR, pages, PTR, None, 0, 1.0, PTR, None, PTR, 1 << 50,
                                    None) == EINVAL
    assert lib.pi0x_cache_attention_workspace(c, B, heads, pages) == 0


@no_gpu
@pytest.mark.parametrize("t", [3, -5, 2 ** 62 + 1])
def test_attention_does_not_use_the_token_stride(lib, t):
    call = [cache(), 0, 1, 8, rows(t=t), PTR, 4, PTR, None, 0, 1.0, PTR, None, None, 0, None]
    assert lib.pi0x_cache_attention(*call) != EINVAL
    call[4] = rows(t=t, h=100)
    assert lib.pi0x_cache_attention(*call) == EINVAL


# ---- the sampler beside another torch, or none ---------------------------------------------

WITHOUT = {
    "a torch without the exchange interface": "import torch; del torch.Tensor.__dlpack_c_exchange_api__",
    "no binding": "import sys; sys.modules['vla_flow_matching_b200._binding'] = None",
    "no torch": "import sys; sys.modules['torch'] = None",
}
LOADS = """
from vla_flow_matching_b200 import pi0x
assert pi0x.load().pi0x_version() >= 1 and pi0x.Sampler is not None
try:
    pi0x.qk_norm_rope(None)
except ImportError as e:
    print("refused:", e)
"""


@pytest.mark.parametrize("name", WITHOUT)
def test_the_library_loads_without_what_only_the_cache_calls_need(lib, name):
    r = subprocess.run([sys.executable, "-c", WITHOUT[name] + LOADS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "refused: the paged-cache calls" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("how", ["error", "missing"])
def test_a_binding_that_does_not_compile_leaves_the_library(monkeypatch, tmp_path, capsys, how):
    compiled = []

    def run(cmd, **kw):
        if cmd[0] == "gcc":
            if how == "missing":
                raise FileNotFoundError("gcc")
            return subprocess.CompletedProcess(cmd, 1, "", "no such type")
        open(cmd[cmd.index("-o") + 1], "w").close()
        compiled.append(cmd)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name in ("BUILD", "LIB", "BINDING", "NO_BINDING"):
        monkeypatch.setattr(B, name, str(tmp_path / name), raising=False)
    open(B.BINDING, "w").close()  # of an earlier build
    monkeypatch.setattr(B.subprocess, "run", run)
    assert B.build() == B.LIB and os.path.exists(B.LIB) and not os.path.exists(B.BINDING)
    assert "paged-cache" in capsys.readouterr().err
    n = len(compiled)
    assert B.up_to_date() and B.build() == B.LIB and len(compiled) == n  # not again and again
