"""What the paged prefix cache's calls take and refuse, seen from the host before any launch (CPU
only; a call that is taken ends at its launch where there is no device)."""
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
