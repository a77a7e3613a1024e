"""When the attention step shares a cache's slots among blocks, seen in the
workspace that it asks for (none for one block): far from where the two forms'
measured times cross, on both sides, at each headdim and type."""
from __future__ import annotations

import ctypes
import os

import pytest

import mamba_chunked_ssd_amd as ssd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ssd.LIB_PATH):
        from mamba_chunked_ssd_amd import build
        build.build()
    return ssd.load_library()


def blocks(lib, d, dtype, batch, kv, slots, group=4):
    shape = ssd.AttnShape(batch, 1, group * kv, kv, d, slots, 0, d ** -0.5, dtype)
    need = lib.ssd_window_attn_step_workspace_size(ctypes.byref(shape))
    # (rows of headdim + 2 floats for each block and head, two regions of whole 256 bytes)
    per = batch * group * kv * (d + 2) * 4
    return 1 if need == 0 else need // per


BF16, F32 = ssd.SSD_DTYPE_BF16, ssd.SSD_DTYPE_F32


# (headdim, type, slots that one block takes in about 9 us of the device's and 11 of a call, in 25 for 9 and 15)
@pytest.mark.parametrize("d,dtype,few,many", [(32, BF16, 2048, 8192), (64, BF16, 1536, 6144), (128, BF16, 512, 2816),
                                              (32, F32, 512, 2560), (64, F32, 256, 1152), (128, F32, 64, 320)])
def test_few_sequences(lib, d, dtype, few, many):
    for batch, kv in ((1, 1), (1, 8), (4, 8)):
        assert blocks(lib, d, dtype, batch, kv, few) == 1
        assert blocks(lib, d, dtype, batch, kv, many) >= 4


# enough walks that memory, or the compute units, are busy with one block each
@pytest.mark.parametrize("d,dtype,slots", [(32, BF16, 4096), (64, BF16, 6144), (128, BF16, 2560), (32, F32, 4096), (128, F32, 4096)])
def test_many_sequences(lib, d, dtype, slots):
    for batch in (32, 64, 512):
        assert blocks(lib, d, dtype, batch, 8, slots) == 1


# half of the second round's compute units would have none
@pytest.mark.parametrize("d,dtype,slots", [(64, F32, 4096), (128, F32, 2052)])
def test_walks_that_leave_units_idle(lib, d, dtype, slots):
    assert blocks(lib, d, dtype, 48, 8, slots) > 1


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F32)])
def test_no_more_blocks_than_four_rounds(lib, d, dtype):
    for batch, kv, group in ((1, 1, 1), (3, 8, 4), (7, 4, 40), (15, 8, 1), (20, 8, 2)):
        n = blocks(lib, d, dtype, batch, kv, 20000, group)
        assert n * batch * kv * -(-group // 32) <= 1024
