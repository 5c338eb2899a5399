"""Refusals of the beam operators, before anything is launched (stand-in addresses, never dereferenced)."""
import ctypes

import pytest
import torch

import rank_lm_head_amd as lr
from rank_lm_head_amd import _lib
from test_beam import _states


@pytest.mark.parametrize("parent,length", [
    (0x20010, None),        # inside the destination (2 x 2 x 16 bytes from 0x20000)
    (0x1fff4, None),        # its last word is the destination's first
    (0x50000, 0x2003c),     # a length is the destination's last word
    (0x50000, 0x1fffc),
])
def test_reorder_refuses_indexes_inside_a_destination(parent, length):
    arr = _states((0x10000, 0x20000, 1, 1, 16))
    rc = _lib.load().lrhead_reorder(arr, 1, ctypes.c_void_p(parent), None if length is None else ctypes.c_void_p(length),
                                    2, 2, 2, None)
    assert rc == _lib.EINVAL


@pytest.mark.parametrize("kwargs", [dict(nb=2 ** 32 + 2), dict(nb=-2 ** 32 + 2), dict(nb=2, end_id=2 ** 31),
                                    dict(nb=2, end_id=-2 ** 40)])
def test_select_refuses_integers_past_32_bits(kwargs):
    with pytest.raises(ValueError, match="does not fit"):
        lr.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), **kwargs)
