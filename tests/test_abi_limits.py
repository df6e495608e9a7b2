"""Sizes at which 32-bit counts end come back as a status before the GPU is
touched (fake, never-dereferenced addresses; needs no GPU)."""
import ctypes
import os

import pytest

import gated_delta_rule_34_amd as gdn

pytestmark = pytest.mark.skipif(not os.path.exists(gdn.lib_path), reason="libgdn.so not built")

FAKE = 0x7F0000000000
BF16 = 1


@pytest.mark.parametrize("C", [(1 << 31) - 1, (1 << 31) - 8, (1 << 31) - 16])
@pytest.mark.parametrize("packed", [False, True])
def test_conv_refuses_channels_beyond_32_bits(packed, C):
    lib = gdn.load()
    n = 7 if packed else 6
    p = [ctypes.c_void_p(FAKE + (i << 40)) for i in range(n)]
    fn = lib.gdn_causal_conv_varlen if packed else lib.gdn_causal_conv
    assert fn(*p, 1, 1, C, 4, BF16, 2, None) == 2
