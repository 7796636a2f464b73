"""Host-side check of strides whose products pass 64 bits (no GPU needed)."""
import ctypes
import os

import pytest

from moe_routing_capacity_gb300 import abi


@pytest.fixture(scope="module", autouse=True)
def built_library():
    if not os.path.exists(abi.LIB_PATH):
        from moe_routing_capacity_gb300 import build
        build.build()
    return abi.lib()


P = ctypes.c_void_p(0x10000)          # a 16-byte aligned address nobody reads


@pytest.mark.parametrize("name", ["q", "o"])
def test_heads_that_share_elements_are_refused(name):
    """Heads 2^37 apart, tokens 2^36: (T - 1) 2^36 is negative in 64 bits."""
    c = abi.Attention()
    c.T, c.n_seqs, c.n_heads, c.n_kv_heads, c.head_dim, c.scale = 1 << 30, 1, 2, 1, 64, 0.125
    for n in ("q", "k", "v", "o"):
        setattr(c, n + "_t", 128)
        setattr(c, n + "_h", 64)
    setattr(c, name + "_t", 1 << 36)
    setattr(c, name + "_h", 1 << 37)
    assert abi.lib().moe_attention_forward(ctypes.byref(c), P, P, P, P, P, None, P, P,
                                           None) == abi.MOE_EINVAL
