"""CPU check of the number of weight parts that the sink-window entry points take."""
import ctypes

import pytest

from fixed_pattern_sparse_sa_b200 import _lib, api, build


@pytest.mark.parametrize("parts", [-1, 3, 1 << 30])
def test_the_library_refuses(parts):
    build.build()
    s = _lib.sa_sink_shape(dtype=0, B=1, Hq=4, Hkv=2, d=64, window=8, sinks=2, scale=0.1, Tq=16, L=16, weight_parts=parts)
    for name, heads in (("q_stride", 4), ("k_stride", 2), ("v_stride", 2), ("dout_stride", 4)):
        for i, x in enumerate((16 * heads * 64, heads * 64, 64)):
            getattr(s, name)[i] = x
    p = ctypes.c_void_p(1 << 20)                                  # never dereferenced: refused first
    lib = _lib.load()
    assert lib.sa_sink_attn_fwd(ctypes.byref(s), p, p, p, None, None, p, p, None) == 1
    assert lib.sa_sink_attn_bwd(ctypes.byref(s), p, p, p, p, p, p, None, None, p, p, p, p, 1 << 40, None) == 1


def test_the_binding_names_them():
    assert [api._parts(x) for x in (None, 1, 2)] == [0, 1, 2]
    for bad in (0, 3, "2"):
        with pytest.raises(ValueError, match="weight_parts"):
            api._parts(bad)
