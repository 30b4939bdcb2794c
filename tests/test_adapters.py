"""The adapters' calls on the host (CPU only): workspace sizes and refusals,
all of which return before anything is launched (the fake addresses never
reach a kernel)."""
import ctypes
import os

import pytest
import torch

from dit_dequant_gemm_amd import api

OK, E_ARG, E_SHAPE, E_ALIGN, E_WS = 0, -1, -2, -3, -4
FAKE = 0x10000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(api.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return api.load_library()


def _bytes(lib, m, n=256, k=512, r=16, split=0):
    b = ctypes.c_size_t()
    return lib.ddg_adapter_workspace_bytes(m, n, k, r, split, ctypes.byref(b)), b.value


def _up256(b):
    return -(-b // 256) * 256


def test_workspace_bytes(lib):
    # at most 64 rows: T in float32, once per part of K (16 groups of 128 to a
    # part, at most 8 parts); more rows: three bf16 parts of T
    for m, k, parts in [(1, 512, 1), (16, 5120, 3), (64, 13824, 7), (64, 1 << 20, 8), (3, 128, 1), (16, 2176, 2)]:
        assert _bytes(lib, m, 256, k, 24) == (OK, _up256(parts * m * 24 * 4)), (m, k)
    for m in (65, 1001, 32760):
        assert _bytes(lib, m, 256, 5120, 24) == (OK, _up256(3 * m * 24 * 2)), m
    assert _bytes(lib, 0) == (OK, 0)
    plain = ctypes.c_size_t()
    for m, n, k in [(16, 1024, 8192), (512, 5120, 5120), (16, 15360, 5120)]:
        assert lib.ddg_workspace_bytes(m, n, k, 0, ctypes.byref(plain)) == OK
        assert _bytes(lib, m, n, k, 8, 1)[1] == _bytes(lib, m, n, k, 8, 0)[1] + plain.value
    for bad in (dict(m=-1), dict(m=1 << 28), dict(m=1, n=-1), dict(m=1, n=1 << 31), dict(m=1, k=0), dict(m=1, k=100),
                dict(m=1, k=(1 << 20) + 128), dict(m=1, r=4), dict(m=1, r=12), dict(m=1, r=136)):
        assert _bytes(lib, **bad)[0] == E_SHAPE, bad
    assert lib.ddg_adapter_workspace_bytes(1, 16, 128, 8, 0, None) == E_ARG


def _gemm(lib, **kw):
    a = dict(x=FAKE, m=16, k=512, packed=2 * FAKE, scales=3 * FAKE, bits=4, n=256, down=4 * FAKE, up=5 * FAKE,
             ascales=6 * FAKE, adapters=3, r=16, rows=7 * FAKE, y=8 * FAKE, y_dtype=0, ws=9 * FAKE, ws_bytes=0)
    a.update(kw)
    return lib.ddg_adapter_gemm(*a.values(), None)


def test_refusals(lib):
    # every pointer in place and the shapes right: only the workspace is short
    assert _gemm(lib) == E_WS
    need = _bytes(lib, 16)[1]
    assert _gemm(lib, ws_bytes=need - 1) == E_WS
    assert _gemm(lib, m=0) == OK
    for name in ("x", "packed", "scales", "down", "up", "ascales", "rows", "y", "ws"):
        assert _gemm(lib, **{name: None}) == E_ARG, name
    for name in ("x", "packed", "down", "up", "y", "ws"):
        assert _gemm(lib, **{name: FAKE + 8}) == E_ALIGN, name
    for name in ("scales", "ascales", "rows"):
        assert _gemm(lib, **{name: FAKE + 2}) == E_ALIGN, name
    for kw in (dict(bits=2), dict(bits=8), dict(y_dtype=2)):
        assert _gemm(lib, **kw) == E_ARG, kw
    for kw in (dict(m=-1), dict(m=1 << 28), dict(k=0), dict(k=500), dict(k=(1 << 20) + 128), dict(n=0), dict(n=24),
               dict(r=0), dict(r=4), dict(r=20), dict(r=136), dict(adapters=0), dict(adapters=-1),
               dict(adapters=1 << 31)):
        assert _gemm(lib, **kw) == E_SHAPE, kw


def test_binding_refusals_on_the_host():
    with pytest.raises(ValueError, match="GPU tensor"):
        api.AdapterPool(torch.zeros(1, 8, 128).bfloat16(), torch.zeros(1, 16, 8).bfloat16(), torch.ones(1))
    with pytest.raises(ValueError, match="no adapters"):
        api.AdapterPool.stack([], None)
