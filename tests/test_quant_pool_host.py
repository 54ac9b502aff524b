"""Host-side checks of the 4-bit and pool entry points that need no GPU: sizes, and arguments refused
before any CUDA call."""
import ctypes

import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load_library()


def _dims(kh=16, vh=48, d=128, w=4):
    return ctypes.byref(gdn._DimsC(kh, vh, d, w))


def test_sizes(lib):
    # 128 rows x 4 blocks of 16 (nvfp4) or 32 (mxfp4) per 512-byte tile
    assert lib.gdn_quant_scale_bytes(0, 1, 64) == 512
    assert lib.gdn_quant_scale_bytes(0, 129, 5120) == 2 * 80 * 512
    assert lib.gdn_quant_scale_bytes(1, 128, 192) == 2 * 512
    assert lib.gdn_quant_scale_bytes(0, 0, 64) == 0
    for fmt, rows, K in ((2, 1, 64), (-1, 1, 64), (0, -1, 64), (0, 1, 96), (0, 1, 0), (0, 1, -64)):
        assert lib.gdn_quant_scale_bytes(fmt, rows, K) == 0
        assert lib.gdn_proj_quant_workspace_size(fmt, rows, K) == 0
    # past 2^32 bytes
    assert lib.gdn_quant_scale_bytes(0, 2 ** 31 - 1, 5120) == (2 ** 31 // 128) * 80 * 512
    assert lib.gdn_proj_quant_workspace_size(0, 2 ** 21, 5120) >= 2 ** 21 * (2560 + 320 + 4)


def test_quantize_arguments(lib):
    ok = [16, 16, 16, 16, None]
    for fn in (lib.gdn_quantize, lib.gdn_dequantize):
        assert fn(2, 4, 64, *ok) == -1
        assert fn(0, -1, 64, *ok) == -1
        assert fn(0, 4, 0, *ok) == -1
        assert fn(0, 4, 96, *ok) == -2
        assert fn(0, 0, 64, *([None] * 5)) == 0
        for i in range(4):
            args = list(ok)
            args[i] = None
            assert fn(1, 4, 64, *args) == -1
            args[i] = 10  # off every required boundary
            assert fn(1, 4, 64, *args) == -1


def test_projection_arguments(lib):
    big = 1 << 30
    ok_in = [16] * 9 + [big, None]   # x, codes, scales, row_scale, qkv, z, b, a, workspace
    ok_out = [16] * 6 + [big, None]  # y, codes, scales, row_scale, out, workspace
    assert lib.gdn_in_proj_quant(_dims(d=64), 0, 8, 128, *ok_in) == -2
    assert lib.gdn_in_proj_quant(None, 0, 8, 128, *ok_in) == -1
    assert lib.gdn_in_proj_quant(_dims(), 5, 8, 128, *ok_in) == -1
    assert lib.gdn_in_proj_quant(_dims(), 0, -8, 128, *ok_in) == -1
    assert lib.gdn_in_proj_quant(_dims(), 0, 8, 100, *ok_in) == -2
    assert lib.gdn_in_proj_quant(_dims(), 0, 0, 128, *([None] * 9), 0, None) == 0
    assert lib.gdn_out_proj_quant(_dims(), 1, 0, 128, *([None] * 6), 0, None) == 0
    assert lib.gdn_out_proj_quant(_dims(), 1, 8, 0, *ok_out) == -1
    need = lib.gdn_proj_quant_workspace_size(0, 100, 128)
    assert need >= 100 * 64 + 2 * 512 + 400
    assert lib.gdn_in_proj_quant(_dims(), 0, 100, 128, *ok_in[:9], need - 1, None) == -4
    # a few tokens are quantised on chip, while they fit there
    assert lib.gdn_proj_quant_workspace_size(0, 2, 6144) == 0 and lib.gdn_proj_quant_workspace_size(1, 16, 1024) == 0
    for T, K in ((3, 6144), (16, 1088), (17, 64), (1, 6208)):
        assert lib.gdn_proj_quant_workspace_size(0, T, K) >= T * (K // 2 + K // 16 + 4)
    for fn, ok, n, extra in ((lib.gdn_in_proj_quant, ok_in, 9, 128), (lib.gdn_out_proj_quant, ok_out, 6, 64)):
        for i in range(n):
            for bad in (None, 10):
                args = list(ok)
                args[i] = bad
                want = -4 if i == n - 1 and bad is None else -1
                assert fn(_dims(), 0, 100, extra, *args) == want, (fn, i, bad)


def _table(*rows):
    return (ctypes.c_int32 * len(rows))(*rows)


def test_pool_arguments(lib):
    d = _dims(1, 1)
    ok = (16, 16, None)
    copy = lib.gdn_copy_slots
    assert copy(d, 0, None, None, 0, None, None, None) == 0
    assert copy(d, -1, _table(0), _table(1), 4, *ok) == -1
    assert copy(_dims(d=64), 1, _table(0), _table(1), 4, *ok) == -2
    for src, dst, rows in (((0, 1), (2, 2), 4), ((4,), (0,), 4), ((-2,), (0,), 4), ((0,), (4,), 4), ((0,), (-1,), 4),
                           ((0,), (0,), 0)):
        assert copy(d, len(src), _table(*src), _table(*dst), rows, *ok) == -1, (src, dst, rows)
    assert copy(d, 1, None, _table(1), 4, *ok) == -1
    assert copy(d, 1, _table(0), None, 4, *ok) == -1
    for st, cv in ((None, 16), (16, None), (8, 16), (16, 8)):
        assert copy(d, 1, _table(0), _table(1), 4, st, cv, None) == -1
    compact = lib.gdn_compact_slots
    live = (ctypes.c_uint8 * 4)(1, 0, 1, 1)
    remap = _table(7, 7, 7, 7)
    assert compact(d, 0, None, 0, None, None, None, None) == 0
    assert compact(d, -1, live, 0, 16, 16, remap, None) == -1
    assert compact(d, 4, None, 0, 16, 16, remap, None) == -1
    assert compact(d, 4, live, 0, 16, 16, None, None) == -1
    assert compact(d, 4, live, 0, 8, 16, remap, None) == -1
    assert list(remap) == [7, 7, 7, 7]


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(gdn.GdnError):
        gdn.quantize(x)
    with pytest.raises(gdn.GdnError):
        gdn.copy_slots([0], [1], torch.zeros((2, 1, 128, 128)), torch.zeros((2, 3, 384)), dims=gdn.Dims(1, 1))
    with pytest.raises(gdn.GdnError):
        gdn.compact_slots([1, 0], torch.zeros((2, 1, 128, 128)), torch.zeros((2, 3, 384)), dims=gdn.Dims(1, 1))


def test_status_string(lib):
    assert "memory" in gdn.status_string(-6)
