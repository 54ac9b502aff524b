"""More of quantize / dequantize against the formats' definition: every finite bf16 magnitude as a row's largest,
and values written to an output that starts on 16 but not on 32 bytes."""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn

import _quant_ref as ref

pytestmark = pytest.mark.gpu
FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_all_row_maxima(dev, fmt):
    """0x0001 to 0x7f7f, beside smaller elements: every border of the row scale and of the block scales."""
    top = (torch.arange(1, 0x7f80, dtype=torch.int32) << 16).view(torch.float32)
    x = torch.zeros((top.numel(), 64), dtype=torch.bfloat16)
    for i, f in enumerate((1.0, -0.5, 0.375, 0.0625, -2.0 ** -9, 2.0 ** -14)):
        x[:, 11 * i] = (top * f).to(torch.bfloat16)
    q = gdn.quantize(x.to(dev), fmt)
    back = gdn.dequantize(q).double().cpu().numpy()
    codes, sc, row = ref.quantize(x.double().numpy(), fmt)
    got = ref.unpack(q)
    assert np.array_equal(got[2], row) and np.array_equal(got[1], sc) and np.array_equal(got[0], codes)
    want = ref.values(codes, sc, row, fmt)
    assert np.array_equal(back, np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 64), (5, 192), (130, 1088), (3, 9216)])
def test_values_off_32_bytes(dev, fmt, rows, K):
    g = torch.Generator().manual_seed(rows + K)
    x = torch.randn((rows, K), generator=g).to(torch.bfloat16)
    q = gdn.quantize(x.to(dev), fmt)
    buf = torch.full((rows * K + 24,), 3.0, dtype=torch.bfloat16, device=dev)
    out = buf[8:8 + rows * K].view(rows, K)
    assert out.data_ptr() % 32 == 16
    gdn.dequantize(q, out=out)
    want = ref.values(*ref.quantize(x.double().numpy(), fmt), fmt)
    assert np.array_equal(out.double().cpu().numpy(), want)
    assert bool((buf[:8] == 3).all()) and bool((buf[8 + rows * K:] == 3).all())
