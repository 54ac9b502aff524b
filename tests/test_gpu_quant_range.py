"""dequantize of rows whose scales were made elsewhere: block scale times row scale beyond f32's range, where a
code of 0 is still 0 and small codes may still have finite values; against float64.

Bound per element: the product of two exact factors rounded to f32 and then to bf16, and half of bf16's
smallest step: |v - v_ref| <= (2^-8 + 2^-23) |v_ref| + 2^-134; infinite from the number that rounds to 2^128 on."""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn

import _quant_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("g", [2.0 ** 120, 1.7 * 2.0 ** 121, 2.0 ** 127, -2.0 ** 123, 3e38, 1.0, -2.0 ** -149, 1.3 * 2.0 ** -126])
def test_any_finite_row_scale(dev, fmt, g):
    """Every code and every block scale of the format, in rows of the row scale g."""
    B = ref.BLOCK[fmt]
    nscale = 127 if fmt == "nvfp4" else 255
    rows, K = 128, 8 * B
    tiles = ref.scale_tiles(fmt, K)
    gen = torch.Generator().manual_seed(11)
    codes = torch.randint(0, 256, (rows, K // 2), generator=gen, dtype=torch.int64).to(torch.uint8)
    scales = (torch.arange(tiles * 512) % nscale).to(torch.uint8).view(1, tiles, 512)
    q = gdn.QuantTensor(codes.to(dev), scales.to(dev), torch.full((rows,), g, dtype=torch.float32, device=dev), fmt)
    got = gdn.dequantize(q).double().cpu().numpy()
    want = ref.values(*ref.unpack(q), fmt)
    top = 2.0 ** 128 - 2.0 ** 119  # the middle between bf16's largest number and 2^128
    sure = np.abs(want) < top * (1 - 2.0 ** -23)
    bound = (2.0 ** -8 + 2.0 ** -23) * np.abs(want) + 2.0 ** -134
    assert (np.abs(got - want)[sure] <= bound[sure]).all()
    beyond = np.abs(want) >= top * (1 + 2.0 ** -23)
    assert np.array_equal(got[beyond], np.copysign(np.inf, want[beyond]))
    assert (want == 0).any() and gdn.last_device_error() == 0
