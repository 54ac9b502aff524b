"""The 4-bit projections over many tiles, every output element: pairs of SMs that walk several tiles (two
accumulators that share columns, scale buffers and ring stages carried from tile to tile), with odd numbers of K
stages, a ragged last stage, segment ends and outputs off 64 features and off 16 bytes, a last row tile whose
second half holds no token; and the few-token forms on many features.

The float64 product is formed on the device from the values that the quantised operands stand for (test_gpu_quant.py
compares these with the formats' definition bit for bit); the bound is derived in test_gpu_qproj.py."""
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200.synth import Dims

pytestmark = pytest.mark.gpu
FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


def _operands(dev, fmt, T, N, K):
    g = torch.Generator(device=dev).manual_seed(T * 31 + N + K)
    x = torch.randn((T, K), generator=g, device=dev)
    x[:, :: 37] *= 9.0
    w = torch.randn((N, K), generator=g, device=dev) * K ** -0.5
    return x.to(torch.bfloat16), gdn.quantize(w.to(torch.bfloat16), fmt)


def _check(y, x, w, fmt):
    K = x.shape[1]
    xv, wv = gdn.dequantize(gdn.quantize(x, fmt)).double(), gdn.dequantize(w).double()
    for c in range(0, y.shape[1], 4096):  # (in parts of the features)
        wc = wv[c:c + 4096]
        want = xv @ wc.T
        bound = 2.0 ** -8 * want.abs() + (K / 64 + 8) * 2.0 ** -23 * (1 + 2.0 ** -8) * (xv.abs() @ wc.abs().T)
        over = (y[:, c:c + 4096].double() - want).abs() - bound
        worst = over.max().item()
        at = divmod(over.argmax().item(), over.shape[1])
        assert worst <= 0, f"{worst:.3e} above the bound at token {at[0]}, feature {c + at[1]}"
    assert gdn.last_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,hidden,kh,vh", [
    (700, 64, 16, 32),     # 147 tiles of one stage
    (1100, 320, 9, 45),    # 275 tiles of 2 stages, the last of 64 elements; 76 tokens in the last row tile
    (1100, 576, 9, 45),    # 3 stages, the last of 64
    (1281, 1088, 9, 45),   # 330 tiles of 5 stages, the last of 64; one token in the last row tile
    (2305, 704, 5, 25),    # 310 tiles of 3 stages, the last of 192
    (1500, 1280, 9, 45),   # 5 whole stages
    (1500, 1664, 9, 45),   # 7 stages, the last of 128
    (8400, 448, 1, 3)])    # 33 row tiles: more than one sweep, 2 stages
def test_in_proj(dev, fmt, T, hidden, kh, vh):
    dims = Dims(num_k_heads=kh, num_v_heads=vh)
    x, w = _operands(dev, fmt, T, dims.conv_channels + dims.value_width + 2 * vh, hidden)
    qkv, z, a, b = gdn.in_proj_quant(x, w, dims=dims)
    _check(torch.cat([qkv, z, b, a], 1), x, w, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,hidden,vh", [(1100, 14001, 5), (900, 16100, 7), (1025, 12344, 3), (5000, 2308, 9)])
def test_out_proj(dev, fmt, T, hidden, vh):
    dims = Dims(num_k_heads=1 if vh < 9 else 3, num_v_heads=vh)
    x, w = _operands(dev, fmt, T, hidden, dims.value_width)
    _check(gdn.out_proj_quant(x, w, dims=dims), x, w, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 2, 3, 16, 17, 33, 64, 65, 80, 96, 97, 128, 129, 2049, 8192])
def test_layer_shape(dev, fmt, T):
    """The 27B layer's in_proj (16480 x 5120) and out_proj (5120 x 6144)."""
    dims = gdn.MODEL
    x, w = _operands(dev, fmt, T, dims.conv_channels + dims.value_width + 2 * dims.num_v_heads, 5120)
    qkv, z, a, b = gdn.in_proj_quant(x, w, dims=dims)
    _check(torch.cat([qkv, z, b, a], 1), x, w, fmt)
    y, w = _operands(dev, fmt, T, 5120, dims.value_width)
    _check(gdn.out_proj_quant(y, w, dims=dims), y, w, fmt)
