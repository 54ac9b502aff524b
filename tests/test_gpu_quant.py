"""quantize / dequantize on the GPU against the formats' definition in float64: codes, block scales
and row scales equal, the values exact, at the sizes and values where rounding and layout can go
wrong (ties, zeros, subnormals, the ends of the range, rows that are not finite)."""
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


def _check(x, fmt, dev):
    q = gdn.quantize(x.to(dev), fmt)
    back = gdn.dequantize(q)
    torch.cuda.synchronize(dev)
    codes, sc, row = ref.quantize(x.double().numpy(), fmt)
    got = ref.unpack(q)
    assert np.array_equal(got[2], row, equal_nan=True)
    assert np.array_equal(got[1], sc)
    assert np.array_equal(got[0], codes)
    want = ref.values(codes, sc, row, fmt)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 64), (3, 128), (7, 192), (130, 320), (129, 1088), (33, 5120), (2, 8256),
                                    (2, 16384), (3, 16448), (1, 40000)])
def test_random_rows(dev, fmt, rows, K):
    g = torch.Generator().manual_seed(rows * 100003 + K)
    x = torch.randn((rows, K), generator=g) * torch.exp2(torch.randint(-20, 21, (rows, 1), generator=g).float())
    _check((x * torch.exp2(torch.randint(-6, 7, (rows, K), generator=g).float())).to(torch.bfloat16), fmt, dev)


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties(dev, fmt):
    """The values and midpoints of E2M1 times m 2^e, with block maxima 6 m 2^e: quotients on the midpoints
    for every E4M3 fraction m; and block maxima whose sixth is a midpoint of E4M3 (51, 57, 63)."""
    g = torch.Generator().manual_seed(5)
    marks = torch.tensor([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6])
    x = marks[torch.randint(0, 15, (64, 15, 32), generator=g)]
    x = torch.where(torch.rand(x.shape, generator=g) < 0.5, -x, x)
    x[:, :, 7] = 6.0
    x[:, :, 23] = -6.0
    m = (8 + torch.arange(15) % 8).view(1, 15, 1).float() / 8
    rowpow = torch.exp2(torch.randint(-30, 31, (64, 1, 1), generator=g).float())
    y = (x * m * rowpow).view(64, 480)
    y = torch.cat([y, (torch.arange(64).view(64, 1) + 1 + torch.zeros(1, 32)) * rowpow.view(64, 1)], 1)
    assert torch.equal(y.to(torch.bfloat16).float(), y)
    _check(y.to(torch.bfloat16), fmt, dev)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_row_maximum(dev, fmt):
    """Every positive finite bf16 as a row's largest magnitude, beside smaller ones: the row scale's and
    the block scales' borders, from the subnormals to the largest number."""
    bits = torch.arange(1, 0x7f80, 7, dtype=torch.int32)
    top = (bits << 16).view(torch.float32).to(torch.bfloat16)
    x = torch.zeros((top.numel(), 64), dtype=torch.bfloat16)
    for i, f in enumerate((1.0, -0.5, 0.375, 0.0625, -2.0 ** -9, 2.0 ** -14)):
        x[:, 11 * i] = (top.float() * f).to(torch.bfloat16)
    _check(x, fmt, dev)


@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_and_non_finite_rows(dev, fmt):
    g = torch.Generator().manual_seed(6)
    x = torch.randn((9, 192), generator=g).to(torch.bfloat16)
    x[1] = 0
    x[2] = -0.0
    x[3, 17] = float("inf")
    x[4, 0] = float("-inf")
    x[5, 191] = float("nan")
    x[6, 5] = torch.finfo(torch.bfloat16).max
    x[7, :32] = 0
    _check(x, fmt, dev)


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_around_are_left(dev, fmt):
    """The outputs are slices of larger buffers: nothing before or behind them is written, and of the
    last scale tile only the rows that exist."""
    rows, K = 37, 320
    tiles = ref.scale_tiles(fmt, K)
    codes = torch.full((rows + 8, K // 2), 0xA5, dtype=torch.uint8, device=dev)
    scales = torch.full((3, tiles, 512), 0xA5, dtype=torch.uint8, device=dev)
    row = torch.full((rows + 8,), 7.0, device=dev)
    q = gdn.QuantTensor(codes[4:4 + rows], scales[1:2], row[4:4 + rows], fmt)
    x = torch.randn((rows, K), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    assert gdn.quantize(x.to(dev), fmt, out=q) is q
    buf = torch.full((rows + 2, K), 3.0, dtype=torch.bfloat16, device=dev)
    gdn.dequantize(q, out=buf[1:1 + rows])
    torch.cuda.synchronize(dev)
    assert bool((codes[:4] == 0xA5).all()) and bool((codes[4 + rows:] == 0xA5).all())
    assert bool((scales[0] == 0xA5).all()) and bool((scales[2] == 0xA5).all())
    assert bool((row[:4] == 7).all()) and bool((row[4 + rows:] == 7).all())
    assert bool((buf[0] == 3).all()) and bool((buf[-1] == 3).all())
    r = torch.arange(128)
    last = scales[1].cpu().view(tiles, 32, 4, 4).permute(2, 1, 0, 3).reshape(128, tiles * 4)
    assert bool((last[r >= rows] == 0xA5).all())
    want = ref.values(*ref.quantize(x.double().numpy(), fmt), fmt)
    assert np.array_equal(buf[1:1 + rows].double().cpu().numpy(), want)


def test_empty_and_refusals(dev):
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device=dev)
    q = gdn.quantize(x[:0])
    assert q.shape == (0, 128) and tuple(gdn.dequantize(q).shape) == (0, 128)
    with pytest.raises(ValueError):
        gdn.quantize(x[:, :96].contiguous())
    with pytest.raises(ValueError):
        gdn.quantize(x[:, :64])  # not contiguous
    with pytest.raises(TypeError):
        gdn.quantize(x.float())
    with pytest.raises(ValueError):
        gdn.quantize(x, "fp4")
    with pytest.raises(ValueError):
        gdn.quantize(x, out=gdn.quantize(x, "mxfp4"))
    q = gdn.quantize(x)
    with pytest.raises(ValueError):
        gdn.dequantize(gdn.QuantTensor(q.codes, q.scales, q.row_scale[:2], "nvfp4"))
    with pytest.raises(ValueError):
        gdn.dequantize(q, out=torch.empty((4, 64), dtype=torch.bfloat16, device=dev))
