"""The 4-bit projections where the product of a token's and a feature's row scale leaves f32's range and
the result does not: against float64, as in test_gpu_qproj.py.

Bound per element: the one derived there, and where the result is below bf16's normal numbers half of
its smallest step, 2^-134:
    |y - y_ref| <= 2^-8 |y_ref| + (K / 64 + 8) 2^-23 S (1 + 2^-8) + 2^-134.
(The two factors of the token's row scale are powers of two: they round only below f32's normal
numbers, by at most 2^-150, which the step's half covers together with the rounding to bf16 for the
results at 2^-118 and above that are asked for here.)"""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200.synth import Dims

import _quant_ref as ref

pytestmark = pytest.mark.gpu
DIMS = Dims(num_k_heads=1, num_v_heads=4)
K, HIDDEN = 512, 200
TOKENS = [2, 20, 100, 300]  # on chip, few tokens, few or pairs, pairs


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


def _normal(seed, rows, std):
    return torch.randn((rows, K), generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * std


def _run(dev, x, w, factor=1.0):
    """out_proj_quant of x and w (float64, taken to bf16) with the weights' row scales times `factor`, and
    the exact result with its S."""
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    q = gdn.quantize(w.to(dev), "nvfp4")
    scaled = (q.row_scale.double() * factor).float()
    q = gdn.QuantTensor(q.codes, q.scales, scaled, "nvfp4")
    y = gdn.out_proj_quant(x.to(dev), q, dims=DIMS)
    torch.cuda.synchronize(dev)
    xv = ref.values(*ref.quantize(x.double().numpy(), "nvfp4"), "nvfp4")
    codes, sc, row = ref.quantize(w.double().numpy(), "nvfp4")
    wv = ref.values(codes, sc, scaled.double().cpu().numpy(), "nvfp4")
    assert gdn.last_device_error() == 0
    return y.double().cpu().numpy(), xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def _check(y, want, S):
    assert np.abs(want).max() < 2.0 ** 127
    bound = 2.0 ** -8 * np.abs(want) + (K / 64 + 8) * 2.0 ** -23 * S * (1 + 2.0 ** -8) + 2.0 ** -134
    assert (np.abs(y - want) <= bound).all()  # (false for a NaN)


@pytest.mark.parametrize("T", TOKENS)
def test_scales_whose_product_overflows(dev, T):
    """Tokens of 2^125 (row scale 2^114) on features of 2^26 (2^15), where each one's largest element meets
    zeros of the other: results of about 2^122, and zeros for features that meet no other element."""
    x, w = _normal(T, T, 2.0 ** 108), _normal(T + 1, HIDDEN, 2.0 ** 10)
    x[:, 1], w[:, 0] = 0, 0
    x[:, 0], w[:, 1] = 2.0 ** 125, 2.0 ** 26
    w[::7, 2:] = 0
    y, want, S = _run(dev, x, w)
    _check(y, want, S)
    assert (y[:, ::7] == 0).all()


@pytest.mark.parametrize("T", TOKENS)
def test_scales_whose_product_underflows(dev, T):
    """Row scales of 2^-100 and 2^-50, every element the largest of its row: results of 2^-118."""
    x = torch.full((T, K), 2.0 ** -89, dtype=torch.float64)
    w = torch.full((HIDDEN, K), 2.0 ** -39, dtype=torch.float64)
    w[1::2] *= -1
    y, want, S = _run(dev, x, w)
    _check(y, want, S)
    assert np.abs(want).min() > 2.0 ** -120


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("ex,ew,factor", [
    (118, -88, 1.0), (-88, 118, 1.0), (58, 60, 1.0), (-60, -50, 1.0), (88, 30, 1.0), (89, 30, 1.0), (91, 28, 1.0),
    (-68, -40, 1.0), (-70, -40, 1.0), (-72, -40, 1.0), (-90, -20, 1.0), (-80, 0, 1.7 * 2.0 ** 120), (100, 0, -0.3 * 2.0 ** -110),
    (0, 0, 1.3 * 2.0 ** 110), (0, 0, -0.7 * 2.0 ** -115)])
def test_far_scales(dev, T, ex, ew, factor):
    """Tokens of 2^ex, weights of 2^ew, the weights' row scales times any finite factor."""
    _check(*_run(dev, _normal(3 * T, T, 2.0 ** ex), _normal(3 * T + 1, HIDDEN, 2.0 ** ew), factor))
