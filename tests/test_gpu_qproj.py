"""The 4-bit projections against float64: the tokens and weights quantised by the formats' definition
(_quant_ref.py), the product summed in float64.

Bound per element, with S = sum_k |x_k w_k| of the quantised values: the rounding to bf16 is at most
2^-8 of the result's magnitude (half a step: eps / 2 of bf16), and the f32 sum adds at most one error
of 2^-23 of a partial sum (<= S, truncation counted) for each of the K / 64 products that are added
and each of the 6 levels inside one, and 2 roundings by the row scales:
    |y - y_ref| <= 2^-8 |y_ref| + (K / 64 + 8) 2^-23 S (1 + 2^-8)."""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200.synth import Dims

import _quant_ref as ref

pytestmark = pytest.mark.gpu
FORMATS = ["nvfp4", "mxfp4"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


def _draw(seed, shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x[:, :: 37] *= 9.0
    return x.to(torch.bfloat16)


def _ref(x, w, fmt):
    xv = ref.values(*ref.quantize(x.double().numpy(), fmt), fmt)
    wv = ref.values(*ref.quantize(w.double().numpy(), fmt), fmt)
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def _check(y, want, S, K):
    bound = 2.0 ** -8 * np.abs(want) + (K / 64 + 8) * 2.0 ** -23 * S * (1 + 2.0 ** -8)
    err = np.abs(y.double().cpu().numpy() - want)
    worst = float((err - bound).max())
    assert worst <= 0, f"{worst:.3e} above the bound, at {np.unravel_index((err - bound).argmax(), err.shape)}"


def _split(full, dims):
    C, VD, Vh = dims.conv_channels, dims.value_width, dims.num_v_heads
    return full[:, :C], full[:, C:C + VD], full[:, C + VD + Vh:], full[:, C + VD:C + VD + Vh]  # qkv, z, a, b


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,hidden,kh,vh", [
    (1, 64, 1, 1), (1, 1088, 3, 9), (2, 128, 1, 3), (15, 192, 2, 4), (16, 256, 1, 8), (17, 320, 3, 9),
    (33, 448, 1, 2), (64, 512, 2, 2), (65, 576, 1, 5), (127, 640, 3, 9), (128, 64, 2, 6), (129, 704, 1, 1),
    (200, 1600, 1, 3), (256, 256, 2, 4), (257, 320, 1, 1), (300, 1088, 4, 12), (513, 192, 3, 9), (1025, 512, 1, 2)])
def test_in_proj(dev, fmt, T, hidden, kh, vh):
    dims = Dims(num_k_heads=kh, num_v_heads=vh)
    N = dims.conv_channels + dims.value_width + 2 * vh
    x, w = _draw(T * 7 + hidden, (T, hidden)), _draw(T * 11 + hidden, (N, hidden), hidden ** -0.5)
    outs = gdn.in_proj_quant(x.to(dev), gdn.quantize(w.to(dev), fmt), dims=dims)
    torch.cuda.synchronize(dev)
    want, S = _ref(x, w, fmt)
    for got, a, b in zip(outs, _split(want, dims), _split(S, dims)):
        _check(got, a, b, hidden)
    assert gdn.last_device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,hidden,vh", [(1, 64, 1), (3, 5120, 1), (8, 192, 48), (31, 1024, 12), (64, 320, 9),
                                         (100, 64, 3), (130, 448, 8), (600, 1088, 5), (1, 1, 2), (40, 37, 3),
                                         (300, 259, 4), (9, 2304, 48), (9, 2688, 48), (40, 2944, 48), (2, 3200, 48),
                                         (17, 3584, 48), (9, 4736, 48), (5, 128, 48), (1, 1000, 48)])
def test_out_proj(dev, fmt, T, hidden, vh):
    dims = Dims(num_k_heads=1 if vh < 9 else 3 if vh < 12 else vh // 3, num_v_heads=vh)
    K = dims.value_width
    y, w = _draw(T + hidden, (T, K)), _draw(T * 3 + hidden, (hidden, K), K ** -0.5)
    out = gdn.out_proj_quant(y.to(dev), gdn.quantize(w.to(dev), fmt), dims=dims)
    torch.cuda.synchronize(dev)
    _check(out, *_ref(y, w, fmt), K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 64, 100, 600, 8192, 8500])
def test_layer_shape_sampled(dev, fmt, T):
    """The 27B layer's in_proj (16480 x 5120) and out_proj (5120 x 6144) on sampled tokens and features."""
    dims, hidden = gdn.MODEL, 5120
    N, VD = dims.conv_channels + dims.value_width + 2 * dims.num_v_heads, dims.value_width
    rng = np.random.default_rng(T)
    rows = np.unique(np.concatenate([rng.integers(0, T, 30), [0, T - 1]]))
    for name, n, k in (("in", N, hidden), ("out", hidden, VD)):
        g = torch.Generator(device=dev).manual_seed(T + n)
        x = torch.randn((T, k), generator=g, device=dev).to(torch.bfloat16)
        w = (torch.randn((n, k), generator=g, device=dev) * k ** -0.5).to(torch.bfloat16)
        q = gdn.quantize(w, fmt)
        if name == "in":
            qkv, z, a, b = gdn.in_proj_quant(x, q, dims=dims)
            y = torch.cat([qkv[rows], z[rows], b[rows], a[rows]], 1)
        else:
            y = gdn.out_proj_quant(x, q, dims=dims)[rows]
        torch.cuda.synchronize(dev)
        cols = np.unique(np.concatenate([rng.integers(0, n, 300), [0, n - 1]]))
        want, S = _ref(x[rows].cpu(), w[cols].cpu(), fmt)
        _check(y[:, cols], want, S, k)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [5, 300])
def test_rows_apart(dev, fmt, T):
    """A token with an infinity or a NaN gives NaN in its own outputs and leaves the others' bits; so does a
    row of the weights; a zero token gives zeros."""
    dims = Dims(num_k_heads=1, num_v_heads=3)
    K, hidden = dims.value_width, 200
    y, w = _draw(1, (T, K)), _draw(2, (hidden, K), K ** -0.5)
    clean = gdn.out_proj_quant(y.to(dev), gdn.quantize(w.to(dev), fmt), dims=dims)
    y[1, 3], y[3, K - 1], y[2] = float("inf"), float("nan"), 0.0
    w[150, 7] = float("-inf")
    out = gdn.out_proj_quant(y.to(dev), gdn.quantize(w.to(dev), fmt), dims=dims)
    torch.cuda.synchronize(dev)
    bad = torch.zeros((T, hidden), dtype=torch.bool, device=dev)
    bad[1] = bad[3] = True
    bad[:, 150] = True
    assert bool(out[bad].isnan().all())
    assert bool((out[2][~bad[2]] == 0).all())
    keep = ~bad
    keep[2] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("fmt", FORMATS)
def test_any_row_scales_of_the_weights(dev, fmt):
    """Weights quantised elsewhere: row scales that are no powers of two (here 0.3 and 1.7 of ours)."""
    dims = Dims(num_k_heads=1, num_v_heads=2)
    K, hidden = dims.value_width, 130
    for T in (3, 400):
        y, w = _draw(3, (T, K)), _draw(4, (hidden, K), K ** -0.5)
        q = gdn.quantize(w.to(dev), fmt)
        f = torch.where(torch.arange(hidden) % 2 == 0, 0.3, 1.7)
        q = gdn.QuantTensor(q.codes, q.scales, q.row_scale * f.to(dev), fmt)
        out = gdn.out_proj_quant(y.to(dev), q, dims=dims)
        torch.cuda.synchronize(dev)
        want, S = _ref(y, w, fmt)
        f64 = f.double().numpy()
        _check(out, want * f64, S * f64, K)


@pytest.mark.parametrize("T", [3, 130, 1000])
def test_outputs_around_are_left(dev, T):
    """Outputs as slices of larger buffers: no element before or behind them is written; scale bytes of
    rows that do not exist play no part (the weights' last tile is filled with NaN scales there)."""
    dims = Dims(num_k_heads=1, num_v_heads=3)
    hidden, N = 192, 5 * 128 + 3 * 128 + 6
    x, w = _draw(T, (T, hidden)), _draw(T + 1, (N, hidden), hidden ** -0.5)
    q = gdn.quantize(w.to(dev), "nvfp4")
    ref_out = gdn.in_proj_quant(x.to(dev), q, dims=dims)
    view = q.scales[-1].view(-1, 32, 4, 4).permute(0, 2, 1, 3).reshape(-1, 128, 4).clone()
    view[:, N % 128:] = 0x7F
    q.scales[-1] = view.view(-1, 4, 32, 4).permute(0, 2, 1, 3).reshape(-1, 512)
    # (8 rows before the output: a whole number of 16 bytes for any width)
    wide = [torch.full((T + 2 * 8, t.shape[1]), 5.0, dtype=torch.bfloat16, device=dev) for t in ref_out]
    out = gdn.in_proj_quant(x.to(dev), q, dims=dims, out=[t[8:8 + T] for t in wide])
    torch.cuda.synchronize(dev)
    for got, want, buf in zip(out, ref_out, wide):
        assert torch.equal(got, want)
        assert bool((buf[:8] == 5).all()) and bool((buf[8 + T:] == 5).all())


@pytest.mark.parametrize("T", [1, 20, 700])
def test_graph_streams_and_repeats(dev, T):
    """The same bits from a second call, from another stream at the same time, and from a captured graph
    replayed on changed tokens."""
    dims = Dims(num_k_heads=3, num_v_heads=9)
    hidden = 576
    N = dims.conv_channels + dims.value_width + 18
    q = gdn.quantize(_draw(5, (N, hidden), hidden ** -0.5).to(dev), "mxfp4")
    x1, x2 = _draw(6, (T, hidden)).to(dev), _draw(7, (T, hidden)).to(dev)
    want1, want2 = gdn.in_proj_quant(x1, q, dims=dims), gdn.in_proj_quant(x2, q, dims=dims)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize(dev)
    with torch.cuda.stream(s1):
        got1 = [gdn.in_proj_quant(x1, q, dims=dims) for _ in range(4)]
    with torch.cuda.stream(s2):
        got2 = [gdn.in_proj_quant(x2, q, dims=dims) for _ in range(4)]
    torch.cuda.synchronize(dev)
    for got, want in ((got1, want1), (got2, want2)):
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))
    xs = x1.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gdn.in_proj_quant(xs, q, dims=dims)
    for x, want in ((x2, want2), (x1, want1)):
        xs.copy_(x)
        graph.replay()
        torch.cuda.synchronize(dev)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_empty_and_refusals(dev):
    dims = Dims(num_k_heads=1, num_v_heads=1)
    K = 128
    w = gdn.quantize(_draw(8, (96, K)).to(dev))
    y = _draw(9, (4, K)).to(dev)
    assert tuple(gdn.out_proj_quant(y[:0], w, dims=dims).shape) == (0, 96)
    with pytest.raises(TypeError):
        gdn.out_proj_quant(y, y, dims=dims)
    with pytest.raises(TypeError):
        gdn.out_proj_quant(y.float(), w, dims=dims)
    with pytest.raises(ValueError):
        gdn.out_proj_quant(y[:, :64].contiguous(), w, dims=dims)
    with pytest.raises(ValueError):
        gdn.out_proj_quant(y, w, dims=Dims(num_k_heads=1, num_v_heads=2))
    with pytest.raises(ValueError):
        gdn.in_proj_quant(y, w, dims=dims)
    with pytest.raises(ValueError):
        gdn.out_proj_quant(y, w, dims=dims, out=torch.empty((4, 95), dtype=torch.bfloat16, device=dev))
    with pytest.raises(gdn.GdnError):  # outputs start on 16 bytes
        buf = torch.empty((4 * 96 + 1,), dtype=torch.bfloat16, device=dev)
        gdn.out_proj_quant(y, w, dims=dims, out=buf[1:].view(4, 96))
