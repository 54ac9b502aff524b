"""The 4-bit projections and the pool moves as a server uses them around the mixer: a prompt prefilled into
a pool row, forked into continuations, decoded step by step, reordered as beams, ended ones freed and the
pool compacted.  Every step is compared with the same step on a plain copy of the pool (torch indexing) and
the projections with the float64 product of the quantised operands; and the calls back to back, captured
and on joined streams give the same bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200 import synth
from gated_deltanet_mixer_gdn_b200.synth import Dims

import _quant_ref as ref

pytestmark = pytest.mark.gpu
DIMS = Dims(num_k_heads=2, num_v_heads=4)
HIDDEN = 320
# bf16 result of the f32 sum of quantised products (derivation in test_gpu_qproj.py), K = 512 at most
REL, SUM = 2.0 ** -8, (512 / 64 + 8) * 2.0 ** -23 * (1 + 2.0 ** -8)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda", 0)


def _model(dev, fmt):
    g = torch.Generator().manual_seed(31)
    C, VD, Vh = DIMS.conv_channels, DIMS.value_width, DIMS.num_v_heads
    w_in = (torch.randn((C + VD + 2 * Vh, HIDDEN), generator=g) * HIDDEN ** -0.5).to(torch.bfloat16)
    w_out = (torch.randn((HIDDEN, VD), generator=g) * VD ** -0.5).to(torch.bfloat16)
    weights = gdn.weights_to(synth.draw_weights(g, DIMS), dev)
    return w_in, w_out, gdn.quantize(w_in.to(dev), fmt), gdn.quantize(w_out.to(dev), fmt), weights


def _values(x, fmt):
    return ref.values(*ref.quantize(x.double().cpu().numpy(), fmt), fmt)


def _check(y, x, w, fmt):
    xv, wv = _values(x, fmt), _values(w, fmt)
    want, S = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= REL * np.abs(want) + SUM * S).all()


def _same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_serving_loop(dev, fmt):
    w_in, w_out, q_in, q_out, weights = _model(dev, fmt)
    P = 9
    g = torch.Generator().manual_seed(32)
    state = torch.randn((P, DIMS.num_v_heads, 128, 128), generator=g).to(dev)  # what earlier sequences left
    conv = torch.randn((P, 3, DIMS.conv_channels), generator=g).to(dev)
    hidden = lambda n: torch.randn((n, HIDDEN), generator=g).to(torch.bfloat16).to(dev)

    # two prompts into cleared rows 2 and 5
    gdn.free_slots([2, 5], state, conv, dims=DIMS)
    x = hidden(150)
    qkv, z, a, b = gdn.in_proj_quant(x, q_in, dims=DIMS)
    _check(torch.cat([qkv, z, b, a], 1), x, w_in, fmt)
    cu = torch.tensor([0, 97, 150], dtype=torch.int32)
    y = gdn.prefill_varlen_slots(cu, [2, 5], qkv, z, a, b, weights, state, conv, dims=DIMS)
    y0, s0, c0 = gdn.prefill_varlen(cu, qkv, z, a, b, weights, dims=DIMS)  # from zero
    assert torch.equal(y, y0) and _same(state[[2, 5]], s0) and _same(conv[[2, 5]], c0)
    _check(gdn.out_proj_quant(y, q_out, dims=DIMS), y, w_out, fmt)

    # the first one forked to three continuations
    plain = [state.clone(), conv.clone()]
    gdn.copy_slots([2, 2, 2], [0, 7, 8], state, conv, dims=DIMS)
    for p in plain:
        p[[0, 7, 8]] = p[2].clone()
    slots = [2, 0, 7, 8, 5]

    def step(slots, x):
        qkv, z, a, b = gdn.in_proj_quant(x, q_in, dims=DIMS)
        y = gdn.decode_slots(slots, qkv, z, a, b, weights, state, conv, dims=DIMS)
        st, cv = plain[0][slots].contiguous(), plain[1][slots].contiguous()
        want = gdn.decode(qkv, z, a, b, weights, st, cv, dims=DIMS)
        plain[0][slots], plain[1][slots] = st, cv
        assert torch.equal(y, want)
        out = gdn.out_proj_quant(y, q_out, dims=DIMS)
        _check(torch.cat([qkv, z, b, a], 1), x, w_in, fmt)
        _check(out, y, w_out, fmt)

    for i in range(4):
        step(slots, hidden(len(slots)))
        if i == 1:  # the four beams reordered in place: one kept, one forked twice, one dropped
            src, dst = [0, 0, 7, 0], [2, 0, 7, 8]
            gdn.copy_slots(src, dst, state, conv, dims=DIMS)
            for k in (0, 1):
                plain[k][dst] = plain[k][src].clone()
        if i == 2:  # beams 7 and 8 end; the pool is compacted and the rows behind cleared
            live = [r in (0, 2, 5) for r in range(P)]
            remap = gdn.compact_slots(live, state, conv, clear=True, dims=DIMS).tolist()
            assert remap == [0, -1, 2, -1, -1, 1, -1, -1, -1]
            for k in (0, 1):
                plain[k] = torch.cat([plain[k][[0, 5, 2]], torch.zeros_like(plain[k][3:])])
            slots = [remap[r] for r in (2, 0, 5)]
        assert _same(state, plain[0]) and _same(conv, plain[1])
    assert gdn.last_device_error() == 0


@pytest.mark.parametrize("T", [1, 40, 300])
def test_weights_made_just_before(dev, T):
    """Weights quantised by the call before, tokens written by the call before that: nothing of them is read
    early, over many repeats without a wait between them."""
    w_in, w_out, _, _, _ = _model(dev, "nvfp4")
    ws = [(w_out.to(dev) * s).to(torch.bfloat16) for s in (1, 2, -1, 0.5)]
    y = torch.randn((T, DIMS.value_width), generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(dev)
    base = gdn.out_proj_quant(y, gdn.quantize(ws[0]), dims=DIMS)
    q = gdn.quantize(ws[0])
    pool = torch.zeros((3, DIMS.num_v_heads, 128, 128), device=dev), torch.zeros((3, 3, DIMS.conv_channels), device=dev)
    outs = []
    for i in range(200):
        k = i % 4
        gdn.quantize(ws[k], out=q)
        outs.append(gdn.out_proj_quant(y, q, dims=DIMS))
        pool[0][0, 0, 0, 0] = float(i)
        gdn.copy_slots([0], [1 + i % 2], *pool, dims=DIMS)
        assert pool[0].shape[0] == 3
    torch.cuda.synchronize(dev)
    for i, o in enumerate(outs):  # (scaling by a power of two or -1 is exact)
        assert torch.equal(o, (base.float() * (1, 2, -1, 0.5)[i % 4]).to(torch.bfloat16)), i
    assert pool[0][1, 0, 0, 0].item() == 198 and pool[0][2, 0, 0, 0].item() == 199


@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_after_other_nodes(dev, T):
    """Captured behind a copy, a memset and a join with another stream, each new call as the first kernel
    after them; replayed on changed inputs."""
    w_in, w_out, q_in, q_out, _ = _model(dev, "mxfp4")
    x = torch.zeros((T, HIDDEN), dtype=torch.bfloat16, device=dev)
    src = torch.zeros_like(x)
    flag = torch.zeros((64,), device=dev)
    P = 4
    state = torch.randn((P, DIMS.num_v_heads, 128, 128), device=dev)
    conv = torch.randn((P, 3, DIMS.conv_channels), device=dev)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(2):
        gdn.in_proj_quant(x, q_in, dims=DIMS)
    torch.cuda.synchronize(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        x.copy_(src)
        qkv, z, a, b = gdn.in_proj_quant(x, q_in, dims=DIMS)
        s2.wait_stream(s1)
        with torch.cuda.stream(s2):
            qx = gdn.quantize(x, "nvfp4")
            back = gdn.dequantize(qx)
        flag.zero_()
        gdn.copy_slots([0, 1], [1, 0], state, conv, dims=DIMS)
        s1.wait_stream(s2)
        o = gdn.out_proj_quant(z, q_out, dims=DIMS)
        flag.zero_()
        o2 = gdn.out_proj_quant(z, q_out, dims=DIMS)
    for seed in range(3):
        new = torch.randn((T, HIDDEN), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(dev)
        src.copy_(new)
        before = state.clone()
        torch.cuda.synchronize(dev)
        with torch.cuda.stream(s1):
            graph.replay()
        torch.cuda.synchronize(dev)
        want = gdn.in_proj_quant(new, q_in, dims=DIMS)
        assert all(torch.equal(u, v) for u, v in zip((qkv, z, a, b), want))
        assert torch.equal(o, gdn.out_proj_quant(want[1], q_out, dims=DIMS)) and torch.equal(o, o2)
        assert np.array_equal(back.double().cpu().numpy(), _values(new, "nvfp4"))
        assert torch.equal(state[[1, 0, 2, 3]], before)
