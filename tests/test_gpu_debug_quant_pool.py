"""The 4-bit and pool entry points on the debug build of the library (-DGDN_DEBUG, see
test_gpu_debug_build.py): the same bits as the release build, the error word 0."""
import os
import subprocess
import sys

import pytest
import torch

import gated_deltanet_mixer_gdn_b200 as gdn
from gated_deltanet_mixer_gdn_b200 import build as gdn_build
from gated_deltanet_mixer_gdn_b200.synth import Dims

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run_cases(dev):
    res = {}
    g = torch.Generator().manual_seed(3)
    dims = Dims(num_k_heads=2, num_v_heads=6)
    N = dims.conv_channels + dims.value_width + 12
    w = torch.randn((N, 448), generator=g).to(torch.bfloat16).to(dev)
    for fmt in gdn.QUANT_FORMATS:
        q = gdn.quantize(w, fmt)
        res[fmt + "_values"] = gdn.dequantize(q)
        for T in (1, 40, 100, 300):
            x = torch.randn((T, 448), generator=g).to(torch.bfloat16).to(dev)
            res[f"{fmt}_proj{T}"] = torch.cat(gdn.in_proj_quant(x, q, dims=dims), 1)
    st = torch.randn((20, 6, 128, 128), generator=g).to(dev)
    cv = torch.randn((20, 3, dims.conv_channels), generator=g).to(dev)
    gdn.copy_slots([1, 0, 3, 3, -1], [0, 1, 4, 5, 3], st, cv, dims=dims)
    gdn.compact_slots([i % 3 != 1 for i in range(20)], st, cv, clear=True, dims=dims)
    res.update(state=st, conv=cv)
    torch.cuda.synchronize(dev)
    return {k: v.cpu() for k, v in res.items()}


CHILD = """
import sys, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import gated_deltanet_mixer_gdn_b200 as gdn
from test_gpu_debug_quant_pool import run_cases
assert gdn.LIB_PATH.endswith("libgdn_b200_debug.so"), gdn.LIB_PATH
res = run_cases(torch.device("cuda", 0))
res["error_word"] = torch.tensor([gdn.last_device_error()])
torch.save(res, {out!r})
"""


def test_debug_build_same_bits(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    out = str(tmp_path / "debug.pt")
    env = dict(os.environ, GDN_B200_LIBRARY=gdn_build.build(debug=True))
    subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), out=out)],
                   env=env, check=True, timeout=600)
    dbg = torch.load(out)
    assert int(dbg.pop("error_word")[0]) == 0
    rel = run_cases(torch.device("cuda", 0))
    assert gdn.last_device_error() == 0 and set(rel) == set(dbg)
    for k in rel:
        assert torch.equal(rel[k], dbg[k]), k
