"""Every kernel file of the debug build whose kernels address global memory by computed indices holds index checks
(GDN_CHECK), and in the 4-bit and pool files every kernel and every function that stores does."""
import os
import re

import gated_deltanet_mixer_gdn_b200 as gdn

CSRC = os.path.join(os.path.dirname(gdn.__file__), "csrc")
UNCHECKED = {"common.cuh", "gemm.cuh", "inproj.cuh"}  # helpers; the bf16 projections (TMA boxes, output tiles)


def _text(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_files():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cuh") and name not in UNCHECKED:
            assert "GDN_CHECK(" in _text(name), name


def test_quant_and_pool_functions():
    parts = [("quant.cuh", ["gdn_quantize_kernel", "gdn_dequantize_kernel"]), ("pool.cuh", ["gdn_pool_kernel"]),
             ("qproj.cuh", ["quantize_tokens", "gdn_qproj_few_kernel", "store_tile32x64", "output_at"])]
    for name, functions in parts:
        text = _text(name)
        for f in functions:
            start = re.search(r"\b%s\([^;{]*\{" % f, text)
            body = text[start.start():text.index("\n}", start.start())]
            assert "GDN_CHECK(" in body, (name, f)
