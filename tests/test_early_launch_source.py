"""The kernels that may start before the stream's previous kernel has ended (quantise, dequantise, the 4-bit
projections, the pool move) read their inputs by ordinary loads and bulk copies: the read-only path requires data
that nothing writes while the kernel is resident, and the previous kernel may still be writing it."""
import os
import re

import gated_deltanet_mixer_gdn_b200 as gdn

CSRC = os.path.join(os.path.dirname(gdn.__file__), "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_no_read_only_loads():
    for name in ("quant.cuh", "qproj.cuh", "pool.cuh"):
        code = _code(name)
        assert "grid_wait()" in code
        assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code), name
