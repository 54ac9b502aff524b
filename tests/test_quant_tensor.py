"""QuantTensor as a value of a program: comparisons and containers ask for identity and never compare elements."""
import torch

import gated_deltanet_mixer_gdn_b200 as gdn


def _make(row_scale=1.0):
    return gdn.QuantTensor(torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((1, 1, 512), dtype=torch.uint8),
                           torch.full((2,), row_scale), "nvfp4")


def test_identity():
    a, b = _make(), _make()
    assert a == a and (a == b) is False and (a != b) is True and (a == None) is False  # noqa: E711
    assert a in [b, a] and _make() not in [a, b]
    assert {a: 1, b: 2}[b] == 2 and len({a, b, a}) == 2
