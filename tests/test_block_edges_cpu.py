"""The operators around the layer without a GPU: what they refuse beyond
test_block_cpu, and what their sources must not do."""
import os
import re

import pytest
import torch

from mixture_experts_layer_55_b200 import MoELayer
from mixture_experts_layer_55_b200 import _binding as B
from mixture_experts_layer_55_b200 import build as build_mod

CSRC = os.path.join(os.path.dirname(B.__file__), "csrc")


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def test_rows_scales_are_not_read_through_the_read_only_path():
    """The down product is resident while the gate/up product writes its rows' scales:
    the read-only path, for data that nothing writes while a kernel runs, is left
    to the weights' scales."""
    with open(os.path.join(CSRC, "ffn_mx8.cu")) as f:
        text = f.read()
    calls = re.findall(r"= load_scales(<\w+>)?\((\w+),", text)
    assert len(calls) == 6
    for how, what in calls:
        assert how == ("<false>" if what in ("pa", "px") else "<true>"), what
    assert [line.strip() for line in text.splitlines() if "__ldg(" in line] == [
        "return WEIGHT ? __ldg(reinterpret_cast<const V*>(p)) : *reinterpret_cast<const V*>(p);"]
