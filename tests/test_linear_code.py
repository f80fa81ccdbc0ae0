"""The products' machine code: the main loops of the 256 x 256 kernels, whose
accumulators take half of a wave's registers, spill nothing and move no
accumulator (a kernel that does takes up to twice as long)."""

import re

import pytest

from test_kernel_code import kernels, pytestmark  # noqa: F401 (a fixture, and when it can run)

AWAY = re.compile("scratch_|v_accvgpr_")


def stage_blocks(code):
    """Instructions without a branch between them that hold 60 products or more and load the ring."""
    targets = {target for _, _, target in code if target is not None}
    blocks, block = [], []
    for address, text, target in code:
        if address in targets:
            blocks.append(block)
            block = []
        block.append(text)
        if target is not None:
            blocks.append(block)
            block = []
    return [b for b in (*blocks, block) if sum(t.startswith("v_mfma") for t in b) >= 60
            and any(t.startswith("buffer_load") and t.endswith(" lds") for t in b)]


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("plain", [0, 1])
def test_large_products_keep_their_accumulators(kernels, mode, plain):  # noqa: F811
    found = {n: c for n, c in kernels.items() if f"k_linearILb0ELi{mode}E" in n and "GeoILi256ELi256E" in n and f"ELi16ELb{plain}E" in n}
    assert len(found) == 1
    for name, code in found.items():
        blocks = stage_blocks(code)
        assert len(blocks) >= 15, (name, len(blocks))   # five stages of the whole tile and of the halves in either direction
        for block in blocks:
            away = [t for t in block if AWAY.match(t)]
            assert not away, (name, len(away), away[:3])
