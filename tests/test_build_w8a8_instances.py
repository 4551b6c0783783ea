"""The weight streams that are built are those that a call can reach: no kernel is there,
and counted by the checks of its assembly, that no size runs."""
import re

import pytest

from tests.test_build_registers import _asm, _hipcc, _kernels

pytestmark = pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")

# row blocks, column tiles a wave, K blocks, K runs in a loop, by expert: rows, N, K that run it
DENSE = {
    (1, 1, 4, 0): (1, 16, 128), (1, 1, 8, 0): (1, 16, 1152), (1, 2, 8, 0): (1, 4288, 1152),
    (2, 1, 4, 0): (17, 16, 128), (2, 1, 4, 1): (17, 8304, 2176), (2, 1, 8, 0): (17, 16, 12288), (2, 1, 8, 1): (17, 272, 117632),
    (4, 1, 4, 0): (33, 16, 2176), (4, 1, 4, 1): (33, 80, 93184), (4, 1, 8, 1): (33, 8304, 12288),
}
GROUPED = {(1, 2, 4, 1), (1, 1, 8, 1)}      # up to K = 256, and past it


def test_streams_that_are_built():
    built = set()
    for name, _ in _kernels(_asm("gemm_w8a8.hip")):
        m = re.search(r"k_w8a8_streamILi(\d+)ELi(\d+)ELi(\d+)ELb([01])ELb([01])E", name)
        if m:
            built.add(tuple(int(x) for x in m.groups()))
    assert built == {d + (0,) for d in DENSE} | {g + (1,) for g in GROUPED}
