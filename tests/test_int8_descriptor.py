"""The inverse of the int8 layout refuses a descriptor whose size is not that of its N
and K, as the product does: callers hold the buffer against total_bytes, the kernel reads
what N and K say.  CPU only."""
import ctypes
import os

import pytest

from block_scaled_precision_04_amd import _binding
from block_scaled_precision_04_amd._binding import WDesc, BS_WDESC_MAGIC, BS_LAYOUT_INT8

FAKE = ctypes.c_void_p(0x10000)


@pytest.mark.parametrize("total", [0, 2048, 256 * 512 - 2048, 256 * 512 + 2048])
def test_unprelayout_refuses_another_size(total):
    if not os.path.exists(_binding.LIB_PATH):
        from block_scaled_precision_04_amd import build
        build.build()
    d = WDesc(BS_WDESC_MAGIC, BS_LAYOUT_INT8, 256, 512, 256 * 512, 0, 0, total)
    assert _binding.lib().bs_unprelayout_int8(ctypes.byref(d), FAKE, FAKE, None) == -4
