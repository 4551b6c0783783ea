"""Every weight stream that is built, at a size that runs it, bit for bit."""
import pytest

from tests.test_build_w8a8_instances import DENSE
from tests.test_gpu_w8a8 import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", DENSE.values(), ids=["-".join(map(str, d)) for d in DENSE])
def test_each_stream(size):
    M, N, K = size
    _run(M, N, K)
    _run(M, N + 3, K + 16)        # columns and K that end inside a tile
