"""GPU: both code formats with every number of query heads a tile carries (4, 8 and 16, and several
chunks of them) and with heads of one and two 128-channel halves."""
import pytest

import fp8_block_scaled_12_b200 as F
from test_parity_attention import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
@pytest.mark.parametrize("G", [1, 4, 6, 8, 9, 16, 20])
@pytest.mark.parametrize("D", [64, 128, 144, 256])
def test_heads_of_a_tile(cuda_device, fmt, G, D):
    case([300, 5, 0, 1029], 2, G, D, 32, fmt, seed=G + D)


@pytest.mark.parametrize("G", [3, 7, 15, 33])
@pytest.mark.parametrize("D", [80, 192])
def test_windows_of_e5m2(cuda_device, G, D):
    case([1000, 3, 128, 400], 1, G, D, 16, F.E5M2, "NHD", window=129, seed=G)
