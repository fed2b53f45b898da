"""The serving operators at the edges of their ranges, on the GPU, against the
same plain statements in 64 bits as the other tests of them."""
import math

import pytest

torch = pytest.importorskip("torch")
import test_activation_aware_amd as ttq  # noqa: E402
from test_gpu_serving import BF16, F16, Batch, attention_ref, check_attention, say  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ttq.load()
    yield
    torch.cuda.synchronize()


# -- attention -----------------------------------------------------------------
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 30])
@pytest.mark.parametrize("lens", [[(70, 3), (9, 4), (1, 130)], [(3, 0), (200, 100)]])
def test_attention_windows_beyond_every_position(lens, window):
    """With tokens before position 0, whose distance to the window's begin passes 32 bits."""
    check_attention(lens, 4, 2, 64, 16, F16, window=window)
    check_attention(lens, 4, 2, 128, 16, BF16, window=window, prefix=[2, 0, 50][:len(lens)])
