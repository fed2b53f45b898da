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


# -- log probabilities ----------------------------------------------------------
def best_ids(x, top):
    """Indices of the `top` best of each row by (value, lowest index), NaN below everything."""
    x = x.double().cpu()
    value = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    by_value = torch.sort(value, dim=1, descending=True, stable=True).indices
    nan = torch.isnan(x).gather(1, by_value)
    return by_value.gather(1, torch.sort(nan.int(), dim=1, stable=True).indices)[:, :top]


@pytest.mark.parametrize("T,V", [(3, 9000), (3, 70), (3, 1), (2, 33), (3, 4097), (3, 120001), (2, 200003),
                                 (1100, 500)])  # whole rows, rows in chunks, a wave a row
@pytest.mark.parametrize("top", [1, 2, 5])
def test_alternatives_of_rows_with_few_numbers(T, V, top):
    """Rows of NaN but for a few logits, of a length that ends inside a group: every id is written, and right."""
    top = min(top, V)
    for numbers in ([], [V - 1], [V // 2], [0, V - 1], list(range(max(0, V - V % 32 - 1), V))[:top]):
        for value in (1.5, -math.inf):
            x = torch.full((T, V), math.nan)
            for i in numbers:
                x[:, i] = value - i * 1e-6 if math.isfinite(value) else value
            for dtype in (torch.float32, BF16):
                y = x.to(dtype).cuda()
                junk = torch.full((T * top,), 0x1234567812345678, dtype=torch.int64, device="cuda")
                del junk  # what the allocator hands out next
                _, _, ids, lp = ttq.ttq_token_logprobs(y, torch.zeros(T, dtype=torch.int64, device="cuda"), top=top)
                assert torch.equal(ids.cpu(), best_ids(y, top)), (numbers, value, dtype)
                if bool(torch.isnan(x).any()):
                    assert bool(torch.isnan(lp).all())
