"""The bound that the GPU tests hold attention over the 4-bit cache to
(packed_precision.py), on the CPU: roundings to fp16 keep it, and keys, values and
probabilities in bf16, three bits less, do not."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import packed_precision as precision  # noqa: E402
from test_gpu_packed_attention import Batch, TYPES  # noqa: E402

LENS = ((300, 400), (1, 300), (140, 140))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("how", [{}, dict(softcap=30.0), dict(slopes=[0.5, 0.1, 0.02, 0.0], window=200), dict(scale=0.05)],
                         ids=["plain", "cap", "bias", "scale"])
def test_the_bound_tells_fp16_from_bf16(dtype, dim, how):
    b = Batch(LENS, 4, 2, dim, 16, dtype)
    want, noise = precision.attend(b, **how)
    most = precision.bound(TYPES[dtype], noise)
    offs = []
    for low in (torch.float16, torch.bfloat16):
        got, _ = precision.attend(b, low, **how)
        offs.append(precision.off(precision.rounded(got, TYPES[dtype]), want))
    assert offs[0] <= most < offs[1], (offs, most)


def test_the_reference_is_the_other_one():
    """The same as the outputs that the other tests compute."""
    b = Batch(LENS, 4, 2, 64, 16)
    for how in ({}, dict(softcap=5.0, window=7), dict(prefix=[0, 40, 100], slopes=[0.5, 0.1, 0.02, 0.0])):
        assert np.abs(precision.attend(b, **how)[0] - b.want(**how)[0]).max() < 1e-12
