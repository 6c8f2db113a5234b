"""The blended table of rotary frequencies, pair by pair against its definition in 64 bits: pairs
that turn more than beta_fast times over the original length keep their frequency, those that
turn less than beta_slow times have it divided, and the share of the division grows linearly in
the pair's number in between, from the last whole pair before the one bound to the first behind
the other, whether these are pairs of the table or not."""
import math

import numpy as np
import pytest


def share_of(i, rot, base, length, fast, slow):
    def pair(turns):   # where base^(-2 i / rot) * length = 2 pi turns
        return rot / 2 * math.log(length / (2 * math.pi * turns), base)

    first, last = math.floor(pair(fast)), math.ceil(pair(slow))
    return np.clip((i - first) / (last - first), 0, 1)


@pytest.mark.parametrize("rot", [8, 64, 128, 256])
@pytest.mark.parametrize("base", [1e4, 5e5])
@pytest.mark.parametrize("length", [60, 150, 4096, 32768, 131072, 1000003])
@pytest.mark.parametrize("factor,fast,slow", [(8.0, 32.0, 1.0), (1.5, 16.0, 2.0)])
def test_ramp(rot, base, length, factor, fast, slow):
    import gated_linear_attention_chunkwise_b200 as dig
    inv, scale = dig.rope_frequencies(rot, base, "ramp", factor, length, fast, slow)
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    turns = plain * length / (2 * math.pi)
    s = share_of(i, rot, base, length, fast, slow)
    want = plain * (1 - s) + plain / factor * s
    got = inv.numpy().astype(np.float64)
    assert np.allclose(got, want, rtol=2.0 ** -23, atol=0)   # one rounding to fp32, and fp64's
    assert scale == pytest.approx(0.1 * math.log(factor) + 1)
    divided = plain / got
    assert np.allclose(divided[turns > fast], 1, rtol=2.0 ** -23)
    assert np.allclose(divided[turns < slow], factor, rtol=2.0 ** -23)


def test_a_table_that_ends_inside_the_ramp():
    """128 channels, base 1e4, 131072 tokens: the slowest pair turns 2.4 times, more than once, and is
    blended."""
    import gated_linear_attention_chunkwise_b200 as dig
    inv, _ = dig.rope_frequencies(128, 1e4, "ramp", 8.0, 131072)
    plain, _ = dig.rope_frequencies(128, 1e4)
    divided = (plain / inv).numpy()
    # (63 - 45) / (70 - 45) of the way: 1 / (0.28 + 0.72 / 8)
    assert divided[63] == pytest.approx(1 / (0.28 + 0.72 / 8), rel=1e-6)
    assert (np.diff(divided) >= -1e-6).all()


def test_device_zero_is_a_device():
    """An index names a CUDA device, 0 among them."""
    import torch
    import gated_linear_attention_chunkwise_b200 as dig
    assert dig.rope_frequencies(8)[0].device.type == "cpu"
    assert dig.rope_frequencies(8, device="cpu")[0].device.type == "cpu"
    if torch.cuda.is_available():
        assert dig.rope_frequencies(8, device=0)[0].device == torch.device("cuda", 0)
    else:
        with pytest.raises((RuntimeError, AssertionError)):
            dig.rope_frequencies(8, device=0)
