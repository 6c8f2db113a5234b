"""The phase of a rotation in fp32: cos and sin of the exact angle, to their own rounding near
their zeros too, where an angle rounded to fp32 would lose all of it."""
import numpy as np
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dig():
    import gated_linear_attention_chunkwise_b200 as pkg
    pkg.device_status()
    return pkg


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_cos_and_sin_keep_their_relative_accuracy(dig, interleaved, inverse):
    """Pairs (1, 0) turn into (cos, sin).  Both functions to 2 units (4 U), the correction and its
    sum 2 U; the angle itself is formed in fp64: three roundings of 2^-53 of up to 1.6e5 turns,
    3.4e-10 in radians."""
    rows, D = 4096, 64
    q = torch.zeros(rows, 1, D, device="cuda")
    i, j = ref.pair_index(D, interleaved)
    q[..., i] = 1.0
    inv, _ = dig.rope_frequencies(D, device="cuda")
    pos = torch.randint(-10 ** 6, 10 ** 6, (rows,), generator=torch.Generator().manual_seed(1))
    pos[:200] = torch.arange(200)
    got, _ = dig.rope(q, None, pos.cuda(), inv, interleaved=interleaved, inverse=inverse)
    got = got.double().cpu().numpy()
    c, s = ref.phases(pos.numpy(), inv.double().cpu().numpy())   # the products are exact in fp64
    s = -s if inverse else s
    for name, g, want in (("cos", got[..., i], c), ("sin", got[..., j], s)):
        bound = 6 * ref.U * np.abs(want) + 3.4e-10
        assert (np.abs(g - want) / bound).max() <= 1, name
