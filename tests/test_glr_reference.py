"""The 64-bit forms of the sequence operators against independent statements of the same
mathematics (unrolled sums, finite differences, complex rotation), on the CPU; and the
host-side table of rotary frequencies."""
import math

import numpy as np
import pytest

import seq_reference as ref


def make(rng, rows, C, nseq, gate_norm):
    x = rng.standard_normal((rows, C))
    g = rng.standard_normal((rows, C))
    gate = g if gate_norm else -np.abs(g) / 4
    return x, gate, rng.standard_normal((nseq, C))


@pytest.mark.parametrize("gate_norm", [None, 1.0, 16.0])
@pytest.mark.parametrize("complement", [False, True])
def test_forward_is_the_unrolled_sum(gate_norm, complement):
    rng = np.random.default_rng(0)
    x, gate, h0 = make(rng, 12, 3, 2, gate_norm)
    cu = [0, 5, 12]
    out, last, *_ = ref.glr_fwd(x, gate, gate_norm, complement, h0, ref.runs(None, cu=cu))
    a = np.exp(gate) if gate_norm is None else (1 / (1 + np.exp(-gate))) ** (1 / gate_norm)
    s = 1 - a if complement else np.ones_like(a)
    for n in range(2):
        for t in range(cu[n], cu[n + 1]):
            want = np.prod(a[cu[n]:t + 1], 0) * h0[n]
            for j in range(cu[n], t + 1):
                want = want + np.prod(a[j + 1:t + 1], 0) * s[j] * x[j]
            assert np.allclose(out[t], want, rtol=1e-12, atol=1e-13)
        assert np.allclose(last[n], out[cu[n + 1] - 1])


@pytest.mark.parametrize("d", range(12))
def test_scan_orders_agree_with_the_oracle(d):
    import oracle
    assert np.array_equal(ref.scan_order(5, 7, d), oracle.scan_order(d, 5, 7))


@pytest.mark.parametrize("gate_norm", [None, 1.0, 16.0])
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
def test_backward_is_the_difference_quotient(gate_norm, complement, reverse):
    rng = np.random.default_rng(1)
    x, gate, h0 = make(rng, 9, 2, 3, gate_norm)
    where = ref.runs(None, cu=[0, 4, 4, 9], reverse=reverse)
    dout, dlast = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)

    def loss(x, gate, h0):
        out, last, *_ = ref.glr_fwd(x, gate, gate_norm, complement, h0, where)
        return np.sum(out * dout) + np.sum(last * dlast)

    h = ref.glr_fwd(x, gate, gate_norm, complement, h0, where)[0]
    got, _ = ref.glr_bwd(x, gate, h, dout, gate_norm, complement, h0, dlast, where)
    args = [x, gate, h0]
    for k in range(3):
        for at in np.ndindex(args[k].shape):
            up, down = [t.copy() for t in args], [t.copy() for t in args]
            up[k][at] += 1e-6
            down[k][at] -= 1e-6
            assert abs((loss(*up) - loss(*down)) / 2e-6 - got[k][at]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication_and_inverse_its_transpose(interleaved):
    rng = np.random.default_rng(2)
    t, d = rng.standard_normal((4, 3, 16)), rng.standard_normal((4, 3, 16))
    pos, inv = np.array([0, 1, -7, 100000]), 100.0 ** -(np.arange(5) / 5)
    out, _ = ref.rotate(t, pos, inv, interleaved, 1.25)
    i, j = ref.pair_index(10, interleaved)
    z = (t[..., i] + 1j * t[..., j]) * 1.25 * np.exp(1j * (pos[:, None] * inv))[:, None]
    assert np.allclose(out[..., i] + 1j * out[..., j], z) and np.array_equal(out[..., 10:], t[..., 10:])
    back, _ = ref.rotate(d, pos, inv, interleaved, 1.25, inverse=True)
    assert np.isclose(np.sum(out * d), np.sum(t * back))


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradient_is_the_difference_quotient(interleaved):
    rng = np.random.default_rng(3)
    t, d, w = rng.standard_normal((2, 2, 8)), rng.standard_normal((2, 2, 8)), rng.standard_normal(8)
    how = (np.array([3, 50]), 100.0 ** -(np.arange(3) / 3), 1e-3, interleaved, 1.1)
    (dx, dw), _ = ref.norm_rope_bwd(d, t, w, *how)

    def loss(t, w):
        return np.sum(ref.norm_rope(t, w, *how)[0] * d)

    for got, k in ((dx, 0), (dw, 1)):
        args = [t, w]
        for at in np.ndindex(args[k].shape):
            up, down = [v.copy() for v in args], [v.copy() for v in args]
            up[k][at] += 1e-6
            down[k][at] -= 1e-6
            assert abs((loss(*up) - loss(*down)) / 2e-6 - got[at]) < 1e-7


def test_rope_frequencies():
    import gated_linear_attention_chunkwise_b200 as dig
    inv, scale = dig.rope_frequencies(8)
    assert scale == 1.0 and np.allclose(inv, [1, 1e-1, 1e-2, 1e-3])
    inv, scale = dig.rope_frequencies(8, scaling="linear", factor=4)
    assert scale == 1.0 and np.allclose(inv, np.array([1, 1e-1, 1e-2, 1e-3]) / 4)
    inv, scale = dig.rope_frequencies(8, scaling="base", factor=4)
    assert np.isclose(inv[0], 1) and np.isclose(inv[3], 1e-3 / 4)    # fastest as it was, slowest as linear
    inv, scale = dig.rope_frequencies(64, scaling="ramp", factor=4, original_length=4096)
    plain, _ = dig.rope_frequencies(64)
    ratio = (plain / inv).numpy()
    assert np.isclose(scale, 0.1 * math.log(4) + 1)
    assert np.isclose(ratio[0], 1) and np.isclose(ratio[-1], 4) and np.all(np.diff(ratio) >= -1e-6)
    turns = plain.numpy() * 4096 / (2 * math.pi)
    assert np.allclose(ratio[turns > 40], 1) and np.allclose(ratio[turns < 0.7], 4)
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="ramp"), dict(rot=8, base=0.0), dict(rot=2, scaling="base")):
        with pytest.raises(ValueError):
            dig.rope_frequencies(**bad)
