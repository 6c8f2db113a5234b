"""Accuracy of the forget gates, read from the recurrence itself: of alpha near 1, which decides
how long a state lasts, and of 1 - alpha.  U = 2^-24; numbers in [1/2, 1) round by at most U / 2."""
import numpy as np
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu
U = ref.U
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dig():
    import gated_linear_attention_chunkwise_b200 as pkg
    pkg.device_status()
    return pkg


def np64(t):
    return t.detach().double().cpu().numpy()


def alpha_and_rest(dig, gate, gate_norm, dtype):
    """alpha: the state that is left of 1 when nothing comes in; 1 - alpha: what an input of 1
    leaves in an empty state; alpha once more without the complement.  All as the kernels hold
    them, in fp32."""
    def left(x, state, complement):
        x = torch.full(gate.shape, x, dtype=dtype, device="cuda")
        state = torch.full(gate.shape, state, device="cuda")
        return dig.glr_step(x, gate, state, gate_norm=gate_norm, complement=complement)[1]

    alpha, rest, alone = left(0.0, 1.0, True), left(1.0, 0.0, True), left(0.0, 1.0, False)
    return np64(alpha), np64(rest), np64(alone)


def log_gates():
    g = torch.Generator().manual_seed(0)
    near = -torch.rand(4096, generator=g) * 0.15
    tiny = -torch.exp(-torch.rand(4096, generator=g) * 40)
    far = -torch.rand(4096, generator=g) * 80
    edge = torch.tensor([0.0, -0.0, -2.0 ** -24, -2.0 ** -25, -1e-30, -0.1499, -0.15, -0.1501, -0.4999, -0.5, -0.5001, -80.0])
    t = torch.cat([near, tiny, far, edge.repeat(4)])
    return t[:t.numel() // 32 * 32].view(4, -1).contiguous().cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_log_gates(dig, dtype):
    """1 - alpha near alpha = 1 (|x| < 0.15, in fp32 calls 1/2): a polynomial in Horner's form whose
    roundings and remainder are below 3 U of it.  alpha there: that, and one rounding (without
    the complement: for |x| < 1/16).  Elsewhere e^x to 2^-22 with an argument rounded twice,
    (4 + 2 |x|) U, and 1 - e^x that and one rounding."""
    gate = log_gates()
    alpha, rest, alone = alpha_and_rest(dig, gate, None, DT[dtype])
    la = np64(gate)
    want, want_rest = np.exp(la), -np.expm1(la)
    exp_error = want * (4 + 2 * np.abs(la)) * U
    near = np.abs(la) < (0.15 if dtype == "bf16" else 0.5)
    for name, got, close in (("alpha", alpha, near), ("alone", alone, np.abs(la) < 1 / 16)):
        bound = np.where(close, U / 2 + 3 * U * want_rest, exp_error) + 2.0 ** -149
        assert (np.abs(got - want) / bound).max() <= 1, name
    bound = np.where(near, 3 * U * want_rest, exp_error + U * want_rest) + 2.0 ** -149
    assert (np.abs(rest - want_rest) / bound).max() <= 1
    assert dig.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate_norm", [1.0, 16.0])
def test_logits_of_gates_that_hardly_forget(dig, dtype, gate_norm):
    """g >= 2: e = e^-g to 4 U in fp32 calls, to (4 + 2 g) U in bf16 ones; 1 + e, its reciprocal, the
    product: 5 U more (logits / norm: log(1 + e) to 4 U, the division, the polynomial: 8 U);
    alpha = 1 - that, with one rounding."""
    g = torch.linspace(2, 80, 4096).to(DT[dtype]).view(8, 512).contiguous().cuda()
    alpha, rest, alone = alpha_and_rest(dig, g, gate_norm, DT[dtype])
    v = np64(g)
    la = -np.log1p(np.exp(-v)) / gate_norm
    want, want_rest = np.exp(la), -np.expm1(la)
    bound = (12 + 2 * v * (dtype == "bf16")) * U * want_rest + 2.0 ** -149
    assert (np.abs(rest - want_rest) / bound).max() <= 1
    for a in (alpha, alone):
        assert (np.abs(a - want) / (U / 2 + bound)).max() <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("log_alpha,T", [(-1e-4, 32768), (-1e-6, 65536), (-3e-3, 20011)])
def test_slow_decay_of_a_constant_input(dig, dtype, log_alpha, T):
    """h_n = (1 - alpha^n) / (1 - alpha).  A token's terms are scaled by alpha (U / 2 + 3 U (1 - alpha)
    off), by a rounded product and by a rounded sum: 3 U a token, and 32 U for the order of the
    folds.  A sum that forgets nothing lies far outside."""
    C = 16
    x = torch.ones(1, T, C, dtype=DT[dtype], device="cuda")
    la = torch.full((1, T, C), log_alpha, device="cuda")
    out, last = dig.glr_fwd(x, la, 1, T, 0)
    a = np.exp(np.float64(np.float32(log_alpha)))
    n = np.arange(1, T + 1)
    want = -np.expm1(n * np.log(a)) / (1 - a)
    # sum over j < n of alpha^j (3 U j + 33 U)
    weighted = np.cumsum(np.exp(n * np.log(a)) * n)
    bound = 3 * U * np.concatenate([[0], weighted[:-1]]) + 33 * U * want
    assert (np.abs(np.arange(1, T + 1) - want) > 3 * bound)[T // 2:].all()
    got = np64(last)[0]
    assert (np.abs(got - want[-1]) <= bound[-1]).all(), (got[0], want[-1], bound[-1])
    b = bound + (ref.EPS16 * want if dtype == "bf16" else 0)
    assert (np.abs(np64(out)[0] - want[:, None]) <= b[:, None]).all()
    dout = torch.ones_like(x)
    dx, dg, dh0 = dig.glr_bwd(x, la, out, dout, 1, T, 0)
    assert (np.abs(np64(dx)[0, ::-1] - want[:, None]) <= b[:, None]).all()
    assert dig.device_status() == 0
