"""Rows of no sequence (padding) before the first and behind the last packed sequence, longer
than what a block walks at once: their outputs are left or zeroed, whatever they hold."""
import pytest
import torch

from test_gpu_glr import inputs, normal, packed_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dig():
    import gated_linear_attention_chunkwise_b200 as pkg
    pkg.device_status()
    return pkg


# Few channels are walked by wide clusters, many by single blocks.
@pytest.mark.parametrize("gap,C", [(129, 8), (200, 8), (1500, 8), (5000, 8), (20011, 8), (129, 520), (200, 520), (5000, 520),
                                   (200, 16384), (1500, 16384)])
@pytest.mark.parametrize("d", [0, 1])
def test_rows_before_the_first_sequence(dig, gap, C, d):
    """Against the definition, zeros in new outputs and untouched rows in given ones."""
    cu = [gap, gap + 1, gap + 1, gap + 40, gap + 90]
    packed_case(dig, cu, gap + 97, C, "f32" if d else "bf16", d, None if d else 16.0, not d, True, seed=gap + C)
    if C == 520:
        packed_case(dig, cu, gap + 2500, C, "bf16", d, 1.0, False, False, fused=True, seed=gap)


@pytest.mark.parametrize("d", [0, 1])
def test_gradients_summed_over_all_rows_see_no_padding(dig, d):
    """What a caller reduces over the rows: the gradients of new outputs are zero in the padding."""
    rows, C, cu = 9000, 64, [7000, 7600, 8100]
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    x, gate = inputs(3, (rows,), C, torch.float32, 1.0)
    for t in (x, gate):
        t[:7000], t[8100:] = float("nan"), float("nan")
    dout = normal(5, (rows, C))
    out, _ = dig.glr_fwd_packed(x, gate, dcu, d, 1.0, True)
    dx, dg, _ = dig.glr_bwd_packed(x, gate, out, dout, dcu, d, 1.0, True)
    for t in (out, dx, dg):
        assert bool((t[:7000] == 0).all()) and bool((t[8100:] == 0).all())
        assert bool(torch.isfinite(t.sum(0)).all())
    assert dig.device_status() == 0


@pytest.mark.parametrize("d", [0, 1])
@pytest.mark.parametrize("gap", [70, 3000])
@pytest.mark.parametrize("junk", [float("inf"), -float("inf"), float("nan"), 3e38, 100.0])
def test_padding_of_any_value_changes_neither_results_nor_the_status(dig, junk, gap, d):
    """Bit for bit what the same call gives with zeros in the padding, and no error recorded."""
    C, cu = 72, [gap, gap + 1, gap + 330, gap + 331, gap + 760]
    rows = cu[-1] + 513
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    for gate_norm, comp in ((None, False), (None, True), (1.0, False), (16.0, True)):
        x, gate = inputs(30, (rows,), C, torch.float32, gate_norm)
        h0, dout, dlast = normal(31, (4, C)), normal(32, (rows, C)), normal(33, (4, C))
        clean = [x, gate, dout]
        for t in clean:
            t[:gap], t[cu[-1]:] = 0, 0
        out, last = dig.glr_fwd_packed(x, gate, dcu, d, gate_norm, comp, h0=h0)
        grads = dig.glr_bwd_packed(x, gate, out, dout, dcu, d, gate_norm, comp, h0=h0, dh_last=dlast)
        bad = [t.clone() for t in (x, gate, out, dout)]
        for t in bad:
            t[:gap], t[cu[-1]:] = junk, junk
        again = dig.glr_fwd_packed(bad[0], bad[1], dcu, d, gate_norm, comp, h0=h0)
        more = dig.glr_bwd_packed(*bad, dcu, d, gate_norm, comp, h0=h0, dh_last=dlast)
        assert dig.device_status() == 0
        for p, q in zip((out, last, *grads), (*again, *more)):
            assert torch.equal(p, q)
