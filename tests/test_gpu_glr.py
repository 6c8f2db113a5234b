"""GPU parity of the gated linear recurrence (glr_fwd, glr_bwd, their packed forms, glr_step)
against the 64-bit loops of seq_reference.py, element by element within a-priori bounds."""
import numpy as np
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dig():
    import gated_linear_attention_chunkwise_b200 as pkg
    pkg.device_status()
    return pkg


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def normal(seed, shape, dtype=torch.float32, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) + mean).to(dtype).cuda()


def inputs(seed, lead, C, dtype, gate_norm, fused=False):
    if fused:
        both = normal(seed, (*lead, 3 * C), dtype)
        return both[..., C:2 * C], both[..., 2 * C:] if gate_norm else -normal(seed + 1, (*lead, 2 * C)).abs()[..., :C] / 8
    x = normal(seed, (*lead, C), dtype)
    if gate_norm:
        return x, normal(seed + 1, (*lead, C), dtype, 1.0)
    return x, -normal(seed + 1, (*lead, C)).abs() / 8


def flat(t):
    t = np64(t)
    return t.reshape(-1, t.shape[-1])


def compare(got, want, bounds, names, dtypes):
    for g, w, b, name, dt in zip(got, want, bounds, names, dtypes):
        ref.check(np64(g).reshape(w.shape), w, b, name, bf16=dt == torch.bfloat16)


def check_fwd(dig, x, gate, gate_norm, complement, h0, call, where):
    out, last = call(h0=h0, gate_norm=gate_norm, complement=complement)
    assert out.dtype == x.dtype and last.dtype == torch.float32 and out.shape == x.shape
    w = ref.glr_fwd(flat(x), flat(gate), gate_norm, complement, np64(h0), where)
    compare((out, last), w[:2], w[2:], ("out", "h_last"), (x.dtype, torch.float32))
    return out


def check_bwd(dig, x, gate, gate_norm, complement, h0, h, dout, dlast, call, where):
    got = call(h0=h0, dh_last=dlast, gate_norm=gate_norm, complement=complement)
    assert got[0].dtype == x.dtype and got[1].dtype == gate.dtype and got[2].dtype == torch.float32
    want, bounds = ref.glr_bwd(flat(x), flat(gate), flat(h), flat(dout), gate_norm, complement, np64(h0), np64(dlast), where)
    compare(got, want, bounds, ("dx", "dgate", "dh0"), (x.dtype, gate.dtype, torch.float32))


def grid_case(dig, B, Hg, Wg, C, dtype, d, gate_norm, complement, with_h0, fused=False, seed=0):
    dtype = DT[dtype]
    x, gate = inputs(seed, (B, Hg * Wg), C, dtype, gate_norm, fused)
    h0 = normal(seed + 2, (B, C)) if with_h0 else None
    where = ref.runs((B, Hg * Wg), order=ref.scan_order(Hg, Wg, d))
    h = check_fwd(dig, x, gate, gate_norm, complement, h0, lambda **k: dig.glr_fwd(x, gate, Hg, Wg, d, **k), where)
    dout, dlast = normal(seed + 3, x.shape, dtype), normal(seed + 4, (B, C)) if with_h0 else None
    check_bwd(dig, x, gate, gate_norm, complement, h0, h, dout, dlast,
              lambda **k: dig.glr_bwd(x, gate, h, dout, Hg, Wg, d, **k), where)
    assert dig.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate_norm", [None, 1.0, 16.0, 0.5])
@pytest.mark.parametrize("complement", [False, True])
def test_gates_and_types(dig, dtype, gate_norm, complement):
    grid_case(dig, 2, 9, 23, 72, dtype, 0, gate_norm, complement, True)
    grid_case(dig, 1, 1, 77, 200, dtype, 1, gate_norm, complement, False, fused=True, seed=10)


@pytest.mark.parametrize("d", range(12))
def test_scan_orders(dig, d):
    grid_case(dig, 2, 13, 11, 64, "f32", d, None, False, True, seed=d)
    grid_case(dig, 1, 7, 40, 136, "bf16", d, 16.0, True, False, seed=d)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 31, 63, 64, 65, 127, 129, 255, 256, 257, 511, 513, 1025, 2049])
@pytest.mark.parametrize("C", [8, 64, 328])
def test_lengths(dig, T, C):
    grid_case(dig, 1 + (T < 100), 1, T, C, "bf16", T % 2, None if T % 3 else 1.0, T % 2 == 0, T % 5 != 0, seed=T)


@pytest.mark.parametrize("B,T,C", [(1, 9001, 40), (1, 4999, 1152), (3, 3001, 520), (64, 65, 264), (300, 5, 72), (1, 1, 65536)])
def test_shapes(dig, B, T, C):
    grid_case(dig, B, 1, T, C, "f32" if C < 100 else "bf16", 0, 16.0, True, True, seed=B + T)


def packed_case(dig, cu, rows, C, dtype, d, gate_norm, complement, with_h0, fused=False, seed=0):
    dtype = DT[dtype]
    x, gate = inputs(seed, (rows,), C, dtype, gate_norm, fused)
    n = len(cu) - 1
    h0 = normal(seed + 2, (n, C)) if with_h0 else None
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    where = ref.runs(None, cu=cu, reverse=d == 1)
    h = check_fwd(dig, x, gate, gate_norm, complement, h0, lambda **k: dig.glr_fwd_packed(x, gate, dcu, d, **k), where)
    dout, dlast = normal(seed + 3, x.shape, dtype), normal(seed + 4, (n, C)) if with_h0 else None
    check_bwd(dig, x, gate, gate_norm, complement, h0, h, dout, dlast,
              lambda **k: dig.glr_bwd_packed(x, gate, h, dout, dcu, d, **k), where)
    # rows of no sequence: as they were in given outputs
    outside = torch.ones(rows, dtype=torch.bool)
    outside[cu[0]:cu[-1]] = False
    out = torch.full_like(h, 7.0)
    dig.glr_fwd_packed(x, gate, dcu, d, gate_norm, complement, h0=h0, out=out)
    assert bool((out[outside.cuda()] == 7).all()) and torch.equal(out[~outside.cuda()], h[~outside.cuda()])
    dx, dg = torch.full_like(out, 7.0), torch.full(x.shape, 7.0, dtype=gate.dtype, device="cuda")
    dig.glr_bwd_packed(x, gate, h, dout, dcu, d, gate_norm, complement, h0=h0, dx=dx, dgate=dg)
    assert bool((dx[outside.cuda()] == 7).all()) and bool((dg[outside.cuda()] == 7).all())
    assert dig.device_status() == 0


CUS = {
    "one": ([0, 37], 37),
    "mixed": ([0, 1, 1, 64, 65, 200, 200, 200, 731, 1000], 1000),
    "padded": ([5, 6, 70, 70, 333], 400),
    "all_empty_but_one": ([3, 3, 3, 4, 4], 9),
    "no_tokens": ([4, 4, 4], 8),
    "single_tokens": (list(range(0, 301)), 301),
    "long_and_short": ([0, 2900, 2901, 2902, 2910, 4097], 4100),
    "ends_inside_tiles": ([0, 7, 15, 23, 63, 128, 129, 255, 511, 512, 520, 1024], 1024),
}


@pytest.mark.parametrize("name", CUS)
@pytest.mark.parametrize("d", [0, 1])
def test_packed(dig, name, d):
    cu, rows = CUS[name]
    packed_case(dig, cu, rows, 72, "f32", d, None, False, True, seed=1)
    packed_case(dig, cu, rows, 136, "bf16", d, 16.0, True, d == 0, fused=True, seed=2)


def test_packed_many_sequences(dig):
    rng = np.random.default_rng(0)
    cu = np.sort(rng.integers(0, 5991, 3001))
    cu[0], cu[-1] = 0, 5990
    packed_case(dig, cu.tolist(), 6000, 64, "bf16", 0, 1.0, True, True, seed=3)


def test_states_in_place_and_carried(dig):
    """Two halves with the state carried in one buffer equal the whole; so do the gradients."""
    x, gate = inputs(5, (2, 300), 96, torch.float32, None)
    whole, last = dig.glr_fwd(x, gate, 1, 300, 0)
    h = torch.zeros(2, 96, device="cuda")
    a, _ = dig.glr_fwd(x[:, :140].contiguous(), gate[:, :140].contiguous(), 1, 140, 0, h0=h, h_last=h)
    mid = h.clone()
    b, got = dig.glr_fwd(x[:, 140:].contiguous(), gate[:, 140:].contiguous(), 1, 160, 0, h0=h, h_last=h)
    assert got.data_ptr() == h.data_ptr()
    assert torch.allclose(torch.cat([a, b], 1), whole, rtol=1e-5, atol=1e-5) and torch.allclose(h, last, rtol=1e-5, atol=1e-5)
    dout = normal(6, x.shape)
    dx, dg, _ = dig.glr_bwd(x, gate, whole, dout, 1, 300, 0)
    r = torch.zeros(2, 96, device="cuda")
    tail = dig.glr_bwd(*(t[:, 140:].contiguous() for t in (x, gate, whole, dout)), 1, 160, 0, h0=mid, dh_last=r, dh0=r)
    head = dig.glr_bwd(*(t[:, :140].contiguous() for t in (x, gate, whole, dout)), 1, 140, 0, dh_last=r, dh0=r)
    assert torch.allclose(torch.cat([head[0], tail[0]], 1), dx, rtol=1e-5, atol=1e-5)
    assert torch.allclose(torch.cat([head[1], tail[1]], 1), dg, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("complement", [False, True])
def test_resets_and_non_finite_values(dig, complement):
    """-inf log gates reset the state; a NaN input or gate stays in its channel and sequence and
    ends at a reset by a full gate in the complement form or at the sequence's end."""
    rows, C, cu = 700, 64, [0, 333, 700]
    x, gate = inputs(7, (rows,), C, torch.float32, None)
    gate[::50, ::3] = -float("inf")
    gate[5:9] = 0.0
    gate[100, 1] = float("nan")
    x[400, 2] = float("nan")
    x[20, 4] = float("inf")
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    where = ref.runs(None, cu=cu)
    out, last = dig.glr_fwd_packed(x, gate, dcu, complement=complement)
    w = ref.glr_fwd(flat(x), flat(gate), None, complement, None, where)
    compare((out, last), w[:2], w[2:], ("out", "h_last"), (torch.float32,) * 2)
    assert dig.device_status() == 0


@pytest.mark.parametrize("gate_norm", [1.0, 16.0])
def test_extreme_logits(dig, gate_norm):
    x, gate = inputs(8, (1, 300), 64, torch.bfloat16, gate_norm)
    for k, v in enumerate((float("inf"), -float("inf"), 300.0, -300.0, 88.0, -88.0, 0.0, 20.0)):
        gate[:, k::40] = v
    where = ref.runs((1, 300), order=np.arange(300))
    for comp in (False, True):
        out, last = dig.glr_fwd(x, gate, 1, 300, 0, gate_norm=gate_norm, complement=comp)
        w = ref.glr_fwd(flat(x), flat(gate), gate_norm, comp, None, where)
        compare((out, last), w[:2], w[2:], ("out", "h_last"), (torch.bfloat16, torch.float32))
        dout = normal(9, x.shape, torch.bfloat16)
        got = dig.glr_bwd(x, gate, out, dout, 1, 300, 0, gate_norm=gate_norm, complement=comp)
        want, b = ref.glr_bwd(flat(x), flat(gate), flat(out), flat(dout), gate_norm, comp, None, None, where)
        compare(got, want, b, ("dx", "dgate", "dh0"), (torch.bfloat16, torch.bfloat16, torch.float32))


def test_no_decay_and_slow_decay(dig):
    """alpha = 1 (a running sum) and alpha within 1e-6 of 1."""
    x, gate = inputs(11, (1, 3000), 64, torch.float32, None)
    gate[..., :32] = 0
    gate[..., 32:] = -1e-6
    where = ref.runs((1, 3000), order=np.arange(3000))
    check_fwd(dig, x, gate, None, False, None, lambda **k: dig.glr_fwd(x, gate, 1, 3000, 0, **k), where)
    check_fwd(dig, x, gate, None, True, None, lambda **k: dig.glr_fwd(x, gate, 1, 3000, 0, **k), where)


def test_repeats_bit_for_bit_on_streams_and_in_graphs(dig):
    x, gate = inputs(12, (2, 2500), 200, torch.bfloat16, 16.0)
    h0, dout = normal(13, (2, 200)), normal(14, x.shape, torch.bfloat16)
    cu = torch.tensor([0, 100, 1900, 2500], dtype=torch.int32).cuda()

    def all_of():
        a = dig.glr_fwd(x, gate, 50, 50, 2, gate_norm=16.0, h0=h0)
        b = dig.glr_bwd(x, gate, a[0], dout, 50, 50, 2, gate_norm=16.0, h0=h0, dh_last=h0)
        c = dig.glr_fwd_packed(x[0], gate[0], cu, gate_norm=16.0, complement=True)
        return (*a, *b, *c)

    want = all_of()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(all_of(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = all_of()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(again, want))
    out = torch.empty_like(x)
    side.wait_stream(torch.cuda.current_stream())
    dig.glr_fwd(x, gate, 50, 50, 2, gate_norm=16.0, h0=h0, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = all_of()
        graphs.append((g, got))
    for g, _ in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_guards_around_the_outputs(dig):
    """Nothing is written outside the outputs: odd sizes inside poisoned buffers."""
    for B, T, C in ((1, 77, 72), (2, 513, 8), (3, 5, 200)):
        x, gate = inputs(15, (B, T), C, torch.bfloat16, None)
        n = B * T * C
        raw = torch.full((n + 2048,), -3.0, dtype=torch.bfloat16, device="cuda")
        last = torch.full((B * C + 2048,), -3.0, device="cuda")
        out = raw[1024:1024 + n].view(B, T, C)
        dig.glr_fwd(x, gate, 1, T, 0, out=out, h_last=last[1024:1024 + B * C].view(B, C))
        raw2, raw3 = torch.full_like(raw, -3.0), torch.full((n + 2048,), -3.0, device="cuda")
        last2 = torch.full_like(last, -3.0)
        dig.glr_bwd(x, gate, out, x, 1, T, 0, dx=raw2[1024:1024 + n].view(B, T, C), dgate=raw3[1024:1024 + n].view(B, T, C),
                    dh0=last2[1024:1024 + B * C].view(B, C))
        for t, m in ((raw, n), (raw2, n), (raw3, n), (last, B * C), (last2, B * C)):
            assert bool((t[:1024] == -3).all()) and bool((t[1024 + m:] == -3).all())


def test_bad_sequence_lengths_are_reported(dig):
    """Descending lengths, or lengths beyond the rows: the device status says so, and nothing is
    read or written out of range (addresses never depend on the lengths)."""
    x, gate = inputs(16, (100,), 64, torch.float32, None)
    for cu in ([0, 60, 40, 100], [0, 50, 101], [-4, 50, 100], [2 ** 30, -2 ** 30, 5]):
        dcu = torch.tensor(cu, dtype=torch.int32).cuda()
        out, _ = dig.glr_fwd_packed(x, gate, dcu)
        assert dig.device_status() == -1, cu
        dig.glr_bwd_packed(x, gate, out, x, dcu)
        assert dig.device_status() == -1, cu
    dig.glr_fwd_packed(x, gate, torch.tensor([0, 100], dtype=torch.int32).cuda())
    assert dig.device_status() == 0


def test_growth_beyond_fp32_is_reported(dig):
    x, gate = inputs(17, (1, 64), 64, torch.float32, None)
    dig.glr_fwd(x, gate * 0 + 0.01, 1, 64, 0)
    assert dig.device_status() == 0
    dig.glr_fwd(x, gate * 0 + 100.0, 1, 64, 0)
    assert dig.device_status() == -7
    dig.glr_bwd(x, gate * 0 + 100.0, x, x, 1, 64, 0)
    assert dig.device_status() == -7


def test_offsets_beyond_32_bits(dig):
    """2.2e9 elements: the last tokens against the definition, restarted behind a reset."""
    T, C = 1_100_000, 2048
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    gate = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").fill_(1.5)
    k = T - 300
    gate[:, k] = -float("inf")
    out, last = dig.glr_fwd(x, gate, 1, T, 0, gate_norm=16.0)
    tx, tg = x[0, k:], gate[0, k:]
    where = [(0, np.arange(300))]
    w = ref.glr_fwd(np64(tx), np64(tg), 16.0, False, None, where)
    compare((out[0, k:], last), w[:2], w[2:], ("out", "h_last"), (torch.bfloat16, torch.float32))
    dx, dg, _ = dig.glr_bwd(x, gate, out, x, 1, T, 0, gate_norm=16.0)
    want, b = ref.glr_bwd(np64(tx), np64(tg), np64(out[0, k:]), np64(tx), 16.0, False, np64(out[0, k - 1:k]), None, where)
    compare((dx[0, k:], dg[0, k:]), want[:2], b[:2], ("dx", "dgate"), (torch.bfloat16,) * 2)


# ---- one token ---------------------------------------------------------------------------


def step_reference(x, gate, state, slots, gate_norm, complement):
    _, alpha, rest, _ = ref.gates(np64(gate), gate_norm)
    la = ref.gates(np64(gate), gate_norm)[0]
    xs, after = np64(x), np64(state).copy()
    out, bound, b_after = np.zeros_like(xs), np.zeros_like(xs), np.zeros_like(after)
    for i, s in enumerate(slots):
        if s < 0 or s >= len(after):
            continue
        u = rest[i] * xs[i] if complement else xs[i]
        mag = np.abs(alpha[i] * after[s]) + np.abs(u)
        b_after[s] = alpha[i] * b_after[s] + (ref.gate_error(la[i]) + 4 * ref.U) * mag
        after[s] = alpha[i] * after[s] + u
        out[i], bound[i] = after[s], b_after[s]
    return out, after, bound, b_after


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate_norm", [None, 1.0, 16.0])
@pytest.mark.parametrize("N,nslots,C", [(1, 1, 8), (3, 7, 72), (40, 100, 1152), (257, 300, 520), (5, 5, 8200)])
def test_step(dig, dtype, gate_norm, N, nslots, C):
    dt = DT[dtype]
    complement = C % 16 == 0
    x, gate = inputs(20, (N,), C, dt, gate_norm, fused=N == 40)
    state = normal(22, (nslots, C))
    slots = torch.randperm(nslots, generator=torch.Generator().manual_seed(1))[:N].to(torch.int32)
    if N > 2:
        slots[1] = -1
    w = step_reference(x, gate, state, slots.tolist(), gate_norm, complement)
    apart = torch.full_like(state, 9.0)
    out, after = dig.glr_step(x, gate, state, slots.cuda(), gate_norm, complement, state_out=apart)
    named = sorted(s for s in slots.tolist() if s >= 0)
    compare((out, after[named]), (w[0], w[1][named]), (w[2], w[3][named]), ("out", "state"), (dt, torch.float32))
    rest = [s for s in range(nslots) if s not in named]
    assert bool((apart[rest] == 9).all())
    before = state.clone()
    out2, same = dig.glr_step(x, gate, state, slots.cuda(), gate_norm, complement)
    assert same.data_ptr() == state.data_ptr() and torch.equal(out2, out) and torch.equal(state[named], apart[named])
    assert torch.equal(state[rest], before[rest])
    assert dig.device_status() == 0


def test_step_rows_without_slots_and_padding(dig):
    x, gate = inputs(23, (6,), 64, torch.float32, None)
    state = normal(24, (9, 64))
    w = step_reference(x, gate, state, range(6), None, False)
    out, after = dig.glr_step(x, gate, state.clone())
    compare((out, after), w[:2], w[2:], ("out", "state"), (torch.float32,) * 2)
    given = torch.full_like(x, 5.0)
    slots = torch.tensor([2, -1, 9, 0, -7, 4], dtype=torch.int32).cuda()   # 9 is out of range
    after = state.clone()
    dig.glr_step(x, gate, after, slots, out=given)
    assert dig.device_status() == -1
    assert bool((given[[1, 2, 4]] == 5).all()) and torch.equal(after[[1, 3, 5, 6, 7, 8]], state[[1, 3, 5, 6, 7, 8]])
    out, _ = dig.glr_step(x, gate, state.clone(), torch.full((6,), -1, dtype=torch.int32).cuda())
    assert bool((out == 0).all()) and dig.device_status() == 0


@pytest.mark.parametrize("N", [2, 33, 300, 1500])
def test_step_rows_of_one_slot_are_successive_tokens(dig, N):
    x, gate = inputs(25, (N,), 136, torch.float32, None)
    state = normal(26, (N // 2 + 1, 136))
    slots = torch.randint(-1, N // 2 + 1, (N,), generator=torch.Generator().manual_seed(N)).to(torch.int32)
    slots[0] = slots[-1] = 1
    w = step_reference(x, gate, state, slots.tolist(), None, True)
    after = state.clone()
    out, _ = dig.glr_step(x, gate, after, slots.cuda(), complement=True)
    compare((out, after), w[:2], w[2:], ("out", "state"), (torch.float32,) * 2)


def test_prompts_then_tokens_equal_the_whole(dig):
    """Packed prompts, their states placed in a pool, then single tokens: the outputs of the whole
    sequences, within twice the bounds of either."""
    lens, more, C = [37, 0, 130, 1], 6, 72
    total = [n + more for n in lens]
    cu_all = np.concatenate([[0], np.cumsum(total)])
    x, gate = inputs(27, (int(cu_all[-1]),), C, torch.float32, 16.0)
    w = ref.glr_fwd(np64(x), np64(gate), 16.0, True, None, ref.runs(None, cu=cu_all))
    at = [np.arange(cu_all[i], cu_all[i] + n) for i, n in enumerate(lens)]
    rows = torch.tensor(np.concatenate(at)).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    out, last = dig.glr_fwd_packed(x[rows].contiguous(), gate[rows].contiguous(), cu, gate_norm=16.0, complement=True)
    r = rows.cpu().numpy()
    ref.check(np64(out), w[0][r], w[2][r], "prompt")
    slots = torch.tensor([5, 2, 0, 3], dtype=torch.int32).cuda()
    pool = torch.zeros(6, C, device="cuda")
    pool[slots.long()] = last
    for t in range(more):
        here = torch.tensor([int(cu_all[i]) + lens[i] + t for i in range(4)]).cuda()
        got, _ = dig.glr_step(x[here].contiguous(), gate[here].contiguous(), pool, slots, gate_norm=16.0, complement=True)
        h = here.cpu().numpy()
        ref.check(np64(got), w[0][h], 2 * w[2][h], f"token {t}")


@pytest.mark.parametrize("d", [0, 1])
def test_padding_may_hold_anything(dig, d):
    """NaN and infinities in rows of no sequence, before the first and behind the last, change nothing."""
    rows, C, cu = 900, 72, [70, 71, 400, 401, 830]
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    for gate_norm, comp in ((None, False), (16.0, True)):
        x, gate = inputs(30, (rows,), C, torch.float32, gate_norm)
        h0, dout, dlast = normal(31, (4, C)), normal(32, (rows, C)), normal(33, (4, C))
        out, last = dig.glr_fwd_packed(x, gate, dcu, d, gate_norm, comp, h0=h0)
        grads = dig.glr_bwd_packed(x, gate, out, dout, dcu, d, gate_norm, comp, h0=h0, dh_last=dlast)
        junk = [t.clone() for t in (x, gate, out, dout)]
        for t, v in zip(junk, (float("nan"), float("inf"), float("nan"), -float("inf"))):
            t[:70], t[830:] = v, v
        junk[1][40:60] = float("nan")
        again = dig.glr_fwd_packed(junk[0], junk[1], dcu, d, gate_norm, comp, h0=h0)
        more = dig.glr_bwd_packed(*junk, dcu, d, gate_norm, comp, h0=h0, dh_last=dlast)
        for p, q in zip((out, last, *grads), (*again, *more)):
            assert torch.allclose(p, q, rtol=1e-5, atol=1e-6) and not bool(torch.isnan(q).any())
    dig.device_status()   # infinite log gates in the padding count as growth


@pytest.mark.parametrize("reverse", [0, 1])
def test_a_nan_ends_with_its_sequence(dig, reverse):
    """Whatever the cut: a NaN at any place of a sequence leaves its neighbours as they were."""
    rows, C = 600, 64
    cu = [0, 3, 130, 131, 260, 264, 600]
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    x, gate = inputs(34, (rows,), C, torch.float32, 1.0)
    dout = normal(35, (rows, C))
    out, last = dig.glr_fwd_packed(x, gate, dcu, reverse, 1.0)
    dx, dg, dh0 = dig.glr_bwd_packed(x, gate, out, dout, dcu, reverse, 1.0)
    for n, at in ((0, 1), (1, 3), (1, 129), (2, 130), (3, 200), (4, 263)):
        bad = x.clone()
        bad[at] = float("nan")
        o, l = dig.glr_fwd_packed(bad, gate, dcu, reverse, 1.0)
        keep = torch.ones(rows, dtype=torch.bool)
        keep[cu[n]:cu[n + 1]] = False
        keep = keep.cuda()
        assert torch.allclose(o[keep], out[keep], rtol=1e-5, atol=1e-6), (n, at)
        assert bool(torch.isnan(o[at]).all()) and bool(torch.isnan(l[n]).all())
        others = [k for k in range(6) if k != n]
        assert torch.allclose(l[others], last[others], rtol=1e-5, atol=1e-6)
        bad = dout.clone()
        bad[at] = float("nan")
        px, pg, p0 = dig.glr_bwd_packed(x, gate, out, bad, dcu, reverse, 1.0)
        assert torch.allclose(px[keep], dx[keep], rtol=1e-5, atol=1e-6) and torch.allclose(pg[keep], dg[keep], rtol=1e-5, atol=1e-6)
        assert torch.allclose(p0[others], dh0[others], rtol=1e-5, atol=1e-6) and bool(torch.isnan(p0[n]).all())
    assert dig.device_status() == 0


@pytest.mark.parametrize("value", [3e37, float("inf"), 1e25])
def test_an_overflow_ends_with_its_sequence(dig, value):
    """Values that overflow inside one sequence leave the others as they were."""
    rows, C = 700, 64
    cu = [0, 90, 333, 350, 700]
    dcu = torch.tensor(cu, dtype=torch.int32).cuda()
    x, gate = inputs(36, (rows,), C, torch.float32, None)
    out, last = dig.glr_fwd_packed(x, gate, dcu)
    bad = x.clone()
    bad[90:333] = value
    o, l = dig.glr_fwd_packed(bad, gate, dcu)
    dx, dg, dh0 = dig.glr_bwd_packed(x, gate, out, x, dcu)
    px, pg, p0 = dig.glr_bwd_packed(x, gate, out, bad, dcu)
    for s in (slice(0, 90), slice(333, 700)):
        for p, q in ((o, out), (px, dx), (pg, dg)):
            assert torch.allclose(p[s], q[s], rtol=1e-5, atol=1e-6)
    assert torch.allclose(l[[0, 2, 3]], last[[0, 2, 3]], rtol=1e-5, atol=1e-6)
    assert torch.allclose(p0[[0, 2, 3]], dh0[[0, 2, 3]], rtol=1e-5, atol=1e-6)


def test_after_release(dig):
    """dig_gla_release forgets what was set up; wide clusters and the workspace come back."""
    x, gate = inputs(37, (1, 9000), 64, torch.bfloat16, 16.0)
    want = dig.glr_fwd(x, gate, 1, 9000, 0, gate_norm=16.0)
    torch.cuda.synchronize()
    dig.lib().dig_gla_release()
    got = dig.glr_fwd(x, gate, 1, 9000, 0, gate_norm=16.0)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and dig.device_status() == 0


def test_two_calls_at_once(dig):
    """Long and short calls on two streams at the same time, each with its own results."""
    xs = [inputs(40 + i, (1, T), 512, torch.bfloat16, 16.0) for i, T in enumerate((20000, 700))]
    want = [dig.glr_fwd(x, g, 1, x.shape[1], 0, gate_norm=16.0) for x, g in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (x, g) in enumerate(xs):
            with torch.cuda.stream(streams[i]):
                got[i].append(dig.glr_fwd(x, g, 1, x.shape[1], 0, gate_norm=16.0))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_first_call_of_a_process_inside_a_capture():
    """Nothing a first call sets up needs an eager call before."""
    import subprocess
    import sys
    code = """
import torch, gated_linear_attention_chunkwise_b200 as dig
x, g = torch.randn(1, 3000, 256, device="cuda"), -torch.rand(1, 3000, 256, device="cuda")
q, w, inv = torch.randn(40, 4, 64, device="cuda"), torch.ones(64, device="cuda"), dig.rope_frequencies(64, device="cuda")[0]
s = torch.zeros(3, 256, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    o, l = dig.glr_fwd(x, g, 1, 3000, 0)
    d = dig.glr_bwd(x, g, o, x, 1, 3000, 0)
    n = dig.qk_norm_rope(q, None, w, None, None, inv)
    b = dig.qk_norm_rope_bwd(n[0], None, q, None, w, None, None, inv)
    t = dig.glr_step(x[0, :3], g[0, :3], s, state_out=torch.empty_like(s))
graph.replay(); graph.replay()
got = [v.clone() for v in (o, l, *d, n[0], b[0], b[2], *t)]
o, l = dig.glr_fwd(x, g, 1, 3000, 0)
n = dig.qk_norm_rope(q, None, w, None, None, inv)
b = dig.qk_norm_rope_bwd(n[0], None, q, None, w, None, None, inv)
want = (o, l, *dig.glr_bwd(x, g, o, x, 1, 3000, 0), n[0], b[0], b[2], *dig.glr_step(x[0, :3], g[0, :3], s, state_out=torch.empty_like(s)))
assert all(torch.equal(p, q) for p, q in zip(got, want))
print("same")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
