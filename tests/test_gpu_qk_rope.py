"""GPU parity of rope, qk_norm_rope and qk_norm_rope_bwd against the 64-bit forms of
seq_reference.py, element by element within a-priori bounds; and a run of the operators
together with the GLA forward and backward."""
import numpy as np
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dig():
    import gated_linear_attention_chunkwise_b200 as pkg
    return pkg


def np64(t):
    return t.detach().double().cpu().numpy()


def normal(seed, shape, dtype=torch.float32, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) + mean).to(dtype).cuda()


def heads(seed, rows, Hq, Hk, D, dtype, fused):
    if fused:
        qkv = normal(seed, (rows, (Hq + 2 * Hk) * D + 16), dtype)
        q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        return q, qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)) if Hk else None
    return normal(seed, (rows, Hq, D), dtype), normal(seed + 1, (rows, Hk, D), dtype) if Hk else None


def case(dig, rows, Hq, Hk, D, rot, dtype, interleaved, scale=1.0, fused=False, far=5000, p32=False, seed=0):
    dt = DT[dtype]
    bf = dt == torch.bfloat16
    q, k = heads(seed, rows, Hq, Hk, D, dt, fused)
    pos = torch.randint(-far, far, (rows,), generator=torch.Generator().manual_seed(seed)).to(
        torch.int32 if p32 else torch.int64).cuda()
    inv = dig.rope_frequencies(rot, device="cuda")[0] if rot else None
    wq, wk = normal(seed + 2, (D,), mean=1.0), normal(seed + 3, (D,), mean=1.0) if Hk else None
    how = dict(interleaved=interleaved, scale=scale)
    P, F = np64(pos), None if inv is None else np64(inv)
    pairs = [("q", q, wq)] + ([("k", k, wk)] if Hk else [])
    if rot:
        for inverse in (False, True):
            got = dig.rope(q, k, pos, inv, inverse=inverse, **how)
            assert len(got) == 2 and (got[1] is None) == (not Hk)
            for (name, t, _), g in zip(pairs, got):
                want, mag = ref.rotate(np64(t), P, F, interleaved, scale, inverse)
                ref.check(np64(g), want, mag * ref.TURN, f"rope {name} inverse={inverse}", bf)
                if D > rot:
                    assert torch.equal(g[..., rot:], t[..., rot:])
    got = dig.qk_norm_rope(q, k, wq, wk, pos, inv, eps=1e-5, **how)
    for (name, t, w), g in zip(pairs, got):
        ref.check(np64(g), *ref.norm_rope(np64(t), np64(w), P, F, 1e-5, interleaved, scale), f"norm {name}", bf)
    dq, dk = heads(seed + 7, rows, Hq, Hk, D, dt, fused)
    got = dig.qk_norm_rope_bwd(dq, dk, q, k, wq, wk, pos, inv, eps=1e-5, **how)
    for i, ((name, t, w), d) in enumerate(zip(pairs, (dq, dk))):
        want, bounds = ref.norm_rope_bwd(np64(d), np64(t), np64(w), P, F, 1e-5, interleaved, scale)
        ref.check(np64(got[i]), want[0], bounds[0], f"d{name}", bf)
        ref.check(np64(got[2 + i]), want[1], bounds[1], f"d{name}_weight")
    if not Hk:
        assert got[1] is None and got[3] is None
    assert dig.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(8, 8), (16, 8), (32, 32), (40, 24), (64, 64), (64, 32), (72, 72), (80, 40), (88, 88),
                                   (96, 96), (128, 128), (128, 64), (136, 8), (160, 160), (192, 128), (200, 200),
                                   (256, 256), (256, 64), (64, 0), (72, 0), (248, 240)])
def test_heads(dig, dtype, interleaved, D, rot):
    case(dig, 13, 4, 2, D, rot, dtype, interleaved, fused=rot % 16 == 0, p32=D % 16 == 0, seed=D + rot)


@pytest.mark.parametrize("rows,Hq,Hk", [(1, 1, 0), (1, 32, 8), (2, 5, 1), (37, 3, 3), (300, 16, 2), (1000, 6, 0), (4099, 1, 1),
                                        (17, 64, 64), (3, 1, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_and_heads(dig, rows, Hq, Hk, dtype):
    case(dig, rows, Hq, Hk, 64, 64, dtype, rows % 2 == 0, scale=1.1, seed=rows)
    case(dig, rows, Hq, Hk, 72, 48, dtype, rows % 2 == 1, scale=0.9, fused=True, seed=rows + 1)


def test_positions_left_out_are_the_rows_of_a_batch(dig):
    q, k = normal(1, (3, 7, 2, 32)), normal(2, (3, 7, 1, 32))
    inv, _ = dig.rope_frequencies(32, device="cuda")
    pos = torch.arange(7).repeat(3, 1).cuda()
    for a, b in zip(dig.rope(q, k, None, inv), dig.rope(q, k, pos, inv)):
        assert torch.equal(a, b) and a.shape[:2] == (3, 7)
    for a, b in zip(dig.rope(q[0], k[0], None, inv), dig.rope(q[0], k[0], pos[0], inv)):
        assert torch.equal(a, b)


def test_far_positions_keep_their_phase(dig):
    """Positions up to 2^40 and of both signs: cos and sin of the exact product."""
    q = torch.ones(8, 1, 64, device="cuda")
    pos = torch.tensor([0, 1, -1, 10 ** 6, -10 ** 6 - 1, 2 ** 31, 2 ** 40 + 12345, -2 ** 40], dtype=torch.int64).cuda()
    inv, _ = dig.rope_frequencies(64, device="cuda")
    got, _ = dig.rope(q, None, pos, inv)
    # the exact product modulo a turn, in integers: inv is m 2^e with a 24-bit m
    from fractions import Fraction
    import math
    turn = Fraction(math.pi) + Fraction(1.2246467991473532e-16)     # pi to 106 bits
    want = np.zeros((8, 1, 64))
    for r, p in enumerate(pos.tolist()):
        for i, f in enumerate(inv.cpu().numpy()):
            a = Fraction(p) * Fraction(float(f))
            a = float(a - 2 * turn * round(a / (2 * turn)))
            want[r, 0, i], want[r, 0, i + 32] = math.cos(a) - math.sin(a), math.cos(a) + math.sin(a)
    # fp64 carries the turns to 2^-53 of them: 2^40 / 2 pi turns leave 2^-15 of a turn there, the others 2^-24
    bound = np.full(want.shape, 2 * ref.TURN)
    bound[6:] += 2 * 2 * math.pi * 2.0 ** 38 * 2.0 ** -53 * 2
    ref.check(np64(got), want, bound, "far")


def test_in_place_and_strided_outputs(dig):
    for D, inter in ((128, False), (72, True), (40, False)):
        Hq, Hk, rows = 4, 2, 21
        qkv = normal(3, (rows, (Hq + 2 * Hk) * D), torch.bfloat16)
        was = qkv.clone()
        q, k = qkv[:, :Hq * D].unflatten(1, (Hq, D)), qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        inv, _ = dig.rope_frequencies(D - 8, device="cuda")
        w = normal(4, (D,), mean=1.0)
        pos = torch.arange(rows).cuda()
        want = dig.qk_norm_rope(q, k, w, w, pos, inv, interleaved=inter)
        back = dig.qk_norm_rope_bwd(*want, q, k, w, w, pos, inv, interleaved=inter)
        dig.qk_norm_rope(q, k, w, w, pos, inv, interleaved=inter, q_out=q, k_out=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(qkv[:, (Hq + Hk) * D:], was[:, (Hq + Hk) * D:])       # the values beside them
        orig = was[:, :Hq * D].unflatten(1, (Hq, D)), was[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        dig.qk_norm_rope_bwd(q, k, *orig, w, w, pos, inv, interleaved=inter, dq=q, dk=k)   # over the gradients
        assert torch.equal(q, back[0]) and torch.equal(k, back[1])
        turned = dig.rope(*orig, pos, inv, interleaved=inter)
        a = torch.full((rows, 2, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
        dig.rope(orig[0], None, pos, inv, interleaved=inter, q_out=a[:, 0])
        assert torch.equal(a[:, 0], turned[0]) and bool((a[:, 1] == 5).all())


def test_extreme_heads(dig):
    """Zeros give zeros (eps carries the norm), huge and tiny heads stay finite, a NaN stays in its head."""
    q = normal(5, (6, 3, 64))
    q[0] = 0
    q[1] *= 1e15
    q[2] *= 1e-15
    q[3, 1, 5] = float("nan")
    w = torch.ones(64, device="cuda")
    inv, _ = dig.rope_frequencies(64, device="cuda")
    pos = torch.arange(6).cuda()
    got, _ = dig.qk_norm_rope(q, None, w, None, pos, inv, eps=1e-6)
    want, b = ref.norm_rope(np64(q), np64(w), np64(pos), np64(inv), 1e-6, False, 1.0)
    ref.check(np64(got), np.where(np.isnan(want), np.nan, want), np.nan_to_num(b), "extreme")
    assert bool((got[0] == 0).all()) and bool(torch.isnan(got[3, 1]).all()) and not bool(torch.isnan(got[3, [0, 2]]).any())
    dq, _, dw, _ = dig.qk_norm_rope_bwd(q * 0 + 1, None, q, None, w, None, pos, inv, eps=1e-6)
    assert not bool(torch.isnan(dq[[0, 1, 2, 4, 5]]).any()) and not bool(torch.isnan(dq[3, [0, 2]]).any())


def test_repeats_streams_and_graphs(dig):
    q, k = heads(6, 700, 8, 2, 72, torch.bfloat16, True)
    dq, dk = heads(7, 700, 8, 2, 72, torch.bfloat16, False)
    w = normal(8, (72,), mean=1.0)
    inv, _ = dig.rope_frequencies(72, device="cuda")
    pos = torch.arange(700).cuda()

    def all_of():
        return (*dig.rope(q, k, pos, inv), *dig.qk_norm_rope(q, k, w, w, pos, inv),
                *dig.qk_norm_rope_bwd(dq, dk, q, k, w, w, pos, inv))

    want = all_of()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(all_of(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = all_of()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    side.wait_stream(torch.cuda.current_stream())
    given = [dig.qk_norm_rope_bwd(dq, dk, q, k, w, w, pos, inv, stream=side) for _ in range(3)]
    side.synchronize()
    for got in given:
        assert all(torch.equal(a, b) for a, b in zip(got, want[4:]))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = all_of()
        graphs.append((g, got))
    for g, _ in graphs * 2:
        g.replay()
    # the two graphs at once, each on a stream of its own
    other = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_beyond_32_bits(dig):
    """2.15e9 elements of queries: the last rows."""
    rows, H, D = 131_100, 128, 128
    q = torch.empty(rows, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    inv, _ = dig.rope_frequencies(128, device="cuda")
    w = normal(9, (128,), mean=1.0)
    pos = torch.arange(rows).cuda()
    got, _ = dig.qk_norm_rope(q, None, w, None, pos, inv)
    t = slice(rows - 5, rows)
    ref.check(np64(got[t]), *ref.norm_rope(np64(q[t]), np64(w), np64(pos[t]), np64(inv), 1e-6, False, 1.0), "tail", True)
    dq, *_ = dig.qk_norm_rope_bwd(got, None, q, None, w, None, pos, inv)
    want, b = ref.norm_rope_bwd(np64(got[t]), np64(q[t]), np64(w), np64(pos[t]), np64(inv), 1e-6, False, 1.0)
    ref.check(np64(dq[t]), want[0], b[0], "tail gradient", True)


def test_a_layer_of_them_together(dig):
    """The token mixer of one layer and its gradient: norm and rotation of q and k, the GLA
    over them, a gated recurrence over its output; backwards through all three, each gradient
    against the same chain in fp64 (torch autograd), at the GLA path's bf16 gates: relative
    RMS 2e-2 per tensor."""
    B, T, H, d = 2, 70, 2, 64
    torch.manual_seed(0)
    q, k, v, x = (torch.randn(B, T, H, d).bfloat16() for _ in range(4))
    la, gate = -torch.rand(B, T, H, d) / 8, torch.randn(B, T, H * d).bfloat16()
    wq, wk = 1 + torch.randn(d) / 5, (1 + torch.randn(d) / 5) / 8
    dy = torch.randn(B, T, H * d).bfloat16()
    inv, _ = dig.rope_frequencies(d)
    dev = [t.cuda() for t in (q, k, v, la, gate, wq, wk, dy, inv)]
    Q, K, V, LA, G, WQ, WK, DY, INV = dev
    qn, kn = dig.qk_norm_rope(Q, K, WQ, WK, None, INV)
    o = dig.gla_fwd(qn, kn, V, LA, 1, T, 0)
    y, _ = dig.glr_fwd(o.view(B, T, H * d), G, 1, T, 0, gate_norm=1.0, complement=True)
    do, dG, _ = dig.glr_bwd(o.view(B, T, H * d), G, y, DY, 1, T, 0, gate_norm=1.0, complement=True)
    dqn, dkn, dV, dLA = dig.gla_bwd(qn, kn, V, LA, do.view(B, T, H, d), 1, T, 0)
    dQ, dK, dWQ, dWK = dig.qk_norm_rope_bwd(dqn, dkn, Q, K, WQ, WK, None, INV)
    got = dict(y=y, q=dQ, k=dK, v=dV, la=dLA, gate=dG, wq=dWQ, wk=dWK)

    leaf = {n: t.double().requires_grad_() for n, t in dict(q=q, k=k, v=v, la=la, gate=gate, wq=wq, wk=wk).items()}
    ang = torch.arange(T).double()[:, None] * inv.double()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

    def turn(t, w):
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    qs, ks = turn(leaf["q"], leaf["wq"]), turn(leaf["k"], leaf["wk"])
    S, outs = torch.zeros(B, H, d, d, dtype=torch.float64), []
    for t in range(T):
        S = leaf["la"][:, t].exp()[..., None] * S + ks[:, t, :, :, None] * leaf["v"][:, t, :, None]
        outs.append((qs[:, t, :, None] @ S)[:, :, 0])
    oo = torch.stack(outs, 1).reshape(B, T, H * d)
    h, ys = torch.zeros(B, H * d, dtype=torch.float64), []
    for t in range(T):
        a = torch.sigmoid(leaf["gate"][:, t])
        h = a * h + (1 - a) * oo[:, t]
        ys.append(h)
    yy = torch.stack(ys, 1)
    yy.backward(dy.double())
    want = dict(y=yy.detach(), **{n: t.grad for n, t in leaf.items()})
    for n, t in got.items():
        e = (t.double().cpu().reshape(want[n].shape) - want[n]).norm() / want[n].norm()
        assert e <= 2e-2, (n, float(e))
    assert dig.device_status() == 0
