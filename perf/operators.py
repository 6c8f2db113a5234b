"""The sequence operators of the language-model path, each as a measured case.

    glr_fwd, glr_bwd      gated linear recurrence over a scan order or packed sequences
    glr_step              the same recurrence for one token of every running sequence
    qk_norm_rope(_bwd)    RMS norm of every query and key head, then the rotary position
    rope                  the rotary position alone (inverse: its gradient)

`run` has two forms of every pass.  The plain one is written with elementary torch
operations in 32 bits (angles and positions in 64) and rounds once at the end; the other
makes the calls a user of this package makes.  `exact` is the definition once more, in 64
bits and as a loop over the tokens where the plain form folds pairs of spans.

Recurrence, along the scan order:  h_p = a_p h_{p-1} + s_p x_p,  a = exp(log_alpha), with
log_alpha given in fp32 or as logsigmoid(gate) / gate_norm, and s = 1 or (complement) 1 - a.
"""
import math

import numpy as np
import torch

own = False
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    """The grids are the bench's c4 and the fp32 c1 shape; head counts and widths of the
    others are the usual ones of decoders with shared key heads."""
    return [
        # A recurrent mixer over the 112 x 112 token grid, scanned by columns (one layer, training or sampling).
        dict(name="glr_fwd_c4_columns", op="glr_fwd", B=2, Hg=112, Wg=112, C=1152, dtype="bf16", dir=2, gate_norm=0.0,
             complement=False, h0=False, fused=False),
        # The prompts of a serving batch (or a packed training batch): 41 sequences of very different lengths, gates as
        # logits beside the inputs in one projection, states carried in and out.
        dict(name="glr_fwd_packed_64k", op="glr_fwd", total=65536, seqs=41, pad=0, C=2048, dtype="bf16", dir=0,
             gate_norm=16.0, complement=True, h0=True, fused=True),
        # The smallest training step: fp32, 16 x 16 tokens, right to left by columns.
        dict(name="glr_bwd_c1_f32", op="glr_bwd", B=2, Hg=16, Wg=16, C=384, dtype="f32", dir=3, gate_norm=0.0,
             complement=False, h0=True, fused=False),
        # Training on a packed batch whose last rows are padding.
        dict(name="glr_bwd_packed_32k", op="glr_bwd", total=32749, seqs=19, pad=13, C=2048, dtype="bf16", dir=0,
             gate_norm=16.0, complement=True, h0=True, fused=True),
        # One token of one sequence: latency.
        dict(name="glr_step_1", op="glr_step", N=1, slots=1, pad=0, C=1152, dtype="bf16", gate_norm=0.0, complement=False),
        # One token of 250 running sequences, in a graph captured for 256 rows, over a pool of 1024 states.
        dict(name="glr_step_256", op="glr_step", N=256, slots=1024, pad=6, C=4096, dtype="bf16", gate_norm=1.0,
             complement=True),
        # One token of 16 sequences, far into their contexts: latency.
        dict(name="qk_norm_rope_decode", op="qk_norm_rope", rows=16, Hq=32, Hk=8, D=128, rot=128, dtype="bf16",
             interleaved=False, fused=True, far=131072, scale=1.0),
        # A prompt batch, queries and keys read from the fused projection; positions up to a million.
        dict(name="qk_norm_rope_prompt", op="qk_norm_rope", rows=16381, Hq=32, Hk=8, D=128, rot=128, dtype="bf16",
             interleaved=False, fused=True, far=1000000, scale=1.0),
        # The training step of the c4 grid's heads (72 channels: half of the pair span is 36).
        dict(name="qk_norm_rope_bwd_c4", op="qk_norm_rope_bwd", rows=25088, Hq=16, Hk=16, D=72, rot=72, dtype="bf16",
             interleaved=False, fused=False, far=12544, scale=1.0),
        # A small fp32 training step, a part of each head rotated, pairs interleaved.
        dict(name="qk_norm_rope_bwd_f32", op="qk_norm_rope_bwd", rows=1000, Hq=6, Hk=2, D=64, rot=32, dtype="f32",
             interleaved=True, fused=False, far=4096, scale=1.1),
        # Rotation alone of a long fp32 sequence, interleaved, half of the head.
        dict(name="rope_f32_interleaved", op="rope", rows=8191, Hq=16, Hk=16, D=80, rot=40, dtype="f32", interleaved=True,
             fused=False, far=65536, scale=1.0, inverse=False),
        # The gradient of a rotation of wide heads, one shared key head.
        dict(name="rope_inverse_d256", op="rope", rows=1237, Hq=8, Hk=1, D=256, rot=64, dtype="bf16", interleaved=False,
             fused=True, far=32768, scale=0.9, inverse=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_bwd", "glr_step", "qk_norm_rope", "qk_norm_rope_bwd", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("glr_fwd", "glr_bwd"):
        C = 8 * _log_int(rng, 4, 512)
        most = 30_000_000 // C  # tokens: at the most 24 bytes an element
        gate_norm = rng.choice([0.0, 1.0, 16.0])
        case = dict(op=op, C=C, dtype=dtype, gate_norm=gate_norm, complement=rng.random() < 0.5, h0=rng.random() < 0.5,
                    fused=gate_norm > 0 and rng.random() < 0.5)
        if rng.random() < 0.5:
            B = _log_int(rng, 1, 8)
            Hg = _log_int(rng, 1, 256)
            Wg = _log_int(rng, 1, max(1, min(65536, most // B) // Hg))
            case.update(B=B, Hg=Hg, Wg=Wg, dir=rng.randrange(4))
        else:
            total = _log_int(rng, 1, min(65536, most))
            case.update(total=total, seqs=_log_int(rng, 1, 300), pad=rng.choice([0, 0, min(total - 1, rng.randrange(70))]),
                        dir=rng.randrange(2))
        return case
    if op == "glr_step":
        N = _log_int(rng, 1, 512)
        return dict(op=op, N=N, slots=N + rng.randrange(600), pad=rng.choice([0, rng.randrange(N)]), C=8 * _log_int(rng, 4, 1024),
                    dtype=dtype, gate_norm=rng.choice([0.0, 1.0, 16.0]), complement=rng.random() < 0.5)
    D = 8 * _log_int(rng, 4, 32)
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 8])
    rot = D if rng.random() < 0.5 else 8 * rng.randrange(1, D // 8 + 1)
    rows = _log_int(rng, 1, min(16384, 60_000_000 // ((Hq + Hk) * D)))
    case = dict(op=op, rows=rows, Hq=Hq, Hk=Hk, D=D, rot=rot, dtype=dtype, interleaved=rng.random() < 0.5,
                fused=rng.random() < 0.5, far=_log_int(rng, 64, 1000000), scale=rng.choice([1.0, 1.1]))
    if op == "rope":
        case["inverse"] = rng.random() < 0.5
    return case


# ---- inputs --------------------------------------------------------------------------


def _lengths(case, seed):
    """Cumulative lengths: wide-spread, with sequences of no token and of one among them."""
    r = np.random.RandomState(seed % (1 << 32))
    tokens, n = case["total"] - case["pad"], case["seqs"]
    w = np.exp(1.5 * r.randn(n))
    w[r.rand(n) < 0.1] = 0.0
    w[r.randint(n)] += 1.0
    cu = np.floor(np.concatenate([[0.0], np.cumsum(w) / np.sum(w)]) * tokens).astype(np.int32)
    cu[-1] = tokens
    if n >= 3 and tokens >= 3:
        cu[1] = min(int(cu[2]), 1)
    return cu


def _normal(gen, shape, dtype, mean=0.0, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * std + mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(int(seed))
    dtype, op = TYPES[case["dtype"]], case["op"]
    s = dict(case=case)
    if op in ("glr_fwd", "glr_bwd"):
        packed = "total" in case
        lead = (case["total"],) if packed else (case["B"], case["Hg"] * case["Wg"])
        C, n = case["C"], case["seqs"] if packed else case["B"]
        if case["fused"]:  # both are halves of one projection's rows
            both = _normal(gen, lead + (2 * C,), dtype)
            s["x"], s["gate"] = both[..., :C], both[..., C:]
        else:
            s["x"] = _normal(gen, lead + (C,), dtype)
            g = _normal(gen, lead + (C,), dtype)
            s["gate"] = g if case["gate_norm"] else _log_sigmoid(g.float()) / 16
        s["cu"] = torch.from_numpy(_lengths(case, int(seed))).to(DEVICE) if packed else None
        s["h0"] = _normal(gen, (n, C), torch.float32) if case["h0"] else None
        if op == "glr_bwd":
            s["h"] = _plain_glr_fwd(s)[0]
            s["dout"] = _normal(gen, lead + (C,), dtype)
            s["dlast"] = _normal(gen, (n, C), torch.float32) if case["h0"] else None
    elif op == "glr_step":
        N, C = case["N"], case["C"]
        s["x"] = _normal(gen, (N, C), dtype)
        g = _normal(gen, (N, C), dtype)
        s["gate"] = g if case["gate_norm"] else _log_sigmoid(g.float()) / 16
        s["state"] = _normal(gen, (case["slots"], C), torch.float32)
        s["after"] = s["state"].clone()  # a server that may take a token back keeps the state before it
        slots = torch.randperm(case["slots"], generator=gen, device=DEVICE)[:N].to(torch.int32)
        slots[N - case["pad"]:] = -1
        s["slots"] = slots
    else:
        rows, Hq, Hk, D = case["rows"], case["Hq"], case["Hk"], case["D"]
        if case["fused"]:  # queries, keys (and values) of one projection
            qkv = _normal(gen, (rows, (Hq + 2 * Hk) * D), dtype)
            s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
            s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
        else:
            s["q"] = _normal(gen, (rows, Hq, D), dtype)
            s["k"] = _normal(gen, (rows, Hk, D), dtype)
        s["positions"] = torch.randint(0, case["far"], (rows,), generator=gen, device=DEVICE)
        pairs = torch.arange(case["rot"] // 2, device=DEVICE, dtype=torch.float64)
        s["inv_freq"] = torch.pow(10000.0, pairs * (-2.0 / case["rot"])).float()
        if op != "rope":
            s["wq"] = _normal(gen, (D,), torch.float32, 1.0, 0.2)
            s["wk"] = _normal(gen, (D,), torch.float32, 1.0, 0.2)
        if op == "qk_norm_rope_bwd":
            s["dq"] = _normal(gen, (rows, Hq, D), dtype)
            s["dk"] = _normal(gen, (rows, Hk, D), dtype)
    return s


# ---- plain forms ---------------------------------------------------------------------


def _log_sigmoid(g):
    return torch.clamp(g, max=0) - torch.log1p(torch.exp(-torch.abs(g)))


def _log_alpha(gate, gate_norm):
    return _log_sigmoid(gate.float()) / gate_norm if gate_norm else gate


def _order(case):
    """Token at each position of the scan order (grids); 0 and 1 only turn a packed batch round."""
    if "total" in case:
        p = torch.arange(case["total"], device=DEVICE)
    else:
        p = torch.arange(case["Hg"] * case["Wg"], device=DEVICE)
        if case["dir"] >= 2:
            p = p % case["Hg"] * case["Wg"] + torch.div(p, case["Hg"], rounding_mode="floor")
    return p.flip(0) if case["dir"] % 2 else p


def _fold(a, x):
    """h_p = a_p h_{p-1} + x_p along dim 1 from h = 0: spans of 1, 2, 4, ... positions folded."""
    span = 1
    while span < x.shape[1]:
        x = torch.cat([x[:, :span], x[:, span:] + a[:, span:] * x[:, :-span]], 1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], 1)
        span *= 2
    return x


def _marks(s):
    """For every position of the scan (batch, position): is its token in a sequence, does it
    begin one, does it end one; and for every sequence that has tokens, its number and the
    (batch, position) where it begins and ends."""
    case = s["case"]
    if s["cu"] is None:
        B, T = s["x"].shape[:2]
        n = torch.arange(B, device=DEVICE)
        return torch.ones(B, T, dtype=torch.bool, device=DEVICE), n, (n, n * 0), (n, n * 0 + T - 1)
    cu, T = s["cu"].long(), case["total"]
    n = torch.nonzero(cu[1:] > cu[:-1]).flatten()
    first, last = cu[:-1][n], cu[1:][n] - 1
    order = _order(case)
    inside = ((order >= cu[0]) & (order < cu[-1]))[None]
    if case["dir"] % 2:
        first, last = T - 1 - last, T - 1 - first
    return inside, n, (n * 0, first), (n * 0, last)


def _scan_view(t, order):
    t = t if t.dim() == 3 else t[None]
    return t[:, order].float()


def _back(t, order, like, dtype):
    out = torch.empty_like(t)
    out[:, order] = t
    return out.reshape(like).to(dtype)


def _plain_glr_fwd(s):
    case, x = s["case"], s["x"]
    order = _order(case)
    inside, n, first, last = _marks(s)
    la = _scan_view(_log_alpha(s["gate"], case["gate_norm"]), order)
    a, u = torch.exp(la), _scan_view(x, order)
    if case["complement"]:
        u = -torch.expm1(la) * u
    if s["h0"] is not None:
        u[first] += a[first] * s["h0"][n]
    a[first] = 0
    h = _fold(a, u)
    h_last = torch.zeros(s["cu"].numel() - 1 if s["cu"] is not None else x.shape[0], case["C"], device=DEVICE)
    if s["h0"] is not None:
        h_last.copy_(s["h0"])  # a sequence of no token keeps its state
    h_last[n] = h[last]
    return _back(torch.where(inside[..., None], h, torch.zeros_like(h)), order, x.shape, x.dtype), h_last


def _plain_glr_bwd(s):
    case, x = s["case"], s["x"]
    order = _order(case)
    inside, n, first, last = _marks(s)
    la = _scan_view(_log_alpha(s["gate"], case["gate_norm"]), order)
    a, u, h = torch.exp(la), _scan_view(x, order), _scan_view(s["h"], order)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    before[first] = s["h0"][n] if s["h0"] is not None else 0
    d = _scan_view(s["dout"], order)
    if s["dlast"] is not None:
        d[last] += s["dlast"][n]
    # delta_p = d_p + a_{p+1} delta_{p+1} inside a sequence
    carry = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    carry[last] = 0
    delta = _fold(carry.flip(1), d.flip(1)).flip(1)
    dh0 = torch.zeros(s["cu"].numel() - 1 if s["cu"] is not None else x.shape[0], case["C"], device=DEVICE)
    if s["dlast"] is not None:
        dh0.copy_(s["dlast"])
    dh0[n] = (a * delta)[first]
    dla = a * delta * ((before - u) if case["complement"] else before)
    dx = -torch.expm1(la) * delta if case["complement"] else delta
    if case["gate_norm"]:
        dla = dla * torch.sigmoid(-_scan_view(s["gate"], order)) / case["gate_norm"]
    zero = torch.zeros_like(delta)
    dx, dla = (torch.where(inside[..., None], t, zero) for t in (dx, dla))
    return _back(dx, order, x.shape, x.dtype), _back(dla, order, x.shape, s["gate"].dtype), dh0


def _plain_glr_step(s):
    case = s["case"]
    on = s["slots"] >= 0
    at = torch.clamp(s["slots"], min=0).long()
    la = _log_alpha(s["gate"], case["gate_norm"])
    u = s["x"].float()
    if case["complement"]:
        u = -torch.expm1(la) * u
    h = torch.exp(la) * s["state"][at] + u
    after = s["after"].clone()
    after[at[on]] = h[on]
    return torch.where(on[:, None], h, torch.zeros_like(h)).to(s["x"].dtype), after


def _angles(s):
    turn = s["positions"].double()[:, None] * s["inv_freq"].double()
    scale = s["case"]["scale"]
    return (torch.cos(turn) * scale).float()[:, None], (torch.sin(turn) * scale).float()[:, None]


def _pairs(case, t):
    rot = case["rot"]
    if case["interleaved"]:
        return t[..., 0:rot:2], t[..., 1:rot:2]
    return t[..., :rot // 2], t[..., rot // 2:rot]


def _rotate(s, t, sign):
    case = s["case"]
    cos, sin = _angles(s)
    sin = sign * sin
    a, b = _pairs(case, t)
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, t[..., case["rot"]:]], -1)


EPS = 1e-6


def _plain_norm_rope(s, t, w):
    t = t.float()
    t = t / torch.sqrt(torch.mean(t * t, -1, keepdim=True) + EPS) * w
    return _rotate(s, t, 1.0)


def _plain_norm_rope_bwd(s, d, t, w):
    d, t32 = _rotate(s, d.float(), -1.0), t.float()
    r = 1 / torch.sqrt(torch.mean(t32 * t32, -1, keepdim=True) + EPS)
    n = t32 * r
    dw = torch.sum(d * n, (0, 1))
    d = d * w
    return (r * (d - n * torch.mean(d * n, -1, keepdim=True))).to(t.dtype), dw


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        return _own_run(s, case, op)
    if op == "glr_fwd":
        return _plain_glr_fwd(s)
    if op == "glr_bwd":
        return _plain_glr_bwd(s)
    if op == "glr_step":
        return _plain_glr_step(s)
    if op == "qk_norm_rope":
        return tuple(_plain_norm_rope(s, t, w).to(t.dtype) for t, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if op == "qk_norm_rope_bwd":
        dq, dwq = _plain_norm_rope_bwd(s, s["dq"], s["q"], s["wq"])
        dk, dwk = _plain_norm_rope_bwd(s, s["dk"], s["k"], s["wk"])
        return dq, dk, dwq, dwk
    sign = -1.0 if case["inverse"] else 1.0
    return tuple(_rotate(s, t.float(), sign).to(t.dtype) for t in (s["q"], s["k"]))


# ---- the package's calls -------------------------------------------------------------


def _own_run(s, case, op):
    import gated_linear_attention_chunkwise_b200 as dig
    if op in ("glr_fwd", "glr_bwd"):
        how = dict(gate_norm=case["gate_norm"] or None, complement=case["complement"], h0=s["h0"])
        if s["cu"] is None:
            where, fwd, bwd = (case["Hg"], case["Wg"], case["dir"]), dig.glr_fwd, dig.glr_bwd
        else:
            where, fwd, bwd = (s["cu"], case["dir"]), dig.glr_fwd_packed, dig.glr_bwd_packed
        if op == "glr_fwd":
            return fwd(s["x"], s["gate"], *where, **how)
        return bwd(s["x"], s["gate"], s["h"], s["dout"], *where, dh_last=s["dlast"], **how)
    if op == "glr_step":
        return dig.glr_step(s["x"], s["gate"], s["state"], s["slots"], gate_norm=case["gate_norm"] or None,
                            complement=case["complement"], state_out=s["after"])
    how = dict(interleaved=case["interleaved"], scale=case["scale"])
    if op == "qk_norm_rope":
        return dig.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], eps=EPS, **how)
    if op == "qk_norm_rope_bwd":
        return dig.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"],
                                    eps=EPS, **how)
    return dig.rope(s["q"], s["k"], s["positions"], s["inv_freq"], inverse=case["inverse"], **how)


# ---- what a pass cannot do without -----------------------------------------------------


def work(case):
    size, op = (2 if case["dtype"] == "bf16" else 4), case["op"]
    if op in ("glr_fwd", "glr_bwd", "glr_step"):
        gate = size if case["gate_norm"] else 4
        C = case["C"]
        if op == "glr_step":
            n = (case["N"] - case["pad"]) * C
            return {"bytes": n * (size + gate + 8) + case["N"] * (C * size + 4), "flops": 3 * n}
        packed = "total" in case
        tokens = case["total"] - case["pad"] if packed else case["B"] * case["Hg"] * case["Wg"]
        seqs = case["seqs"] if packed else case["B"]
        ends = seqs * C * 4 * (2 if case["h0"] else 1)
        n = tokens * C
        filled = case["pad"] * C if packed else 0
        if op == "glr_fwd":
            return {"bytes": n * (2 * size + gate) + filled * size + ends, "flops": 3 * n}
        reads = size * (3 if case["complement"] else 2) + gate  # dout, h (and x), gate
        return {"bytes": n * (reads + size + gate) + filled * (size + gate) + ends + (seqs * C * 4 if case["h0"] else 0),
                "flops": 6 * n}
    n = case["rows"] * (case["Hq"] + case["Hk"]) * case["D"]
    table = case["rows"] * 8 + case["rot"] * 2
    if op == "qk_norm_rope_bwd":
        return {"bytes": 3 * n * size + table + 16 * case["D"], "flops": 14 * n}
    if op == "qk_norm_rope":
        return {"bytes": 2 * n * size + table + 8 * case["D"], "flops": 8 * n}
    part = n * case["rot"] // case["D"]
    return {"bytes": 2 * n * size + table, "flops": 3 * part}


# ---- the definitions in 64 bits --------------------------------------------------------


def _exact_order(case):
    """The scan order as a list of tokens, from the grid laid out and transposed or turned."""
    grid = np.arange(case["total"]).reshape(1, -1) if "total" in case else \
        np.arange(case["Hg"] * case["Wg"]).reshape(case["Hg"], case["Wg"])
    flat = (grid.T if case["dir"] in (2, 3) else grid).reshape(-1)
    return (flat[::-1] if case["dir"] in (1, 3) else flat).tolist()


def _exact_runs(s):
    """[(sequence, its tokens in scan order)]; on grids all batches walk the same tokens at once."""
    case = s["case"]
    if s["cu"] is None:
        return [(None, _exact_order(case))]
    cu = s["cu"].tolist()
    runs = [(i, list(range(cu[i], cu[i + 1]))) for i in range(len(cu) - 1)]
    return [(i, t[::-1]) for i, t in runs] if case["dir"] == 1 else runs


def _exact_glr(s):
    case = s["case"]
    g, x = s["gate"].double(), s["x"].double()
    la = -torch.logaddexp(torch.zeros_like(g), -g) / case["gate_norm"] if case["gate_norm"] else g
    alpha = la.exp()
    gain = -torch.expm1(la) if case["complement"] else torch.ones_like(alpha)
    packed = s["cu"] is not None
    n = case["seqs"] if packed else case["B"]
    at = (lambda v, t: v[t]) if packed else (lambda v, t: v[:, t])
    start = s["h0"].double() if s["h0"] is not None else torch.zeros(n, case["C"], dtype=torch.float64, device=DEVICE)
    if case["op"] == "glr_fwd":
        drive = gain * x
        out, ends = torch.zeros_like(x), start.clone()
        for i, tokens in _exact_runs(s):
            h = start[i] if packed else start
            for t in tokens:
                h = torch.addcmul(at(drive, t), at(alpha, t), h)
                at(out, t).copy_(h)
            if packed:
                ends[i] = h
            else:
                ends = h
        return out, ends
    h, dout = s["h"].double(), s["dout"].double()
    delta, before = torch.zeros_like(x), torch.zeros_like(x)
    r0 = s["dlast"].double() if s["dlast"] is not None else torch.zeros_like(start)
    dh0 = r0.clone()
    for i, tokens in _exact_runs(s):
        r, prev = (r0[i], start[i]) if packed else (r0, start)
        for t in reversed(tokens):
            d = at(dout, t) + r
            at(delta, t).copy_(d)
            r = at(alpha, t) * d
        if packed:
            dh0[i] = r
        else:
            dh0 = r
        if tokens:
            at(before, tokens[0]).copy_(prev)
            here = torch.tensor(tokens, device=DEVICE)
            if packed:
                before[here[1:]] = h[here[:-1]]
            else:
                before[:, here[1:]] = h[:, here[:-1]]
    dx = gain * delta
    dla = alpha * delta * (before - x) if case["complement"] else alpha * delta * before
    return dx, dla / (1 + g.exp()) / case["gate_norm"] if case["gate_norm"] else dla, dh0


def _exact_heads(s, t, w, d=None):
    """One tensor of heads by complex numbers: norm and rotation, or (with d) their gradient."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    first = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    phase = torch.polar(torch.full((case["rows"], 1, half), case["scale"], dtype=torch.float64, device=DEVICE),
                        (s["positions"].double()[:, None] * s["inv_freq"].double()[None])[:, None])

    def turn(v, phase):
        z = torch.complex(v[..., first], v[..., second]) * phase
        v = v.clone()
        v[..., first], v[..., second] = z.real, z.imag
        return v

    t = t.double()
    if w is None:
        return turn(t, phase.conj() if case["inverse"] else phase)
    w = w.double()
    r = torch.rsqrt(t.square().sum(-1, keepdim=True) / case["D"] + EPS)
    if d is None:
        return turn(t * r * w, phase)
    d = turn(d.double(), phase.conj())
    wd = w * d
    return wd * r - t * r ** 3 * (wd * t).sum(-1, keepdim=True) / case["D"], (d * t * r).sum((0, 1))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("glr_fwd", "glr_bwd"):
        return _exact_glr(s)
    if op == "glr_step":
        g = s["gate"].double()
        alpha = (1 / (1 + torch.exp(-g))) ** (1 / case["gate_norm"]) if case["gate_norm"] else g.exp()
        out, after = torch.zeros_like(s["x"], dtype=torch.float64), s["after"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                gain = 1 - alpha[i] if case["complement"] else 1.0
                out[i] = alpha[i] * s["state"][slot].double() + gain * s["x"][i].double()
                after[slot] = out[i]
        return out, after
    if op == "rope":
        return _exact_heads(s, s["q"], None), _exact_heads(s, s["k"], None)
    if op == "qk_norm_rope":
        return _exact_heads(s, s["q"], s["wq"]), _exact_heads(s, s["k"], s["wk"])
    dq, dwq = _exact_heads(s, s["q"], s["wq"], s["dq"])
    dk, dwk = _exact_heads(s, s["k"], s["wk"], s["dk"])
    return dq, dk, dwq, dwk
