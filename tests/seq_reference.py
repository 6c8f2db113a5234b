"""Plain 64-bit forms of the sequence operators (gated linear recurrence, rotary positions,
query/key norm) with a-priori bounds on what fp32 arithmetic may deviate from them.

Bounds.  u = 2^-24 is half a unit in the last place of fp32, relative.  Every quantity below
is a sum of products of computed factors, so its error is at most its sum of absolute
values times the roundings a term passes through:
  - a gate alpha = exp(la): exp itself 4u, its argument (a product, a logarithm and a
    division for logits) at most 10u |la|, and for logits 2^-22 / gate_norm < 4u of absolute
    error in a fast logarithm: GATE = 16u + 16u |la| bounds them all, and 1 - alpha too;
  - one step of the recurrence multiplies and adds: 2u more; spans may be folded in any
    order, so a term passes each gate once and at most 32 further additions.
Rounding a result to bf16 adds at most 2^-8 of it.
"""
import numpy as np

U = 2.0 ** -24
EPS16 = 2.0 ** -8


def scan_order(Hg, Wg, d):
    """Token at each scan position, from the grid written out (codes 0..11)."""
    grid = np.arange(Hg * Wg).reshape(Hg, Wg)
    if d < 4:
        flat = (grid.T if d >= 2 else grid).reshape(-1)
        return flat[::-1] if d % 2 else flat
    j = d - 4
    lines = [list(r) for r in (grid.T if j >= 4 else grid)]
    if j & 2:
        lines = lines[::-1]
    out = []
    for i, line in enumerate(lines):
        out += line[::-1] if (i + j) % 2 else line
    return np.array(out)


def gates(gate, gate_norm):
    """(log_alpha, alpha, 1 - alpha, d log_alpha / d gate) in 64 bits."""
    g = np.asarray(gate, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if gate_norm is None:
            la, slope = g, np.ones_like(g)
        else:
            la = np.where(g < 0, g, 0.0) - np.log1p(np.exp(-np.abs(g)))
            la = np.where(np.isnan(g), g, la) / gate_norm
            slope = np.where(g < 0, 1.0, np.exp(-np.abs(g))) / (1 + np.exp(-np.abs(g))) / gate_norm
            slope = np.where(np.isnan(g), g, slope)
        return la, np.exp(la), -np.expm1(la), slope


def gate_error(la):
    return 16 * U * (1 + np.where(np.isfinite(la), np.abs(la), 0.0))


def runs(shape, order=None, cu=None, reverse=False):
    """[(sequence, token rows in scan order)] over rows [B * T] or packed rows."""
    if cu is None:
        B, T = shape
        return [(b, b * T + order) for b in range(B)]
    r = [(n, np.arange(cu[n], cu[n + 1])) for n in range(len(cu) - 1)]
    return [(n, t[::-1]) for n, t in r] if reverse else r


def glr_fwd(x, gate, gate_norm, complement, h0, where, out0=None):
    """x, gate [rows, C]; where = runs(...).  Returns (out, h_last, bound_out, bound_last), the
    bounds those of fp32 arithmetic before a final rounding."""
    x = np.asarray(x, np.float64)
    la, alpha, rest, _ = gates(gate, gate_norm)
    s = rest if complement else np.ones_like(alpha)
    n, C = len(where), x.shape[1]
    out = np.zeros_like(x) if out0 is None else np.array(out0, np.float64)
    last, b_out, b_last = np.zeros((n, C)), np.zeros_like(x), np.zeros((n, C))
    with np.errstate(invalid="ignore", over="ignore"):
        for i, tokens in where:
            h = np.zeros(C) if h0 is None else np.asarray(h0[i], np.float64).copy()
            H, E = np.abs(h), np.zeros(C)
            for t in tokens:
                e = gate_error(la[t])
                h = alpha[t] * h + s[t] * x[t]
                E = alpha[t] * E + (e + 2 * U) * (alpha[t] * H + np.abs(s[t] * x[t]))
                H = alpha[t] * H + np.abs(s[t] * x[t])
                out[t], b_out[t] = h, E + 32 * U * H
            last[i], b_last[i] = h, E + 32 * U * H
    return out, last, b_out, b_last


def glr_bwd(x, gate, h, dout, gate_norm, complement, h0, dh_last, where):
    """Returns (dx, dgate, dh0) and their bounds."""
    x, h, dout = (np.asarray(t, np.float64) for t in (x, h, dout))
    la, alpha, rest, slope = gates(gate, gate_norm)
    s = rest if complement else np.ones_like(alpha)
    n, C = len(where), x.shape[1]
    dx, dg, dh0 = np.zeros_like(x), np.zeros_like(x), np.zeros((n, C))
    bx, bg, b0 = np.zeros_like(x), np.zeros_like(x), np.zeros((n, C))
    for i, tokens in where:
        r = np.zeros(C) if dh_last is None else np.asarray(dh_last[i], np.float64).copy()
        R, E = np.abs(r), np.zeros(C)
        for k in range(len(tokens) - 1, -1, -1):
            t = tokens[k]
            before = h[tokens[k - 1]] if k else (np.zeros(C) if h0 is None else np.asarray(h0[i], np.float64))
            m, M = (before - x[t], np.abs(before) + np.abs(x[t])) if complement else (before, np.abs(before))
            e = gate_error(la[t])
            d, D = dout[t] + r, np.abs(dout[t]) + R
            ED = E + 34 * U * D
            dx[t], bx[t] = s[t] * d, s[t] * ED + 2 * e * s[t] * D
            r, R, E = alpha[t] * d, alpha[t] * D, alpha[t] * E + (e + 2 * U) * alpha[t] * D
            ER = alpha[t] * ED + (e + 2 * U) * R
            dg[t], bg[t] = r * m * slope[t], (ER + (4 * U + e) * R) * M * slope[t]
        dh0[i], b0[i] = r, E + 34 * U * R
    return (dx, dg, dh0), (bx, bg, b0)


def phases(positions, inv_freq):
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    return np.cos(a)[:, None], np.sin(a)[:, None]


def pair_index(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(t, positions, inv_freq, interleaved, scale, inverse=False):
    """(rotated [rows, H, D], sum of the absolute terms)."""
    t = np.array(t, np.float64)
    mag = np.abs(t)
    if inv_freq is None or len(inv_freq) == 0:
        return t, mag
    i, j = pair_index(2 * len(inv_freq), interleaved)
    c, s = phases(positions, inv_freq)
    if inverse:
        s = -s
    out = t.copy()
    out[..., i] = scale * (t[..., i] * c - t[..., j] * s)
    out[..., j] = scale * (t[..., j] * c + t[..., i] * s)
    both = abs(scale) * (mag[..., i] + mag[..., j])
    mag[..., i], mag[..., j] = both, both
    return out, mag


#: cos and sin: 2 units each, of an angle rounded to fp32 within half a turn: pi u.  Products,
#: sums, the scale: 5u.  The sum of D squares in any order of 32 lanes and more: (D/8 + 6) u;
#: the square root's reciprocal, weights, means: 12u.
TURN = 16 * U


def norm_error(D):
    return (D / 8 + 18) * U


def norm_rope(t, w, positions, inv_freq, eps, interleaved, scale):
    t = np.asarray(t, np.float64)
    r = 1 / np.sqrt(np.mean(t * t, -1, keepdims=True) + eps)
    out, mag = rotate(t * r * np.asarray(w, np.float64), positions, inv_freq, interleaved, scale)
    return out, mag * (TURN + norm_error(t.shape[-1]))


def norm_rope_bwd(d, t, w, positions, inv_freq, eps, interleaved, scale):
    """((dx, dw), bounds)."""
    t, w = np.asarray(t, np.float64), np.asarray(w, np.float64)
    D = t.shape[-1]
    g, G = rotate(d, positions, inv_freq, interleaved, scale, inverse=True)
    r = 1 / np.sqrt(np.mean(t * t, -1, keepdims=True) + eps)
    n = t * r
    dx = r * (w * g - n * np.mean(w * g * n, -1, keepdims=True))
    Dx = r * (np.abs(w) * G + np.abs(n) * np.mean(np.abs(w) * G * np.abs(n), -1, keepdims=True))
    e = TURN + 3 * norm_error(D)
    terms = t.shape[0] * t.shape[1]
    return (dx, (g * n).sum((0, 1))), (Dx * e, (G * np.abs(n)).sum((0, 1)) * (e + (terms + 8) * U))


def check(got, ref, bound, what, bf16=False, least=1e-35):
    """Every element within its bound (and the rounding to bf16); same non-finite values."""
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN pattern"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{what}: infinities"
    b = bound + least
    if bf16:
        b = b + EPS16 * (np.abs(ref) + b) + 2.0 ** -134
    err = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) / np.where(fine, b, 1), 0)
    if err.size:
        at = np.unravel_index(np.argmax(err), err.shape)
        assert err.max() <= 1.0, f"{what}: {err.max():.3g} of the bound at {at}: {got[at]!r} against {ref[at]!r}"
