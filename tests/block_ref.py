"""The gated scan, the norms around a block and 8-bit activations in float64, each with bounds on what float32 arithmetic may
add, counted in roundings.

U = 2^-24 is half a step of float32.  The hardware's exponential, reciprocal and reciprocal square root are taken as
2 U off (one unit in the last place)."""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 1e-36


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def values(codes, scales):
    """What int8 codes and the scales of groups of 128 stand for."""
    c, s = f64(codes), f64(scales)
    return c * np.repeat(s, 128, axis=-1)[..., :c.shape[-1]]


def pack(x):
    """Codes and scales of float32 x [R, D], in the format's own float32 steps."""
    f = np.float32
    R, D = x.shape
    n = (D + 127) // 128
    codes, scales = np.zeros((R, D), np.int8), np.zeros((R, n), f)
    for j in range(n):
        part = x[:, 128 * j:128 * j + 128].astype(f)
        amax = np.abs(part).max(1) if R else np.zeros(0, f)
        bad, some = ~np.isfinite(amax), amax >= f(2.0 ** -118)
        inv = np.where(bad | ~some, f(0), f(127) / np.where(some & ~bad, amax, f(1))).astype(f)
        with np.errstate(invalid="ignore"):
            q = np.where(bad[:, None], f(0), np.rint((part * inv[:, None]).astype(f)))
        codes[:, 128 * j:128 * j + 128] = np.where(bad[:, None], 0, q).astype(np.int8)
        scales[:, j] = np.where(bad, f(np.nan), np.where(some, (amax * f(1 / 127)).astype(f), f(0)))
    return codes, scales


def _sigmoid(y):
    e = np.exp(-np.abs(y))
    return np.where(y >= 0, 1, e) / (1 + e), np.where(y >= 0, e, 1) / (1 + e)


class Decay:
    """Log-decays g, a = e^g, 1 - a and the relative errors of each that float32 may make."""

    def __init__(self, z, A_log, g_min):
        if A_log is None:
            self.g, eg, self.slope, self.e_slope = np.minimum(z, 0.0), 0.0, np.ones_like(z), 0.0
        else:
            y = np.exp(A_log) * z
            s, r = _sigmoid(y)
            self.g = g_min * s
            # e^A: its argument times log2(e) rounds twice; y: one product more
            ey = np.abs(y) * (np.abs(A_log) * 2 * U + 3 * U + 4 * U)
            # the Sigmoid: the exponential (its argument rounds twice), a sum, a reciprocal
            es = r * (ey + np.abs(y) * 2 * U + 2 * U) + 3 * U
            eg = es + U
            self.slope = g_min * s * r * np.exp(A_log)
            self.e_slope = 2 * (ey + np.abs(y) * 2 * U) + (np.abs(A_log) * 2 + 20) * U
        fin = np.where(np.isfinite(self.g), np.abs(self.g), 0.0)
        self.a, self.rest = np.exp(self.g), -np.expm1(self.g)
        # e^g: g's error, two roundings of its argument, the exponential
        self.e_a = fin * (eg + 2 * U) + 2 * U
        near = self.g > -0.1
        # e^g - 1 by a cubic where e^g is near 1: five steps at most and its own error (below U / 2); else by subtraction
        e_rest = np.where(near, eg + 7 * U, (self.e_a * self.a + U) / np.maximum(self.rest, 0.09))
        self.e_rest = e_rest
        # error of a h relative to |h|: through e^g - 1 or through e^g
        self.e_step = np.where(near, self.rest * e_rest, self.a * self.e_a)


def scan(x, z, A_log, g_min, complement, cu, h0):
    """h, final states and bounds of both; x, z [T, C] float64, cu a list, h0 [N, C] or None."""
    d = Decay(z, A_log, g_min)
    m = d.rest if complement else np.ones_like(x)
    em = d.e_rest + U if complement else np.zeros_like(x)
    N = len(cu) - 1
    h, tol = np.zeros_like(x), np.zeros_like(x)
    hT = np.zeros((N, x.shape[1])) if h0 is None else h0.copy()
    tT = np.zeros_like(hT)
    for s in range(N):
        H, M, E = hT[s].copy(), np.abs(hT[s]), np.zeros(x.shape[1])
        for t in range(cu[s], cu[s + 1]):
            b = np.abs(m[t] * x[t])
            # per token: two roundings of each side's product and sum; joining slices and tiles, as many again (they carry a
            # decay product whose exponent rounds once a token)
            with np.errstate(invalid="ignore"):
                H = np.where(d.a[t] == 0, 0.0, d.a[t] * H) + m[t] * x[t]
                E = d.a[t] * E + d.e_step[t] * M + b * em[t] + 10 * U * (d.a[t] * M + b) + U * np.abs(d.g[t].clip(-100)) * d.a[t] * M
            M = d.a[t] * M + b
            h[t], tol[t] = H, E
        if cu[s + 1] > cu[s]:
            hT[s], tT[s] = H, E
    return h, hT, tol, tT


def scan_bwd(x, z, h, d_h, A_log, g_min, complement, cu, h0, dhT):
    """(dx, dg, dA, dh0) and their bounds (without the rounding to the results' types)."""
    d = Decay(z, A_log, g_min)
    N, C = len(cu) - 1, z.shape[1]
    dx, dg, tx, tg = (np.zeros_like(z) for _ in range(4))
    dh0 = np.zeros((N, C)) if dhT is None else dhT.copy()
    t0 = np.zeros_like(dh0)
    for s in range(N):
        e, M, E = dh0[s].copy(), np.abs(dh0[s]), np.zeros(C)
        for t in reversed(range(cu[s], cu[s + 1])):
            D, MD, ED = d_h[t] + e, np.abs(d_h[t]) + M, E + 4 * U * (np.abs(d_h[t]) + M)
            e = np.where(d.a[t] == 0, 0.0, d.a[t] * D)
            M = d.a[t] * MD
            E = d.a[t] * ED + d.e_step[t] * MD + 8 * U * M + U * np.abs(d.g[t].clip(-100)) * M
            m, em = (d.rest[t], d.e_rest[t] + U) if complement else (1.0, 0.0)
            dx[t], tx[t] = m * D, m * ED + np.abs(m * MD) * em
            prev = h[t - 1] if t > cu[s] else 0.0 * e if h0 is None else h0[s]
            size = np.abs(prev)
            if complement:
                prev, size = prev - x[t], size + np.abs(x[t])
            sl = d.slope[t]
            dg[t] = e * prev * sl
            tg[t] = np.abs(sl) * (E * np.abs(prev) + M * size * 4 * U) + np.abs(sl) * M * np.abs(prev) * (np.broadcast_to(d.e_slope, z.shape)[t] + 4 * U)
        if cu[s + 1] > cu[s]:
            dh0[s], t0[s] = e, E
    dA = tA = None
    if A_log is not None:
        dA = (dg * z).sum(0)
        # partial sums of at most 64 steps in float32, joined in float64
        tA = (np.abs(z) * tg).sum(0) + 70 * U * np.abs(dg * z).sum(0)
    return (dx, dg, dA, dh0), (tx, tg, tA, t0)


def close(got, want, tol, dtype, what):
    """|got - want| within the bound and half a step of the type."""
    g = f64(got)
    limit = 1.01 * (tol + HALF[dtype] * (np.abs(want) + tol)) + TINY
    bad = ~(np.abs(g - want) <= limit)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / limit, 0)), g.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond the bound, worst at {i}: {g[i]} for {want[i]} (bound {limit[i]})")


def norm_fwd(x, y, gate, post, res, scale, eps):
    """x' and its bound."""
    D = y.shape[1]
    u, e = y, np.zeros_like(y)                     # value, relative error
    if post is not None:
        rs = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps)
        # sum of squares: a square and up to 32 additions a lane, 10 across lanes and waves; the mean and eps; the root halves it
        u, e = post * (y * rs), np.full_like(y, ((43 + 3) / 2 + 2 + 2) * U)
    if gate is not None:
        s, r = _sigmoid(gate)
        u, e = u * s, e + (r * (np.abs(gate) * 2 * U + 2 * U) + 4 * U)
    if res is not None:
        u, e = u * res, e + U
    v = x + scale * u
    return v, np.abs(scale * u) * (e + 2 * U) + np.abs(v) * U


def norm_n(x, pre, eps):
    """n of the rounded x' and its bound."""
    rs = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    n = pre * x * rs
    return n, np.abs(n) * ((43 + 3) / 2 + 4) * U


def norm_bwd(x, y, gate, post, res, pre, scale, eps, dx, dn):
    """dx, dy, dgate, dpost, dres, dpre and bounds: results' magnitudes (every product and sum taken without its sign)
    times 64 roundings: a sum over a row is 45 deep at most, the rest of any path below 20."""
    K = 64 * U
    G, mG = dx.copy(), np.abs(dx)
    out, tol = {}, {}
    if dn is not None:
        rx = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
        xh, w = x * rx, pre * dn
        G = G + rx * (w - xh * (w * xh).mean(1, keepdims=True))
        mG = mG + rx * (np.abs(w) + np.abs(xh) * np.abs(w * xh).mean(1, keepdims=True))
        out["dpre"], tol["dpre"] = (dn * xh).sum(0), 2 * K * np.abs(dn * xh).sum(0)
    out["dx"], tol["dx"] = G, K * mG
    if y is None:
        return out, tol
    ry = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if post is not None else 1.0
    yh = y * ry
    u = yh if post is None else post * yh
    s, r = (np.ones_like(y), np.zeros_like(y)) if gate is None else _sigmoid(gate)
    Kg = K + (0 if gate is None else np.abs(gate) * 4 * U)
    if res is not None:
        out["dres"] = (scale * G * s * u).sum(0)
        tol["dres"] = 2 * (Kg * np.abs(scale * mG * s * u)).sum(0)
    q = scale * (1.0 if res is None else res)
    dr, mr = q * G, np.abs(q) * mG
    if gate is not None:
        out["dgate"], tol["dgate"] = dr * u * s * r, Kg * mr * np.abs(u) * s * r
    du, mu = dr * s, mr * s
    if post is None:
        out["dy"], tol["dy"] = du, Kg * mu
        return out, tol
    out["dpost"], tol["dpost"] = (du * yh).sum(0), 2 * (Kg * mu * np.abs(yh)).sum(0)
    w, mw = post * du, np.abs(post) * mu
    out["dy"] = ry * (w - yh * (w * yh).mean(1, keepdims=True))
    tol["dy"] = 2 * ry * (Kg * mw + np.abs(yh) * (Kg * mw * np.abs(yh)).mean(1, keepdims=True))
    return out, tol
