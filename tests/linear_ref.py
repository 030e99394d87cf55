"""Plain float64 forms of linear attention with a decay per head and of the cache's
page operators, token by token and page by page, for the tests."""
import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # a rounding: at most half a step, relative


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def widen(x, H):
    """[..., Hk, D] -> [..., H, D]: value head h reads head h // (H // Hk)."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def decay(g, rows, H):
    """exp(g) as [rows, H] float64; values above 0 count as 0, -inf forgets."""
    g = np.broadcast_to(np.minimum(f64(g) if isinstance(g, torch.Tensor) else g, 0.0), (rows, H))
    return np.exp(g)


def forward(q, k, v, g, scale, cu, h0=None, every=None):
    """q, k [R, Hk, Dk], v [R, H, Dv], g [R, H] or [H] (float64 arrays); cu: offsets.
    Returns o [R, H, Dv], states [N, H, Dk, Dv] and, with every, {(sequence, tokens): state}."""
    R, H, Dv = v.shape
    q, k = widen(q, H), widen(k, H)
    a = decay(g, R, H)
    N = len(cu) - 1
    o, out, snaps = np.zeros_like(v), np.zeros((N, H, q.shape[-1], Dv)), {}
    for s in range(N):
        S = np.zeros((H, q.shape[-1], Dv)) if h0 is None else h0[s].copy()
        for t in range(cu[s], cu[s + 1]):
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
            if every and (t + 1 - cu[s]) % every == 0 and t + 1 < cu[s + 1]:
                snaps[s, t + 1 - cu[s]] = S.copy()
        out[s] = S
    return (o, out, snaps) if every else (o, out)


def backward(q, k, v, g, do, scale, cu, h0=None, dhT=None):
    """Gradients by the recurrence's own chain rule: dq, dk, dv, dg [R, H] (or [H] for g [H]), dh0."""
    R, H, Dv = v.shape
    Hk, Dk = q.shape[-2:]
    qw, kw = widen(q, H), widen(k, H)
    a = decay(g, R, H)
    N = len(cu) - 1
    dq, dk, dv, dg = np.zeros_like(qw), np.zeros_like(kw), np.zeros_like(v), np.zeros((R, H))
    dh0 = np.zeros((N, H, Dk, Dv))
    for s in range(N):
        S = [np.zeros((H, Dk, Dv)) if h0 is None else h0[s]]
        for t in range(cu[s], cu[s + 1]):
            S.append(a[t][:, None, None] * S[-1] + kw[t][:, :, None] * v[t][:, None, :])
        dS = np.zeros((H, Dk, Dv)) if dhT is None else dhT[s].copy()
        for t in reversed(range(cu[s], cu[s + 1])):
            i = t - cu[s] + 1
            dq[t] = scale * np.einsum("hkv,hv->hk", S[i], do[t])
            dS = dS + scale * qw[t][:, :, None] * do[t][:, None, :]
            dk[t] = np.einsum("hkv,hv->hk", dS, v[t])
            dv[t] = np.einsum("hkv,hk->hv", dS, kw[t])
            dg[t] = a[t] * np.einsum("hkv,hkv->h", S[i - 1], dS)
            dS = a[t][:, None, None] * dS
        dh0[s] = dS
    share = lambda x: x.reshape(R, Hk, H // Hk, Dk).sum(2)  # noqa: E731
    return share(dq), share(dk), dv, (dg.sum(0) if np.ndim(g) == 1 else dg), dh0


# ---- pages: lists, one page after the other ------------------------------------------------------------------------

def pages_copy(dst, src, dst_pages, src_pages):
    """numpy pools; pairs in order, so the last of several with one destination counts."""
    old = [x.copy() for x in src]
    for d, s in zip(dst_pages, src_pages):
        if 0 <= d < dst[0].shape[0] and 0 <= s < old[0].shape[0]:
            for x, y in zip(dst, old):
                x[d] = y[s]


def pages_fork(pools, table, count, parents, children):
    n_pages, rows = len(count), table.shape[0]
    free = [p for p in range(n_pages) if count[p] <= 0]
    start = table.copy()
    new = []
    for i, (a, c) in enumerate(zip(parents, children)):
        if not (0 <= a < rows and 0 <= c < rows) or c in list(parents) or c in list(children[:i]):
            new.append(-1)
            continue
        held = [j for j in range(table.shape[1]) if 0 <= start[a, j] < n_pages]
        table[c] = -1
        if not held or not free:
            new.append(-1)
            continue
        p = free.pop(0)
        for j in held[:-1]:
            table[c, j] = start[a, j]
            count[start[a, j]] += 1
        table[c, held[-1]] = p
        count[p] = 1
        for x in pools:
            x[p] = x[start[a, held[-1]]]
        new.append(p)
    return new


def pages_free(table, count, rows):
    for r in rows:
        if not 0 <= r < table.shape[0]:
            continue
        for j in range(table.shape[1]):
            p, table[r, j] = table[r, j], -1
            if 0 <= p < len(count):
                count[p] = max(count[p] - 1, 0) if count[p] > 0 else count[p]


def pages_compact(pools, table, count):
    n_pages = len(count)
    live = [p for p in range(n_pages) if count[p] > 0]
    n = len(live)
    moved = np.full(n_pages, -1, np.int32)
    moved[live] = live
    holes = [p for p in range(n) if count[p] <= 0]
    for p, h in zip([p for p in live if p >= n], holes):
        moved[p] = h
        count[h], count[p] = count[p], 0
        for x in pools:
            x[h] = x[p]
    for j in np.ndindex(table.shape):
        p = table[j]
        table[j] = moved[p] if 0 <= p < n_pages else -1
    return moved, n


# ---- bounds for the chunked form -------------------------------------------------------------------------------------
#
# Every result is a sum of products of inputs and decays, so running the same formulas on absolute
# values bounds the sum of its terms' magnitudes ("mags").  With u = 2^-24:
#  * float32 arithmetic: a term passes through a sum over the contracted width, one over the chunk and one product and
#    addition per chunk it is carried (its decay shrinks the error it carries with it); each rounds by u.  The decay of
#    a token pair is the exponential of a difference of float64 sums held in two floats (2^-22 relative for |G| below
#    the underflow, with the hardware exponential's error).  ACC counts them: 128 + 64 + 64 plus three a chunk.
#  * bf16 operands: the decayed score or the state's operand of an output term is rounded once (2^-8).
#  * the output's own rounding, to its type.

def acc(tokens):
    return (256 + 16 + 3 * (tokens // 32 + 1)) * 2.0 ** -24


def bound(ref, mags, dtype, tokens):
    """Largest |error| of an output of type dtype, of value ref and term magnitudes mags."""
    t = mags * (acc(tokens) + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0))
    return 1.02 * (t + HALF[dtype] * (np.abs(ref) + t)) + 1e-35


def rel2(got, ref):
    """Difference over result in the 2-norm."""
    n = np.linalg.norm(ref)
    return float(np.linalg.norm(got - ref) / n) if n else float(np.linalg.norm(got))
