"""Workloads of the gated scan, of the norms around a block and of activations kept in 8 bits.

Per channel, the gated scan is  h_t = a_t h_{t-1} + m_t x_t  with a_t = exp(min(g_t, 0)); g is given, or made from logits
as g_t = g_min * Sigmoid(exp(A) z_t); m_t = 1, or 1 - a_t ("complement").  The norms around a block are

    u = w_post * y / rms(y),   x' = x + scale * s * Sigmoid(gate) * u,   n = w_pre * x' / rms(x')

with x' rounded to its type before n is formed from it.  Activations in 8 bits are int8 codes with one float32 scale for
each 128 consecutive channels of a row: scale = amax * (1 / 127), code = rint(x * (127 / amax)), each step in float32.
``scan_fwd`` / ``scan_bwd`` run packed sequences, ``scan_step`` one token a sequence on states in slots, ``norm_fwd`` /
``norm_bwd`` rows, ``act`` packs and unpacks.  With ``own`` the calls go to the library's kernels; without it they are
plain torch operations in float32 (float64 for products of many decays), rounded once at the end.
"""
import math
import random

import numpy
import torch

own = False
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GROUP = 128      # channels that share a scale
G_MIN = -5.0
EPS = 1e-6


def _kda():
    import gated_delta_rule_20_amd as kda
    return kda


# ---- cases -------------------------------------------------------------------------------------------------------

def _scan(kind, name, dtype, C, n, lo, hi, len_seed, logits, complement, states, wide_g=False, fused=False, packed=False):
    """n packed sequences of lo..hi tokens (drawn from len_seed) and C channels; logits: the decay's gate is part of the
    call; wide_g: decays in float32 next to bf16 values; fused: x and g are the halves of one projection's rows; packed: scan_bwd
    reads h (and x) from 8 bits."""
    return {"kind": kind, "name": name, "dtype": dtype, "C": C, "n": n, "lo": lo, "hi": hi, "len_seed": len_seed,
            "logits": logits, "complement": complement, "states": states, "wide_g": wide_g, "fused": fused, "packed": packed}


def _step(name, dtype, C, n, pad, slots, logits, complement):
    """n sequences, the last `pad` of them empty places of a padded batch, on a pool of `slots` states."""
    return {"kind": "scan_step", "name": name, "dtype": dtype, "C": C, "n": n, "pad": pad, "slots": slots,
            "logits": logits, "complement": complement}


def _norm(kind, name, dtype, R, D, gate, post, pre, res, wide_x=False, packed=False):
    """R rows of D channels; gate, post, pre, res: which parts there are; wide_x: the residual stream is float32 next to
    bf16 blocks; packed: norm_bwd reads x', y and the gate from 8 bits."""
    return {"kind": kind, "name": name, "dtype": dtype, "R": R, "D": D, "gate": gate, "post": post, "pre": pre, "res": res,
            "wide_x": wide_x, "packed": packed}


def _act(name, dtype, R, D):
    return {"kind": "act", "name": name, "dtype": dtype, "R": R, "D": D}


def listed():
    return [
        # short prompts of a small model in float32, among them empty and one-token ones: launch latency
        _scan("scan_fwd", "scan_fwd_short_fp32", "fp32", 100, 16, 0, 200, 3, False, False, True),
        # one long context, values and decay logits from one fused projection
        _scan("scan_fwd", "scan_fwd_128k_bf16", "bf16", 2048, 1, 131072, 131072, 0, True, True, False, fused=True),
        # gradients of a small float32 layer on ragged sequences, an odd number of channels
        _scan("scan_bwd", "scan_bwd_ragged_fp32", "fp32", 257, 24, 1, 300, 5, True, False, True),
        # gradients of one training sequence, its activations kept in 8 bits
        _scan("scan_bwd", "scan_bwd_8k_bf16", "bf16", 4096, 1, 8192, 8192, 0, True, True, False, packed=True),
        # a decode step of a few sequences: latency
        _step("scan_step_3", "bf16", 2048, 3, 0, 16, False, False),
        # a decode step of a full batch with a padded end
        _step("scan_step_512", "bf16", 8192, 512, 7, 640, True, True),
        # between two blocks of a decode step of a few sequences: latency
        _norm("norm_fwd", "norm_fwd_4", "bf16", 4, 2560, True, True, True, False),
        # between two blocks of a prefill or a training step
        _norm("norm_fwd", "norm_fwd_8k", "bf16", 8192, 4096, True, True, True, True),
        # gradients of a small float32 model, odd sizes
        _norm("norm_bwd", "norm_bwd_ragged_fp32", "fp32", 333, 1000, True, True, True, True),
        # gradients of a training step, its activations kept in 8 bits
        _norm("norm_bwd", "norm_bwd_8k", "bf16", 8192, 4096, True, True, True, True, packed=True),
        # a few odd rows
        _act("act_37", "fp32", 37, 1001),
        # the activations of one layer of a training step
        _act("act_8k", "bf16", 8192, 4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd", "act"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    wide = rng.random() < 0.3 and dtype == "bf16"
    packed = rng.random() < 0.35
    flag = lambda p=0.6: rng.random() < p  # noqa: E731
    if kind in ("scan_fwd", "scan_bwd"):
        C = rng.choice([_log_int(rng, 1, 8192), 64 * _log_int(rng, 1, 128)])
        total = _log_int(rng, 16, max(17, min(131072, (1 << 27) // C)))
        n = min(_log_int(rng, 1, 96), total)
        mean = max(1, total // n)
        lo = rng.choice([0 if n > 3 else 1, 1, mean, max(1, mean // 8)])
        c = _scan(kind, "", dtype, C, n, lo, max(lo, 2 * mean - lo), rng.randrange(1 << 20), flag(), flag(0.5), flag(),
                  wide, kind == "scan_fwd" and not wide and flag(0.4), kind == "scan_bwd" and packed)
    elif kind == "scan_step":
        n = _log_int(rng, 1, 1024)
        c = _step("", dtype, _log_int(rng, 1, 16384), n, rng.choice([0, 0, n // 9]), n + rng.randrange(0, 65), flag(), flag())
    else:
        D = rng.choice([_log_int(rng, 1, 16384), 64 * _log_int(rng, 1, 256)])
        R = _log_int(rng, 1, min(65536, (1 << 26) // D))
        c = _act("", dtype, R, D) if kind == "act" else _norm(kind, "", dtype, R, D, flag(), flag(0.75), flag(0.75), flag(), wide,
                                                             kind == "norm_bwd" and packed)
    del c["name"]
    return c


def _lengths(c):
    g = torch.Generator().manual_seed(c["len_seed"])
    return torch.randint(c["lo"], c["hi"] + 1, (c["n"],), generator=g).tolist()


# ---- inputs ------------------------------------------------------------------------------------------------------

def _codes(x):
    """x [..., D] in 8 bits: codes [..., D] int8 and scales [..., groups] float32."""
    D = x.shape[-1]
    n = (D + GROUP - 1) // GROUP
    w = torch.nn.functional.pad(x.float(), (0, n * GROUP - D)).unflatten(-1, (n, GROUP))
    amax = w.abs().amax(-1, keepdim=True)
    inv = torch.where(amax > 0, torch.full_like(amax, 127.0) / amax, 0.0)
    codes = torch.round(w * inv).to(torch.int8).flatten(-2)[..., :D].contiguous()
    return codes, (amax * torch.full_like(amax, 1.0 / 127.0))[..., 0].contiguous()


def _values(p):
    """The values that codes and scales stand for, float32."""
    codes, scales = p
    return codes.float() * scales.repeat_interleave(GROUP, -1)[..., :codes.shape[-1]]


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    unit = lambda *shape: torch.rand(shape, generator=gen, device=dev)  # noqa: E731
    c, dt = case, DTYPES[case["dtype"]]
    s = {"case": case}
    if c["kind"] == "act":
        # activations with a few channels far larger than the rest
        s["x"] = (normal(c["R"], c["D"]) * torch.exp2(3.0 * unit(c["D"]) ** 8)).to(dt)
        return s
    if c["kind"] in ("norm_fwd", "norm_bwd"):
        R, D = c["R"], c["D"]
        tx = torch.float32 if c["wide_x"] else dt
        s["y"] = (2.0 * normal(R, D)).to(dt)
        s["x"] = (3.0 * normal(R, D)).to(tx)
        s["gate"] = (normal(R, D)).to(dt) if c["gate"] else None
        s["post"] = 1.0 + 0.2 * normal(D) if c["post"] else None
        s["pre"] = 1.0 + 0.2 * normal(D) if c["pre"] else None
        s["res"] = 0.5 + 0.1 * normal(D) if c["res"] else None
        s["scale"] = 0.25
        if c["kind"] == "norm_bwd":
            s["dx"] = normal(R, D).to(tx)
            s["dn"] = normal(R, D).to(dt) if c["pre"] else None
            if c["packed"]:
                for k in ("x", "y", "gate"):
                    s[k] = None if s[k] is None else _codes(s[k])
        return s
    C = c["C"]
    tg = torch.float32 if c.get("wide_g") else dt
    if c["kind"] == "scan_step":
        R = c["n"]
    else:
        lens = _lengths(c)
        R = sum(lens)
        s["lens"] = lens
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(device=dev, dtype=torch.int32)
    x = normal(R, C)
    if c["logits"]:
        # memories from a few tokens to thousands
        s["A"] = torch.log(0.5 + unit(C))
        g = 1.5 * normal(R, C) - 2.0 - 5.0 * unit(C)
    else:
        # data-dependent log-decays, now and then (a new document) one that forgets everything
        s["A"] = None
        g = -torch.nn.functional.softplus(normal(R, C) - 2.0 - 5.0 * unit(C))
        g = torch.where(unit(R, 1) < 2e-3, torch.full_like(g, -40.0), g)
    if c.get("fused"):
        rows = torch.cat([x.to(dt), g.to(dt)], 1)
        s["x"], s["g"] = rows[:, :C], rows[:, C:]
    else:
        s["x"], s["g"] = x.to(dt), g.to(tg)
    if c["kind"] == "scan_step":
        n, pad, slots = c["n"], c["pad"], c["slots"]
        s["state"] = normal(slots, C)
        s["new_state"] = torch.zeros_like(s["state"])
        pick = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
        pick[n - pad:] = -1
        s["slots"] = pick.to(dev)
        return s
    s["h0"] = normal(c["n"], C) if c["states"] else None
    if c["kind"] == "scan_bwd":
        # what the forward pass has kept, the gradients that arrive
        h = _forward(s)[0].to(dt)
        s["h"] = _codes(h) if c["packed"] else h
        if c["complement"] and c["packed"]:
            s["x"] = _codes(s["x"])
        elif not c["complement"]:
            s["x"] = None
        s["dh"] = normal(R, C).to(dt)
        s["dhT"] = normal(c["n"], C) if c["states"] else None
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    kind = s["case"]["kind"]
    if own:
        return _OWN[kind](s)
    return _PLAIN[kind](s)


def _packed(p):
    return _kda().Packed(*p) if isinstance(p, tuple) else p


def _own_scan_fwd(s):
    return _kda().gated_scan_fwd(s["x"], s["g"], A_log=s["A"], g_min=G_MIN, complement=s["case"]["complement"],
                                 cu_seqlens=s["cu"], initial_state=s["h0"])


def _own_scan_bwd(s):
    return _kda().gated_scan_bwd(_packed(s["x"]), s["g"], _packed(s["h"]), s["dh"], A_log=s["A"], g_min=G_MIN,
                                 complement=s["case"]["complement"], cu_seqlens=s["cu"], initial_state=s["h0"],
                                 dfinal_state=s["dhT"])


def _own_scan_step(s):
    h = _kda().gated_scan_step(s["x"], s["g"], s["state"], A_log=s["A"], g_min=G_MIN, complement=s["case"]["complement"],
                               slots=s["slots"], new_state=s["new_state"])
    return h, s["new_state"]


def _own_norm_fwd(s):
    return _kda().block_norm_fwd(s["x"], s["y"], gate=s["gate"], post_weight=s["post"], res_scale=s["res"], scale=s["scale"],
                                 pre_weight=s["pre"], eps=EPS)


def _own_norm_bwd(s):
    # codes and scales do not say which type the block has, and without pre no gradient of n does
    return tuple(_kda().block_norm_bwd(_packed(s["x"]), _packed(s["y"]), s["dx"], s["dn"], gate=_packed(s["gate"]),
                                       post_weight=s["post"], res_scale=s["res"], scale=s["scale"], pre_weight=s["pre"], eps=EPS,
                                       dtype=DTYPES[s["case"]["dtype"]]))


def _own_act(s):
    kda = _kda()
    p = kda.act_pack(s["x"])
    return kda.act_unpack(p, dtype=s["x"].dtype), p.scales


# ---- plain forms -------------------------------------------------------------------------------------------------

def _decay(s):
    """Log-decays and, with logits, the gate's Sigmoid, in float32."""
    g = s["g"].float()
    if s["A"] is None:
        return g.clamp_max(0.0), None
    sig = torch.sigmoid(torch.exp(s["A"]) * g)
    return G_MIN * sig, sig


def _scan_rows(a, b):
    """All h_t = a_t h_{t-1} + b_t along the first axis from h_{-1} = 0: spans double, products of decays in float64."""
    n, d = a.shape[0], 1
    while d < n:
        b = torch.cat([b[:d], b[d:] + (a[d:] * b[:-d]).float()])
        if 2 * d < n:
            a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _bounds(s):
    """First and last rows of the sequences that have any, and which these are."""
    cu = s["cu"].long()
    there = torch.tensor([i for i, n in enumerate(s["lens"]) if n > 0], dtype=torch.long, device=cu.device)
    return cu[:-1][there], cu[1:][there] - 1, there


def _forward(s):
    c = s["case"]
    g, _ = _decay(s)
    a = torch.exp(g.double())
    x = s["x"].float()
    if c["complement"]:
        x = -torch.expm1(g) * x
    first, last, there = _bounds(s)
    if s["h0"] is not None:
        x = x.index_add(0, first, (a[first] * s["h0"][there]).float())
    a.index_fill_(0, first, 0.0)
    h = _scan_rows(a, x)
    hT = torch.zeros((c["n"], c["C"]), device=x.device) if s["h0"] is None else s["h0"].clone()
    hT[there] = h[last]
    return h, hT


def _plain_scan_fwd(s):
    h, hT = _forward(s)
    return h.to(s["x"].dtype), hT


def _plain_scan_bwd(s):
    c = s["case"]
    wide = lambda t: _values(t) if isinstance(t, tuple) else t.float()  # noqa: E731
    g, sig = _decay(s)
    a = torch.exp(g.double())
    first, last, there = _bounds(s)
    d = s["dh"].float()
    if s["dhT"] is not None:
        d = d.index_add(0, last, s["dhT"][there])
    # D_t = d_t + a_{t+1} D_{t+1}, cut where a sequence ends
    nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])
    nxt.index_fill_(0, last, 0.0)
    D = _scan_rows(nxt.flip(0), d.flip(0)).flip(0)
    e = (a * D).float()
    h = wide(s["h"])
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[first] = 0.0 if s["h0"] is None else s["h0"][there]
    dx = D
    if c["complement"]:
        dx = -torch.expm1(g) * D
        prev = prev - wide(s["x"])
    dg, dA = e * prev, None
    if sig is not None:
        z = s["g"].float()
        dg = dg * (G_MIN * sig * (1.0 - sig)) * torch.exp(s["A"])
        dA = (dg * z).double().sum(0).float()
    dh0 = torch.zeros((c["n"], c["C"]), device=h.device) if s["dhT"] is None else s["dhT"].clone()
    dh0[there] = e[first]
    return dx.to(s["dh"].dtype), dg.to(s["g"].dtype), dA, dh0


def _plain_scan_step(s):
    g, _ = _decay(s)
    x = s["x"].float()
    if s["case"]["complement"]:
        x = -torch.expm1(g) * x
    slots = s["slots"].long()
    h = torch.exp(g) * s["state"][slots.clamp_min(0)] + x
    n = slots.numel() - s["case"]["pad"]
    s["new_state"].index_copy_(0, slots[:n], h[:n])
    return torch.where((slots >= 0)[:, None], h, 0.0).to(s["x"].dtype), s["new_state"]


def _rstd(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm_fwd(s):
    r = s["y"].float()
    if s["post"] is not None:
        r = s["post"] * (r * _rstd(r))
    if s["gate"] is not None:
        r = torch.sigmoid(s["gate"].float()) * r
    if s["res"] is not None:
        r = s["res"] * r
    x = (s["x"].float() + s["scale"] * r).to(s["x"].dtype)
    n = None
    if s["pre"] is not None:
        w = x.float()
        n = (s["pre"] * (w * _rstd(w))).to(s["y"].dtype)
    return x, n


def _plain_norm_bwd(s):
    wide = lambda t: _values(t) if isinstance(t, tuple) else t.float()  # noqa: E731
    G = s["dx"].float()
    dpre = dpost = dres = dgate = None
    total = lambda t: t.double().sum(0).float()  # noqa: E731
    if s["pre"] is not None:
        x, dn = wide(s["x"]), s["dn"].float()
        r = _rstd(x)
        x = x * r
        dpre = total(dn * x)
        dn = s["pre"] * dn
        G = G + r * (dn - x * (dn * x).mean(-1, keepdim=True))
    dx = G.to(s["dx"].dtype)
    y = wide(s["y"])
    ry = _rstd(y)
    u = y if s["post"] is None else s["post"] * (y * ry)
    sig = None if s["gate"] is None else torch.sigmoid(wide(s["gate"]))
    if s["res"] is not None:
        dres = s["scale"] * total(G * (u if sig is None else sig * u))
        G = s["res"] * G
    G = s["scale"] * G
    tb = DTYPES[s["case"]["dtype"]]
    if sig is not None:
        dgate = (G * u * sig * (1.0 - sig)).to(tb)
        G = G * sig
    if s["post"] is not None:
        y = y * ry
        dpost = total(G * y)
        G = s["post"] * G
        G = ry * (G - y * (G * y).mean(-1, keepdim=True))
    return dx, G.to(tb), dgate, dpost, dres, dpre


def _plain_act(s):
    codes, scales = _codes(s["x"])
    return _values((codes, scales)).to(s["x"].dtype), scales


_PLAIN = {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step, "norm_fwd": _plain_norm_fwd,
          "norm_bwd": _plain_norm_bwd, "act": _plain_act}
_OWN = {"scan_fwd": _own_scan_fwd, "scan_bwd": _own_scan_bwd, "scan_step": _own_scan_step, "norm_fwd": _own_norm_fwd,
        "norm_bwd": _own_norm_bwd, "act": _own_act}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    eight = 1.0 + 4.0 / GROUP
    if c["kind"] == "act":
        n = c["R"] * c["D"]
        return {"bytes": n * 2 * (size + eight), "flops": 5 * n}
    if c["kind"] in ("norm_fwd", "norm_bwd"):
        n = c["R"] * c["D"]
        tx = 4 if c["wide_x"] else size
        weights = 4 * c["D"] * (c["post"] + c["pre"] + c["res"])
        if c["kind"] == "norm_fwd":
            return {"bytes": n * (2 * tx + size * (1 + c["gate"] + c["pre"])) + weights, "flops": 14 * n}
        saved = (2 + c["gate"]) * eight if c["packed"] else tx + size * (1 + c["gate"])
        return {"bytes": n * (2 * tx + saved + size * (c["pre"] + 1 + c["gate"])) + 2 * weights, "flops": 32 * n}
    tg = 4 if c.get("wide_g") else size
    if c["kind"] == "scan_step":
        n = (c["n"] - c["pad"]) * c["C"]
        return {"bytes": n * (8 + 3 * size), "flops": 4 * n}
    n = sum(_lengths(c)) * c["C"]
    state = 4 * c["n"] * c["C"]
    if c["kind"] == "scan_fwd":
        return {"bytes": n * (2 * size + tg) + state * (1 + c["states"]), "flops": 4 * n}
    saved = (1 + c["complement"]) * (eight if c["packed"] else size)
    return {"bytes": n * (2 * size + 2 * tg + saved) + state * (1 + 2 * c["states"]), "flops": 10 * n}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _exact_decay(s):
    g = s["g"].double()
    if s["A"] is None:
        return torch.minimum(g, torch.zeros_like(g)), None
    sig = 1.0 / (1.0 + torch.exp(-torch.exp(s["A"].double()) * g))
    return G_MIN * sig, sig


def _exact_values(p):
    if not isinstance(p, tuple):
        return p.double()
    at = torch.arange(p[0].shape[-1], device=p[0].device) // GROUP
    return p[0].double() * p[1].double()[..., at]


def _exact_codes(x):
    """Packing as its float32 steps define it, in numpy; the values in 64 bits."""
    f = numpy.float32
    w = x.float().cpu().numpy()
    out = numpy.zeros(w.shape, numpy.float64)
    scales = []
    for at in range(0, w.shape[-1], GROUP):
        part = w[..., at:at + GROUP]
        amax = numpy.abs(part).max(-1, keepdims=True)
        with numpy.errstate(divide="ignore"):
            inv = numpy.where(amax > 0, f(127.0) / amax, f(0.0)).astype(f)
        scale = amax * f(1.0 / 127.0)
        out[..., at:at + GROUP] = numpy.rint(part * inv).astype(numpy.float64) * scale.astype(numpy.float64)
        scales.append(scale)
    return (torch.from_numpy(out).to(x.device), torch.from_numpy(numpy.concatenate(scales, -1).astype(numpy.float64)).to(x.device))


def _exact_scan(case, s):
    """Token by token; sequences from the longest to the shortest, so that those with a token t are the first ones."""
    lens = s["lens"]
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    start = s["cu"].long()[:-1][order]
    ends, alive, over = sorted(lens), [], 0
    for t in range(max(lens)):
        while ends[over] <= t:
            over += 1
        alive.append(len(lens) - over)
    back = torch.empty(len(order), dtype=torch.long)
    back[order] = torch.arange(len(order))
    back = back.to(start.device)
    g, sig = _exact_decay(s)
    a = torch.exp(g)
    N, C = case["n"], case["C"]
    state = lambda t: torch.zeros((N, C), dtype=torch.float64, device=g.device) if t is None else t.double()[order]  # noqa: E731
    if case["kind"] == "scan_fwd":
        b = s["x"].double()
        b = -torch.expm1(g) * b if case["complement"] else b
        H, h = state(s["h0"]), torch.zeros_like(b)
        for t, m in enumerate(alive):
            at = start[:m] + t
            H[:m] = a[at] * H[:m] + b[at]
            h[at] = H[:m]
        return h, H[back]
    d, E = s["dh"].double(), state(s["dhT"])
    D, e = torch.zeros_like(d), torch.zeros_like(d)
    for t in reversed(range(len(alive))):
        at = start[:alive[t]] + t
        D[at] = d[at] + E[:alive[t]]
        E[:alive[t]] = a[at] * D[at]
        e[at] = E[:alive[t]]
    h = _exact_values(s["h"])
    dg = torch.zeros_like(e)
    h0 = state(s["h0"])[back]
    cu = s["cu"].tolist()
    for i in range(N):
        lo, hi = cu[i], cu[i + 1]
        if hi > lo:
            dg[lo] = e[lo] * h0[i]
            dg[lo + 1:hi] = e[lo + 1:hi] * h[lo:hi - 1]
    dx = D
    if case["complement"]:
        dg = dg - e * _exact_values(s["x"])
        dx = -torch.expm1(g) * D
    dA = None
    if sig is not None:
        eA = torch.exp(s["A"].double())
        dg = dg * G_MIN * sig * (1.0 - sig) * eA
        dA = (dg * s["g"].double()).sum(0)
    return dx, dg, dA, E[back]


def _exact_norm(case, s):
    def block(x, y, gate, post, res):
        u = y
        if post is not None:
            u = post * y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + EPS)
        if gate is not None:
            u = u / (1.0 + torch.exp(-gate))
        if res is not None:
            u = res * u
        u = s["scale"] * u
        return x(u) if callable(x) else x + u

    def after(x, pre):
        return pre * x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + EPS)

    f = lambda t: None if t is None else _exact_values(t)  # noqa: E731
    if case["kind"] == "norm_fwd":
        x = block(f(s["x"]), f(s["y"]), f(s["gate"]), f(s["post"]), f(s["res"]))
        # n is of x' as it was rounded
        n = None if s["pre"] is None else after(x.to(s["x"].dtype).double(), f(s["pre"]))
        return x, n
    leaf = {k: f(s[k]) for k in ("y", "gate", "post", "res", "pre")}
    for t in leaf.values():
        if t is not None:
            t.requires_grad_(True)
    kept = f(s["x"])
    x0 = torch.zeros_like(kept).requires_grad_(True)
    # the residual stream before the block is whatever gives the kept x' behind it
    x1 = block(lambda u: x0 + (kept - u.detach()) + u, **{k: leaf[k] for k in ("y", "gate", "post", "res")})
    loss = (x1 * f(s["dx"])).sum()
    if s["pre"] is not None:
        loss = loss + (after(x1, leaf["pre"]) * f(s["dn"])).sum()
    loss.backward()
    grad = lambda k: None if leaf[k] is None else leaf[k].grad  # noqa: E731
    return x0.grad, grad("y"), grad("gate"), grad("post"), grad("res"), grad("pre")


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "act":
        return _exact_codes(s["x"])
    if kind in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s)
    if kind in ("scan_fwd", "scan_bwd"):
        return _exact_scan(case, s)
    g, _ = _exact_decay(s)
    x = s["x"].double()
    x = -torch.expm1(g) * x if case["complement"] else x
    h, new = torch.zeros_like(x), s["new_state"].double()
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            h[i] = torch.exp(g[i]) * s["state"][slot].double() + x[i]
            new[slot] = h[i]
    return h, new
