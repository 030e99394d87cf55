"""Workloads of linear attention with a decay for each head and of the page operators of a state cache.

Per head, with state S in R^{Dk x Dv}:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t

``fwd`` and ``bwd`` run whole (packed) sequences, ``step`` one token per sequence on states kept in the slots of a
pool, ``copy`` / ``fork`` / ``free`` / ``compact`` move and account for the pages of such a pool.  With ``own`` the
calls go to the library's kernels; without it they are plain torch operations in float32 (float64 for sums of
log-decays), rounded once at the end.
"""
import math
import random

import torch

own = False
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64


def _kda():
    import gated_delta_rule_20_amd as kda
    return kda


# ---- cases -------------------------------------------------------------------------------------------------------

def _linear(kind, name, dtype, H, Hk, Dk, Dv, n, lo, hi, len_seed, per_head, states):
    """n packed sequences of lo..hi tokens (drawn from len_seed); Hk query/key heads serve H value heads; per_head:
    one constant decay a head, else one a token and head; states: carried in (and, for bwd, its gradient)."""
    return {"kind": kind, "name": name, "dtype": dtype, "H": H, "Hk": Hk, "Dk": Dk, "Dv": Dv, "n": n, "lo": lo, "hi": hi,
            "len_seed": len_seed, "per_head": per_head, "states": states}


def _step(name, dtype, H, Hk, Dk, Dv, n, pad, slots, per_head):
    """n sequences, the last `pad` of them empty places of a padded batch, on a pool of `slots` states."""
    return {"kind": "step", "name": name, "dtype": dtype, "H": H, "Hk": Hk, "Dk": Dk, "Dv": Dv, "n": n, "pad": pad,
            "slots": slots, "per_head": per_head}


def _pages(kind, name, H, D, pages, rows, per_row, m, live=0.0):
    """A pool of `pages` pages (an fp32 state [H, D, D] and a bf16 convolution state [H, 3, 3 D] each); `rows` sequences
    that hold up to `per_row` pages; m pages copied or rows forked / freed; live: share of rows that live at compaction."""
    return {"kind": kind, "name": name, "H": H, "D": D, "pages": pages, "rows": rows, "per_row": per_row, "m": m, "live": live}


def listed():
    return [
        # short prompts of a small model in float32, among them empty and one-token ones: launch latency
        _linear("fwd", "fwd_short_fp32", "fp32", 2, 2, 64, 64, 16, 0, 200, 3, False, True),
        # one prompt on a fresh context: few heads, parallel over the tokens
        _linear("fwd", "fwd_8k_bf16", "bf16", 32, 32, 128, 128, 1, 8192, 8192, 0, False, True),
        # packed prompts of mixed lengths, as a prefill batch holds them
        _linear("fwd", "fwd_packed_bf16", "bf16", 32, 32, 128, 128, 64, 128, 4096, 247, False, True),
        # one long context with constant decays
        _linear("fwd", "fwd_128k_bf16", "bf16", 32, 32, 128, 128, 1, 131072, 131072, 0, True, False),
        # gradients of a small float32 layer on ragged sequences, query/key heads shared by two value heads
        _linear("bwd", "bwd_short_fp32", "fp32", 4, 2, 64, 64, 6, 1, 300, 5, False, True),
        # gradients of one training sequence
        _linear("bwd", "bwd_8k_bf16", "bf16", 32, 32, 128, 128, 1, 8192, 8192, 0, False, False),
        # a decode step of a few sequences: latency
        _step("step_4", "bf16", 32, 32, 128, 128, 4, 0, 16, True),
        # a decode step of a full batch with a padded end, on 1 GiB of states
        _step("step_512", "bf16", 32, 32, 128, 128, 512, 7, 640, False),
        # prefix snapshots copied into private states when requests are admitted
        _pages("copy", "copy_256", 32, 128, 640, 64, 8, 256),
        # eight continuations sampled from running sequences
        _pages("fork", "fork_8", 8, 128, 256, 40, 6, 8),
        # a batch of finished sequences gives its pages back: table work only
        _pages("free", "free_64", 2, 64, 4096, 256, 16, 64),
        # the pool is packed to its front after two thirds of the sequences ended
        _pages("compact", "compact_512", 32, 128, 512, 100, 5, 0, 0.35),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "step", "step", "copy", "fork", "free", "compact"])
    Dk, Dv = rng.choice([64, 128]), rng.choice([64, 128])
    H = _log_int(rng, 1, 32)
    Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0] + [H, H])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    per_head = rng.random() < 0.4
    if kind in ("fwd", "bwd"):
        total = _log_int(rng, 16, 65536 if kind == "fwd" else 6000)
        n = min(_log_int(rng, 1, 96), total)
        mean = max(1, total // n)
        lo = rng.choice([0, 1, mean, max(1, mean // 8)])
        hi = max(lo, 2 * mean - lo)
        c = _linear(kind, "", dtype, H, Hk, Dk, Dv, n, lo, hi, rng.randrange(1 << 20), per_head, rng.random() < 0.6)
    elif kind == "step":
        n = _log_int(rng, 1, 512)
        c = _step("", dtype, H, Hk, Dk, Dv, n, rng.choice([0, 0, n // 9]), n + rng.randrange(0, 65), per_head)
    else:
        rows = _log_int(rng, 2, 300)
        per_row = rng.randrange(1, 17)
        pages = rows * per_row + rng.randrange(rows, 2 * rows + 9)
        page = 1 << rng.randrange(15, 21)  # keeps a pool below 1.5 GiB
        D = rng.choice([64, 128])
        Hp = max(1, min(32, page // (4 * D * D), (1500 << 20) // (pages * 4 * D * D)))
        m = rng.randrange(1, max(2, rows // 2)) if kind != "copy" else rng.randrange(1, max(2, pages // 2))
        c = _pages(kind, "", Hp, D, pages, rows, per_row, m, rng.uniform(0.1, 0.9))
    del c["name"]
    return c


def _lengths(c):
    g = torch.Generator().manual_seed(c["len_seed"])
    return torch.randint(c["lo"], c["hi"] + 1, (c["n"],), generator=g).tolist()


# ---- inputs ------------------------------------------------------------------------------------------------------

def _gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = _gen(seed, dev)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    s = {"case": case}
    if case["kind"] in ("copy", "fork", "free", "compact"):
        c, r = case, random.Random(seed)
        P, D, H = c["pages"], c["D"], c["H"]
        s["pools"] = [normal(P, H, D, D), normal(P, H, 3, 3 * D).to(torch.bfloat16)]
        order = list(range(P))
        r.shuffle(order)
        if c["kind"] == "copy":
            # snapshots in one pool, private states in another
            s["snap"] = [normal(P, H, D, D), normal(P, H, 3, 3 * D).to(torch.bfloat16)]
            s["src"] = torch.tensor([r.randrange(P) for _ in range(c["m"])], dtype=torch.int32, device=dev)
            s["dst"] = torch.tensor(order[:c["m"]], dtype=torch.int32, device=dev)
            return s
        live_rows = [i for i in range(c["rows"]) if c["kind"] != "compact" or r.random() < c["live"]]
        if c["kind"] == "fork":
            live_rows = list(range(c["rows"] - min(c["m"], c["rows"] // 2)))
        table = [[-1] * c["per_row"] for _ in range(c["rows"])]
        count = [0] * P
        for i in live_rows:
            for j in range(r.randint(1, c["per_row"])):
                share = j == 0 and r.random() < 0.3 and any(count)  # a prefix snapshot that several sequences hold
                p = r.choice([x for x in range(P) if count[x]]) if share else (order.pop() if order else -1)
                if p >= 0 and p not in table[i]:
                    table[i][j] = p
                    count[p] += 1
        # the table and the counts are one buffer, as a server keeps them
        meta = torch.tensor(sum(table, []) + count, dtype=torch.int32, device=dev)
        s["meta"] = meta
        if c["kind"] == "fork":
            kids = list(range(len(live_rows), c["rows"]))
            s["parents"] = torch.tensor([r.choice(live_rows) for _ in kids], dtype=torch.int32, device=dev)
            s["children"] = torch.tensor(kids, dtype=torch.int32, device=dev)
        if c["kind"] == "free":
            s["rows"] = torch.tensor(r.sample(live_rows, min(c["m"], len(live_rows))), dtype=torch.int32, device=dev)
        return s
    dt, H, Hk, Dk, Dv = DTYPES[case["dtype"]], case["H"], case["Hk"], case["Dk"], case["Dv"]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)  # noqa: E731
    if case["kind"] == "step":
        R = case["n"]
    else:
        lens = _lengths(case)
        R = sum(lens)
        s["lens"] = lens
        s["cu"] = torch.tensor([0] + lens).cumsum(0).to(device=dev, dtype=torch.int32)
    s["q"] = unit(normal(R, Hk, Dk)).to(dt)
    s["k"] = unit(normal(R, Hk, Dk)).to(dt)
    s["v"] = normal(R, H, Dv).to(dt)
    if case["per_head"]:
        # constant decays whose memory reaches from tens to thousands of tokens
        s["g"] = torch.log1p(-torch.exp2(-4.0 - 8.0 * (torch.rand((H,), generator=gen, device=dev) + torch.arange(H, device=dev)) / H))
    else:
        # data-dependent decays, now and then (a new document) one that forgets everything
        g = -torch.nn.functional.softplus(normal(R, H) - 3.0)
        s["g"] = torch.where(torch.rand((R, H), generator=gen, device=dev) < 2e-3, torch.full_like(g, -40.0), g)
    s["scale"] = 1.0 if Dk == 128 else 0.5
    if case["kind"] == "step":
        n, pad, slots = case["n"], case["pad"], case["slots"]
        s["state"] = 0.3 * normal(slots, H, Dk, Dv)
        s["new_state"] = torch.zeros_like(s["state"])
        pick = torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
        pick[n - pad:] = -1
        s["slots"] = pick.to(dev)
        return s
    N = case["n"]
    s["h0"] = 0.3 * normal(N, H, Dk, Dv) if case["states"] else None
    if case["kind"] == "bwd":
        s["do"] = normal(R, H, Dv).to(dt)
        s["dhT"] = 0.1 * normal(N, H, Dk, Dv) if case["states"] else None
    return s


def _meta(s):
    """This pass's own copy of the page table and the reference counts, so that a pass can be made again."""
    c, meta = s["case"], s["meta"].clone()
    cut = c["rows"] * c["per_row"]
    return meta[:cut].view(c["rows"], c["per_row"]), meta[cut:]


# ---- one pass ----------------------------------------------------------------------------------------------------

def run(s):
    kind = s["case"]["kind"]
    if own:
        return _OWN[kind](s)
    return _PLAIN[kind](s)


def _own_fwd(s):
    return _kda().linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], cu_seqlens=s["cu"],
                                   initial_state=s["h0"])


def _own_bwd(s):
    return _kda().linear_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], scale=s["scale"], cu_seqlens=s["cu"],
                                   initial_state=s["h0"], dfinal_state=s["dhT"])


def _own_step(s):
    o = _kda().linear_recurrent_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"], slots=s["slots"],
                                     new_state=s["new_state"])
    return o, s["new_state"]


def _own_copy(s):
    _kda().cache_copy(s["pools"], s["snap"], s["dst"], s["src"])
    return s["pools"]


def _own_fork(s):
    table, count = _meta(s)
    pages = _kda().cache_fork(s["pools"], table, count, s["parents"], s["children"])
    return table, count, pages, s["pools"]


def _own_free(s):
    table, count = _meta(s)
    _kda().cache_free(table, count, s["rows"])
    return table, count


def _own_compact(s):
    table, count = _meta(s)
    moved, n_live = _kda().cache_compact(s["pools"], table, count)
    return table, count, moved, n_live, s["pools"]


# ---- plain forms -------------------------------------------------------------------------------------------------

def _chunks(s):
    """Packed tokens cut into chunks that restart at every sequence: token index, which of them are there, the
    sequence of each chunk, each sequence's chunk count and first chunk."""
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    counts = (lens + CHUNK - 1) // CHUNK
    first = counts.cumsum(0) - counts
    nc = sum((n + CHUNK - 1) // CHUNK for n in s["lens"])
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=cu.device), counts, output_size=nc)
    pos = (torch.arange(nc, device=cu.device) - first[seq])[:, None] * CHUNK + torch.arange(CHUNK, device=cu.device)
    ok = pos < lens[seq][:, None]
    return torch.where(ok, cu[:-1][seq][:, None] + pos, 0), ok, seq, counts, first


def _cut(x, idx, ok, H):
    """[R, heads, D] -> [chunks, H, CHUNK, D] in float32, zero where no token is; shared heads repeated."""
    x = (x.float() * 1.0)[idx] * ok[..., None, None]
    return x.transpose(1, 2).repeat_interleave(H // x.shape[2], dim=1)


def _decays(s, idx, ok, seq, first):
    """In-chunk sums G, the lower triangle exp(G_i - G_j), chunk totals and the decay from the end of chunk b to the
    start of chunk a (b < a, same sequence), all from sums in float64."""
    c = s["case"]
    g = s["g"].double()
    g = g.expand(idx.shape + (c["H"],)) if g.dim() == 1 else g[idx]
    G = (g * ok[..., None]).transpose(1, 2).cumsum(-1)
    i = torch.arange(CHUNK, device=G.device)
    D = torch.where(i[:, None] >= i, torch.exp((G[..., :, None] - G[..., None, :]).clamp_max(0.0)).float(), 0.0)
    tot = G[..., -1]
    B = tot.cumsum(0).T                                   # [H, chunks], through chunk c
    before = torch.nn.functional.pad(B, (1, 0))[:, :-1]   # through chunk c - 1
    n = torch.arange(seq.numel(), device=G.device)
    M = torch.where((n[:, None] > n) & (seq[:, None] == seq),
                    torch.exp((before[:, :, None] - B[:, None, :]).clamp_max(0.0)).float(), 0.0)
    enter = torch.exp(before - before[:, first[seq].clamp_max(seq.numel() - 1)]).float().T  # from the sequence's start
    return G, D, tot, B, M, enter


def _states_in(M, U, enter, h0, seq):
    S = (M @ U.transpose(0, 1).flatten(2)).view(U.shape[1], U.shape[0], *U.shape[2:]).transpose(0, 1)
    return S if h0 is None else S + enter[..., None, None] * h0[seq]


def _put(x, idx, ok, like):
    """[chunks, H, CHUNK, D] -> rows [R, H, D] in like's type."""
    out = torch.empty((like.shape[0],) + (x.shape[1], x.shape[3]), dtype=torch.float32, device=x.device)
    out[idx[ok]] = x.transpose(1, 2)[ok]
    return out.to(like.dtype)


def _plain_fwd(s):
    c = s["case"]
    H = c["H"]
    idx, ok, seq, counts, first = _chunks(s)
    q, k, v = (_cut(s[x], idx, ok, H) for x in "qkv")
    if seq.numel():
        G, D, tot, _, M, enter = _decays(s, idx, ok, seq, first)
        o = s["scale"] * ((q @ k.transpose(-1, -2)) * D) @ v
        U = (k * torch.exp(tot[..., None] - G).float()[..., None]).transpose(-1, -2) @ v
        S = _states_in(M, U, enter, s["h0"], seq)
        o = o + s["scale"] * torch.exp(G).float()[..., None] * (q @ S)
        o = _put(o, idx, ok, s["v"])
        hT = torch.exp(tot).float()[..., None, None] * S + U
        hT = hT[(first + counts - 1).clamp_min(0)]
    else:
        o, hT = torch.empty_like(s["v"]), torch.zeros((c["n"], H, c["Dk"], c["Dv"]), device=q.device)
    empty = torch.zeros_like(hT) if s["h0"] is None else s["h0"]
    return o, torch.where((counts > 0)[:, None, None, None], hT, empty)


def _plain_bwd(s):
    c = s["case"]
    H, Hk, scale = c["H"], c["Hk"], s["scale"]
    idx, ok, seq, counts, first = _chunks(s)
    q, k, v, do = (_cut(s[x], idx, ok, H) for x in ("q", "k", "v", "do"))
    if not seq.numel():
        zero = torch.zeros((c["n"], H, c["Dk"], c["Dv"]), device=q.device) if s["dhT"] is None else s["dhT"]
        dg = torch.zeros_like(s["g"])
        return torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"]), dg, zero
    G, D, tot, B, M, enter = _decays(s, idx, ok, seq, first)
    w_in, w_out = torch.exp(G).float()[..., None], torch.exp(tot[..., None] - G).float()[..., None]
    qk, dv_ = q @ k.transpose(-1, -2), do @ v.transpose(-1, -2)
    S = _states_in(M, (k * w_out).transpose(-1, -2) @ v, enter, s["h0"], seq)
    U = scale * (q * w_in).transpose(-1, -2) @ do
    last = (first + counts - 1)[seq]
    leave = torch.exp(B[:, last] - B).float().T
    dS = _states_in(M.transpose(-1, -2), U, leave, s["dhT"], seq)
    dq_in = scale * w_in * (do @ S.transpose(-1, -2))
    dk_in = w_out * (v @ dS.transpose(-1, -2))
    dA = scale * dv_ * D
    dq, dk = dA @ k + dq_in, dA.transpose(-1, -2) @ q + dk_in
    dv = (scale * qk * D).transpose(-1, -2) @ do + w_out * (k @ dS)
    x = torch.tril(scale * qk * dv_ * D, -1)
    y = (q * dq_in).sum(-1) + x.sum(-1) - x.sum(-2)
    z = (k * dk_in).sum(-1)
    dg = y.flip(-1).cumsum(-1).flip(-1) + z.cumsum(-1) - z
    dg = dg + (torch.exp(tot).float() * (S * dS).sum((-1, -2)))[..., None]
    dg = _put(dg[..., None], idx, ok, s["g"].new_empty((s["q"].shape[0], 1)))[..., 0]
    if c["per_head"]:
        dg = dg.double().sum(0).float()
    share = lambda t: t.view(t.shape[0], Hk, H // Hk, *t.shape[2:]).sum(2)  # noqa: E731
    dh0 = (torch.exp(tot).float()[..., None, None] * dS + U)[first.clamp_max(seq.numel() - 1)]
    empty = torch.zeros_like(dh0) if s["dhT"] is None else s["dhT"]
    dh0 = torch.where((counts > 0)[:, None, None, None], dh0, empty)
    return _put(share(dq), idx, ok, s["q"]), _put(share(dk), idx, ok, s["k"]), _put(dv, idx, ok, s["v"]), dg, dh0


def _plain_step(s):
    H, slots = s["case"]["H"], s["slots"].long()
    there = slots >= 0
    q, k = (x.float().repeat_interleave(H // x.shape[1], dim=1) for x in (s["q"], s["k"]))
    S = s["state"][slots.clamp_min(0)]
    g = s["g"].expand(slots.numel(), H)
    S = torch.exp(g)[..., None, None] * S + k[..., None] * s["v"].float()[:, :, None, :]
    o = s["scale"] * (q[..., None] * S).sum(-2)
    n = slots.numel() - s["case"]["pad"]
    s["new_state"].index_copy_(0, slots[:n], S[:n])
    return torch.where(there[:, None, None], o, 0.0).to(s["v"].dtype), s["new_state"]


def _plain_copy(s):
    a, b = s["pools"]
    src, dst = s["src"].long(), s["dst"].long()
    a.index_copy_(0, dst, s["snap"][0].index_select(0, src))
    b.index_copy_(0, dst, s["snap"][1].index_select(0, src))
    return s["pools"]


def _plain_fork(s):
    table, count = _meta(s)
    rows = table[s["parents"].long()]
    cols = torch.arange(table.shape[1], device=table.device)
    tail = torch.where(rows >= 0, cols, -1).amax(-1)
    free = torch.sort((count > 0).to(torch.int8), stable=True).indices  # free pages first, lowest first
    need = tail >= 0
    at = need.cumsum(0) - 1
    fits = need & (at < (count == 0).sum())
    new = torch.where(fits, free[at.clamp(0, count.numel() - 1)], -1)
    shared = (rows >= 0) & (cols < tail[:, None]) & fits[:, None]
    count.scatter_add_(0, rows.clamp_min(0).long().flatten(), shared.int().flatten())
    count.scatter_add_(0, new.clamp_min(0), fits.int())
    kids = torch.where(cols == tail[:, None], new[:, None].int(), torch.where(shared, rows, -1))
    table.index_copy_(0, s["children"].long(), torch.where(fits[:, None], kids, -1))
    src = torch.gather(rows, 1, tail.clamp_min(0)[:, None])[:, 0].long()[fits]
    a, b = s["pools"]
    a[new[fits]] = a[src]
    b[new[fits]] = b[src]
    return table, count, new.int(), s["pools"]


def _plain_free(s):
    table, count = _meta(s)
    rows = s["rows"].long()
    held = table[rows].flatten()
    count.scatter_add_(0, held.clamp_min(0).long(), -(held >= 0).int())
    table.index_fill_(0, rows, -1)
    return table, count.clamp_min_(0)


def _plain_compact(s):
    table, count = _meta(s)
    live = count > 0
    n_live = live.sum()
    page = torch.arange(count.numel(), device=count.device)
    holes = (~live & (page < n_live)).nonzero()[:, 0]
    movers = (live & (page >= n_live)).nonzero()[:, 0]
    moved = torch.where(live, page, -1).index_copy_(0, movers, holes).int()
    a, b = s["pools"]
    a[holes] = a[movers]
    b[holes] = b[movers]
    count[holes] = count[movers]
    count[movers] = 0
    table.copy_(torch.where(table >= 0, moved[table.clamp_min(0).long()], -1))
    return table, count, moved, n_live.int().view(1), s["pools"]


_PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "copy": _plain_copy, "fork": _plain_fork,
          "free": _plain_free, "compact": _plain_compact}
_OWN = {"fwd": _own_fwd, "bwd": _own_bwd, "step": _own_step, "copy": _own_copy, "fork": _own_fork, "free": _own_free,
        "compact": _own_compact}


# ---- what a pass cannot do without ---------------------------------------------------------------------------------

def work(case):
    c = case
    if c["kind"] in ("copy", "fork", "free", "compact"):
        page = c["H"] * (4 * c["D"] * c["D"] + 2 * 9 * c["D"])
        tables = 4 * (c["rows"] * c["per_row"] + c["pages"])
        if c["kind"] == "copy":
            return {"bytes": 2 * c["m"] * page + 8 * c["m"], "flops": 0}
        if c["kind"] == "fork":
            return {"bytes": 2 * min(c["m"], c["rows"] // 2) * (page + 4 * c["per_row"]) + 4 * c["pages"], "flops": 0}
        if c["kind"] == "free":
            return {"bytes": 4 * 4 * c["m"] * c["per_row"], "flops": 0}
        # of the live pages (live * rows * (1 + per_row) / 2 of them), the share behind the front moves
        held = min(c["pages"], c["live"] * c["rows"] * (1 + c["per_row"]) / 2)
        return {"bytes": 2 * held * (1 - held / c["pages"]) * page + 2 * tables, "flops": 0}
    size = 2 if c["dtype"] == "bf16" else 4
    state = 4 * c["H"] * c["Dk"] * c["Dv"]
    if c["kind"] == "step":
        n = c["n"] - c["pad"]
        return {"bytes": n * (2 * state + size * (2 * c["Hk"] * c["Dk"] + 2 * c["H"] * c["Dv"])),
                "flops": 5 * n * c["H"] * c["Dk"] * c["Dv"]}
    R = sum(_lengths(c))
    g = 4 * c["H"] * (1 if c["per_head"] else R)
    if c["kind"] == "fwd":
        return {"bytes": R * size * (2 * c["Hk"] * c["Dk"] + 2 * c["H"] * c["Dv"]) + g + c["n"] * state * (1 + c["states"]),
                "flops": 4 * R * c["H"] * c["Dk"] * c["Dv"]}
    return {"bytes": R * size * (4 * c["Hk"] * c["Dk"] + 3 * c["H"] * c["Dv"]) + 2 * g + c["n"] * state * (1 + 2 * c["states"]),
            "flops": 10 * R * c["H"] * c["Dk"] * c["Dv"]}


# ---- the definition in 64 bits, token by token -----------------------------------------------------------------------

def exact(case, seed):
    if case["kind"] in ("copy", "fork", "free", "compact"):
        return None  # nothing is computed: values are moved
    s = prepare(case, seed)
    H = case["H"]
    wide = lambda x: x.double().repeat_interleave(H // x.shape[1], dim=1)  # noqa: E731
    q, k, v = wide(s["q"]) * s["scale"], wide(s["k"]), s["v"].double()
    a = torch.exp(s["g"].double()).expand(q.shape[0], H)[..., None, None]
    if case["kind"] == "step":
        o, new = torch.zeros_like(v), s["new_state"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                new[slot] = a[i] * s["state"][slot].double() + k[i][:, :, None] * v[i][:, None, :]
                o[i] = (q[i][:, :, None] * new[slot]).sum(1)
        return o, new
    lens = s["lens"]
    if max(lens) * (1 if case["kind"] == "fwd" else 3) > 140000:
        return None
    # sequences from the longest to the shortest: those that still have a token at step t are the first ones
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    start = s["cu"].long()[:-1][order]
    more = [0] * (max(lens) + 1)
    for n in lens:
        more[n] += 1
    active, alive = [], len(lens) - more[0]
    for t in range(max(lens)):
        active.append(alive)
        alive -= more[t + 1]
    S = torch.zeros((case["n"], H, case["Dk"], case["Dv"]), dtype=torch.float64, device=q.device)
    if s["h0"] is not None:
        S += s["h0"].double()[order]
    back = torch.empty(len(order), dtype=torch.long)
    back[order] = torch.arange(len(order))
    back = back.to(q.device)
    if case["kind"] == "fwd":
        o = torch.zeros_like(v)
        for t, m in enumerate(active):
            at = start[:m] + t
            X = S[:m].mul_(a[at]).addcmul_(k[at][..., None], v[at][:, :, None, :])
            o[at] = (q[at][..., None] * X).sum(-2)
        return o, S[back]
    do = s["do"].double()
    dq, dk, dv, dg = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(a[..., 0, 0])
    for t, m in enumerate(active):
        at = start[:m] + t
        X = S[:m].mul_(a[at]).addcmul_(k[at][..., None], v[at][:, :, None, :])
        dq[at] = (do[at][:, :, None, :] * X).sum(-1)
    dS = torch.zeros_like(S)
    if s["dhT"] is not None:
        dS += s["dhT"].double()[order]
    # R = <S_t, dL/dS_t>: scaling S_t scales what every earlier decay contributes
    R = (S * dS).sum((-1, -2))
    for t in reversed(range(len(active))):
        m = active[t]
        at = start[:m] + t
        X = dS[:m].addcmul_(q[at][..., None], do[at][:, :, None, :])
        dk[at] = (v[at][:, :, None, :] * X).sum(-1)
        dv[at] = (k[at][..., None] * X).sum(-2)
        r = R[:m] + (q[at] * dq[at]).sum(-1) - (k[at] * dk[at]).sum(-1)
        dg[at] = r
        R[:m] = r
        X.mul_(a[at])
    dq = dq * s["scale"]
    share = lambda t: t.view(t.shape[0], case["Hk"], -1, t.shape[-1]).sum(2)  # noqa: E731
    return share(dq), share(dk), dv, (dg.sum(0) if case["per_head"] else dg), dS[back]
