"""GPU test of the gated scan, the norms around a block, 8-bit activations and the state cache as a recurrent model uses them:
a training step of two blocks (all gradients against float64 autograd of the definition), the same step from 8-bit
activations, prefill and decode on slots with a forked state."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FP, BF = torch.float32, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


def _kda():
    import gated_delta_rule_20_amd as kda
    return kda


def _params(D, C, layers, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    layer = lambda: dict(pre=1 + 0.1 * rnd(D), win=rnd(D, 2 * C) / D ** 0.5, A=0.3 * rnd(C), wout=rnd(C, D) / C ** 0.5,  # noqa: E731
                         wgate=rnd(D, D) / D ** 0.5, post=1 + 0.1 * rnd(D), res=0.7 + 0.1 * rnd(D))
    return [layer() for _ in range(layers)], 1 + 0.1 * rnd(D)


def _forward(kda, params, last, x, cu, pack=False):
    """Blocks: n = norm(x); (v, z) = n Win; h = scan(v, z); x = x + res Sigmoid(n Wgate) norm(h Wout).  Returns the last norm's
    output and what the backward pass needs."""
    kept = []
    x, n = kda.block_norm_fwd(x, pre_weight=params[0]["pre"])
    first = x
    for i, p in enumerate(params):
        rows = n @ p["win"]
        C = p["A"].shape[0]
        h, hT, *h8 = kda.gated_scan_fwd(rows[:, :C], rows[:, C:], A_log=p["A"], complement=True, cu_seqlens=cu, pack=pack)
        y, gate = h @ p["wout"], n @ p["wgate"]
        nxt = params[i + 1]["pre"] if i + 1 < len(params) else last
        x, n2, *saved = kda.block_norm_fwd(x, y, gate=gate, post_weight=p["post"], res_scale=p["res"], pre_weight=nxt, pack=pack)
        kept.append(dict(n=n, rows=rows, h=h, h8=h8[0] if pack else h, x8=kda.act_pack(rows[:, :C]) if pack else rows[:, :C],
                         saved=saved[0] if pack else (x, y, gate)))
        n = n2
    return n, (first, kept)


def _backward(kda, params, last, state, dn, cu):
    first, kept = state
    grads = [{} for _ in params]
    dx = torch.zeros_like(first)
    for i in reversed(range(len(params))):
        p, k, g = params[i], kept[i], grads[i]
        nxt = params[i + 1]["pre"] if i + 1 < len(params) else last
        xs, ys, gs = k["saved"]
        b = kda.block_norm_bwd(xs, ys, dx, dn, gate=gs, post_weight=p["post"], res_scale=p["res"], pre_weight=nxt, dtype=FP)
        g["post"], g["res"], g["next"] = b.dpost_weight, b.dres_scale, b.dpre_weight
        dx = b.dx
        g["wout"], g["wgate"] = k["h"].t() @ b.dy, k["n"].t() @ b.dgate
        C = p["A"].shape[0]
        drows = torch.empty_like(k["rows"])
        _, _, g["A"], _ = kda.gated_scan_bwd(k["x8"], k["rows"][:, C:], k["h8"], b.dy @ p["wout"].t(), A_log=p["A"], complement=True,
                                             cu_seqlens=cu, dx=drows[:, :C], dg=drows[:, C:])
        g["win"] = k["n"].t() @ drows
        dn = drows @ p["win"].t() + b.dgate @ p["wgate"].t()
    b = kda.block_norm_bwd(first, None, dx, dn, pre_weight=params[0]["pre"])
    return b.dx, b.dpre_weight, grads


def _definition(params, last, x, lens):
    rms = lambda v: v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)  # noqa: E731
    n = params[0]["pre"] * rms(x)
    for i, p in enumerate(params):
        v, z = (n @ p["win"]).chunk(2, -1)
        a = torch.exp(-5.0 * torch.sigmoid(torch.exp(p["A"]) * z))
        hs, at = [], 0
        for length in lens:
            h = torch.zeros_like(v[0])
            for t in range(at, at + length):
                h = a[t] * h + (1 - a[t]) * v[t]
                hs.append(h)
            at += length
        y = torch.stack(hs) @ p["wout"]
        x = x + p["res"] * torch.sigmoid(n @ p["wgate"]) * (p["post"] * rms(y))
        n = (params[i + 1]["pre"] if i + 1 < len(params) else last) * rms(x)
    return n


def _training(D=48, C=40, lens=(70, 1, 0, 100), seed=0):
    params, last = _params(D, C, 2, seed)
    gen = torch.Generator().manual_seed(seed + 1)
    T = sum(lens)
    x, dn = torch.randn(T, D, generator=gen), torch.randn(T, D, generator=gen)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    dev = [{k: v.cuda() for k, v in p.items()} for p in params]
    return params, last, dev, last.cuda(), x, dn, lens, cu


def test_training_step():
    """float32 against float64 autograd.  Every step is a few roundings (2^-24 each) and products of 48 terms (48 2^-24 = 3e-6 at
    worst); over two blocks and back 2e-5 in the 2-norm."""
    kda = _kda()
    params, last, dev, dlast, x, dn, lens, cu = _training()
    n, state = _forward(kda, dev, dlast, x.cuda(), cu)
    dx, dpre0, grads = _backward(kda, dev, dlast, state, dn.cuda(), cu)
    wide = [{k: v.double().requires_grad_(True) for k, v in p.items()} for p in params]
    wlast, wx = last.double().requires_grad_(True), x.double().requires_grad_(True)
    out = _definition(wide, wlast, wx, lens)
    (out * dn.double()).sum().backward()

    def near(a, b, what):
        b = b.detach()
        assert (a.double().cpu() - b).norm() <= 2e-5 * b.norm(), what
    near(n, out, "n")
    near(dx, wx.grad, "dx")
    near(dpre0, wide[0]["pre"].grad, "pre 0")
    for i, g in enumerate(grads):
        for k in ("post", "res", "wout", "wgate", "A", "win"):
            near(g[k], wide[i][k].grad, (i, k))
        near(g["next"], wide[i + 1]["pre"].grad if i + 1 < len(grads) else wlast.grad, (i, "next"))


def test_training_step_from_8_bits():
    """The same step with its activations kept in 8 bits: the forward pass is unchanged, the gradients are those that the values
    of the codes give (bit for bit but for the order of a product's roundings), and near the exact ones."""
    kda = _kda()
    params, last, dev, dlast, x, dn, lens, cu = _training(seed=5)
    n, state = _forward(kda, dev, dlast, x.cuda(), cu)
    n8, state8 = _forward(kda, dev, dlast, x.cuda(), cu, pack=True)
    assert torch.equal(n, n8)
    exact = _backward(kda, dev, dlast, state, dn.cuda(), cu)
    got = _backward(kda, dev, dlast, state8, dn.cuda(), cu)
    un = lambda t: kda.act_unpack(t, dtype=FP)  # noqa: E731
    values = (state8[0], [dict(k, h8=un(k["h8"]), x8=un(k["x8"]), saved=tuple(un(t) for t in k["saved"])) for k in state8[1]])
    want = _backward(kda, dev, dlast, values, dn.cuda(), cu)
    flat = lambda r: [r[0], r[1]] + [g[k] for g in r[2] for k in sorted(g)]  # noqa: E731
    for a, b, c in zip(flat(got), flat(want), flat(exact)):
        # a product contracted into the sum behind it saves one rounding of 2^-24 here and there
        assert (a - b).norm() <= 4e-6 * b.norm()
        # a code is off by amax / 254 at most, 1 / 254 of 3 to 4 standard deviations: 1% of each value in the 2-norm; the
        # gradients are products of a few of them, in two blocks
        assert (a - c).norm() <= 0.1 * c.norm()


def test_captured_training_step():
    """The whole step in a graph, replayed on fresh inputs, with eager work between the replays."""
    kda = _kda()
    params, last, dev, dlast, x, dn, lens, cu = _training(D=64, C=130, lens=(300, 5, 64), seed=9)
    x, dn = x.cuda(), dn.cuda()

    def step():
        n, state = _forward(kda, dev, dlast, x, cu, pack=True)
        dx, dpre, grads = _backward(kda, dev, dlast, state, dn, cu)
        return [n, dx, dpre] + [g[k] for g in grads for k in sorted(g)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(torch.randn_like(x))
        dn.copy_(torch.randn_like(dn))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b), i


def test_serving_with_state_cache():
    """Prefill of packed prompts into a pool of states, a fork of one sequence, decode steps on slots (with an empty place): as the
    whole sequences run at once, to float32."""
    kda = _kda()
    D, C = 32, 24
    params, last = _params(D, C, 1, 3)
    p = {k: v.cuda() for k, v in params[0].items()}
    last = last.cuda()
    lens, more = (17, 70, 5), 9
    gen = torch.Generator().manual_seed(4)
    xs = [torch.randn(n + more, D, generator=gen).cuda() for n in lens]
    fork = torch.cat([xs[1][:lens[1]], torch.randn(more, D, generator=gen).cuda()])

    def block(x, scan):
        x, n = kda.block_norm_fwd(x, pre_weight=p["pre"])
        rows = n @ p["win"]
        h = scan(rows[:, :C], rows[:, C:])
        return kda.block_norm_fwd(x, h @ p["wout"], gate=n @ p["wgate"], post_weight=p["post"], res_scale=p["res"], pre_weight=last)[1]
    whole = [block(x, lambda a, g: kda.gated_scan_fwd(a[None], g[None], A_log=p["A"])[0][0]) for x in xs + [fork]]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    states = torch.empty(3, C, device="cuda")
    prompt = torch.cat([x[:n] for x, n in zip(xs, lens)])
    out = block(prompt, lambda a, g: kda.gated_scan_fwd(a, g, A_log=p["A"], cu_seqlens=cu, final_state=states)[0])
    assert torch.allclose(out, torch.cat([w[:n] for w, n in zip(whole, lens)]), rtol=1e-4, atol=1e-4)
    # sequence s lives in page s of a pool of 8; row 3 continues row 1
    pool = torch.full((8, C), float("nan"), device="cuda")
    pool[:3] = states
    table = torch.full((4, 1), -1, dtype=torch.int32, device="cuda")
    table[:3, 0] = torch.arange(3)
    count = torch.tensor([1, 1, 1, 0, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kda.cache_fork([pool], table, count, ints(1), ints(3))
    slots = torch.cat([table[:, 0], ints(-1)])
    for t in range(more):
        x = torch.stack([s[n + t] for s, n in zip(xs + [fork], (*lens, lens[1]))] + [torch.zeros(D, device="cuda")])
        got = block(x, lambda a, g: kda.gated_scan_step(a, g, pool, A_log=p["A"], slots=slots))
        want = torch.stack([w[n + t] for w, n in zip(whole, (*lens, lens[1]))])
        assert torch.allclose(got[:4], want, rtol=1e-4, atol=1e-4), t


def test_linear_attention_from_8_bits():
    """linear_chunk_bwd takes q, k, v as they were kept in 8 bits."""
    kda = _kda()
    gen = torch.Generator().manual_seed(0)
    for dtype, D in ((BF, 128), (FP, 64)):
        q, k, v, do = (torch.randn(1, 200, 4, D, generator=gen).to(dtype).cuda() for _ in range(4))
        g = -torch.rand(1, 200, 4, generator=gen).cuda()
        qp, kp, vp = (kda.act_pack(t) for t in (q, k, v))
        got = kda.linear_chunk_bwd(qp, kp, vp, g, do)
        want = kda.linear_chunk_bwd(*(kda.act_unpack(t, dtype=dtype) for t in (qp, kp, vp)), g, do)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        mixed = kda.linear_chunk_bwd(q, kp, v, g, do)
        assert torch.equal(mixed[2], kda.linear_chunk_bwd(q, kda.act_unpack(kp, dtype=dtype), v, g, do)[2])
    with pytest.raises(ValueError):
        kda.linear_chunk_bwd((q, k), k, v, g, do)
