"""GPU test of the linear-attention and cache entry points together, as a server uses them: a packed prefill that
leaves snapshots, private states copied out of them, forks, decode steps on slots, freed rows, a compaction in
between, and a training step (forward, then gradients) on what was generated.  Every sequence is followed token by token
in float64; tables and counts by plain page operations."""
import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_20_amd as kda
    kda.load_library()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("own_stream", [False, True])
def test_serve(dtype, own_stream):
    import gated_delta_rule_20_amd as kda
    H, Hk, D, pages, per_row, rows = 4, 2, 64, 24, 4, 10
    lens = [300, 64, 129, 700]
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    g = (-torch.rand(H, generator=gen) * 0.2)
    scale = 0.5
    stream = torch.cuda.Stream() if own_stream else torch.cuda.current_stream()

    # each sequence's tokens, as float64 arrays of what the kernels got
    def tokens(n):
        return dict(q=rnd(n, Hk, D).to(dtype), k=(rnd(n, Hk, D) / 8).to(dtype), v=rnd(n, H, D).to(dtype))
    prompts = [tokens(n) for n in lens]
    packed = {x: torch.cat([p[x] for p in prompts]).cuda() for x in "qkv"}
    cu = [0] + np.cumsum(lens).tolist()
    gd, cud = g.cuda(), _i32(cu)
    pool = torch.zeros((pages, H, D, D), device="cuda")
    extra = torch.randint(0, 100, (pages, 5), generator=gen).to(torch.int8).cuda()     # a second, odd-sized pool
    ck = torch.zeros((4, 3, H, D, D), device="cuda")
    torch.cuda.synchronize()
    history = {s: {x: ref.f64(p[x]) for x in "qkv"} for s, p in enumerate(prompts)}   # row -> its tokens

    def check(out, state, hist):
        a = [hist["q"], hist["k"], hist["v"], ref.f64(g)]
        n = a[0].shape[0]
        ro, rs = ref.forward(*a, scale, [0, n])
        mo, ms = ref.forward(np.abs(a[0]), np.abs(a[1]), np.abs(a[2]), a[3], scale, [0, n])
        assert np.all(np.abs(ref.f64(state) - rs[0]) <= ref.bound(rs[0], ms[0], torch.float32, n))
        if out is not None:
            assert np.all(np.abs(ref.f64(out) - ro[-1]) <= ref.bound(ro[-1], mo[-1], dtype, n))

    with torch.cuda.stream(stream):
        kw = dict(stream=stream if own_stream else None)
        # prefill, a snapshot every 128 tokens
        o, final = kda.linear_chunk_fwd(packed["q"], packed["k"], packed["v"], gd, scale=scale, cu_seqlens=cud,
                                        checkpoints=ck, checkpoint_every=2, **kw)
        # pages: row s holds its snapshots in order, then its private state
        table = np.full((rows, per_row), -1, np.int32)
        count = np.zeros(pages, np.int32)
        src, dst, nxt = [], [], 3
        for s, n in enumerate(lens):
            snaps = [j for j in range(3) if 128 * (j + 1) < n]
            for c, j in enumerate(snaps):
                src.append(s * 3 + j)
                dst.append(nxt)
                table[s, c], count[nxt], nxt = nxt, 1, nxt + 1
            table[s, len(snaps)], count[nxt], nxt = nxt, 1, nxt + 1
        kda.cache_copy(pool, ck.view(-1, H, D, D), _i32(dst), _i32(src), **kw)
        last = [int(table[s][table[s] >= 0][-1]) for s in range(4)]
        kda.cache_copy(pool, final, _i32(last), _i32([0, 1, 2, 3]), **kw)
        td, cd = torch.from_numpy(table).cuda(), torch.from_numpy(count).cuda()

        def slots_of(live):
            t = td.cpu().numpy()
            return [int(t[r][t[r] >= 0][-1]) for r in live]

        def decode(live, steps):
            for _ in range(steps):
                tok = tokens(len(live) + 2)                    # the batch is padded by two empty places
                d = {x: y.cuda() for x, y in tok.items()}
                slots = _i32(slots_of(live) + [-1, -1])
                out = kda.linear_recurrent_step(d["q"], d["k"], d["v"], gd, pool, scale=scale, slots=slots, **kw)
                assert float(out[len(live):].abs().max()) == 0.0
                for i, r in enumerate(live):
                    for x in "qkv":
                        history[r][x] = np.concatenate([history[r][x], ref.f64(tok[x][i:i + 1])])
            for i, (r, s) in enumerate(zip(live, slots_of(live))):
                check(out[i], pool[s], history[r])

        for s in range(4):
            check(o[cu[s + 1] - 1], pool[last[s]], history[s])
        decode([0, 1, 2, 3], 3)
        # two continuations of sequence 3, one of sequence 1
        wt, wc = td.cpu().numpy(), cd.cpu().numpy()
        new = kda.cache_fork([pool, extra], td, cd, _i32([3, 1, 3]), _i32([4, 5, 6]), **kw)
        assert new.tolist() == ref.pages_fork([], wt, wc, [3, 1, 3], [4, 5, 6])
        for a, c in ((3, 4), (1, 5), (3, 6)):
            history[c] = {x: y.copy() for x, y in history[a].items()}
        assert torch.equal(extra[new.long()], extra[_i32([slots_of([a])[0] for a in (3, 1, 3)]).long()])
        decode([0, 1, 2, 3, 4, 5, 6], 2)
        # sequences 0 and 3 end; the snapshots that 4 and 6 share with 3 stay
        kda.cache_free(td, cd, _i32([0, 3]), **kw)
        ref.pages_free(wt, wc, [0, 3])
        moved, n_live = kda.cache_compact([pool, extra], td, cd, **kw)
        wm, wn = ref.pages_compact([], wt, wc)
        assert n_live.tolist() == [wn] and moved.tolist() == wm.tolist()
        assert np.array_equal(td.cpu().numpy(), wt) and np.array_equal(cd.cpu().numpy(), wc)
        live = [1, 2, 4, 5, 6]
        decode(live, 2)
        # a snapshot still holds the prompt's state
        for r, c in ((4, 0), (6, 1)):
            check(None, pool[int(wt[r, c])], {x: y[:128 * (c + 1)] for x, y in history[3].items()})
        # a training step on the longest continuation
        h = history[4]
        n = h["q"].shape[0]
        x = {y: torch.from_numpy(h[y]).to(dtype).cuda()[None] for y in "qkv"}
        do = rnd(1, n, H, D).to(dtype).cuda()
        of, _ = kda.linear_chunk_fwd(x["q"], x["k"], x["v"], gd, scale=scale, **kw)
        check(of[0, -1], pool[slots_of([4])[0]], h)
        got = kda.linear_chunk_bwd(x["q"], x["k"], x["v"], gd, do, scale=scale, **kw)
        want = ref.backward(h["q"], h["k"], h["v"], ref.f64(g), ref.f64(do[0]), scale, [0, n])
        mags = ref.backward(*(np.abs(h[y]) for y in "qkv"), ref.f64(g), np.abs(ref.f64(do[0])), scale, [0, n])
        for a, b, m in zip(got[:3], want, mags):
            assert np.all(np.abs(ref.f64(a).reshape(b.shape) - b) <= ref.bound(b, m, dtype, n))
