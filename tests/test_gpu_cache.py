"""GPU tests of the cache's page operators against plain page-by-page forms: contents and tables equal bit for bit."""
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


def _pools(n_pages, shapes, seed=0):
    """One pool per (dtype, page shape), random bits of small integers."""
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(-100, 100, (n_pages,) + s, generator=gen).to(dt).cuda() for dt, s in shapes]


# pages of 16-byte, 4-byte, 2-byte and 1-byte units, one byte to several slices
SHAPES = [(torch.float32, (2, 64, 64)), (torch.bfloat16, (3, 384)), (torch.float32, (5,)), (torch.bfloat16, (7,)),
          (torch.int8, (1,)), (torch.float32, (3, 5000)), (torch.int8, (33000 + 17,))]


def _np(pools):
    return [p.to(torch.float32).cpu().numpy() for p in pools]


def _same(pools, want):
    for i, (p, w) in enumerate(zip(pools, want)):
        assert np.array_equal(p.to(torch.float32).cpu().numpy(), w), i


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("n", [0, 1, 7, 300, 5000])
def test_copy_between_pools(n):
    import gated_delta_rule_20_amd as kda
    src, dst = _pools(40, SHAPES, 1), _pools(53, SHAPES, 2)
    r = np.random.RandomState(n)
    d, s = r.randint(-2, 55, n).tolist(), r.randint(-2, 42, n).tolist()   # repeats and pages out of range among them
    want, frm = _np(dst), _np(src)
    ref.pages_copy(want, frm, d, s)
    kda.cache_copy(dst, src, _i32(d), _i32(s))
    _same(dst, want)
    _same(src, frm)


def test_copy_within_a_pool_and_one_tensor():
    import gated_delta_rule_20_amd as kda
    pool = _pools(20, SHAPES[:1], 3)[0]
    want = _np([pool])
    ref.pages_copy(want, want, [10, 11, 12, 10], [0, 0, 1, 2])
    kda.cache_copy(pool, None, _i32([10, 11, 12, 10]), _i32([0, 0, 1, 2]))
    _same([pool], want)


def test_copy_beyond_4_gib():
    import gated_delta_rule_20_amd as kda
    pool = torch.zeros((4200, 1 << 18), device="cuda")     # 1 MiB pages
    pool[4199] = 3.0
    kda.cache_copy(pool, None, _i32([4100, 0]), _i32([4199, 4199]))
    assert float(pool[4100].min()) == 3.0 and float(pool[0].min()) == 3.0
    assert float(pool[1:4100].abs().max()) == 0.0 and float(pool[4101:4199].abs().max()) == 0.0


def _tables(rows, per_row, n_pages, seed, fill=0.6):
    """A random page table with shared pages, odd entries among them (-1 inside a row, a page out of range)."""
    r = np.random.RandomState(seed)
    table = np.full((rows, per_row), -1, np.int32)
    free = list(r.permutation(n_pages))
    count = np.zeros(n_pages, np.int32)
    for i in range(rows):
        if r.rand() > fill:
            continue
        for j in range(r.randint(0, per_row + 1)):
            if r.rand() < 0.2 and count.any():
                p = int(r.choice(np.nonzero(count)[0]))
            elif free and r.rand() < 0.95:
                p = int(free.pop())
            else:
                continue
            table[i, j] = p
            count[p] += 1
    return table, count


SIZES = [(1, 1, 1), (2, 3, 4), (12, 5, 60), (40, 70, 3000), (300, 4, 5000), (7, 1, 9)]   # rows, per_row, n_pages


def _fork(table, count, pools, parents, children):
    import gated_delta_rule_20_amd as kda
    wt, wc, wp = table.copy(), count.copy(), _np(pools)
    new = ref.pages_fork(wp, wt, wc, parents, children)
    t, c = torch.from_numpy(table).cuda(), torch.from_numpy(count).cuda()
    got = kda.cache_fork(pools, t, c, _i32(parents), _i32(children))
    assert got.tolist() == new
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(c.cpu().numpy(), wc)
    _same(pools, wp)
    return new


@pytest.mark.parametrize("rows,per_row,n_pages", SIZES)
def test_fork(rows, per_row, n_pages):
    table, count = _tables(rows, per_row, n_pages, rows + per_row)
    r = np.random.RandomState(rows)
    empty = [i for i in range(rows) if (table[i] < 0).all()]
    r.shuffle(empty)
    full = [i for i in range(rows) if i not in empty] or [0]
    parents = [int(r.choice(full)) for _ in empty]
    _fork(table, count, _pools(n_pages, SHAPES[:3], 4), parents, empty)


def test_fork_refuses_row_by_row():
    """Rows out of range, a child that is a parent, a child named twice, an empty parent, its own child."""
    table, count = _tables(10, 4, 40, 5, fill=1.0)
    table[6:] = -1
    count[:] = np.bincount(table[table >= 0], minlength=40)
    new = _fork(table, count, _pools(40, SHAPES[:2], 6), [0, 1, 2, -1, 0, 10, 3, 7, 4, 2], [6, 0, 7, 8, 6, 8, 7, 8, 4, 9])
    assert new[0] >= 0 and new[9] >= 0 and new.count(-1) == 8


def test_fork_when_pages_run_out():
    table = np.array([[0, 1, -1], [2, -1, -1], [-1, -1, -1], [-1, -1, -1], [5, 5, 5], [4, -1, -1]], np.int32)
    count = np.array([1, 1, 1, 0, 1, 3], np.int32)
    # page 3 alone is free: the first fork takes it, the fork of an empty row needs none, the next finds none
    new = _fork(table, count, _pools(6, SHAPES[:2], 7), [0, 2, 1], [3, 5, 2])
    assert new == [3, -1, -1]


def test_fork_many():
    """More forks than one planning pass holds (1024), more rows than pages left."""
    rows, n_pages = 2600, 1500
    table = np.full((rows, 2), -1, np.int32)
    table[0], table[1] = [0, 1], [2, -1]
    count = np.zeros(n_pages, np.int32)
    count[:3] = 1
    count[7] = -5                                       # a count below zero is a free page
    kids = list(range(2, rows))
    _fork(table, count, _pools(n_pages, SHAPES[2:3], 8), [i % 2 for i in kids], kids)


@pytest.mark.parametrize("rows,per_row,n_pages", SIZES)
def test_free(rows, per_row, n_pages):
    import gated_delta_rule_20_amd as kda
    table, count = _tables(rows, per_row, n_pages, 3 * rows)
    r = np.random.RandomState(rows)
    pick = r.randint(-1, rows + 1, max(1, rows // 2)).tolist() + [0, 0]
    count[0] = min(count[0], 1)                          # a broken count does not fall below 0
    wt, wc = table.copy(), count.copy()
    ref.pages_free(wt, wc, pick)
    t, c = torch.from_numpy(table).cuda(), torch.from_numpy(count).cuda()
    kda.cache_free(t, c, _i32(pick))
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(c.cpu().numpy(), wc)


@pytest.mark.parametrize("rows,per_row,n_pages", SIZES + [(50, 9, 4097), (3, 3, 12345)])
@pytest.mark.parametrize("fill", [0.0, 0.4, 1.0])
def test_compact(rows, per_row, n_pages, fill):
    import gated_delta_rule_20_amd as kda
    table, count = _tables(rows, per_row, n_pages, 5 * rows, fill)
    table.flat[0] = n_pages + 3                          # an entry out of range becomes -1
    pools = _pools(n_pages, SHAPES[:3], 9)
    wt, wc, wp = table.copy(), count.copy(), _np(pools)
    moved, n = ref.pages_compact(wp, wt, wc)
    t, c = torch.from_numpy(table).cuda(), torch.from_numpy(count).cuda()
    got, n_live = kda.cache_compact(pools, t, c)
    assert n_live.tolist() == [n] and np.array_equal(got.cpu().numpy(), moved)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(c.cpu().numpy(), wc)
    _same(pools, wp)


def test_pages_graph_replays():
    """Fork, free, compact and copy captured in one graph; each replay equals the eager calls."""
    import gated_delta_rule_20_amd as kda
    pools, snap = _pools(60, SHAPES[:3], 10), _pools(10, SHAPES[:3], 11)
    table, count = _tables(12, 5, 60, 17)
    empty = [i for i in range(12) if (table[i] < 0).all()]
    full = [i for i in range(12) if i not in empty]
    t, c = torch.from_numpy(table).cuda(), torch.from_numpy(count).cuda()
    pa, ch, fr = _i32([full[0]] * len(empty)), _i32(empty), _i32(full[:2])
    dp, sp = _i32([59, 58]), _i32([3, 9])

    def calls(pools, t, c):
        kda.cache_copy(pools, snap, dp, sp)
        new = kda.cache_fork(pools, t, c, pa, ch)
        kda.cache_free(t, c, fr)
        return new, *kda.cache_compact(pools, t, c)

    keep = [x.clone() for x in (*pools, t, c)]
    calls(pools, t, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(pools, t, c)
    for _ in range(3):
        for x, y in zip((*pools, t, c), keep):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        e = [x.clone() for x in keep]
        want = calls(e[:3], e[3], e[4])
        for x, y in zip((*pools, t, c, *out), (*e, *want)):
            assert torch.equal(x, y)
