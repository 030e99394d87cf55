"""The entry points of linear attention and of the cache's pages reject bad arguments with a status before anything
is enqueued (CPU only: no call here reaches a kernel launch)."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_20_amd as kda


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_20_amd import build
        build.build()
    return kda.load_library()


def _message(lib):
    return lib.kda_last_error_message().decode()


def _step_args(**over):
    a = kda.LinearStepArgs(N=4, H=4, Hk=2, Dk=128, Dv=64, dtype=kda.KDA_BF16, scale=1.0, n_slots=8, g_per_head=0)
    for f in ("q", "k", "v", "g", "slots", "o"):
        setattr(a, f, 0x10000)
    a.state, a.new_state = 0x1000000, 0x1000000
    for key, val in over.items():
        setattr(a, key, val)
    return a


@pytest.mark.parametrize("over,status,msg", [
    (dict(Dk=96), 2, "head dims"),
    (dict(Dv=256), 2, "head dims"),
    (dict(dtype=2), 1, "dtype"),
    (dict(H=0), 1, "multiple"),
    (dict(Hk=0), 1, "multiple"),
    (dict(Hk=3), 1, "multiple"),
    (dict(N=-1), 1, "N >= 0"),
    (dict(N=1 << 29), 2, "too large"),
    (dict(n_slots=-1), 1, "n_slots"),
    (dict(slots=None, n_slots=3), 1, "at least N"),
    (dict(slots=0x10002), 1, "slots"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(g=None), 1, "g is NULL"),
    (dict(g=0x10001), 1, "g is not"),
    (dict(q=None), 1, "q is NULL"),
    (dict(k=0x10008), 1, "k is not 16-byte"),
    (dict(v=None), 1, "v is NULL"),
    (dict(state=None), 1, "state is NULL"),
    (dict(new_state=0x1000004), 1, "new_state is not"),
    (dict(new_state=0x1000000 + 8 * 4 * 128 * 64 * 4 - 16), 1, "overlaps"),
    (dict(new_state=0x1000000 - 16), 1, "overlaps"),
    (dict(o=None), 1, "o is NULL"),
])
def test_step_rejects(lib, over, status, msg):
    assert lib.kda_linear_recurrent_step(ctypes.byref(_step_args(**over)), None) == status
    assert msg in _message(lib)


def test_step_null_and_empty(lib):
    assert lib.kda_linear_recurrent_step(None, None) == 1
    assert lib.kda_linear_recurrent_step(ctypes.byref(_step_args(N=0, q=None, g=None, state=None)), None) == 0


def _pool(dst=0x100000, src=None, page=64):
    return (kda.CachePool * 1)(kda.CachePool(dst, src, page))


A = 0x10000  # an aligned address that nothing dereferences


@pytest.mark.parametrize("args,status,msg", [
    ((_pool(), -1, 4, 4, A, A, 1), 1, "n_pools"),
    ((_pool(), 9, 4, 4, A, A, 1), 1, "n_pools"),
    ((None, 1, 4, 4, A, A, 1), 1, "pools is NULL"),
    ((_pool(dst=None), 1, 4, 4, A, A, 1), 1, "pool 0 is NULL"),
    ((_pool(page=0), 1, 4, 4, A, A, 1), 1, "no page bytes"),
    ((_pool(page=1 << 41), 1, 4, 4, A, A, 1), 2, "1 TiB"),
    ((_pool(), 1, -1, 4, A, A, 1), 1, "page counts"),
    ((_pool(), 1, 4, 4, A, A, -1), 1, "n=-1"),
    ((_pool(), 1, 4, 4, None, A, 1), 1, "dst_pages is NULL"),
    ((_pool(), 1, 4, 4, A, A + 2, 1), 1, "src_pages is not"),
    ((_pool(src=0x100040), 1, 4, 4, A, A, 1), 1, "overlaps"),
    ((_pool(page=1 << 39), 1, 4, 4, A, A, 1 << 20), 2, "too many"),
])
def test_copy_rejects(lib, args, status, msg):
    assert lib.kda_cache_copy(*args, None) == status
    assert msg in _message(lib)


def test_cache_noops(lib):
    assert lib.kda_cache_copy(_pool(), 1, 4, 4, None, None, 0, None) == 0
    assert lib.kda_cache_copy(None, 0, 4, 4, A, A, 3, None) == 0
    assert lib.kda_cache_fork(_pool(), 1, 4, A, 2, 2, A, None, None, 0, None, None, None) == 0
    assert lib.kda_cache_free(A, 2, 2, A, 4, None, 0, None) == 0
    assert lib.kda_cache_free(None, 0, 2, A, 4, A, 3, None) == 0


@pytest.mark.parametrize("args,msg", [
    ((_pool(), 1, -1, A, 2, 2, A, A, A, 1, A, A), "n_pages"),
    ((_pool(), 1, 1 << 30, A, 2, 2, A, A, A, 1, A, A), "n_pages"),
    ((_pool(), 1, 4, A, -2, 2, A, A, A, 1, A, A), "rows"),
    ((_pool(), 1, 4, None, 2, 2, A, A, A, 1, A, A), "table is NULL"),
    ((_pool(), 1, 4, A, 2, 2, None, A, A, 1, A, A), "refcount is NULL"),
    ((_pool(), 1, 4, A + 1, 2, 2, A, A, A, 1, A, A), "4-byte"),
    ((_pool(), 1, 4, A, 2, 2, A, None, A, 1, A, A), "parents"),
    ((_pool(), 1, 4, A, 2, 2, A, A, None, 1, A, A), "children"),
    ((_pool(), 1, 4, A, 2, 2, A, A, A, -1, A, A), "n=-1"),
    ((_pool(), 1, 4, A, 2, 2, A, A, A, 1, None, A), "old_pages"),
    ((_pool(), 1, 4, A, 2, 2, A, A, A, 1, A, None), "new_pages"),
])
def test_fork_rejects(lib, args, msg):
    assert lib.kda_cache_fork(*args, None) == 1
    assert msg in _message(lib)


@pytest.mark.parametrize("args,msg", [
    ((A, 2, -1, A, 4, A, 1), "per_row"),
    ((None, 2, 2, A, 4, A, 1), "table is NULL"),
    ((A, 2, 2, None, 4, A, 1), "refcount is NULL"),
    ((A, 2, 2, A, 4, None, 1), "free_rows"),
])
def test_free_rejects(lib, args, msg):
    assert lib.kda_cache_free(*args, None) == 1
    assert msg in _message(lib)


@pytest.mark.parametrize("args,msg", [
    ((_pool(), 1, 4, None, 2, 2, A, A, A, A), "table is NULL"),
    ((_pool(), 1, 4, A, 2, 2, A, None, A, A), "moved_to"),
    ((_pool(), 1, 4, A, 2, 2, A, A, None, A), "moves"),
    ((_pool(), 1, 4, A, 2, 2, A, A, A, None), "counts"),
])
def test_compact_rejects(lib, args, msg):
    assert lib.kda_cache_compact(*args, None) == 1
    assert msg in _message(lib)


def test_binding_requires_device_tensors(lib):
    x, s = torch.zeros(3, 2, 64), torch.zeros(3, 2, 64, 64)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        kda.linear_recurrent_step(x, x, x, torch.zeros(2), s)
    with pytest.raises(ValueError, match="g must be"):
        kda.linear_recurrent_step(x, x, x, None, s)
    with pytest.raises(ValueError, match="k must be"):
        kda.linear_chunk_fwd(x, None, x, torch.zeros(2))
    with pytest.raises(ValueError, match="unsupported dtype"):
        kda.linear_recurrent_step(x.half(), x.half(), x.half(), torch.zeros(2), s)
    with pytest.raises(ValueError, match="device tensor"):
        kda.cache_copy(s, None, i, i)
    with pytest.raises(ValueError, match="pools"):
        kda.cache_copy([], None, i, i)
    with pytest.raises(ValueError, match="device tensor"):
        kda.cache_free(i.view(1, 3), i, i)


def _fwd_args(**over):
    a = kda.LinearFwdArgs(B=1, T=1000, H=4, Hk=2, Dk=128, Dv=64, dtype=kda.KDA_BF16, scale=1.0)
    for f in ("q", "k", "v", "g", "o"):
        setattr(a, f, 0x10000)
    a.workspace, a.workspace_bytes = 0x100000, 1 << 40
    for key, val in over.items():
        setattr(a, key, val)
    return a


def _bwd_args(**over):
    a = kda.LinearBwdArgs(B=1, T=1000, H=4, Hk=2, Dk=128, Dv=64, dtype=kda.KDA_BF16, scale=1.0)
    for f in ("q", "k", "v", "g", "d_o", "dq", "dk", "dv", "dg"):
        setattr(a, f, 0x10000)
    a.workspace, a.workspace_bytes = 0x100000, 1 << 40
    for key, val in over.items():
        setattr(a, key, val)
    return a


SHAPE_REFUSALS = [
    (dict(Dk=32), 2, "head dims"),
    (dict(Dv=100), 2, "head dims"),
    (dict(dtype=-1), 1, "dtype"),
    (dict(H=5), 1, "multiple"),
    (dict(Hk=0), 1, "multiple"),
    (dict(B=0), 1, "B >= 1"),
    (dict(T=-1), 1, "T >= 0"),
    (dict(scale=float("inf")), 1, "scale"),
    (dict(cu_seqlens=0x20000, B=2, N=1), 1, "B == 1"),
    (dict(cu_seqlens=0x20000, N=0), 1, "N >= 1"),
    (dict(cu_seqlens=0x20002, N=1), 1, "cu_seqlens"),
    (dict(B=1 << 16, T=1 << 16), 2, "too large"),
    (dict(cu_seqlens=0x20000, N=1 << 28), 2, "too large"),
]


@pytest.mark.parametrize("over,status,msg", SHAPE_REFUSALS + [
    (dict(q=None), 1, "q is NULL"),
    (dict(k=0x10008), 1, "k is not 16-byte"),
    (dict(o=None), 1, "o is NULL"),
    (dict(g=None), 1, "g is NULL"),
    (dict(g=0x10002), 1, "g is not 4-byte"),
    (dict(initial_state=0x10004), 1, "initial_state"),
    (dict(final_state=0x10004), 1, "final_state"),
    (dict(checkpoints=0x10004, checkpoint_every=1, checkpoint_slots=1), 1, "checkpoints is not"),
    (dict(checkpoints=0x10000, checkpoint_every=0, checkpoint_slots=1), 1, "checkpoint_every"),
    (dict(checkpoints=0x10000, checkpoint_every=1, checkpoint_slots=0), 1, "checkpoint_slots"),
    (dict(workspace=None), 3, "workspace is NULL"),
    (dict(workspace_bytes=1024), 3, "needs"),
    (dict(workspace=0x100010), 3, "256-byte"),
])
def test_forward_rejects(lib, over, status, msg):
    assert lib.kda_linear_chunk_fwd(ctypes.byref(_fwd_args(**over)), None) == status
    assert msg in _message(lib)


@pytest.mark.parametrize("over,status,msg", SHAPE_REFUSALS + [
    (dict(d_o=None), 1, "d_o is NULL"),
    (dict(dq=None), 1, "dq is NULL"),
    (dict(dv=0x10008), 1, "dv is not 16-byte"),
    (dict(dg=0x10002), 1, "dg is not"),
    (dict(d_final_state=0x10004), 1, "d_final_state"),
    (dict(d_initial_state=0x10004), 1, "d_initial_state"),
    (dict(workspace=None), 3, "workspace is NULL"),
    (dict(workspace_bytes=1 << 16), 3, "needs"),
])
def test_backward_rejects(lib, over, status, msg):
    assert lib.kda_linear_chunk_bwd(ctypes.byref(_bwd_args(**over)), None) == status
    assert msg in _message(lib)


def test_chunk_null_and_empty(lib):
    n = ctypes.c_size_t(0)
    assert lib.kda_linear_chunk_fwd(None, None) == 1 and lib.kda_linear_chunk_bwd(None, None) == 1
    assert lib.kda_linear_chunk_fwd_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.kda_linear_chunk_bwd_workspace_size(ctypes.byref(_bwd_args()), None) == 1
    assert lib.kda_linear_chunk_fwd(ctypes.byref(_fwd_args(T=0, q=None, g=None, o=None, workspace=None)), None) == 0


def test_workspace_sizes(lib):
    """No workspace for sequences that stay whole; otherwise one state per head for every segment that another follows,
    so that many short sequences need none per sequence."""
    def size(fn, a):
        n = ctypes.c_size_t(0)
        assert getattr(lib, fn)(ctypes.byref(a), ctypes.byref(n)) == 0, _message(lib)
        return n.value
    fwd, bwd = "kda_linear_chunk_fwd_workspace_size", "kda_linear_chunk_bwd_workspace_size"
    assert size(fwd, _fwd_args(T=128)) == 0
    one = 4 * 4 * 128 * 64                              # a state of every head
    assert size(fwd, _fwd_args(T=1000)) >= one
    packed = _fwd_args(T=1 << 20, cu_seqlens=0x20000, N=1 << 16)
    assert size(fwd, packed) <= ((1 << 20) // 256 + 1) * (one + 4096)
    assert size(bwd, _bwd_args(T=64, Hk=4, dg=None)) == 0
    assert size(bwd, _bwd_args(T=64, dg=None)) == 2 * 64 * 4 * 128 * 4    # shared heads: dq, dk per value head
    assert size(bwd, _bwd_args(T=64, Hk=4)) == 1024                       # y [64, 4]


def test_plans_of_the_largest_calls(lib):
    """Token and head counts at the limits plan without overflow."""
    n = ctypes.c_size_t(0)
    for over in (dict(T=2 ** 31 - 1, H=1 << 15, Hk=1), dict(T=2 ** 31 - 1, H=1, Hk=1), dict(T=1, H=1 << 15, Hk=1 << 15),
                 dict(T=2 ** 31 - 1, cu_seqlens=0x20000, N=(1 << 13) - 1, H=1 << 15, Hk=1), dict(B=1 << 12, T=1 << 18, H=1 << 12, Hk=1)):
        for fn, a in (("kda_linear_chunk_fwd_workspace_size", _fwd_args(**over)),
                      ("kda_linear_chunk_bwd_workspace_size", _bwd_args(dg=None, Hk=over["H"], **{k: v for k, v in over.items() if k != "Hk"}))):
            assert getattr(lib, fn)(ctypes.byref(a), ctypes.byref(n)) == 0, _message(lib)
            assert n.value < 1 << 50


# A launch has fewer than 2^32 threads: 2^24 - 1 workgroups of 256 or 2^23 - 1 of 512.  What is beyond is refused with the
# other checks, before the first of a call's kernels.

@pytest.mark.parametrize("over", [dict(H=64, N=1 << 18), dict(H=1, Hk=1, N=1 << 24), dict(H=1 << 15, N=(1 << 13) - 1)])
def test_forward_refuses_more_workgroups_than_a_launch_holds(lib, over):
    a = _fwd_args(cu_seqlens=0x20000, T=0, **over)
    assert lib.kda_linear_chunk_fwd(ctypes.byref(a), None) == 2
    assert "too many segments" in _message(lib)


@pytest.mark.parametrize("over", [dict(H=32, N=1 << 18), dict(H=1, Hk=1, N=1 << 23), dict(H=1 << 15, N=(1 << 13) - 1)])
def test_backward_refuses_more_workgroups_than_a_launch_holds(lib, over):
    a = _bwd_args(cu_seqlens=0x20000, T=0, **over)
    assert lib.kda_linear_chunk_bwd(ctypes.byref(a), None) == 2
    assert "too many segments" in _message(lib)


def test_largest_calls_of_one_launch_pass_the_check(lib):
    """One less, and the next check speaks (or, without anything to write, nothing does)."""
    fwd = _fwd_args(cu_seqlens=0x20000, T=0, H=1, Hk=1, N=(1 << 24) - 1)
    assert lib.kda_linear_chunk_fwd(ctypes.byref(fwd), None) == 0
    fwd.initial_state = 0x10004
    assert lib.kda_linear_chunk_fwd(ctypes.byref(fwd), None) == 1 and "initial_state" in _message(lib)
    bwd = _bwd_args(cu_seqlens=0x20000, T=0, H=1, Hk=1, N=(1 << 23) - 1, initial_state=0x10004)
    assert lib.kda_linear_chunk_bwd(ctypes.byref(bwd), None) == 1 and "initial_state" in _message(lib)


def test_step_and_pages_refuse_more_workgroups_than_a_launch_holds(lib):
    a = _step_args(N=1 << 22, q=None)
    assert lib.kda_linear_recurrent_step(ctypes.byref(a), None) == 2 and "too large" in _message(lib)
    a.N -= 1
    assert lib.kda_linear_recurrent_step(ctypes.byref(a), None) == 1 and "q is NULL" in _message(lib)
    big = _pool(page=(1 << 25) + 1)                         # 1025 pieces
    n = (1 << 24) // 1025 + 1
    assert lib.kda_cache_copy(big, 1, 4, 4, A, A, n, None) == 2 and "too many" in _message(lib)
    assert lib.kda_cache_fork(big, 1, 4, A, 2, 2, A, A, A, n, A, A, None) == 2 and "too many" in _message(lib)
    assert lib.kda_cache_copy(_pool(), 1, 4, 4, A, A, 1 << 24, None) == 2


def test_binding_refuses_missing_tensors(lib):
    """None in the place of a tensor that has to be given is a ValueError, as any other wrong argument."""
    s, i = torch.zeros(3, 2, 64, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="pool 0 must be a device tensor"):
        kda.cache_copy([None], None, i, i)
    with pytest.raises(ValueError, match="pool 0 must be a device tensor"):
        kda.cache_copy([s], [None], i, i)
    with pytest.raises(ValueError, match="table must be a device tensor"):
        kda.cache_free(None, i, i)
    for table, count, name in ((None, i, "table"), (i.view(1, 3), None, "table|refcount")):
        with pytest.raises(ValueError, match=name):
            kda.cache._tables(table, count, torch.device("cuda", 0))
    with pytest.raises(ValueError, match="rows must be a device tensor"):
        kda.cache._list(None, "rows", torch.device("cuda", 0))


class _Stream:
    device = torch.device("cuda", 1)


@pytest.mark.parametrize("call", [
    lambda t, i, s: kda.linear_recurrent_step(t, t, t, t, t, stream=s),
    lambda t, i, s: kda.linear_recurrent_step(scale=1.0, q=t, k=t, v=t, g=t, state=t, stream=s),
    lambda t, i, s: kda.linear_chunk_fwd(cu_seqlens=None, scale=0.5, q=t, k=t, v=t, g=t, stream=s),
    lambda t, i, s: kda.linear_chunk_bwd(need_dg=False, q=t, k=t, v=t, g=t, d_o=t, stream=s),
    lambda t, i, s: kda.cache_copy(t, None, i, i, stream=s),
    lambda t, i, s: kda.cache_copy([t], None, i, i, stream=s),
    lambda t, i, s: kda.cache_copy(src_pools=None, pools=[t], dst_pages=i, src_pages=i, stream=s),
    lambda t, i, s: kda.cache_free(rows=i, table=i, refcount=i, stream=s),
])
def test_stream_of_another_device(lib, call):
    """A stream that is not of the tensors' device is refused, in whatever order the call names its arguments."""
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cpu"):
        call(torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32), _Stream())
