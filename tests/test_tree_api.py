"""Drafted trees over a cache of pages on the CPU: pins of the oracle, the table of axes, and every refusal of the C ABI
and of engine.TreeBatch. Nothing is launched: refused calls return before, and the others have nothing to do."""
import contextlib
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as O

A = 1 << 20  # an aligned address that nobody reads


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


# ---- the oracle -------------------------------------------------------------------------------------
def test_chain_equals_the_causal_oracle():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(2, 12, 8)), rng.normal(size=(2, 12, 8))
    ref, _ = O.live_attn(q, k, v)
    np.testing.assert_allclose(O.tree_attn(q, k, v, np.tri(5, dtype=bool)), ref, rtol=1e-12)


def test_a_branch_equals_its_chain():
    """A node's output is that of the chain of its ancestors alone; a row that sees nothing gives zeros."""
    rng = np.random.default_rng(1)
    parent = [-1, 0, 0, 1, 2, 4]
    see, depth = O.ancestors(parent)
    assert depth.tolist() == [0, 1, 1, 2, 2, 3]
    q, k, v = rng.normal(size=(6, 2, 8)), rng.normal(size=(1, 9, 8)), rng.normal(size=(1, 9, 8))
    o = O.tree_attn(q, k, v, see)
    branch = [0, 2, 4, 5]
    rows = [0, 1, 2] + [3 + j for j in branch]
    chain, _ = O.live_attn(q[branch], k[:, rows], v[:, rows])
    np.testing.assert_allclose(o[branch], chain, rtol=1e-12)
    see[3] = False
    assert not O.tree_attn(q, k[:, 3:], v[:, 3:], see)[3].any()


def test_ancestors_by_hand():
    see, depth = O.ancestors([-1, 0, 5, 1, -1, 4])  # node 2's parent comes behind it: a root of its own
    want = ["100000", "110000", "001000", "110100", "000010", "000011"]
    assert ["".join("01"[int(x)] for x in row) for row in see] == want and depth.tolist() == [0, 1, 0, 2, 0, 1]
    assert O.pack_mask(np.eye(40, dtype=bool), 2)[[0, 31, 32, 39]].tolist() == [[1, 0], [-2 ** 31, 0], [0, 1], [0, 128]]


def test_axes_and_rotation():
    assert O.axes([2, 1, 1], False) == [0, 0, 1, 2] and O.axes([3, 1, 2], True) == [0, 1, 2, 0, 2, 0]
    rng = np.random.default_rng(2)
    x, f = rng.normal(size=(7, 2, 32)), O.rope_freqs("none", 16, 1e4)
    pos = rng.integers(0, 1000, size=7)
    for inter in (False, True):
        same = O.rope_axes(x, [pos, pos, pos], f, O.axes([4, 2, 2], True), inter, 1.25)
        np.testing.assert_array_equal(same, O.rope(x, pos, f, inter, 1.25))
    y = O.rope_axes(x, [pos, 0 * pos], f, O.axes([3, 5], False), False)
    np.testing.assert_array_equal(y[..., 3:8], x[..., 3:8])  # pairs of the axis that stands still
    np.testing.assert_allclose(y[..., 0] ** 2 + y[..., 8] ** 2, x[..., 0] ** 2 + x[..., 8] ** 2)


def test_acceptance_of_a_chain_equals_accept():
    rng = np.random.default_rng(3)
    for L in range(6):
        for _ in range(20):
            logits = rng.integers(0, 3, size=(L + 1, 4)).astype(np.float32)  # ties
            draft = rng.integers(0, 4, size=L)
            tokens, n = O.accept(logits, draft, L)
            path, out = O.accept_tree(logits, [9] + draft.tolist(), list(range(-1, L)), L + 1)
            assert out == list(tokens)[:n] and path == list(range(n))


def test_acceptance_takes_the_lowest_child_and_skips_nan():
    nan = float("nan")
    logits = np.array([[nan, 1, 5, 5], [nan] * 4, [0, 0, 0, 0], [9, 1, 2, 3]], np.float32)
    assert O.accept_tree(logits, [0, 2, 2, 0], [-1, 0, 0, 2], 4) == ([0, 1], [2, 0])
    assert O.accept_tree(logits, [0, 1, 2, 0], [-1, 0, 0, 2], 4) == ([0, 2, 3], [2, 0, 0])
    assert O.accept_tree(logits, [0, 1, 2, 0], [-1, 0, 0, 2], 0) == ([], [])


def test_pages_by_hand():
    p = O.Pages(8, 4, 3, 4, *(np.zeros((8, 1, 4, 2)) for _ in range(2)))
    p.reserve([(0, 6)])
    assert p.table[0, :2].tolist() == [0, 1] and p.n_free == 6
    for t in range(6):
        p.put(0, t, np.full((1, 1, 2), t + 1.0), np.full((1, 1, 2), -t - 1.0))
    p.commit([(0, 6, None, None, -1)])
    p.fork([(0, 1), (0, 2)])
    assert p.refs[:2].tolist() == [3, 3] and p.len.tolist() == [6, 6, 6]
    p.reserve([(1, 1), (2, 0), (0, 3)])  # 1 copies page 1, 2 asks for nothing, 0 copies it too and takes another
    assert p.table[1, :2].tolist() == [0, 2] and p.table[0, :3].tolist() == [0, 3, 4] and p.refs[:5].tolist() == [3, 1, 1, 1, 1]
    assert p.k[2, 0, :, 0].tolist() == [5, 6, 0, 0] and p.v[3, 0, :2, 1].tolist() == [-5, -6]
    for t, x in ((6, 7.0), (7, 8.0), (8, 9.0)):
        p.put(0, t, np.full((1, 1, 2), x), np.full((1, 1, 2), -x))
    p.commit([(0, 3, [0, 2, 1], 2, -1)])  # rows 6 and 8
    assert p.len[0] == 8 and p.k[3, 0, :, 0].tolist() == [5, 6, 7, 9]
    p.trim([(0, 5, 77), (1, 0, 0)])
    assert p.next.tolist() == [77, 0, 6] and p.held.tolist() == [2, 0, 2] and p.free[: p.n_free].tolist() == [7, 6, 5, 4, 2]
    p.check()
    p.compact()
    assert p.table[0, :2].tolist() == [0, 2] and p.table[2, :2].tolist() == [0, 1] and p.k[2, 0, 2, 0] == 7
    assert p.free[: p.n_free].tolist() == [7, 6, 5, 4, 3]
    p.check()
    p.reserve([(1, 17), (2, 99)])
    assert p.faults == 2


def test_pages_of_any_life_stay_counted():
    rng = np.random.default_rng(4)
    p = O.Pages(30, 16, 6, 12)
    for _ in range(400):
        s, t = rng.choice(6, 2, replace=False)
        op = rng.integers(5)
        if op == 0:
            p.reserve([(s, int(rng.integers(60)))])
        elif op == 1:
            p.fork([(s, t)])
        elif op == 2:
            p.trim([(s, int(rng.integers(100)), 0)])
        elif op == 3:
            p.compact()
        else:
            room = p.held[s] * 16 - p.len[s]
            p.commit([(s, int(rng.integers(room + 1)), None, None, -1)])
        p.check()


def test_a_commit_of_rows_that_are_not_there_leaves_the_sequence():
    """A page that others hold, or fewer pages than the rows take: nothing becomes context, with a path and without."""
    p = O.Pages(4, 4, 3, 4, *(np.zeros((4, 1, 4, 2)) for _ in range(2)))
    p.reserve([(0, 6)])
    p.commit([(0, 6, None, None, -1)])
    p.fork([(0, 1)])
    p.reserve([(2, 8), (1, 1)])  # none is left for 1's copy of the second page
    p.commit([(1, 1, None, None, 5), (0, 2, [0, 1], 2, -1), (2, 9, None, 1, -1)])
    assert p.faults == 4 and p.len.tolist() == [6, 6, 0] and p.next.tolist() == [6, 6, 0]
    p.trim([(2, 0, 0)])
    p.reserve([(1, 1)])
    p.commit([(1, 1, None, None, 5), (0, 2, [0, 1], 2, -1), (2, 0, None, None, 9)])
    assert p.faults == 4 and p.len.tolist() == [8, 7, 0] and p.next.tolist() == [8, 11, 0]
    p.check()


# ---- the table of axes ----------------------------------------------------------------------------
@pytest.mark.parametrize("sections", [[32], [16, 16], [12, 10, 10], [0, 32, 0], [8, 8, 8, 8], [1, 30, 1]])
@pytest.mark.parametrize("dealt", [False, True])
def test_axes_init(vc, sections, dealt):
    rope = vc.vc_rope_init(vc.VC_ROPE_NONE, 64, base=500000.0)
    t = vc.vc_rope_axes_init(rope, sections, dealt)
    assert list(t.axis)[:32] == O.axes(sections, dealt) and t.n_axes == len(sections)
    assert list(t.rope.freq) == list(rope.freq)


def test_axes_init_refusals(vc):
    rope = vc.vc_rope_init(vc.VC_ROPE_NONE, 64)
    for sections in ([], [31], [33], [-1, 33], [8] * 5, [2 ** 31 - 1, 2 ** 31 - 1]):
        with pytest.raises(vc.VCError):
            vc.vc_rope_axes_init(rope, sections)
    lib, out, sec = vc.lib_handle(), vc.vc_rope_axes(), (ctypes.c_int32 * 1)(32)
    ref = ctypes.byref
    assert lib.vc_rope_axes_init(None, 1, sec, 0, ref(out)) == vc.VC_ERR_INVALID
    assert lib.vc_rope_axes_init(ref(rope), 1, None, 0, ref(out)) == vc.VC_ERR_INVALID
    assert lib.vc_rope_axes_init(ref(rope), 1, sec, 0, None) == vc.VC_ERR_INVALID
    assert lib.vc_rope_axes_init(ref(rope), 1, sec, 2, ref(out)) == vc.VC_ERR_INVALID
    rope.rot_dim = 24
    assert lib.vc_rope_axes_init(ref(rope), 1, sec, 0, ref(out)) == vc.VC_ERR_UNSUPPORTED


# ---- refusals of the C ABI ------------------------------------------------------------------------
def _pool(vc, **kw):
    f = dict(k=A, v=2 * A, refs=3 * A, free_pages=4 * A, n_free=5 * A, table=6 * A, len=7 * A, held=8 * A, next=9 * A,
             n_pages=100, page=16, n_seq=10, max_pages=20)
    return vc.vc_paged_kv(**{**f, **kw})


def _calls(vc, shape=None, kv=None):
    """Every call of a pool with one request that has nothing wrong, by name."""
    shape, kv = shape or vc.vc_shape(1, 8, 2, 64), kv or _pool(vc)
    kw = dict(stream=0, raise_on_error=False)
    n = max(1, min(shape.B, 64))
    reqs = lambda t, make: (t * n)(*[make(b) for b in range(n)])
    axes = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, 64), [32])
    rope = lambda b: vc.vc_rope_page_req(seq=b % 10)
    return {
        "reserve": lambda: vc.vc_pages_reserve(shape, kv, reqs(vc.vc_reserve_req, lambda b: vc.vc_reserve_req(b % 10, 1)), **kw),
        "fork": lambda: vc.vc_pages_fork(shape, kv, reqs(vc.vc_fork_req, lambda b: vc.vc_fork_req(5, 5)), **kw),
        "trim": lambda: vc.vc_pages_trim(shape, kv, reqs(vc.vc_trim_req, lambda b: vc.vc_trim_req(b % 10, -1, 0)), **kw),
        "compact": lambda: vc.vc_pages_compact(shape, kv, **kw),
        "rope": lambda: vc.vc_rope_pages(shape, axes, kv, reqs(vc.vc_rope_page_req, rope), **kw),
        "attn": lambda: vc.vc_tree_attn(shape, kv, reqs(vc.vc_tree_req, lambda b: vc.vc_tree_req(seq=b % 10)), **kw),
        "commit": lambda: vc.vc_tree_commit(shape, kv, reqs(vc.vc_commit_req, lambda b: vc.vc_commit_req(seq=b % 10)), **kw),
    }


@pytest.mark.parametrize("dims,err", [((0, 8, 2, 64), 1), ((33, 8, 2, 64), 1), ((1, 8, 3, 64), 1), ((1, 2, 4, 64), 1),
                                      ((1, 8, 0, 64), 1), ((1, 8, 2, 96), 2), ((1, 65536, 65536, 64), 2)])
def test_shapes_refused(vc, dims, err):
    s = vc.vc_shape(*dims)
    for name, call in _calls(vc, shape=s).items():
        assert call() == err, name
    assert vc.vc_pages_init(s, _pool(vc), stream=0, raise_on_error=False) == err
    assert vc.vc_pages_workspace_size(s, _pool(vc)) == 0 and vc.vc_tree_workspace_size(s, 1) == 0


@pytest.mark.parametrize("field,value,err", [
    *[(f, v, 1) for f in ("k", "v") for v in (None, A + 8)],
    *[(f, v, 1) for f in ("refs", "free_pages", "n_free", "table", "len", "held", "next") for v in (None, A + 2)],
    ("n_pages", 0, 1), ("n_seq", 0, 1), ("max_pages", 0, 1), ("n_pages", -1, 1),
    *[("page", p, 2) for p in (0, 1, 8, 17, 24, 256, -16)],
    ("n_pages", 2 ** 30, 2), ("n_pages", 2 ** 30 - 1, 2), ("max_pages", 2 ** 26 + 1, 2)])
def test_pools_refused(vc, field, value, err):
    kv = _pool(vc, **{field: value})
    for name, call in _calls(vc, kv=kv).items():
        assert call() == err, name
    assert vc.vc_pages_init(vc.vc_shape(1, 8, 2, 64), kv, stream=0, raise_on_error=False) == err
    assert vc.vc_pages_workspace_size(vc.vc_shape(1, 8, 2, 64), kv) == 0


def test_calls_with_nothing_wrong_but_what_they_lack(vc):
    got = {name: call() for name, call in _calls(vc).items()}
    ok, inv, ws = vc.VC_OK, vc.VC_ERR_INVALID, vc.VC_ERR_WORKSPACE
    # no workspace; a fork onto itself; fewer than no rows; nothing to do
    assert got == {"reserve": ws, "fork": inv, "trim": inv, "compact": ws, "rope": ok, "attn": ok, "commit": ok}


def test_requests_name_sequences_of_the_pool_once(vc):
    shape, kv, kw = vc.vc_shape(2, 8, 2, 64), _pool(vc), dict(stream=0, raise_on_error=False)
    axes = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, 64), [32])
    for a, b in ((3, 3), (0, 10), (-1, 0)):
        for call, t, extra in ((vc.vc_pages_reserve, vc.vc_reserve_req, ()), (vc.vc_pages_trim, vc.vc_trim_req, ()),
                               (vc.vc_tree_commit, vc.vc_commit_req, ()), (vc.vc_rope_pages, vc.vc_rope_page_req, (axes,))):
            arr = (t * 2)(t(seq=a), t(seq=b))
            assert call(shape, *extra, kv, arr, **kw) == vc.VC_ERR_INVALID, (call, a, b)
    one = (vc.vc_tree_req * 2)(vc.vc_tree_req(seq=0), vc.vc_tree_req(seq=10))
    assert vc.vc_tree_attn(shape, kv, one, **kw) == vc.VC_ERR_INVALID
    fork = lambda *pairs: vc.vc_pages_fork(vc.vc_shape(len(pairs), 8, 2, 64), kv,
                                           (vc.vc_fork_req * len(pairs))(*[vc.vc_fork_req(*p) for p in pairs]), **kw)
    for pairs in (((1, 1),), ((1, 2), (3, 2)), ((1, 2), (2, 3)), ((2, 3), (1, 2)), ((0, 10),), ((-1, 0),), ((10, 1),)):
        assert fork(*pairs) == vc.VC_ERR_INVALID, pairs
    for call, t in ((vc.vc_pages_reserve, vc.vc_reserve_req), (vc.vc_pages_fork, vc.vc_fork_req), (vc.vc_pages_trim, vc.vc_trim_req),
                    (vc.vc_tree_attn, vc.vc_tree_req), (vc.vc_tree_commit, vc.vc_commit_req)):
        assert call(shape, kv, None, **kw) == vc.VC_ERR_INVALID
    assert vc.vc_pages_reserve(vc.vc_shape(1, 8, 2, 64), kv, (vc.vc_reserve_req * 1)(vc.vc_reserve_req(0, -1)), **kw) == 1


def test_trim_counts_its_pages_in_32_bits(vc):
    kv = _pool(vc, max_pages=2 ** 26, n_seq=32)
    arr = (vc.vc_trim_req * 32)(*[vc.vc_trim_req(i, 0, 0) for i in range(32)])
    assert vc.vc_pages_trim(vc.vc_shape(32, 8, 2, 64), kv, arr, stream=0, raise_on_error=False) == vc.VC_ERR_UNSUPPORTED


@pytest.mark.parametrize("B,max_pages,err", [(32, 2 ** 26 - 1, 2), (32, 2 ** 26 - 32, 2), (32, 2 ** 26 - 33, 1), (31, 2 ** 26, 1)])
def test_trim_steps_stay_in_32_bits(vc, B, max_pages, err):
    """The kernel goes through the pages 1024 at a time: the number behind the last step counts too. (Sizes within the
    limit get as far as the request for fewer than no rows.)"""
    arr = (vc.vc_trim_req * B)(*[vc.vc_trim_req(i, -1, 0) for i in range(B)])
    kv = _pool(vc, max_pages=max_pages, n_seq=32)
    assert vc.vc_pages_trim(vc.vc_shape(B, 8, 2, 64), kv, arr, stream=0, raise_on_error=False) == err


def _rope(vc, axes="ok", **kw):
    if axes == "ok":
        axes = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, 64), [16, 16])
    f = dict(q=10 * A, k=11 * A, v=12 * A, q_stride=0, k_stride=0, v_stride=0, off=None, off_stride=0, q_out=13 * A, seq=3, n_rows=2)
    arr = (vc.vc_rope_page_req * 1)(vc.vc_rope_page_req(**{**f, **kw}))
    return vc.vc_rope_pages(vc.vc_shape(1, 8, 2, 64), axes, _pool(vc), arr, stream=0, raise_on_error=False)


def test_rope_pages_refusals(vc):
    ok, inv, uns = vc.VC_OK, vc.VC_ERR_INVALID, vc.VC_ERR_UNSUPPORTED
    assert _rope(vc, n_rows=0) == ok and _rope(vc, n_rows=-1) == inv
    for f in ("q", "k", "v", "q_out"):
        assert _rope(vc, **{f: A + 8}) == inv and _rope(vc, **{f: None}) == inv
    assert _rope(vc, off=A + 2) == inv and _rope(vc, off=A, off_stride=1) == inv and _rope(vc, off=A, off_stride=-2) == inv
    assert _rope(vc, q_stride=8 * 64 - 8) == inv and _rope(vc, k_stride=2 * 64 + 4) == inv and _rope(vc, v_stride=64) == inv
    assert _rope(vc, q_out=10 * A, q_stride=1024) == inv  # in place needs packed rows
    assert _rope(vc, axes=None) == inv and _rope(vc, n_rows=2 ** 30 + 1) == uns
    make = lambda rot=64: vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, rot), [rot // 2])
    assert _rope(vc, axes=make(128)) == uns  # more rotated channels than d
    for change in (lambda t: setattr(t, "n_axes", 0), lambda t: setattr(t, "n_axes", 5), lambda t: t.axis.__setitem__(3, 1),
                   lambda t: t.axis.__setitem__(3, -1), lambda t: setattr(t.rope, "layout", 5),
                   lambda t: setattr(t.rope, "amp", 1e300), lambda t: t.rope.freq.__setitem__(3, math.nan)):
        t = make()
        change(t)
        assert _rope(vc, axes=t) == inv


def _attn(vc, shape=None, kv=None, **kw):
    f = dict(q=10 * A, o=11 * A, mask=None, mask_words=0, seq=3, n_rows=2)
    arr = (vc.vc_tree_req * 1)(vc.vc_tree_req(**{**f, **kw}))
    return vc.vc_tree_attn(shape or vc.vc_shape(1, 8, 2, 64), kv or _pool(vc), arr, stream=0, raise_on_error=False)


def test_tree_attn_refusals(vc):
    inv, uns = vc.VC_ERR_INVALID, vc.VC_ERR_UNSUPPORTED
    assert _attn(vc, n_rows=0) == vc.VC_OK and _attn(vc, n_rows=-1) == inv
    for f in ("q", "o"):
        assert _attn(vc, **{f: A + 8}) == inv and _attn(vc, **{f: None}) == inv
    assert _attn(vc, mask=A + 2, mask_words=1) == inv and _attn(vc, mask=A) == inv
    assert _attn(vc, mask=A, mask_words=1, n_rows=33) == inv and _attn(vc, mask=A, mask_words=-1) == inv
    assert _attn(vc) == vc.VC_ERR_WORKSPACE
    assert _attn(vc, n_rows=2 ** 26 + 1) == uns
    assert _attn(vc, shape=vc.vc_shape(1, 2048, 2048, 64), kv=_pool(vc, page=128, max_pages=2 ** 23)) == uns  # 2^34 tiles
    assert vc.vc_tree_workspace_size(vc.vc_shape(1, 8, 2, 64), 0) == 0


@pytest.mark.parametrize("B,Hq,Hkv,n_rows", [(1, 8, 8, 1), (1, 8, 2, 256), (1, 4, 4, 300), (32, 2, 2, 9), (4, 64, 8, 40),
                                             (1, 64, 64, 200)])
def test_tree_attn_takes_tables_up_to_the_headers_sum(vc, B, Hq, Hkv, n_rows):
    """Accepted (up to the workspace that is not there) at 2^29 of the header's sum, refused from 2^32 on."""
    kw = dict(stream=0, raise_on_error=False)
    arr = (vc.vc_tree_req * B)(*[vc.vc_tree_req(q=A, o=A, seq=b % 10, n_rows=n_rows) for b in range(B)])
    call = lambda rows: vc.vc_tree_attn(vc.vc_shape(B, Hq, Hkv, 64), _pool(vc, max_pages=rows // 128, page=128), arr, **kw)
    per = B * Hkv * -(-(n_rows * Hq // Hkv) // 256)  # sixteenths of the sum for each row of the table
    most = min(2 ** 30, 2 ** 29 * 16 // per // 128 * 128)
    assert call(most) == vc.VC_ERR_WORKSPACE
    if 2 ** 32 * 16 // per <= 2 ** 30:
        assert call(2 ** 32 * 16 // per) == vc.VC_ERR_UNSUPPORTED


def test_tree_workspace_does_not_grow_with_the_call(vc):
    """Two slots a CTA hold every partial, however many requests, heads and rows there are."""
    size = lambda B, Hq, Hkv, rows: vc.vc_tree_workspace_size(vc.vc_shape(B, Hq, Hkv, 128), rows)
    assert 0 < size(1, 8, 1, 1) <= size(1, 8, 1, 2) <= size(1, 8, 1, 40)
    assert size(1, 8, 1, 40) == size(32, 64, 8, 40) == size(32, 64, 8, 100000) < 64 << 20


def test_trees_refused(vc):
    inv, uns, kw = vc.VC_ERR_INVALID, vc.VC_ERR_UNSUPPORTED, dict(stream=0, raise_on_error=False)
    mask = lambda B=1, N=4, a=(A, 2 * A, 3 * A, 4 * A): vc.vc_tree_mask(B, N, *a, **kw)
    accept = lambda B=1, N=4, V=10, a=(A,) * 7: vc.vc_tree_accept(B, N, V, *a, **kw)
    for call in (mask, accept):
        assert call(B=0) == inv and call(N=0) == inv and call(N=1025) == uns and call(B=2 ** 21, N=1024) == uns
    for i in range(3):
        assert mask(a=tuple(None if j == i else A for j in range(4))) == inv
    for i in range(4):
        assert mask(a=tuple(A + 2 if j == i else A for j in range(4))) == inv
    assert accept(V=0) == inv
    for i in range(7):
        for bad in (None, A + 2):
            assert accept(a=tuple(bad if j == i else A for j in range(7))) == inv


def test_commit_refusals(vc):
    kw = dict(stream=0, raise_on_error=False)
    call = lambda **f: vc.vc_tree_commit(vc.vc_shape(1, 8, 2, 64), _pool(vc),
                                         (vc.vc_commit_req * 1)(vc.vc_commit_req(**{**dict(seq=1, n_rows=2), **f})), **kw)
    for f in (dict(n_rows=-1), dict(path=A + 2), dict(n_acc=A + 1)):
        assert call(**f) == vc.VC_ERR_INVALID


def test_descriptors_have_the_headers_sizes(vc, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ["vc_paged_kv", "vc_reserve_req", "vc_fork_req", "vc_trim_req", "vc_rope_axes", "vc_rope_page_req", "vc_tree_req",
             "vc_commit_req"]
    src = tmp_path / "s.cpp"
    src.write_text('#include <stdio.h>\n#include "vc.h"\nint main() {\n' +
                   "".join('printf("%%zu\\n", sizeof(%s));\n' % n for n in names) + "}\n")
    subprocess.run(["g++", "-I", os.path.join(root, "include"), "-I", "/usr/local/cuda/include", str(src), "-o",
                    str(tmp_path / "s")], check=True)
    out = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(getattr(vc, n)) for n in names]


def test_paged_kv_refuses_what_is_too_small(vc):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    k = torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16)
    good = [k, k.clone(), i(6), i(6), i(1), i(3, 4), i(3), i(3), i(3)]
    kv = vc.paged_kv(*good)
    assert (kv.n_pages, kv.page, kv.n_seq, kv.max_pages) == (6, 16, 3, 4)
    for at, bad in ((0, k[:, :, ::2]), (1, k[:3]), (2, i(5)), (3, i(5)), (4, i(0)), (5, i(3, 8)[:, ::2]), (6, i(2)), (7, i(2)), (8, i(2))):
        with pytest.raises(ValueError):
            vc.paged_kv(*[bad if j == at else t for j, t in enumerate(good)])


# ---- the engine, with the library's calls recorded -------------------------------------------------
class _Event:
    def record(self, *_):
        pass


@pytest.fixture
def calls(vc, monkeypatch):
    from lossless_compressed_kv_vc_gb300 import engine
    made = []
    monkeypatch.setattr(torch.cuda, "Event", _Event)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    for name, at in (("vc_pages_reserve", 2), ("vc_pages_fork", 2), ("vc_pages_trim", 2), ("vc_rope_pages", 3), ("vc_tree_attn", 2),
                     ("vc_tree_commit", 2), ("vc_pages_init", None), ("vc_pages_compact", None), ("vc_tree_mask", None),
                     ("vc_tree_accept", None)):
        def call(*args, _name=name, _at=at, **kw):
            made.append((_name, [type(e).from_buffer_copy(e) for e in args[_at]] if _at else args))
            return 0
        monkeypatch.setattr(engine, name, call)
    return made


HQ, HKV, D = 8, 2, 64


def trees(vc, axes=(32,), **kw):
    from lossless_compressed_kv_vc_gb300 import engine
    table = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, D), list(axes))
    return engine.TreeBatch(HQ, HKV, D, **{**dict(n_seq=4, n_pages=20, page=16, axes=table, max_rows=8, device="cpu"), **kw})


def new(heads, B=2, R=8):
    return torch.zeros((B, R, heads, D), dtype=torch.bfloat16)


def test_engine_passes_its_tensors_on(vc, calls):
    tb = trees(vc, axes=(12, 10, 10))
    x = torch.zeros((2, 8, (HQ + 2 * HKV) * D), dtype=torch.bfloat16)
    q, k, v = (t.unflatten(2, (-1, D)) for t in x.split([HQ * D, HKV * D, HKV * D], 2))
    off = torch.zeros((2, 3, 8), dtype=torch.int32)
    tb.append([3, 1], q, k, v, [8, 2], off)
    name, arr = calls[-1]
    assert name == "vc_rope_pages" and [(e.seq, e.n_rows) for e in arr] == [(3, 8), (1, 2)]
    for b, e in enumerate(arr):
        assert (e.q, e.k, e.v) == (q[b].data_ptr(), k[b].data_ptr(), v[b].data_ptr()) and e.q_out == tb.q_rot[b].data_ptr()
        assert (e.q_stride, e.k_stride, e.v_stride) == ((HQ + 2 * HKV) * D,) * 3
        assert (e.off, e.off_stride) == (off[b].data_ptr(), 8)
    depth = torch.zeros((2, 8), dtype=torch.int32)
    tb.append([3, 1], q, k, v, [8, 2], depth)
    assert [(e.off, e.off_stride) for e in calls[-1][1]] == [(depth[b].data_ptr(), 0) for b in range(2)]
    o, mask = new(HQ), torch.zeros((2, 8, 2), dtype=torch.int32)
    tb.attend([3, 1], o, [8, 2], mask)
    assert [(e.q, e.o, e.mask, e.mask_words, e.seq, e.n_rows) for e in calls[-1][1]] == \
        [(tb.q_rot[b].data_ptr(), o[b].data_ptr(), mask[b].data_ptr(), 2, (3, 1)[b], (8, 2)[b]) for b in range(2)]
    path, n_acc = torch.zeros((2, 8), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    tb.commit([3, 1], [8, 2], path, n_acc, [5, 0])
    assert [(e.path, e.n_acc, e.seq, e.n_rows, e.advance) for e in calls[-1][1]] == \
        [(path[b].data_ptr(), n_acc.data_ptr() + 4 * b, (3, 1)[b], (8, 2)[b], (5, 0)[b]) for b in range(2)]
    tb.commit([2], [1])
    assert [(e.path, e.n_acc, e.advance) for e in calls[-1][1]] == [(None, None, -1)]
    tb.trim([1, 2], [5, 7], [9, 11])
    assert [(e.seq, e.rows, e.next) for e in calls[-1][1]] == [(1, 5, 9), (2, 7, 11)]
    tb.fork([(0, 1), (0, 2)])
    assert [(e.src, e.dst) for e in calls[-1][1]] == [(0, 1), (0, 2)]


def test_engine_steps_make_their_calls_in_order(vc, calls):
    tb = trees(vc)
    calls.clear()
    tb.step([0, 1], new(HQ, R=1), new(HKV, R=1), new(HKV, R=1), new(HQ, R=1))
    assert [c[0] for c in calls] == ["vc_pages_reserve", "vc_rope_pages", "vc_tree_attn", "vc_tree_commit"]
    calls.clear()
    parent, n = torch.zeros((2, 8), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    tb.step([0, 1], new(HQ), new(HKV), new(HKV), new(HQ), [8, 3], parent, n)
    assert [c[0] for c in calls] == ["vc_tree_mask", "vc_pages_reserve", "vc_rope_pages", "vc_tree_attn"]
    calls.clear()
    tb.accept([0, 1], torch.zeros((2, 8, 30)), parent, parent, n, [8, 3])
    assert [c[0] for c in calls] == ["vc_tree_accept", "vc_tree_commit"]


def test_engine_refusals(vc, calls):
    tb = trees(vc, max_rows=1100)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    calls.clear()
    with pytest.raises(ValueError):  # more nodes than a tree has
        tb.step([0], *(torch.empty((1, 1100, h, D), dtype=torch.bfloat16) for h in (HQ, HKV, HKV, HQ)), [1], i(1, 1100), i(1))
    with pytest.raises(ValueError):
        tb.accept([0], torch.zeros(8), i(1, 8), i(1, 8), i(1), [1])
    assert not calls
    tb = trees(vc)
    calls.clear()
    good = dict(q=new(HQ), k=new(HKV), v=new(HKV))

    def refused(f, *a, **kw):
        with pytest.raises(ValueError):
            f(*a, **kw)
        assert not calls

    for seqs in ([], [0, 0], [0, 4], [-1, 0]):
        refused(tb.reserve, seqs, [1] * len(seqs))
        refused(tb.trim, seqs)
        refused(tb.append, seqs, **good, rows=[1] * len(seqs))
        refused(tb.attend, seqs, new(HQ), [1] * len(seqs))
        refused(tb.commit, seqs, [1] * len(seqs))
    refused(tb.reserve, [0, 1], [1])
    refused(tb.reserve, [0], [-1])
    refused(tb.trim, [0], [-1])
    refused(tb.trim, [0], [1], [2 ** 31])
    for pairs in ([], [(0, 0)], [(0, 1), (2, 1)], [(0, 1), (1, 2)], [(0, 4)], [(-1, 0)]):
        refused(tb.fork, pairs)
    for rows in ([1], [9, 1], [-1, 1]):
        refused(tb.append, [0, 1], **good, rows=rows)
        refused(tb.attend, [0, 1], new(HQ), rows)
        refused(tb.commit, [0, 1], rows)
    refused(tb.append, [0, 1], **{**good, "q": new(HQ, R=4), "k": new(HKV, R=4), "v": new(HKV, R=4)}, rows=[5, 1])
    for name, heads in (("q", HQ), ("k", HKV), ("v", HKV)):
        for bad in (new(heads).float(), new(heads + 1), new(heads)[:1], new(heads, R=7), new(heads, R=1).expand(2, 8, heads, D),
                    new(heads).transpose(2, 3).contiguous().transpose(2, 3), new(heads).to("meta")):
            refused(tb.append, [0, 1], **{**good, name: bad}, rows=[2, 2])
    for off in (i(2, 7), i(2, 2, 8), i(2, 8).long(), i(8, 2).t()):
        refused(tb.append, [0, 1], **good, rows=[2, 2], off=off)
    for o in (new(HQ).float(), new(HQ, R=1), new(HQ + 1), new(HQ)[:1], new(HQ, R=16)[:, ::2], new(HQ, B=1).expand(2, -1, -1, -1),
              torch.zeros(2 * 8 * HQ * D + 4, dtype=torch.bfloat16)[4:].view(2, 8, HQ, D)):
        refused(tb.attend, [0, 1], o, [2, 2])
    for mask in (i(2, 1, 1), i(2, 8, 0), i(2, 8), i(1, 8, 1), i(2, 8, 1).long(), i(2, 8, 2)[:, :, ::2]):
        refused(tb.attend, [0, 1], new(HQ), [2, 2], mask)
    refused(tb.commit, [0, 1], [2, 2], i(2, 1))
    refused(tb.commit, [0, 1], [2, 2], i(1, 8))
    refused(tb.commit, [0, 1], [2, 2], i(2, 8), i(3))
    refused(tb.commit, [0, 1], [2, 2], advance=[1])
    refused(tb.commit, [0, 1], [2, 2], advance=[1, -1])
    for parent, n in ((i(2, 1), i(2)), (i(3, 8), i(3)), (i(2, 8), i(1)), (i(2, 9), i(2)), (i(2, 8).long(), i(2)), (i(8), i(2))):
        refused(tb.step, [0, 1], **good, o=new(HQ), rows=[2, 2], parent=parent, n_nodes=n)
    for logits, token in ((torch.zeros(2, 8, 5).double(), i(2, 8)), (torch.zeros(2, 8, 5), i(2, 7)), (torch.zeros(1, 8, 5), i(2, 8)),
                          (torch.zeros(2, 1, 5), i(2, 1)), (torch.zeros(2, 8, 10)[:, :, ::2], i(2, 8))):
        refused(tb.accept, [0, 1], logits, token, i(2, 8)[:, : token.shape[1]].contiguous(), i(2), [2, 2])
    for kw in (dict(page=8), dict(n_seq=0), dict(n_pages=0), dict(max_rows=0), dict(max_pages=0)):
        with pytest.raises(ValueError):
            trees(vc, **kw)


def test_engine_steps_look_at_their_tokens_before_the_pool_changes(vc, calls):
    """Nothing is called for a step whose tokens append would refuse, or whose trees are not as wide as they."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    tb = trees(vc)
    calls.clear()
    good = dict(q=new(HQ), k=new(HKV), v=new(HKV))
    for name, heads in (("q", HQ), ("k", HKV), ("v", HKV)):
        flat = torch.zeros(2 * 8 * heads * D + 64, dtype=torch.bfloat16)
        wide = torch.zeros((2, 8, heads * D + 4), dtype=torch.bfloat16)
        for bad in (new(heads).float(), new(heads + 1), new(heads)[:1], new(heads, R=7), new(heads, R=1).expand(2, 8, heads, D),
                    new(heads).transpose(2, 3).contiguous().transpose(2, 3), new(heads).to("meta"), new(heads)[0],
                    flat[4 : 4 + 2 * 8 * heads * D].view(2, 8, heads, D), wide[..., : heads * D].unflatten(2, (heads, D)),
                    flat.as_strided((2, 8, heads, D), (8 * heads * D + 4, heads * D, D, 1))):
            for tree in ({}, dict(parent=i(2, 8), n_nodes=i(2))):
                for rows in ([2, 2], [8, 1]):
                    with pytest.raises(ValueError):
                        tb.step([0, 1], **{**good, name: bad}, o=new(HQ), rows=rows, **tree)
                    with pytest.raises(ValueError):
                        tb.append([0, 1], **{**good, name: bad}, rows=rows)
                    assert not calls, (name, bad.shape, bad.stride())
    for R in (2, 7):  # trees narrower than their tokens
        with pytest.raises(ValueError):
            tb.step([0, 1], **good, o=new(HQ), rows=[2, 2], parent=i(2, R), n_nodes=i(2))
        assert not calls
    with pytest.raises(ValueError):
        tb.step([0, 1], *(new(h, R=4) for h in (HQ, HKV, HKV)), o=new(HQ), rows=[5, 1])
    assert not calls
    tb.step([0, 1], **{**good, "q": torch.zeros(2 * 8 * HQ * D + 4, dtype=torch.bfloat16)[: 2 * 8 * HQ * D].view(2, 8, HQ, D)}, o=new(HQ), rows=[8, 1])
    one = torch.zeros((2, 1, HQ * D + 4), dtype=torch.bfloat16)[:1, :, : HQ * D].unflatten(2, (HQ, D))
    tb.step([2], one, new(HKV, 1, 1), new(HKV, 1, 1), new(HQ, 1, 1))  # one token's stride does not matter
    odd = torch.zeros(8 * HQ * D + 4, dtype=torch.bfloat16).as_strided((2, 8, HQ, D), (4, HQ * D, D, 1))
    tb.step([0, 1], **{**good, "q": odd}, o=new(HQ), rows=[8, 0])  # nor where a sequence without tokens starts


def test_engine_refuses_a_table_of_axes_that_does_not_fit(vc):
    """At once, not in a step's append behind its reserve."""
    from lossless_compressed_kv_vc_gb300 import engine
    wide = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, 2 * D), [D])
    broken = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, D), [D // 2])
    broken.axis[3] = 1
    for axes in (wide, broken, None):
        with pytest.raises(vc.VCError):
            engine.TreeBatch(HQ, HKV, D, n_seq=2, n_pages=4, page=16, axes=axes, device="cpu")


def test_the_default_stream_is_waited_on_itself(vc, monkeypatch):
    """Stream 0 is the default stream, of which ExternalStream would make a new one."""
    from lossless_compressed_kv_vc_gb300 import engine

    class Default:
        cuda_stream, waited = 0, []

        def wait_event(self, e):
            self.waited.append(e)

    class Owner:
        _ordered, _built = set(), "built"
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *_: Default())
    monkeypatch.setattr(torch.cuda, "ExternalStream", None)
    for _ in range(2):
        engine.Batch._order(Owner, 0)
    assert Default.waited == ["built"] and Owner._ordered == {0}
