"""GPU parity of drafted trees over a cache of pages (vc_pages_*, vc_rope_pages, vc_tree_*) and of engine.TreeBatch
against the float64 oracle.

Tolerances. Rotation as in test_gpu_live.py: |err| <= 2^-8 |y| + 2^-20 amp (|a| + |b|). Attention: tests/util.py (bf16
weights and output). Page tables, counts, masks, depths, paths, tokens and all moved rows are compared bit for bit.

Pages that no sequence holds, and the rows behind a sequence's last one, hold NaN and have to stay as they were.
"""
import numpy as np
import pytest
import torch

import oracle as O
from tests.test_gpu_live import NAN, bits, f64, gen, randn
from tests.util import assert_attn_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


def ints(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class Pool:
    """A pool on the GPU, NaN wherever no row has been written, beside the oracle's."""

    def __init__(self, vc, Hq, Hkv, d, n_pages, page, n_seq, max_pages):
        self.vc, self.Hq, self.Hkv, self.d, self.page = vc, Hq, Hkv, d, page
        shape = (n_pages, Hkv, page, d)
        self.k, self.v = (torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.state = {n: ints(*s, fill=-77) for n, s in (("refs", (n_pages,)), ("free_pages", (n_pages,)), ("n_free", (1,)),
                                                        ("table", (n_seq, max_pages)), ("len", (n_seq,)), ("held", (n_seq,)),
                                                        ("next", (n_seq,)))}
        self.kv = vc.paged_kv(self.k, self.v, **self.state)
        self.status = ints(1)
        self.ws = torch.full((max(16, vc.vc_pages_workspace_size(self.shape(32), self.kv)),), 0x5A, dtype=torch.uint8, device="cuda")
        vc.vc_pages_init(self.shape(), self.kv)
        self.ref = O.Pages(n_pages, page, n_seq, max_pages, *(np.array(bits(x)) for x in (self.k, self.v)))
        self.ref.table[:] = -77

    def shape(self, B=1):
        return self.vc.vc_shape(B, self.Hq, self.Hkv, self.d)

    def arr(self, t, reqs):
        return (t * len(reqs))(*[t(*r) for r in reqs])

    def reserve(self, *reqs):
        self.vc.vc_pages_reserve(self.shape(len(reqs)), self.kv, self.arr(self.vc.vc_reserve_req, reqs), self.ws, self.status)
        self.ref.reserve(reqs)

    def fork(self, *pairs):
        self.vc.vc_pages_fork(self.shape(len(pairs)), self.kv, self.arr(self.vc.vc_fork_req, pairs), self.status)
        self.ref.fork(pairs)

    def trim(self, *reqs):
        self.vc.vc_pages_trim(self.shape(len(reqs)), self.kv, self.arr(self.vc.vc_trim_req, reqs), self.status)
        self.ref.trim(reqs)

    def compact(self):
        self.vc.vc_pages_compact(self.shape(), self.kv, self.ws, self.status)
        self.ref.compact()

    def commit(self, *reqs):
        """(seq, rows, path list or None, n_acc or None, advance)"""
        arr, keep = (self.vc.vc_commit_req * len(reqs))(), []
        for e, (seq, rows, path, n_acc, advance) in zip(arr, reqs):
            p = None if path is None else torch.tensor(path, dtype=torch.int32, device="cuda")
            n = None if n_acc is None else ints(1, fill=n_acc)
            keep += [p, n]
            e.path, e.n_acc = (None if t is None else t.data_ptr() for t in (p, n))
            e.seq, e.n_rows, e.advance = seq, rows, advance
        self.vc.vc_tree_commit(self.shape(len(reqs)), self.kv, arr, self.status)
        self.ref.commit(reqs)

    def write(self, seq, a, n, g):
        """Random rows a .. a+n-1 of a sequence, by its table, on both sides."""
        k, v = randn(g, self.Hkv, n, self.d), randn(g, self.Hkv, n, self.d)
        self.ref.put(seq, a, bits(k), bits(v))
        at = torch.arange(a, a + n, device="cuda")
        pages = torch.tensor(self.ref.table[seq], device="cuda").long()[at // self.page]
        self.k[pages, :, at % self.page], self.v[pages, :, at % self.page] = k.transpose(0, 1), v.transpose(0, 1)

    def fill(self, seq, n, extra, g):
        """Room for n + extra rows, n of them context."""
        self.reserve((seq, n + extra))
        self.write(seq, 0, n, g)
        if n:
            self.commit((seq, n, None, None, -1))

    def rows(self, seq, a, b):
        at = torch.arange(a, b, device="cuda")
        pages = self.state["table"][seq].long()[at // self.page]
        return tuple(x[pages, :, at % self.page].transpose(0, 1) for x in (self.k, self.v))

    def same(self):
        torch.cuda.synchronize()
        got = {n: t.cpu().numpy() for n, t in self.state.items()}
        for name in ("refs", "len", "held", "next", "table"):
            assert np.array_equal(got[name], getattr(self.ref, name)), name
        assert int(got["n_free"][0]) == self.ref.n_free
        assert np.array_equal(got["free_pages"], self.ref.free)
        assert np.array_equal(bits(self.k), self.ref.k) and np.array_equal(bits(self.v), self.ref.v)
        self.ref.check()


# ---- pages ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (6, 3, 128)])
def test_pages_of_any_life(vc, page, Hq, Hkv, d):
    """Reserve, fork, trim, compact and commit in random order, several requests a call, the pool now and then full:
    state and rows equal the oracle's after every call."""
    g, rng = gen(1), np.random.default_rng(page + d)
    n_seq, most = 9, 6
    p = Pool(vc, Hq, Hkv, d, 40, page, n_seq, most)
    faults = 0
    for step in range(120):
        B = int(rng.integers(1, 7))
        seqs = rng.choice(n_seq, B, replace=False).tolist()
        op = int(rng.integers(6))
        before = p.ref.faults
        if op <= 1:
            p.reserve(*[(s, int(rng.integers(0, 2 * page))) for s in seqs])
            for s in seqs:  # write what may be written, make some of it context
                n = int(p.ref.len[s])
                own = int(p.ref.held[s]) * page - n
                if n % page and own and p.ref.refs[p.ref.table[s, n // page]] > 1:
                    own = 0
                rows = int(rng.integers(0, own + 1)) if own else 0
                if rows:
                    p.write(s, n, rows, g)
                    p.commit((s, rows, None, int(rng.integers(0, rows + 1)), int(rng.integers(-1, 50))))
        elif op == 2:
            p.fork(*[(seqs[0], s) for s in seqs[1:]] or [(seqs[0], (seqs[0] + 1) % n_seq)])
        elif op == 3:
            p.trim(*[(s, int(rng.integers(0, most * page)) if rng.random() < 0.6 else 0, int(rng.integers(99))) for s in seqs])
        elif op == 4:
            p.compact()
        else:
            p.trim(*[(s, 2 ** 31 - 1, 0) for s in seqs])
        p.same()
        faults += p.ref.faults > before
        assert int(p.status.item()) == (vc.VC_DEV_PAGES if p.ref.faults > before else 0)
        p.status.zero_()
    assert faults > 0


def test_reserve_when_pages_run_short(vc):
    """Requests in order, each served whole or not at all; a request that is not served leaves its shared page shared
    for those behind it."""
    g = gen(2)
    p = Pool(vc, 2, 2, 64, 6, 16, 6, 6)
    p.fill(0, 20, 0, g)           # pages 0, 1
    p.fork((0, 1), (0, 2), (0, 3))
    p.same()
    p.reserve((1, 100), (2, 1), (3, 17), (0, 1))  # not served; a copy; copy and one more; a copy: none left
    p.same()
    assert p.ref.faults == 1 and p.ref.n_free == 0 and int(p.status.item()) == vc.VC_DEV_PAGES
    p.status.zero_()
    p.trim((2, 0, 0))
    p.reserve((3, 60), (1, 12), (0, 20))  # more than there are; its own page does; the one that is left
    p.same()
    assert p.ref.faults == 2 and p.ref.n_free == 0


def test_reserve_of_more_than_2_to_the_25_pages(vc):
    """One request for 35 million pages beside one for more than are left: whole, or not at all. Only the state exists:
    nothing is copied, so that no row of K or V is touched."""
    n_pages, most, page = 40 * 10 ** 6, 36 * 10 ** 6, 16
    k = torch.zeros((16,), dtype=torch.bfloat16, device="cuda")
    st = dict(refs=ints(n_pages), free_pages=ints(n_pages), n_free=ints(1), table=ints(3, most, fill=-77), len=ints(3), held=ints(3),
              next=ints(3))
    kv = vc.vc_paged_kv(k.data_ptr(), k.data_ptr(), *(t.data_ptr() for t in st.values()), n_pages, page, 3, most)
    shape, status = vc.vc_shape(3, 1, 1, 64), ints(1)
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    vc.vc_pages_init(shape, kv)
    take = 35 * 10 ** 6
    reqs = [(0, take * page - 5), (1, 10 ** 7 * page), (2, 17)]
    vc.vc_pages_reserve(shape, kv, (vc.vc_reserve_req * 3)(*[vc.vc_reserve_req(*r) for r in reqs]), ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == vc.VC_DEV_PAGES and st["held"].tolist() == [take, 0, 2] and int(st["n_free"]) == n_pages - take - 2
    assert torch.equal(st["table"][0, :take], torch.arange(take, dtype=torch.int32, device="cuda"))
    assert st["table"][2, :3].tolist() == [take, take + 1, -77] and (st["table"][0, take:] == -77).all() and (st["table"][1] == -77).all()
    assert (st["refs"][: take + 2] == 1).all() and not st["refs"][take + 2 :].any()


def test_thirty_two_forks_of_one(vc):
    """One sequence copied 31 times in one call, room for all in one call: the last one keeps the shared page."""
    g = gen(3)
    p = Pool(vc, 4, 2, 128, 120, 32, 32, 8)
    p.fill(0, 70, 0, g)
    p.fork(*[(0, i) for i in range(1, 32)])
    p.reserve(*[(i, 40) for i in range(31, -1, -1)])
    p.same()
    assert p.ref.faults == 0 and int(p.status.item()) == 0
    assert len(set(p.ref.table[:, 2].tolist())) == 32
    p.trim(*[(i, 0 if i % 2 else 33, 5) for i in range(32)])
    p.same()


@pytest.mark.parametrize("Hkv,d,page,B", [(8, 128, 128, 9), (4, 128, 128, 31), (8, 128, 16, 31), (8, 128, 16, 32), (3, 64, 128, 21),
                                          (8, 64, 64, 17)])
def test_copies_of_either_size(vc, Hkv, d, page, B):
    """Shared last pages of many requests, copied by one launch (up to 2 MB of rows in all) and by two."""
    g = gen(27)
    p = Pool(vc, Hkv, Hkv, d, 2 * B + 6, page, B + 1, 4)
    p.fill(0, 2 * page - 3, 0, g)
    p.fork(*[(0, i) for i in range(1, B)])
    p.reserve(*[(i, 1 + i % 5) for i in range(B)])
    p.same()
    p.trim(*[(i, page + i if i % 2 else 1, 0) for i in range(1, B)])
    p.reserve(*[(i, page) for i in range(1, B)])  # some first pages are shared by all
    p.same()
    assert p.ref.faults == 0 and int(p.status.item()) == 0


def test_trim_of_pages_that_several_requests_hold(vc):
    """A page that several requests of one call give back goes on the stack once, at the place of the last of them."""
    g = gen(4)
    p = Pool(vc, 2, 1, 64, 64, 16, 8, 40)
    p.fill(0, 500, 0, g)
    p.fork((0, 1), (0, 2), (0, 3), (0, 4))
    p.trim((2, 100, 1), (0, 0, 0), (4, 300, 2), (1, 17, 3))
    p.same()
    p.trim((3, 0, 0), (4, 0, 0), (1, 0, 0), (2, 0, 0))
    p.same()
    assert p.ref.n_free == 64 and int(p.status.item()) == 0


def test_broken_state_is_skipped_and_reported(vc):
    """Table entries outside the pool, lengths beyond the pages held, a stack with foreign words: reported, and nothing
    outside is touched (what the calls may leave behind is theirs)."""
    g = gen(5)
    for breakage in ("table", "len", "negative len", "held", "stack", "n_free", "refs"):
        p = Pool(vc, 2, 2, 64, 24, 16, 4, 6)
        for s in range(3):
            p.fill(s, 40, 8, g)
        st = p.state
        if breakage == "table":
            st["table"][0, 1], st["table"][1, 2], st["table"][2, 2] = 24, -1, 2 ** 30
        elif breakage == "len":
            st["len"][:3] = 2 ** 30
        elif breakage == "negative len":
            st["len"][:3] = -5
        elif breakage == "held":
            st["held"][:3] = 1000
        elif breakage == "stack":
            st["free_pages"].fill_(10 ** 9)
        elif breakage == "n_free":
            st["n_free"].fill_(2 ** 30)
        else:
            st["refs"].fill_(0)
        codes = set()
        for call in (lambda: p.vc.vc_pages_reserve(p.shape(3), p.kv, p.arr(vc.vc_reserve_req, [(0, 30), (1, 1), (2, 50)]), p.ws, p.status),
                     lambda: p.vc.vc_pages_fork(p.shape(1), p.kv, p.arr(vc.vc_fork_req, [(0, 3)]), p.status),
                     lambda: p.vc.vc_tree_commit(p.shape(1), p.kv, p.arr(vc.vc_commit_req, [(None, None, 1, 40, -1)]), p.status),
                     lambda: p.vc.vc_pages_compact(p.shape(), p.kv, p.ws, p.status),
                     lambda: p.vc.vc_pages_trim(p.shape(3), p.kv, p.arr(vc.vc_trim_req, [(0, 0, 0), (1, 0, 0), (2, 0, 0)]), p.status)):
            p.status.zero_()
            call()
            torch.cuda.synchronize()
            codes.add(int(p.status.item()))
        assert codes <= {0, vc.VC_DEV_PAGES} and vc.VC_DEV_PAGES in codes, breakage


def test_commit_along_paths(vc):
    """Paths of any ascending nodes, across pages, more rows than the kernel looks up at a time; a path that goes wrong
    ends there."""
    g, rng = gen(6), np.random.default_rng(6)
    p = Pool(vc, 3, 3, 64, 200, 16, 8, 48)
    cases = []
    for s, (n, rows) in enumerate([(0, 1), (15, 9), (16, 40), (33, 700), (5, 600), (100, 30), (7, 12)]):
        p.fill(s, n, rows, g)
        p.write(s, n, rows, g)
        m = [1, 4, 13, 650, 300, 0, 5][s]
        stay = 40 if s == 3 else 0  # rows that lie where they belong
        path = list(range(stay)) + sorted(rng.choice(np.arange(stay, rows), m - stay, replace=False).tolist())
        cases.append((s, rows, path + [-1] * (rows - m), m, -1 if s % 2 else 3))
    p.commit(*cases)
    p.same()
    assert int(p.status.item()) == 0
    s, n = 6, int(p.ref.len[6])
    p.reserve((s, 6))
    p.write(s, n, 6, g)
    p.commit((s, 6, [1, 3, 9, 4, 5, 5], 5, -1))  # 9 is none of the 6
    p.same()
    assert int(p.ref.len[s]) == n + 2 and int(p.status.item()) == vc.VC_DEV_PAGES
    p.status.zero_()
    p.reserve((s, 6))
    p.write(s, n + 2, 6, g)
    p.commit((s, 6, [2, 4, 1, 5, 5, 5], 99, -1))  # 1 lies before its own place
    p.same()
    p.commit((s, 3, None, -4, -1))                # held to none
    p.same()
    assert int(p.ref.len[s]) == n + 4


def test_commit_of_rows_that_were_never_written(vc):
    """Sequences that reserve could not serve are left as they are, whatever the path says: a last page that another one
    holds, room for a part of the rows, pages laid down by hand that are nobody's; the others of the call are served."""
    g = gen(31)
    p = Pool(vc, 4, 2, 64, 9, 16, 6, 6)
    p.fill(0, 20, 0, g)
    p.fill(2, 27, 0, g)
    p.fill(3, 5, 40, g)
    p.write(3, 5, 40, g)
    p.fork((0, 1), (2, 4))
    p.fill(5, 1, 0, g)
    p.reserve((1, 3), (2, 9), (4, 1))  # one page left: 1 gets its copy of it, and the others wait
    p.same()
    assert p.ref.n_free == 0 and p.ref.faults == 2
    for s, rows, path, n_acc, advance in ((2, 9, None, None, -1), (2, 5, [0, 1, 2, 3, 4], 5, -1), (4, 1, [0], 1, 4),
                                          (2, 9, [0, 2, 7, -1, -1, -1, -1, -1, -1], 3, -1), (4, 5, None, 0, 7),
                                          (5, 17, None, 3, -1), (5, 40, [0] * 40, 1, -1)):
        p.status.zero_()
        p.commit((s, rows, path, n_acc, advance), (3, 1, None, None, -1))
        p.same()
        assert int(p.status.item()) == vc.VC_DEV_PAGES
    assert p.ref.len.tolist() == [20, 20, 27, 12, 27, 1]
    p.status.zero_()
    p.write(1, 20, 3, g)
    p.commit((1, 3, [0, 2, -1], 2, -1))
    p.trim((3, 0, 0))
    p.reserve((2, 9), (4, 1))
    p.write(2, 27, 9, g)
    p.write(4, 27, 1, g)
    p.commit((2, 9, [0, 4, 7, 8, -1, -1, -1, -1, -1], 4, -1), (4, 1, None, None, -1))
    p.same()
    assert int(p.status.item()) == 0 and p.ref.len.tolist() == [20, 22, 31, 0, 28, 1]
    mine = int(p.ref.table[5, 0])
    for page, refs in ((9, 1), (-1, 1), (2 ** 30, 1), (mine, 0), (mine, 2)):  # laid down by hand
        p.state["table"][5, 0], p.state["refs"][mine] = page, refs
        p.status.zero_()
        vc.vc_tree_commit(p.shape(), p.kv, p.arr(vc.vc_commit_req, [(None, None, 5, 2, 1)]), p.status)
        torch.cuda.synchronize()
        assert int(p.status.item()) == vc.VC_DEV_PAGES and int(p.state["len"][5]) == int(p.state["next"][5]) == 1


# ---- rotary append ----------------------------------------------------------------------------------
def _rope_close(got, x, pos, freqs, axis, inter, amp, heads, d):
    x = f64(x).reshape(-1, heads, d)
    ref = O.rope_axes(x, pos, freqs, axis, inter, amp)
    rot, mag = 2 * len(freqs), np.abs(x)
    h = rot // 2
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, h), slice(h, rot))
    lim = 2.0 ** -8 * np.abs(ref)
    both = 2.0 ** -20 * abs(amp) * (mag[..., a] + mag[..., b])
    lim[..., a] += both
    lim[..., b] += both
    lim[..., rot:] = 0
    err = np.abs(f64(got).reshape(ref.shape) - ref)
    assert np.all(err <= lim), float((err - lim).max())


@pytest.mark.parametrize("Hq,Hkv,d,rot,inter,sections,dealt,page,fused,keys_only", [
    (8, 2, 64, 64, False, [32], False, 16, False, False),
    (8, 2, 64, 32, True, [6, 5, 5], True, 16, True, False),
    (32, 8, 128, 128, False, [24, 20, 20], False, 64, True, False),
    (40, 8, 128, 128, True, [0, 32, 32, 0], True, 32, False, False),
    (6, 6, 128, 48, False, [1, 23], True, 128, False, True),
    (3, 1, 64, 16, False, [8, 0, 0], False, 16, True, False)])
def test_rope_pages(vc, Hq, Hkv, d, rot, inter, sections, dealt, page, fused, keys_only):
    """Rows into pages at every place of a page, offsets on every axis (negative ones, and far positions), requests without
    rows between the others; all other rows and the state stay as they were."""
    g, rng = gen(7), np.random.default_rng(7)
    p = Pool(vc, Hq, Hkv, d, 60, page, 6, 12)
    lens, rows = [0, 3, page - 1, page, 5 * page + 7, 1], [1, 40, 0, 17, 2, 33]
    amp = 1.25
    rope = vc.vc_rope_init(vc.VC_ROPE_NONE, rot, vc.VC_ROPE_INTERLEAVED if inter else vc.VC_ROPE_HALF, 500000.0, amp=amp)
    axes, axis = vc.vc_rope_axes_init(rope, sections, dealt), O.axes(sections, dealt)
    freqs = O.rope_freqs("none", rot, 500000.0)
    for s in range(6):
        p.fill(s, lens[s], rows[s], g)
    p.state["next"].copy_(torch.tensor([0, 7, 5, 1000003, 100 - 2 ** 30, 2 ** 30 - 2000], dtype=torch.int32))
    p.ref.next[:] = p.state["next"].cpu().numpy()
    arr, keep = (vc.vc_rope_page_req * 6)(), []
    order = [3, 0, 5, 2, 1, 4]
    for e, s in zip(arr, order):
        T = max(rows[s], 1)
        x = randn(g, T, (Hq + 2 * Hkv) * d)
        q, k, v = (t if fused else t.contiguous() for t in x.split([Hq * d, Hkv * d, Hkv * d], 1))
        out = torch.full((T, Hq, d), NAN, dtype=torch.bfloat16, device="cuda")
        kind = s % 3
        off = [None, torch.tensor(rng.integers(-9, 900, (T,)), dtype=torch.int32, device="cuda"),
               torch.tensor(rng.integers(-9, 900, (len(sections), T + 3)), dtype=torch.int32, device="cuda")][kind]
        e.q, e.q_out = (None, None) if keys_only else (q.data_ptr(), out.data_ptr())
        e.k, e.v, e.seq, e.n_rows = k.data_ptr(), v.data_ptr(), s, rows[s]
        e.q_stride, e.k_stride, e.v_stride = (t.stride(0) for t in (q, k, v))
        e.off, e.off_stride = None if off is None else off.data_ptr(), T + 3 if kind == 2 else 0
        o = np.arange(T) if off is None else off.cpu().numpy()
        o = np.broadcast_to(o, (len(sections), T)) if kind < 2 else o[:, :T]
        keep.append((s, q, k, v, out, off, int(p.ref.next[s]) + o.astype(np.int64)))
    old_k, old_v = p.k.clone(), p.v.clone()
    vc.vc_rope_pages(p.shape(6), axes, p.kv, arr, p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    for s, q, k, v, out, _, pos in keep:
        R, n = rows[s], lens[s]
        if R and not keys_only:
            _rope_close(out[:R], q[:R], pos[:, :R], freqs, axis, inter, amp, Hq, d)
        if keys_only or not R:
            assert torch.isnan(out).all()
        if R:
            gk, gv = p.rows(s, n, n + R)
            _rope_close(gk.transpose(0, 1), k[:R], pos[:, :R], freqs, axis, inter, amp, Hkv, d)
            assert np.array_equal(bits(gv.transpose(0, 1)), bits(v[:R].reshape(R, Hkv, d)))
            at = torch.arange(n, n + R, device="cuda")
            pages = p.state["table"][s].long()[at // page]
            old_k[pages, :, at % page], old_v[pages, :, at % page] = p.k[pages, :, at % page], p.v[pages, :, at % page]
    assert np.array_equal(bits(p.k), bits(old_k)) and np.array_equal(bits(p.v), bits(old_v))
    p.ref.k, p.ref.v = bits(p.k), bits(p.v)
    p.same()


def test_rope_pages_writes_only_pages_of_its_own(vc):
    """Tokens without a page, and those whose page another sequence holds, are turned and not written."""
    g = gen(8)
    Hq, Hkv, d = 4, 2, 64
    p = Pool(vc, Hq, Hkv, d, 12, 16, 3, 4)
    p.fill(0, 24, 0, g)   # rows 24 .. 31 of its second page are there
    p.fork((0, 1))        # and now shared
    p.fill(2, 30, 0, g)   # rows 30, 31
    axes = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, d), [d // 2])
    for s, R, written in ((0, 3, 0), (2, 5, 2)):
        q, k, v = randn(g, R, Hq, d), randn(g, R, Hkv, d), randn(g, R, Hkv, d)
        out, old = torch.zeros_like(q), (p.k.clone(), p.v.clone())
        p.status.zero_()
        arr = (vc.vc_rope_page_req * 1)(vc.vc_rope_page_req(q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, 0, None, 0,
                                                            out.data_ptr(), s, R))
        vc.vc_rope_pages(p.shape(), axes, p.kv, arr, p.status)
        torch.cuda.synchronize()
        assert int(p.status.item()) == vc.VC_DEV_PAGES
        n = int(p.ref.len[s])
        pos = [n + np.arange(R)]
        _rope_close(out, q, pos, O.rope_freqs("none", d, 10000.0), [0] * (d // 2), False, 1.0, Hq, d)
        if written:
            gv = p.rows(s, n, n + written)[1]
            assert np.array_equal(bits(gv.transpose(0, 1)), bits(v[:written]))
            at = torch.arange(n, n + written, device="cuda")
            pages = p.state["table"][s].long()[at // 16]
            for x, o in zip((p.k, p.v), old):
                o[pages, :, at % 16] = x[pages, :, at % 16]
        assert np.array_equal(bits(p.k), bits(old[0])) and np.array_equal(bits(p.v), bits(old[1]))


# ---- attention ----------------------------------------------------------------------------------------
def random_tree(rng, N, chain=0.5):
    return [-1] + [i - 1 if rng.random() < chain else int(rng.integers(0, i)) for i in range(1, N)]


def attend(vc, p, reqs, ws=None, stream=None):
    """reqs: (seq, q, mask int32 [N][words] or None). Outputs, NaN before the call."""
    outs = [torch.full_like(q, NAN) for _, q, _ in reqs]
    arr = (vc.vc_tree_req * len(reqs))()
    for e, (seq, q, mask), o in zip(arr, reqs, outs):
        e.q, e.o, e.seq, e.n_rows = q.data_ptr(), o.data_ptr(), seq, q.shape[0]
        if mask is not None:
            e.mask, e.mask_words = mask.data_ptr(), mask.shape[1]
    shape = p.shape(len(reqs))
    if ws is None:
        ws = torch.full((vc.vc_tree_workspace_size(shape, max(q.shape[0] for _, q, _ in reqs)),), 0xFF, dtype=torch.uint8, device="cuda")
    vc.vc_tree_attn(shape, p.kv, arr, ws, p.status, stream)
    return outs


def check(vc, p, Hq, reqs, see, outs, heads=None):
    """Outputs against the oracle; see[b] [N][N]. heads: KV heads compared (all by default)."""
    torch.cuda.synchronize()
    G = p.Hq // p.Hkv
    for (seq, q, _), w, o in zip(reqs, see, outs):
        N, n = q.shape[0], int(p.ref.len[seq])
        if N == 0:
            continue
        k, v = (f64(x) for x in p.rows(seq, 0, n + N))
        hs = range(p.Hkv) if heads is None else heads
        for h in hs:
            ref = O.tree_attn(f64(q)[:, h * G : (h + 1) * G], k[h : h + 1], v[h : h + 1], w)
            assert_attn_close(o[:, h * G : (h + 1) * G], ref, f"sequence {seq}, {n} + {N} rows, head {h}")


def build(vc, g, Hq, Hkv, d, page, sizes, spare=3):
    """A pool whose sequences hold n context rows and N rows behind them; sizes: (n, N)."""
    need = [-(-(n + max(N, 1)) // page) for n, N in sizes]
    p = Pool(vc, Hq, Hkv, d, sum(need) + spare, page, len(sizes), max(need) + 1)
    for s, (n, N) in enumerate(sizes):  # a page at a time in turn, so that their pages lie scattered
        p.reserve((s, 1))
    while any(p.ref.held[s] < need[s] for s in range(len(sizes))):
        for s in range(len(sizes)):
            if p.ref.held[s] < need[s]:
                p.reserve((s, int(p.ref.held[s]) * page + 1))
    for s, (n, N) in enumerate(sizes):
        k, v = randn(g, Hkv, n + N, d), randn(g, Hkv, n + N, d)
        at = torch.arange(n + N, device="cuda")
        pages = torch.tensor(p.ref.table[s], device="cuda").long()[at // page]
        p.k[pages, :, at % page], p.v[pages, :, at % page] = k.transpose(0, 1), v.transpose(0, 1)
    p.ref.len[:] = [n for n, _ in sizes]
    p.state["len"].copy_(torch.tensor(p.ref.len))
    assert int(p.status.item()) == 0
    return p


LENGTHS = [0, 1, 15, 16, 17, 62, 63, 64, 65, 100, 126, 127, 128, 129, 191, 255, 256, 257, 400]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (4, 1, 128), (5, 5, 128), (16, 1, 64)])
def test_single_tokens_of_every_length(vc, Hq, Hkv, d, page):
    g = gen(10)
    sizes = [(n, 1) for n in LENGTHS]
    p = build(vc, g, Hq, Hkv, d, page, sizes)
    reqs = [(s, randn(g, 1, Hq, d), None) for s in range(len(sizes))]
    outs = attend(vc, p, reqs)
    check(vc, p, Hq, reqs, [np.ones((1, 1), bool)] * len(reqs), outs)
    assert int(p.status.item()) == 0


TREES = [  # Hq, Hkv, d, page, (context, tokens) of each request
    (8, 2, 64, 16, [(1000, 8), (0, 8), (1, 1), (127, 30), (64, 64), (200, 33)]),
    (32, 8, 128, 32, [(300, 25), (1027, 16), (5, 32), (128, 12)]),
    (40, 8, 128, 64, [(500, 25), (63, 25), (64, 25)]),
    (64, 8, 128, 64, [(700, 64), (33, 64)]),              # two full units a head: CTAs by unit
    (16, 1, 128, 16, [(2000, 50), (10, 48), (600, 64)]),  # 800, 768 and 1024 rows: units of different numbers
    (16, 1, 64, 128, [(900, 48), (3000, 48)]),            # 768 rows: three full units, CTAs by unit
    (6, 6, 128, 16, [(333, 130), (2, 129), (0, 128), (50, 200)]),
    (12, 2, 64, 32, [(1500, 96), (11, 70)]),
    (4, 4, 64, 16, [(40, 300)]),
    (2, 1, 128, 128, [(5000, 3)]),                        # one piece over many CTAs
]


@pytest.mark.parametrize("case", TREES)
@pytest.mark.parametrize("kind", ["tree", "chain", "random", "mixed"])
def test_trees(vc, case, kind):
    """Trees, chains, masks of any bits (rows without any, tokens that see later ones) and mixtures of them, bits
    behind the last token set."""
    Hq, Hkv, d, page, sizes = case
    g, rng = gen(11), np.random.default_rng(11)
    p = build(vc, g, Hq, Hkv, d, page, sizes)
    reqs, see = [], []
    for s, (n, N) in enumerate(sizes):
        how = kind if kind != "mixed" else ("tree", "chain", "random")[s % 3]
        w = {"tree": lambda: O.ancestors(random_tree(rng, N))[0], "chain": lambda: np.tri(N, dtype=bool),
             "random": lambda: rng.random((N, N)) < 0.3}[how]()
        mask = None
        if how != "chain" or s % 2:
            if how == "random":
                w[rng.random(N) < 0.3] = False
            words = (N + 31) // 32 + s % 2
            bits_ = np.zeros((N, 32 * words), bool)
            bits_[:, :N] = w
            bits_[:, N:] = rng.random((N, 32 * words - N)) < 0.5
            mask = torch.tensor(O.pack_mask(bits_, words), device="cuda")
        see.append(w)
        reqs.append((s, randn(g, N, Hq, d), mask))
    outs = attend(vc, p, reqs)
    check(vc, p, Hq, reqs, see, outs)
    assert int(p.status.item()) == 0
    again = attend(vc, p, reqs)  # the same bits
    assert all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.parametrize("Hq,Hkv,d,page,sizes", [
    (8, 1, 64, 16, [(0, 700), (1, 333), (250, 65)]),           # units of 32 tokens, seven or more of them a head
    (3, 1, 128, 32, [(0, 515), (130, 300)]),                   # a unit ends within a token's heads
    (5, 5, 64, 128, [(127, 520), (0, 0), (0, 513)]),
    (16, 1, 128, 64, [(0, 512)]),                              # 32 full units: most of the square is cut away
    (16, 1, 128, 64, [(9000, 512)]),                           # the same over a context beside which the cut is little
    (14, 2, 128, 16, [(40, 400), (3000, 37), (0, 37), (12, 1)]),
    (24, 1, 64, 16, [(0, 128), (64, 128), (128, 128)])])
@pytest.mark.parametrize("tree", [False, True])
def test_prompt_chunks(vc, Hq, Hkv, d, page, sizes, tree):
    """Chains of several units of query rows, which end at different keys; with `tree` every other request has a mask."""
    g = gen(25)
    p = build(vc, g, Hq, Hkv, d, page, sizes)
    reqs, see = [], []
    for s, (n, N) in enumerate(sizes):
        w = np.tri(N, dtype=bool)
        if tree and s % 2 == 0 and N:
            w = O.ancestors(random_tree(np.random.default_rng(s), N))[0]
        words = -(-N // 32)
        reqs.append((s, randn(g, N, Hq, d), torch.tensor(O.pack_mask(w, words), device="cuda") if tree and s % 2 == 0 and N else None))
        see.append(w)
    outs = attend(vc, p, reqs)
    check(vc, p, Hq, reqs, see, outs)
    assert int(p.status.item()) == 0


def test_a_prompt_chunk_with_too_few_pages(vc):
    """Tokens whose rows lie behind the pages held are seen by none; those that have pages by whom they would be."""
    g = gen(26)
    p = build(vc, g, 8, 1, 64, 16, [(20, 200)])
    held = int(p.ref.held[0])
    q = randn(g, 400, 8, 64)
    N = held * 16 - 20  # tokens whose rows the pages have room for
    at = torch.arange(220, held * 16, device="cuda")
    pages = p.state["table"][0].long()[at // 16]
    p.k[pages, :, at % 16], p.v[pages, :, at % 16] = 0, 0  # rows behind the last token hold NaN: now numbers
    outs = attend(vc, p, [(0, q, None)])
    torch.cuda.synchronize()
    assert int(p.status.item()) == vc.VC_DEV_PAGES
    k, v = (f64(x) for x in p.rows(0, 0, held * 16))
    assert_attn_close(outs[0][:N], O.tree_attn(f64(q)[:N], k, v, np.tri(N, dtype=bool)), "rows with pages")
    tail = min(400 - N, N)
    assert_attn_close(outs[0][400 - tail :], O.tree_attn(np.concatenate([f64(q)[400 - tail :], f64(q)[: N - tail]]), k, v,
                                                         np.ones((N, N), bool))[:tail], "rows without")


def test_a_mask_that_leaves_nothing(vc):
    """No context and an empty row: zeros, whatever K and V hold; beside rows that see themselves."""
    g = gen(12)
    p = build(vc, g, 8, 2, 64, 16, [(0, 40), (0, 1), (0, 3)])
    at = p.state["table"][0].long()[0]
    p.k[at, :, 5], p.v[at, :, 5] = NAN, float("inf")
    w0 = np.eye(40, dtype=bool)
    w0[[0, 5, 7, 39]] = False
    see = [w0, np.zeros((1, 1), bool), np.zeros((3, 3), bool)]
    reqs = [(s, randn(g, len(w), 8, 64), torch.tensor(O.pack_mask(w, 2), device="cuda")) for s, w in enumerate(see)]
    outs = attend(vc, p, reqs)
    torch.cuda.synchronize()
    assert all((o[~w.any(1)] == 0).all() for o, w in zip(outs, see))
    check(vc, p, 8, reqs, see, outs)


BROKEN = [  # Hq, Hkv, d, page, context, tokens, broken tokens
    (8, 2, 64, 16, 96, 64, (24, 63)), (8, 2, 64, 16, 95, 64, tuple(range(23, 64))), (16, 4, 128, 32, 226, 64, (24, 34, 63)),
    (4, 4, 128, 64, 172, 128, (18, 118)), (4, 4, 128, 128, 212, 128, (28, 118)), (32, 4, 128, 16, 420, 40, (12, 30, 39)),
    (4, 4, 64, 16, 392, 128, (8, 58, 108, 127)), (64, 8, 128, 64, 100, 64, (3, 40)), (8, 8, 128, 16, 0, 5, (2,))]


@pytest.mark.parametrize("case", BROKEN)
@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
@pytest.mark.parametrize("tree", [False, True])
def test_broken_rows_reach_only_those_that_see_them(vc, case, bad, tree):
    """K and V of some tokens are not finite, in several steps of a chain: rows that see none of them come out as the
    oracle's, the others not finite (an infinite V by itself; a NaN key whatever V is)."""
    Hq, Hkv, d, page, n, N, broken = case
    g, rng = gen(13), np.random.default_rng(13)
    p = build(vc, g, Hq, Hkv, d, page, [(n, N)] * 3)
    see = O.ancestors(random_tree(rng, N, 0.3))[0] if tree else np.tri(N, dtype=bool)
    hit = see[:, list(broken)].any(1)
    assert hit.any() and not hit.all()
    mask = torch.tensor(O.pack_mask(see, (N + 31) // 32), device="cuda") if tree else None
    for s in range(3):
        for j in broken:
            page_of = int(p.ref.table[s, (n + j) // page])
            p.v[page_of, :, (n + j) % page, d // 3] = bad
            if s == 1 and np.isnan(bad):
                p.k[page_of, :, (n + j) % page] = bad
    reqs = [(s, randn(g, N, Hq, d), mask) for s in range(3)]
    for _ in range(5):
        outs = attend(vc, p, reqs)
        torch.cuda.synchronize()
        for (s, q, _), o in zip(reqs, outs):
            k, v = (np.nan_to_num(f64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in p.rows(s, 0, n + N))
            ref = O.tree_attn(f64(q), k, v, see)
            assert_attn_close(o[torch.tensor(~hit)], ref[~hit])
            seen = o[torch.tensor(hit)]
            assert not torch.isfinite(seen[..., d // 3]).any()
            if s != 1 or not np.isnan(bad):
                fine = [c for c in range(d) if c != d // 3]
                assert_attn_close(seen[..., fine], ref[hit][..., fine])
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("Hq,Hkv,d,page,n,N", [(8, 2, 64, 16, 700, 1), (8, 2, 64, 16, 700, 4), (8, 2, 64, 32, 700, 30),
                                               (4, 4, 128, 64, 900, 200), (32, 4, 128, 64, 1000, 64)])
@pytest.mark.parametrize("shape", ["rising", "falling", "steps", "late", "deep"])
def test_scores_that_outgrow_the_first_ones(vc, Hq, Hkv, d, page, n, N, shape):
    """Scores that rise or fall by a factor of up to 2^70 of weight along the keys, in opposite directions for different
    rows: the maximum moves again and again, or not at all; rows that start far below zero; and a part of a chain that
    sees nothing at first."""
    g, rng = gen(19), np.random.default_rng(19)
    p = build(vc, g, Hq, Hkv, d, page, [(n, N), (0, N)])
    u = torch.nn.functional.normalize(torch.randn(d, generator=g, device="cuda"), dim=0)
    reqs, see = [], []
    for s, ctx in ((0, n), (1, 0)):
        T = ctx + N
        t = torch.arange(T, device="cuda").float()
        c = {"rising": 100 * t / T, "falling": 100 - 100 * t / T, "late": torch.where(t >= T - 3, 100.0, 0.0),
             "deep": torch.where(t < T // 2, -100.0, 0.0) + 20 * t / T,
             "steps": torch.tensor(rng.uniform(-60, 60, T // 50 + 1), device="cuda").float()[(t // 50).long()]}[shape]
        at = torch.arange(T, device="cuda")
        pages = p.state["table"][s].long()[at // page]
        k = 0.3 * torch.randn((T, Hkv, d), generator=g, device="cuda") + c[:, None, None] * u
        p.k[pages, :, at % page] = k.bfloat16()
        sign = torch.where(torch.rand((N, Hq, 1), generator=g, device="cuda") < 0.3, -1.0, 1.0)
        q = (torch.randn((N, Hq, d), generator=g, device="cuda") * 0.5 + sign * u * np.sqrt(d) * 0.5).bfloat16()
        w = rng.random((N, N)) < 0.2 if s else O.ancestors(random_tree(rng, N))[0]
        reqs.append((s, q, torch.tensor(O.pack_mask(w, (N + 31) // 32), device="cuda")))
        see.append(w)
    check(vc, p, Hq, reqs, see, attend(vc, p, reqs))
    assert int(p.status.item()) == 0


def test_infinite_scores(vc):
    """A context key with an infinite channel: rows whose product with it is -inf leave it out, the others are not finite,
    as in the oracle."""
    for Hq, Hkv, d, page, n, N in ((8, 2, 64, 16, 300, 1), (8, 2, 64, 32, 300, 20), (4, 2, 128, 64, 200, 130)):
        g = gen(29)
        p = build(vc, g, Hq, Hkv, d, page, [(n, N)])
        p.k[int(p.ref.table[0, 77 // page]), :, 77 % page, 5] = float("inf")
        q = randn(g, N, Hq, d)
        o = attend(vc, p, [(0, q, None)])[0]
        k, v = (f64(x) for x in p.rows(0, 0, n + N))
        with np.errstate(invalid="ignore"):
            ref = O.tree_attn(f64(q), k, v, np.tri(N, dtype=bool))
        fine = np.isfinite(ref).all(-1)
        assert fine.any() and not fine.all()
        assert np.array_equal(torch.isfinite(o).all(-1).cpu().numpy(), fine)
        assert_attn_close(o[torch.tensor(fine)][:, None], ref[fine][:, None])


@pytest.mark.parametrize("Hq,Hkv,d,page", [(8, 2, 64, 16), (32, 8, 128, 64), (12, 2, 64, 128)])
def test_a_batch_of_thirty_two(vc, Hq, Hkv, d, page):
    """All requests of a call, some without tokens, in an order that is not the sequences', two of one sequence."""
    g, rng = gen(14), np.random.default_rng(14)
    sizes = [(int(rng.integers(0, 900)), int(rng.integers(1, 20))) for _ in range(31)]
    p = build(vc, g, Hq, Hkv, d, page, sizes)
    order = rng.permutation(31).tolist() + [4]
    reqs, see = [], []
    for i, s in enumerate(order):
        N = 0 if i in (3, 17) else sizes[s][1]
        w = O.ancestors(random_tree(rng, N))[0] if N else np.zeros((0, 0), bool)
        reqs.append((s, randn(g, max(N, 1), Hq, d)[:N], torch.tensor(O.pack_mask(w, 1), device="cuda") if N else None))
        see.append(w)
    outs = attend(vc, p, reqs)
    check(vc, p, Hq, reqs, see, outs)
    assert int(p.status.item()) == 0


@pytest.mark.parametrize("G,d,page,n", [(9, 64, 16, 128), (32, 128, 128, 128), (128, 128, 64, 256), (32, 64, 64, 64), (16, 128, 32, 129)])
def test_pieces_of_one_tile_that_all_see_whole(vc, G, d, page, n):
    """One token over n - 1 rows: many heads of a tile or two each, in which a chain needs no V before its next queries."""
    g = gen(36)
    Hkv, B = 24, 20
    p = build(vc, g, G * Hkv, Hkv, d, page, [(n - 1, 1)] * B)
    reqs = [(s, randn(g, 1, G * Hkv, d), None) for s in range(B)]
    ws = torch.empty(vc.vc_tree_workspace_size(p.shape(B), 1), dtype=torch.uint8, device="cuda")
    first = attend(vc, p, reqs, ws)
    check(vc, p, G * Hkv, reqs, [np.ones((1, 1), bool)] * B, first, heads=(0, 11, 23))
    for _ in range(100):
        outs = attend(vc, p, reqs, ws)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0 and all(torch.equal(a, b) for a, b in zip(first, outs))


def test_rows_that_have_no_pages(vc):
    """Tokens behind the pages held are seen by none; a table entry outside the pool reads as nothing; both are reported
    and the other requests come out right."""
    g = gen(15)
    Hq, Hkv, d, page = 8, 2, 64, 16
    p = build(vc, g, Hq, Hkv, d, page, [(200, 8), (30, 10), (100, 4)])
    p.state["held"][1] = 2  # rows 32 and on are gone: tokens 2 .. 9
    reqs = [(s, randn(g, N, Hq, d), None) for s, N in ((0, 8), (1, 10), (2, 4))]
    outs = attend(vc, p, reqs)
    torch.cuda.synchronize()
    assert int(p.status.item()) == vc.VC_DEV_PAGES
    check(vc, p, Hq, [reqs[0], reqs[2]], [np.tri(8, dtype=bool), np.tri(4, dtype=bool)], [outs[0], outs[2]])
    k, v = (f64(x) for x in p.rows(1, 0, 32))
    see = np.tri(10, 2, dtype=bool)
    ref = np.concatenate([O.tree_attn(f64(reqs[1][1])[i : i + 2], k, v, see[i : i + 2]) for i in range(0, 10, 2)])
    assert_attn_close(outs[1], ref)
    p.status.zero_()
    p.state["held"][1] = 3
    p.state["table"][0, 3] = 10 ** 9
    outs = attend(vc, p, reqs)
    torch.cuda.synchronize()
    assert int(p.status.item()) == vc.VC_DEV_PAGES and torch.isfinite(outs[0]).all()
    check(vc, p, Hq, reqs[1:], [np.tri(10, dtype=bool), np.tri(4, dtype=bool)], outs[1:])


@pytest.mark.parametrize("Hq,Hkv,d,page,n,N", [
    (8, 2, 64, 16, 200, 1), (8, 2, 64, 16, 9, 2), (32, 8, 128, 16, 3000, 4), (4, 4, 128, 128, 1, 7), (32, 8, 128, 32, 70, 9),
    (8, 2, 64, 64, 127, 30), (64, 8, 128, 64, 300, 64), (64, 8, 128, 16, 1, 64), (16, 1, 64, 128, 4060, 40), (5, 5, 128, 16, 23, 300)])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("junk", [None, NAN, float("inf")])
def test_tokens_in_a_page_that_others_hold_are_seen_by_none(vc, Hq, Hkv, d, page, n, N, tree, junk):
    """Sequences forked within a page and not made ready: their tokens' rows there were never written, whatever the page
    holds, so all see the context alone, those behind in pages of their own too; reported, and others come out right."""
    g, rng = gen(32), np.random.default_rng(N + n)
    p = Pool(vc, Hq, Hkv, d, 5 + 3 * -(-(n + N) // page), page, 3, 1 + -(-(n + N) // page))
    p.fill(0, n, N, g)
    p.write(0, n, N, g)
    p.fill(2, n, N, g)
    p.write(2, n, N, g)
    p.fork((0, 1))
    last = int(p.ref.table[0, n // page])
    assert p.ref.refs[last] == 2
    if junk is not None:
        p.k[last, :, n % page :], p.v[last, :, n % page :] = junk, junk
    see = O.ancestors(random_tree(rng, N))[0] if tree else np.tri(N, dtype=bool)
    mask = torch.tensor(O.pack_mask(see, -(-N // 32)), device="cuda") if tree else None
    none = np.zeros((N, N), bool)
    for seqs in ([2, 0, 1], [1], [0]):
        p.status.zero_()
        reqs = [(s, randn(g, N, Hq, d), mask) for s in seqs]
        outs = attend(vc, p, reqs)
        torch.cuda.synchronize()
        assert int(p.status.item()) == vc.VC_DEV_PAGES
        check(vc, p, Hq, [r for r in reqs if r[0] == 2], [see], [o for r, o in zip(reqs, outs) if r[0] == 2])
        k, v = (np.concatenate([f64(x), np.zeros((Hkv, N, d))], 1) for x in p.rows(0, 0, n))
        for (s, q, _), o in zip(reqs, outs):
            if s != 2:
                assert_attn_close(o, O.tree_attn(f64(q), k, v, none), f"sequence {s}")


def test_a_sequence_without_pages(vc):
    g = gen(16)
    p = build(vc, g, 8, 2, 64, 16, [(50, 2), (0, 1)])
    p.trim((1, 0, 0))
    reqs = [(1, randn(g, 3, 8, 64), None)]
    assert not attend(vc, p, reqs)[0].any()  # nothing to see: zeros
    assert int(p.status.item()) == vc.VC_DEV_PAGES
    both = [(1, randn(g, 3, 8, 64), None), (0, randn(g, 2, 8, 64), None)]
    outs = attend(vc, p, both)
    assert not outs[0].any()
    check(vc, p, 8, both[1:], [np.tri(2, dtype=bool)], outs[1:])


@pytest.mark.parametrize("Hq,Hkv,d,page,sizes", [(8, 2, 64, 16, [(500, 9), (70, 9), (300, 2)]),
                                                 (64, 8, 128, 64, [(700, 64), (90, 64)]), (4, 4, 128, 32, [(9, 300)])])
def test_the_least_workspace_and_a_byte_less(vc, Hq, Hkv, d, page, sizes):
    g = gen(17)
    p = build(vc, g, Hq, Hkv, d, page, sizes)
    reqs = [(s, randn(g, N, Hq, d), None) for s, (_, N) in enumerate(sizes)]
    full = vc.vc_tree_workspace_size(p.shape(len(sizes)), max(N for _, N in sizes))
    ws = torch.full((full + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    ref = attend(vc, p, reqs, ws)
    ok = lambda b: attend_status(vc, p, reqs, ws[:b]) == 0
    lo, hi = 0, full
    assert not ok(0) and ok(full)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if ok(mid) else (mid, hi)
    ws.fill_(0xFF)
    outs = attend(vc, p, reqs, ws[:hi])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, outs)) and (ws[hi:] == 0xFF).all()


def attend_status(vc, p, reqs, ws):
    outs = [torch.empty_like(q) for _, q, _ in reqs]
    arr = (vc.vc_tree_req * len(reqs))(*[vc.vc_tree_req(q.data_ptr(), o.data_ptr(), None, 0, s, q.shape[0])
                                         for (s, q, _), o in zip(reqs, outs)])
    st = vc.vc_tree_attn(p.shape(len(reqs)), p.kv, arr, ws, p.status, raise_on_error=False)
    torch.cuda.synchronize()
    assert st in (0, vc.VC_ERR_WORKSPACE)
    return st


def test_pages_beyond_32_bit_offsets(vc):
    """A pool of more than 2^32 elements, the sequences' pages at its end: append, attention, a copied page, compaction."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    Hq, Hkv, d, page, n_pages = 16, 8, 128, 128, 36000  # 4.7e9 elements a pool
    g = gen(18)
    k, v = (torch.empty((n_pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = dict(refs=ints(n_pages), free_pages=ints(n_pages), n_free=ints(1), table=ints(3, 8), len=ints(3), held=ints(3), next=ints(3))
    kv = vc.paged_kv(k, v, **st)
    shape, status = vc.vc_shape(1, Hq, Hkv, d), ints(1)
    ws = torch.empty(max(vc.vc_pages_workspace_size(shape, kv), vc.vc_tree_workspace_size(shape, 8)), dtype=torch.uint8, device="cuda")
    vc.vc_pages_init(shape, kv)
    st["free_pages"].copy_(torch.arange(n_pages, device="cuda"))  # the last pages first
    n, N = 300, 5
    one = lambda t, *a: (t * 1)(t(*a))
    vc.vc_pages_reserve(shape, kv, one(vc.vc_reserve_req, 0, n), ws, status)
    axes = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, d), [d // 2])
    xk, xv = randn(g, n, Hkv, d), randn(g, n, Hkv, d)
    rope = lambda x, y, s, R, q=None, o=None: vc.vc_rope_pages(shape, axes, kv, one(
        vc.vc_rope_page_req, q, x.data_ptr(), y.data_ptr(), 0, 0, 0, None, 0, o, s, R), status)
    rope(xk, xv, 0, n)
    vc.vc_tree_commit(shape, kv, one(vc.vc_commit_req, None, None, 0, n, -1), status)
    vc.vc_pages_fork(shape, kv, one(vc.vc_fork_req, 0, 1), status)
    vc.vc_pages_reserve(shape, kv, one(vc.vc_reserve_req, 1, N), ws, status)
    q, q2, yk, yv = randn(g, N, Hq, d), torch.zeros((N, Hq, d), dtype=torch.bfloat16, device="cuda"), randn(g, N, Hkv, d), randn(g, N, Hkv, d)
    rope(yk, yv, 1, N, q.data_ptr(), q2.data_ptr())
    o = torch.zeros_like(q2)
    attn = lambda: vc.vc_tree_attn(shape, kv, one(vc.vc_tree_req, q2.data_ptr(), o.data_ptr(), None, 0, 1, N), ws, status)
    attn()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and st["table"][1, :3].tolist() == [n_pages - 1, n_pages - 2, n_pages - 4]
    freqs, ax = O.rope_freqs("none", d, 10000.0), [0] * (d // 2)
    kk = np.concatenate([O.rope_axes(f64(x), [a + np.arange(len(x))], freqs, ax, False) for x, a in ((xk, 0), (yk, n))]).transpose(1, 0, 2)
    vv = np.concatenate([f64(xv), f64(yv)]).transpose(1, 0, 2)
    kk = f64(torch.tensor(kk).bfloat16())
    ref = O.tree_attn(f64(q2), kk, vv, np.tri(N, dtype=bool))
    assert_attn_close(o, ref)
    before = o.clone()
    o.zero_()
    vc.vc_pages_compact(shape, kv, ws, status)
    attn()
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(o, before)
    # four pages in use, ascending: the copied one, sequence 0's last, the shared second, the shared first
    assert st["table"][1, :3].tolist() == [3, 2, 0] and st["table"][0, :3].tolist() == [3, 2, 1]
    assert int(st["n_free"].item()) == n_pages - 4 and st["free_pages"][n_pages - 5].item() == 4


# ---- masks and acceptance ------------------------------------------------------------------------------
@pytest.mark.parametrize("B,N", [(1, 1), (3, 7), (5, 32), (2, 33), (4, 64), (2, 255), (1, 1024), (40, 20)])
def test_tree_mask(vc, B, N):
    rng = np.random.default_rng(N)
    words = (N + 31) // 32
    parent = np.array([random_tree(rng, N, 0.9 if b % 2 else 0.3) for b in range(B)], np.int32)
    n = rng.integers(0, N + 1, B).astype(np.int32)
    n[0] = N
    if N > 4:
        parent[0, 3], parent[0, 4] = 3, -9  # roots of their own
    if B > 2:
        n[1], n[2] = -3, N + 5
    ref_mask, ref_depth = np.zeros((B, N, words), np.int32), np.zeros((B, N), np.int32)
    for b in range(B):
        m = min(max(int(n[b]), 0), N)
        see, depth = O.ancestors(parent[b, :m].tolist())
        ref_mask[b, :m], ref_depth[b, :m] = O.pack_mask(see, words), depth
    mask, depth = ints(B, N, words, fill=-1), ints(B, N, fill=-1)
    vc.vc_tree_mask(B, N, torch.tensor(parent, device="cuda"), torch.tensor(n, device="cuda"), mask, depth)
    assert np.array_equal(mask.cpu().numpy(), ref_mask) and np.array_equal(depth.cpu().numpy(), ref_depth)
    only = ints(B, N, words, fill=-1)
    vc.vc_tree_mask(B, N, torch.tensor(parent, device="cuda"), torch.tensor(n, device="cuda"), only)
    assert torch.equal(only, mask)


@pytest.mark.parametrize("B,N,V", [(1, 1, 1), (2, 5, 7), (3, 16, 1000), (4, 33, 1003), (2, 200, 50), (1, 1024, 9), (33, 3, 130),
                                   (1, 4, 128257), (5, 2, 32001)])
def test_accept_tree(vc, B, N, V):
    """Ties, infinities, NaN, rows of NaN alone, drafts of which many agree."""
    g, rng = gen(20), np.random.default_rng(N + V)
    logits = torch.randint(0, 6, (B, N, V), generator=g, device="cuda").float()  # many ties
    if V > 4:
        logits[0, 0, V // 2], logits[0, 0, V - 1] = float("inf"), float("inf")
        logits[-1, -1] = NAN
        logits[B // 2, N // 2, : V // 2] = NAN
        logits[0, N - 1] = -float("inf")
    parent = np.array([random_tree(rng, N, 0.4) for _ in range(B)], np.int32)
    host = logits.cpu().numpy()
    token = rng.integers(0, V, (B, N)).astype(np.int32)
    for b in range(B):
        for i in range(1, N):
            if rng.random() < 0.7:
                token[b, i] = O.accept_tree(host[b, parent[b, i]][None], [0], [-1], 1)[1][0]
    n = rng.integers(0, N + 1, B).astype(np.int32)
    n[0] = N
    if B > 2:
        n[1], n[2] = N + 7, -1
    dev = lambda a: torch.tensor(a, device="cuda")
    out, path, n_acc = ints(B, N, fill=9), ints(B, N, fill=9), ints(B, fill=9)
    vc.vc_tree_accept(B, N, V, logits, dev(token), dev(parent), dev(n), out, path, n_acc)
    for b in range(B):
        p, t = O.accept_tree(host[b], token[b], parent[b], min(max(int(n[b]), 0), N))
        assert n_acc[b].item() == len(p)
        assert path[b].tolist() == p + [-1] * (N - len(p)) and out[b].tolist() == t + [-1] * (N - len(p))


# ---- the engine: turns as they are used -------------------------------------------------------------------
def _batch(vc, Hq, Hkv, d, **kw):
    from lossless_compressed_kv_vc_gb300 import engine
    axes = vc.vc_rope_axes_init(vc.vc_rope_init(vc.VC_ROPE_NONE, d, base=500000.0), kw.pop("sections", [d // 2]))
    return engine.TreeBatch(Hq, Hkv, d, axes=axes, **kw)


@pytest.mark.parametrize("Hq,Hkv,d,page", [(8, 2, 64, 16), (32, 8, 128, 32)])
def test_turns_of_trees(vc, Hq, Hkv, d, page):
    """Prompts, then turns of trees that are accepted in part, sequences forked and dropped on the way, the pool compacted
    once: every output against the oracle over the accepted tokens' own keys and values, positions by depth."""
    g, rng = gen(21), np.random.default_rng(21)
    N, V, n_seq = 12, 40, 4
    tb = _batch(vc, Hq, Hkv, d, n_seq=n_seq, n_pages=80, page=page, max_rows=100, max_pages=24)
    freqs, axis = O.rope_freqs("none", d, 500000.0), [0] * (d // 2)
    hist = [[np.zeros((0, Hkv, d))] * 2 for _ in range(n_seq)]  # rotated keys and values of the context

    def turned(x, pos):
        return f64(torch.tensor(O.rope_axes(f64(x), [pos], freqs, axis, False)).bfloat16())

    def compare(s, q, k, v, see, depth, o):
        pos = len(hist[s][0]) + np.asarray(depth)
        rows = [np.concatenate([h, x]) for h, x in zip(hist[s], (turned(k, pos), f64(v)))]
        ref = O.tree_attn(turned(q, pos), *(x.transpose(1, 0, 2) for x in rows), see)
        assert_attn_close(o, ref, f"sequence {s}")
        return rows

    seqs = [2, 0, 3]
    prompt = [100, 37, 1]
    q, k, v = (randn(g, 3, 100, h, d) for h in (Hq, Hkv, Hkv))
    o = torch.zeros((3, 100, Hq, d), dtype=torch.bfloat16, device="cuda")
    tb.step(seqs, q, k, v, o, prompt)
    for b, (s, R) in enumerate(zip(seqs, prompt)):
        hist[s] = compare(s, q[b, :R], k[b, :R], v[b, :R], np.tri(R, dtype=bool), np.arange(R), o[b, :R])
    taken = 0
    for turn in range(5):
        if turn == 2:
            tb.fork([(2, 1)])
            hist[1] = list(hist[2])
            seqs = [2, 1, 3, 0]
        if turn == 3:
            tb.trim([0])
            hist[0] = [np.zeros((0, Hkv, d))] * 2
            tb.compact()
        B = len(seqs)
        rows = [N, N - 3, N, 5][:B]
        parent = torch.tensor(np.array([random_tree(rng, N) for _ in range(B)], np.int32), device="cuda")
        n_nodes = torch.tensor(rows, dtype=torch.int32, device="cuda")
        q, k, v = (randn(g, B, N, h, d) for h in (Hq, Hkv, Hkv))
        o = torch.full((B, N, Hq, d), NAN, dtype=torch.bfloat16, device="cuda")
        tb.step(seqs, q, k, v, o, rows, parent, n_nodes)
        logits = torch.randn((B, N, V), generator=g, device="cuda")
        token = logits.argmax(2).gather(1, parent.clamp(min=0).long()).to(torch.int32)
        token = torch.where(torch.rand((B, N), generator=g, device="cuda") < 0.8, token, (token + 1) % V).contiguous()
        out, path, n_acc = tb.accept(seqs, logits, token, parent, n_nodes, rows)
        torch.cuda.synchronize()
        assert int(tb.dev_status.item()) == 0
        for b, (s, R) in enumerate(zip(seqs, rows)):
            see, depth = O.ancestors(parent[b, :R].tolist())
            full = compare(s, q[b, :R], k[b, :R], v[b, :R], see, depth, o[b, :R])
            p, t = O.accept_tree(logits[b].cpu().numpy(), token[b].tolist(), parent[b].tolist(), R)
            assert path[b, : len(p)].tolist() == p and out[b, : len(p)].tolist() == t and n_acc[b].item() == len(p)
            n = len(hist[s][0])
            hist[s] = [x[list(range(n)) + [n + j for j in p]] for x in full]
            taken += len(p)
            assert int(tb.len[s]) == n + len(p) == int(tb.next[s])
            assert torch.isnan(o[b, R:]).all()
    assert taken > 30


def test_image_tokens_share_positions(vc):
    """A prompt of text, an image on three axes, text behind it: positions go on from the image's largest."""
    Hq, Hkv, d, sections = 8, 2, 64, [12, 10, 10]
    g = gen(22)
    tb = _batch(vc, Hq, Hkv, d, n_seq=1, n_pages=10, page=16, max_rows=24, sections=sections)
    freqs, axis = O.rope_freqs("none", d, 500000.0), O.axes(sections, False)
    rows = np.zeros((2, 0, Hkv, d))
    at = 0
    for R, off, advance in ((5, None, None), (24, np.stack([np.zeros(24), np.arange(24) // 6, np.arange(24) % 6]), 6), (3, None, None)):
        q, k, v = (randn(g, 1, R, h, d) for h in (Hq, Hkv, Hkv))
        o = torch.zeros((1, R, Hq, d), dtype=torch.bfloat16, device="cuda")
        tb.reserve([0], [R])
        tb.append([0], q, k, v, [R], None if off is None else torch.tensor(off[None], dtype=torch.int32, device="cuda"))
        mask = None
        see = np.tri(R, dtype=bool)
        if off is not None:  # the image's tokens see one another
            see = np.ones((R, R), bool)
            mask = torch.tensor(O.pack_mask(see, 1)[None], device="cuda")
        tb.attend([0], o, [R], mask)
        tb.commit([0], [R], advance=None if advance is None else [advance])
        pos = at + (np.tile(np.arange(R), (3, 1)) if off is None else off)
        rot = lambda x: f64(torch.tensor(O.rope_axes(f64(x[0]), pos, freqs, axis, False)).bfloat16())
        rows = np.concatenate([rows, np.stack([rot(k), f64(v[0])])], 1)
        ref = O.tree_attn(rot(q), *(x.transpose(1, 0, 2) for x in rows), see)
        assert_attn_close(o[0], ref)
        at += R if advance is None else advance
    assert int(tb.next[0]) == 5 + 6 + 3 and int(tb.len[0]) == 32 and int(tb.dev_status.item()) == 0


def test_a_captured_turn_follows_the_caches_as_they_grow(vc):
    """One graph of a whole turn (masks, room, append, attention, acceptance, commit), replayed on new inputs while
    lengths and tables move on: the same as eager turns, at every turn."""
    Hq, Hkv, d, N, V, B = 8, 2, 64, 6, 50, 3
    g = gen(23)
    make = lambda: _batch(vc, Hq, Hkv, d, n_seq=B, n_pages=60, page=16, max_rows=40)
    eager, graph = make(), make()
    seqs, rows = [2, 0, 1], [N, N - 2, N]
    x = [randn(g, B, 40, h, d) for h in (Hq, Hkv, Hkv)]
    for tb in (eager, graph):
        tb.step(seqs, *x, torch.zeros_like(x[0]), [40, 13, 16])
    q, k, v = (randn(g, B, N, h, d) for h in (Hq, Hkv, Hkv))
    parent, token = ints(B, N), ints(B, N)
    n_nodes = torch.tensor(rows, dtype=torch.int32, device="cuda")
    logits = torch.zeros((B, N, V), device="cuda")
    outs = [torch.zeros((B, N, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def turn(tb, o):
        tb.step(seqs, q, k, v, o, rows, parent, n_nodes)
        return tb.accept(seqs, logits, token, parent, n_nodes, rows)

    # inputs of the capture: nothing runs, state stays
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        got = turn(graph, outs[1])
    rng = np.random.default_rng(23)
    for _ in range(12):
        for t in (q, k, v):
            t.copy_(randn(g, *t.shape))
        logits.copy_(torch.randn((B, N, V), generator=g, device="cuda"))
        parent.copy_(torch.tensor(np.array([random_tree(rng, N) for _ in range(B)], np.int32)))
        token.copy_(logits.argmax(2).gather(1, parent.clamp(min=0).long()))
        want = turn(eager, outs[0])
        cg.replay()
        torch.cuda.synchronize()
        assert torch.equal(*outs) and all(torch.equal(a, b) for a, b in zip(want, got))
        for name in ("len", "held", "next", "table", "refs", "free_pages", "n_free"):
            assert torch.equal(getattr(eager, name), getattr(graph, name)), name
        assert torch.equal(eager.k, graph.k) and torch.equal(eager.v, graph.v)
    assert int(eager.dev_status.item()) == int(graph.dev_status.item()) == 0 and int(graph.len.sum()) > 69 + 36


def test_two_pools_on_two_streams(vc):
    """Steps of two pools side by side on streams of their own, one given and one current: as one alone."""
    Hq, Hkv, d, B = 32, 8, 128, 4
    g = gen(24)
    make = lambda: _batch(vc, Hq, Hkv, d, n_seq=B, n_pages=160, page=64, max_rows=500)
    alone, one, two = make(), make(), make()
    x = [randn(g, B, 500, h, d) for h in (Hq, Hkv, Hkv)]
    y = [randn(g, B, 1, h, d) for h in (Hq, Hkv, Hkv)]
    outs = [torch.zeros_like(y[0]) for _ in range(3)]
    scratch = [torch.zeros_like(x[0]) for _ in range(3)]
    seqs, rows = [0, 1, 2, 3], [500, 400, 1, 130]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    alone.step(seqs, *x, scratch[0], rows)
    one.step(seqs, *x, scratch[1], rows, stream=s1)
    with torch.cuda.stream(s2):
        two.step(seqs, *x, scratch[2], rows)
    for _ in range(30):
        alone.step(seqs, *y, outs[0])
        one.step(seqs, *y, outs[1], stream=s1.cuda_stream)
        with torch.cuda.stream(s2):
            two.step(seqs, *y, outs[2])
    torch.cuda.synchronize()
    for tb, o in ((one, outs[1]), (two, outs[2])):
        assert torch.equal(o, outs[0]) and torch.equal(tb.k, alone.k) and torch.equal(tb.v, alone.v)
        assert torch.equal(tb.len, alone.len) and int(tb.dev_status.item()) == 0


@pytest.mark.parametrize("stream", [None, 0])
def test_a_pool_built_on_a_stream_that_is_behind(vc, stream):
    """A pool whose construction waits behind other work of its stream, used at once on the default stream."""
    Hq, Hkv, d, B = 8, 2, 64, 3
    g = gen(28)
    make = lambda: _batch(vc, Hq, Hkv, d, n_seq=B, n_pages=40, page=16, max_rows=40)
    x = [randn(g, B, 40, h, d) for h in (Hq, Hkv, Hkv)]
    outs = [torch.zeros_like(x[0]) for _ in range(2)]
    alone = make()
    torch.cuda.synchronize()
    alone.step([0, 1, 2], *x, outs[0], [40, 1, 17])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # about 25 ms of device time
        late = make()
    late.step([0, 1, 2], *x, outs[1], [40, 1, 17], stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(late.len, alone.len) and torch.equal(late.table[:, 0], alone.table[:, 0])
    assert int(late.dev_status.item()) == 0 and int(late.n_free.item()) == int(alone.n_free.item())


def test_a_pool_that_runs_out(vc):
    """Room is asked for beyond the pool: reported, the sequence's rows are not written anywhere, the others go on."""
    Hq, Hkv, d = 8, 2, 64
    g = gen(25)
    tb = _batch(vc, Hq, Hkv, d, n_seq=2, n_pages=4, page=16, max_rows=40)
    x = [randn(g, 2, 40, h, d) for h in (Hq, Hkv, Hkv)]
    o = torch.zeros_like(x[0])
    tb.step([0, 1], *x, o, [40, 40])  # three pages for the first, the second asks for three of the one left
    torch.cuda.synchronize()
    assert int(tb.dev_status.item()) == vc.VC_DEV_PAGES
    assert tb.held.tolist() == [3, 0] and tb.len.tolist() == [40, 0] and not o[1].any()
    tb.dev_status.zero_()
    tb.trim([1])
    y = [t[:1, :1].contiguous() for t in x]
    tb.step([0], *y, o[:1, :1].contiguous())
    torch.cuda.synchronize()
    assert int(tb.dev_status.item()) == 0 and tb.len.tolist() == [41, 0]


def _unserved(vc, shared):
    """A small pool and one that never runs out, as far as the step that the small one cannot serve: sequence 1 has
    forked from 0 within a page (`shared`), or asks for more rows than its own last page has room for. 2 holds the rest."""
    Hq, Hkv, d = 8, 2, 64
    small, large = (_batch(vc, Hq, Hkv, d, n_seq=3, n_pages=n, page=16, max_rows=40, max_pages=9) for n in (7, 40))
    g = gen(33 + shared)
    x = [randn(g, 3, 40, h, d) for h in (Hq, Hkv, Hkv)]
    for tb in (small, large):
        tb.step([0, 1], *(t[:2] for t in x), torch.zeros_like(x[0][:2]), [27, 0 if shared else 5])
        if shared:
            tb.fork([(0, 1)])
        tb.step([2], *(t[2:].contiguous() for t in x), torch.zeros_like(x[0][2:]), [40])
        tb.reserve([2], [40 if shared else 24])
    torch.cuda.synchronize()
    assert int(small.n_free.item()) == 0 and int(small.dev_status.item()) == 0
    return small, large, g


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_a_turn_that_the_pool_cannot_serve_is_made_again(vc, tree, shared):
    """Lengths and positions stay where they were; with pages given back the same turn equals that of a pool that never
    ran out, and so do those that follow."""
    small, large, g = _unserved(vc, shared)
    Hq, Hkv, d, N, V = 8, 2, 64, 14, 30
    parent = torch.tensor([random_tree(np.random.default_rng(5), N)], dtype=torch.int32, device="cuda")
    rows, n_nodes = [N], ints(1, fill=N)

    def turn(tb, q, k, v, logits):
        o = torch.full((1, N, Hq, d), NAN, dtype=torch.bfloat16, device="cuda")
        token = logits.argmax(2).gather(1, parent.clamp(min=0).long()).to(torch.int32)
        tb.step([1], q, k, v, o, rows, *((parent, n_nodes) if tree else ()))
        if tree:
            tb.accept([1], logits, token, parent, n_nodes, rows)
        torch.cuda.synchronize()
        return o

    before = [t.clone() for t in (small.len, small.next, small.held, small.table, small.refs)]
    x = [randn(g, 1, N, h, d) for h in (Hq, Hkv, Hkv)] + [torch.randn((1, N, V), generator=g, device="cuda")]
    turn(small, *x)
    assert int(small.dev_status.item()) == vc.VC_DEV_PAGES
    assert all(torch.equal(a, b) for a, b in zip(before, (small.len, small.next, small.held, small.table, small.refs)))
    small.dev_status.zero_()
    small.trim([2])
    large.trim([2])
    for again in range(3):
        if again:
            x = [randn(g, 1, N, h, d) for h in (Hq, Hkv, Hkv)] + [torch.randn((1, N, V), generator=g, device="cuda")]
        assert torch.equal(turn(small, *x), turn(large, *x))
        assert int(small.dev_status.item()) == int(large.dev_status.item()) == 0
        assert torch.equal(small.len, large.len) and torch.equal(small.next, large.next)
        if again == 0:  # the other one goes on too
            y = [randn(g, 1, 3, h, d) for h in (Hq, Hkv, Hkv)]
            outs = [torch.zeros_like(y[0]) for _ in range(2)]
            for tb, o in zip((small, large), outs):
                tb.step([0], *y, o, [3])
            torch.cuda.synchronize()
            assert torch.equal(*outs)
    n = int(small.len[1])
    assert n > before[0][1]
    for tb in (small, large):
        at = torch.arange(n, device="cuda")
        tb.got = [t[tb.table[1].long()[at // 16], :, at % 16] for t in (tb.k, tb.v)]
    assert all(torch.equal(a, b) for a, b in zip(small.got, large.got))
