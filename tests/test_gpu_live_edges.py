"""GPU tests of the live-cache calls at the places where a masked or broken value could leak: value rows that are
broken in several steps of a chain. Tolerances and helpers are those of test_gpu_live.py.
"""
import numpy as np
import pytest
import torch

import oracle as O
from tests.test_gpu_live import NAN, bits, cache, f64, gen, randn
from tests.util import assert_attn_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


def _attend(vc, Hq, Hkv, d, reqs, scored, prefix=None):
    """reqs: (q, k, v, n, score) each; the outputs and the call's device status."""
    B = len(reqs)
    outs = [torch.zeros_like(r[0]) for r in reqs]
    arr = (vc.vc_live_req * B)(*[vc.vc_live_req(q.data_ptr(), o.data_ptr(), q.shape[0], vc.live_kv(k, v, n, s))
                                 for (q, k, v, n, s), o in zip(reqs, outs)])
    shape, R = vc.vc_shape(B, Hq, Hkv, d), max(r[0].shape[0] for r in reqs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if scored:
        ws = torch.empty(vc.vc_scored_workspace_size(shape, R, max(r[3] for r in reqs)), dtype=torch.uint8, device="cuda")
        vc.vc_scored_attn(shape, arr, ws, status)
    else:
        ws = torch.empty(vc.vc_prefix_workspace_size(shape, R), dtype=torch.uint8, device="cuda")
        vc.vc_prefix_attn(shape, prefix, arr, ws, status)
    torch.cuda.synchronize()
    return outs, int(status.item())


# Hq, Hkv, d, n, query rows, broken own rows: new keys that lie in two or three 64-key steps of a chain, the steps
# one behind the other, with a broken value row in each.
STEPS = [(8, 2, 64, 160, 64, (120, 159)),             # chains of 128 rows each: keys 96..159 in two steps
         (8, 2, 64, 159, 64, tuple(range(118, 159))),  # every row from one on
         (16, 4, 128, 290, 64, (250, 260, 289)),
         (4, 4, 128, 300, 128, (190, 290)),            # both chains the same rows, a half of every tile each
         (4, 4, 128, 340, 128, (240, 330)),
         (32, 4, 128, 460, 40, (432, 450, 459)),       # a unit of 256 rows and one of 64
         (4, 4, 64, 520, 128, (400, 450, 500, 519))]


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("case", STEPS)
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_broken_values_in_consecutive_steps(vc, case, bad, scored):
    """Rows before the first broken token come out as the oracle's over the keys they see, rows from it on are not
    finite, whichever warp of a chain is ahead; weights do not depend on V."""
    Hq, Hkv, d, n, r, broken = case
    if scored and r * (Hq // Hkv) > 256:
        r = 256 // (Hq // Hkv)
    g = gen(41)
    reqs, first = [], broken[0] - (n - r)  # the first row that sees a broken one
    assert 0 < first < r
    for _ in range(4):
        q, (k, v, score, _) = randn(g, r, Hq, d), cache(g, Hkv, d, n, n + 3)
        v[:, list(broken)] = bad
        reqs.append((q, k, v, n, score))
    refs = [O.live_attn(f64(q), f64(k[:, :n]), np.where(np.isfinite(f64(v[:, :n])), f64(v[:, :n]), 0.0))
            for q, k, v, _, _ in reqs]
    old = [s.clone() for *_, s in reqs]
    for _ in range(10):
        for (*_, s), o in zip(reqs, old):
            s.copy_(o)
        outs, status = _attend(vc, Hq, Hkv, d, reqs, scored)
        assert status == 0
        for o, (_, _, _, _, s), was, (ref, w) in zip(outs, reqs, old, refs):
            assert_attn_close(o[:first], ref[:first])
            assert not torch.isfinite(o[first:]).any()
            if scored:
                # a factor within 1 +- (2 d 2^-23 max sum|q k| / sqrt(d) + 2^-20), and the sum's two roundings; with
                # unit normal q and k, sum|q k| / sqrt(d) stays below 16 at these sizes
                lim = w * (2 * d * 2.0 ** -23 * 16 + 2.0 ** -20) + 2.0 ** -23 * (f64(was[:, :n]) + w)
                assert np.all(np.abs(f64(s[:, :n]) - f64(was[:, :n]) - w) <= lim)
            else:
                assert np.array_equal(bits(s), bits(was))


@pytest.mark.parametrize("what", ["query", "key"])
@pytest.mark.parametrize("Hq,Hkv,d,n,r,at", [(8, 2, 64, 300, 5, 0), (8, 2, 64, 257, 5, 2), (32, 2, 128, 1030, 8, 5),
                                             (4, 4, 64, 1100, 120, 40), (4, 4, 128, 64, 64, 1)])
def test_a_broken_row_leaves_the_weights_of_keys_it_does_not_see(vc, Hq, Hkv, d, n, r, at, what):
    """One head of row `at` has a NaN query, or its key an infinite channel that gives it a product of +inf, and so NaN
    weights, and the other rows that see it -inf, a weight of 0: the scores of keys that only other rows see stay
    finite."""
    g = gen(43)
    q, (k, v, score, _) = randn(g, r, Hq, d), cache(g, Hkv, d, n, n + 3)
    if what == "query":
        q[at, 0] = NAN
    else:
        k[:, n - r + at, 3] = float("inf")
        q[..., 3] = -q[..., 3].abs() - 0.125
        q[at, 0, 3] *= -1
    with np.errstate(invalid="ignore"):
        ref, w = O.live_attn(f64(q), f64(k[:, :n]), f64(v[:, :n]))
    was = f64(score[:, :n])
    (o,), status = _attend(vc, Hq, Hkv, d, [(q, k, v, n, score)], True)
    got = f64(score[:, :n])
    assert status == 0
    assert np.array_equal(np.isnan(got), np.isnan(w)) and np.isnan(w).any() and np.isfinite(w).any()
    fine = np.isfinite(w)
    # as above, with the largest |q k| of finite keys below 16
    lim = w * (2 * d * 2.0 ** -23 * 16 + 2.0 ** -20) + 2.0 ** -23 * (was + w)
    assert np.all(np.abs(got - was - w)[fine] <= lim[fine])
    rows = np.isfinite(ref).all(-1)
    assert np.array_equal(torch.isfinite(o).all(-1).cpu().numpy(), rows)
    assert_attn_close(o[torch.tensor(rows)][:, None], ref[rows][:, None])


def _smallest(call, enough, wrong):
    """The smallest workspace, in bytes, that call(bytes) does not turn down with the status `wrong`."""
    lo, hi = 0, enough  # lo is refused
    assert call(0) == wrong and call(enough) == 0
    while hi - lo > 1:
        mid = (lo + hi) // 2
        st = call(mid)
        assert st in (0, wrong)
        lo, hi = (mid, hi) if st == wrong else (lo, mid)
    return hi


@pytest.mark.parametrize("kind", ["prefix", "scored", "evict"])
def test_the_least_workspace_and_a_byte_less(vc, kind):
    """A call needs no more than the size that the library names. With the least that it takes the words behind stay
    as they were and its results are those with all of it; a byte less is refused and nothing is written."""
    Hq, Hkv, d = 8, 2, 64
    ns, rows, B = [500, 70, 300], [9, 9, 2], 3
    g = gen(47)
    shape = vc.vc_shape(B, Hq, Hkv, d)
    state = [cache(g, Hkv, d, n, n + 2) for n in ns]
    for (_, _, _, p), n in zip(state, ns):
        p[:, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
    qs = [randn(g, r, Hq, d) for r in rows]
    outs = [torch.full_like(q, 7.0) for q in qs]
    old = [[t.clone() for t in s] for s in state] + [[o.clone() for o in outs]]
    pk, pv, _, _ = cache(g, Hkv, d, 300, 300)
    prefix = vc.vc_kv_full(pk.data_ptr(), pv.data_ptr(), 300, 300)
    size = {"prefix": vc.vc_prefix_workspace_size(shape, max(rows)), "evict": vc.vc_evict_workspace_size(shape, max(ns)),
            "scored": vc.vc_scored_workspace_size(shape, max(rows), max(ns))}[kind]
    buf = torch.empty(size + 4096, dtype=torch.uint8, device="cuda")

    def restore():
        for now, was in zip(state + [outs], old):
            for a, b in zip(now, was):
                a.copy_(b)

    def call(n):
        restore()
        buf.fill_(0x5A)
        kvs = [vc.live_kv(k, v, m, s, p) for (k, v, s, p), m in zip(state, ns)]
        ws = buf[:n] if n else None
        if kind == "evict":
            arr = (vc.vc_evict_req * B)(*[vc.vc_evict_req(kv, m // 2, 4, m - 9) for kv, m in zip(kvs, ns)])
            st = vc.vc_evict_kv(shape, arr, ws, raise_on_error=False)
        else:
            arr = (vc.vc_live_req * B)(*[vc.vc_live_req(q.data_ptr(), o.data_ptr(), q.shape[0], kv)
                                         for q, o, kv in zip(qs, outs, kvs)])
            st = vc.vc_scored_attn(shape, arr, ws, raise_on_error=False) if kind == "scored" else \
                vc.vc_prefix_attn(shape, prefix, arr, ws, raise_on_error=False)
        torch.cuda.synchronize()
        assert bool((buf[n:] == 0x5A).all())
        if st != vc.VC_OK:
            assert bool((buf == 0x5A).all())
            for now, was in zip(state + [outs], old):
                for a, b in zip(now, was):
                    assert np.array_equal(bits(a), bits(b))
        return st

    assert call(size) == vc.VC_OK
    want = [[t.clone() for t in s] for s in state + [outs]]
    least = _smallest(call, size, vc.VC_ERR_WORKSPACE)
    assert call(least - 1) == vc.VC_ERR_WORKSPACE
    assert call(least) == vc.VC_OK
    for now, was in zip(state + [outs], want):
        for a, b in zip(now, was):
            assert np.array_equal(bits(a), bits(b))


def test_a_batch_keeps_the_index_of_its_device(vc):
    from lossless_compressed_kv_vc_gb300 import engine
    lb = engine.LiveBatch(8, 2, 64, 2, 10, vc.vc_rope_init(vc.VC_ROPE_NONE, 64), device="cuda")
    assert lb.device == torch.device("cuda", torch.cuda.current_device())
    q, k = (torch.zeros((2, h, 1, 64), dtype=torch.bfloat16, device="cuda").transpose(1, 2) for h in (8, 2))
    lb.step(q, k, k, torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16, device="cuda"))  # single tokens, split by heads
    torch.cuda.synchronize()
    assert lb.n == [1, 1] and int(lb.dev_status.item()) == 0


@pytest.mark.parametrize("inter", [False, True])
def test_rope_with_a_table_filled_by_hand(vc, inter):
    """Frequencies of the caller's own: a ramp over the pairs' index between plain and squeezed ones, and a factor on
    every rotated channel (0.1 ln 8 + 1)."""
    Hq, Hkv, d, rot, R, n, pos0 = 8, 2, 128, 96, 9, 4, 70001
    freqs = O.rope_freqs("none", rot, 1e6)
    keep = np.clip((30 - np.arange(rot // 2)) / 20, 0, 1)
    freqs = keep * freqs + (1 - keep) * freqs / 8
    amp = 0.1 * np.log(8) + 1
    table = vc.vc_rope_init(vc.VC_ROPE_NONE, rot, vc.VC_ROPE_INTERLEAVED if inter else vc.VC_ROPE_HALF)
    table.amp = amp
    for j, f in enumerate(freqs):
        table.freq[j] = f
    g = gen(53)
    k, v, score, pos = cache(g, Hkv, d, n, n + R)
    q, kn, vn = randn(g, R, Hq, d), randn(g, R, Hkv, d), randn(g, R, Hkv, d)
    out = torch.empty_like(q)
    e = vc.vc_rope_req(q=q.data_ptr(), k=kn.data_ptr(), v=vn.data_ptr(), pos0=pos0, n_rows=R, q_out=out.data_ptr(),
                       kv=vc.live_kv(k, v, n, score, pos))
    vc.vc_rope_append(vc.vc_shape(1, Hq, Hkv, d), table, (vc.vc_rope_req * 1)(e))
    torch.cuda.synchronize()
    at = pos0 + np.arange(R)
    for got, x in ((out, q), (k[:, n:].transpose(0, 1), kn)):
        ref, mag = O.rope(f64(x), at, freqs, inter, amp), np.abs(f64(x))
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        lim = 2.0 ** -8 * np.abs(ref)  # as at the top of test_gpu_live.py
        both = 2.0 ** -20 * amp * (mag[..., a] + mag[..., b])
        lim[..., a] += both
        lim[..., b] += both
        lim[..., rot:] = 0
        assert np.all(np.abs(f64(got) - ref) <= lim)
