"""GPU parity of the live-cache calls (vc_rope_append, vc_prefix_attn, vc_scored_attn, vc_evict_kv) and of
engine.LiveBatch against the float64 oracle.

Tolerances. Rotation: inputs are bf16, cos and sin within 2^-21, two fp32 products and a sum, one
rounding to bf16 (half a step, 2^-8 of the value at most): |err| <= 2^-8 |y| + 2^-20 amp (|a| + |b|).
Attention outputs: tests/util.py (bf16 weights, bf16 output). Weights gathered in score: a score of d
products accumulated in fp32 with any rounding is off by at most d 2^-23 sum|q k| / sqrt(d), and the
row's log-sum-exp by at most the largest of those; exp2 and the sums over a tile add less than 2^-20.
So a weight is off by a factor within 1 +- (2 d 2^-23 max sum|q k| / sqrt(d) + 2^-20), and the sum with
what was there before by 2^-23 of it (two roundings). Eviction moves bits and is compared bit for bit.

Rows behind a cache's last one hold NaN in every test and have to stay as they were.
"""
import numpy as np
import pytest
import torch

import oracle as O
from tests.util import assert_attn_close

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.detach().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cache(g, Hkv, d, n, cap):
    """k, v with NaN behind row n, score and pos of the rows before it."""
    k, v = randn(g, Hkv, cap, d), randn(g, Hkv, cap, d)
    k[:, n:], v[:, n:] = NAN, NAN
    score = torch.rand((Hkv, cap), generator=g, device="cuda")
    score[:, n:] = NAN
    return k, v, score, torch.full((Hkv, cap), -7, dtype=torch.int32, device="cuda")


# ---- rotary positions ------------------------------------------------------------------------------
ROPE = {"none": {}, "linear": {"factor": 4.0}, "ntk": {"factor": 8.0},
        "bands": {"factor": 8.0, "orig_ctx": 8192, "low": 1.0, "high": 4.0}}


def _rope_case(vc, Hq, Hkv, d, rot, inter, kind, rows, pos0=0, listed=False, fused=False, amp=1.0, in_place=False,
               keep_meta=True, keys_only=False, seed=0):
    g = gen(seed)
    code = {"none": vc.VC_ROPE_NONE, "linear": vc.VC_ROPE_LINEAR, "ntk": vc.VC_ROPE_NTK, "bands": vc.VC_ROPE_BANDS}[kind]
    layout = vc.VC_ROPE_INTERLEAVED if inter else vc.VC_ROPE_HALF
    table = vc.vc_rope_init(code, rot, layout, 500000.0, amp=amp, **ROPE[kind])
    freqs = O.rope_freqs(kind, rot, 500000.0, **ROPE[kind])
    B = len(rows)
    arr, keep = (vc.vc_rope_req * B)(), []
    for b, R in enumerate(rows):
        n, cap = 5 + 3 * b, 5 + 3 * b + R + 2
        k, v, score, pos = cache(g, Hkv, d, n, cap)
        T = max(R, 1)
        if fused:
            x = randn(g, T, (Hq + 2 * Hkv) * d)
            xq, xk, xv = x.split([Hq * d, Hkv * d, Hkv * d], dim=1)
        else:
            xq, xk, xv = randn(g, T, Hq * d), randn(g, T, Hkv * d), randn(g, T, Hkv * d)
        q_in = xq.clone()
        q_out = xq if in_place else torch.full((T, Hq, d), NAN, dtype=torch.bfloat16, device="cuda")
        at = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32) + pos0 if listed else None
        e = arr[b]
        e.kv = vc.live_kv(k, v, n, score if keep_meta else None, pos if keep_meta else None)
        e.q, e.q_out = (None, None) if keys_only else (xq.data_ptr(), q_out.data_ptr())
        e.k, e.v, e.n_rows, e.pos0 = xk.data_ptr(), xv.data_ptr(), R, pos0 + b
        e.q_stride, e.k_stride, e.v_stride = xq.stride(0), xk.stride(0), xv.stride(0)
        e.pos = at.data_ptr() if listed else None
        where = at.cpu().numpy()[:R] if listed else pos0 + b + np.arange(R)
        keep.append((k, v, score, pos, q_in, xk.clone(), xv.clone(), q_out, where, n, R, at, xq, xk, xv,
                     [t.clone() for t in (k, v, score, pos)]))
    vc.vc_rope_append(vc.vc_shape(B, Hq, Hkv, d), table, arr)
    torch.cuda.synchronize()

    def close(got, x, heads, where, what):
        x = f64(x).reshape(len(where), heads, d)
        ref = O.rope(x, where, freqs, inter, amp)
        mag = np.abs(x)
        lim = 2.0 ** -8 * np.abs(ref)
        h = rot // 2
        a = slice(0, rot, 2) if inter else slice(0, h)
        b = slice(1, rot, 2) if inter else slice(h, rot)
        both = 2.0 ** -20 * abs(amp) * (mag[..., a] + mag[..., b])
        lim[..., a] += both
        lim[..., b] += both
        lim[..., rot:] = 0
        err = np.abs(f64(got).reshape(ref.shape) - ref)
        assert np.all(err <= lim), (what, float((err - lim).max()))

    for k, v, score, pos, q_in, xk, xv, q_out, where, n, R, at, xq, _, _, old in keep:
        if not keys_only and R:
            close(q_out[:R], q_in[:R], Hq, where, "q")
        if R:
            close(k[:, n : n + R].transpose(0, 1), xk[:R], Hkv, where, "k")
        assert np.array_equal(bits(v[:, n : n + R]), bits(xv[:R].reshape(R, Hkv, d).transpose(0, 1)))
        if keep_meta:
            assert not score[:, n : n + R].any() and np.array_equal(pos[:, n : n + R].cpu().numpy(), np.tile(where, (Hkv, 1)))
        for t, o in zip((k, v, score, pos), old):  # nothing else is touched
            lo = (n, n + R) if keep_meta or t.dim() == 3 else (n, n)
            assert np.array_equal(bits(t[:, : lo[0]]), bits(o[:, : lo[0]])) and np.array_equal(bits(t[:, lo[1] :]), bits(o[:, lo[1] :]))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 32)])
def test_rope_layouts(vc, d, rot, inter):
    _rope_case(vc, 8, 2, d, rot, inter, "none", [1, 0, 7], pos0=1000)


@pytest.mark.parametrize("kind", list(ROPE))
def test_rope_scalings(vc, kind):
    _rope_case(vc, 5, 5, 128, 128, False, kind, [3, 33], pos0=12345, amp=1.2)


@pytest.mark.parametrize("pos0", [0, 131071, 10_000_000, 2 ** 31 - 40, -5, -2 ** 31])
def test_rope_far_positions(vc, pos0):
    _rope_case(vc, 4, 1, 64, 64, True, "none", [9, 2], pos0=pos0)


def test_rope_listed_positions_fused_projection(vc):
    _rope_case(vc, 40, 8, 128, 64, True, "linear", [25, 1, 17], pos0=65536, listed=True, fused=True)


def test_rope_in_place_and_without_meta(vc):
    _rope_case(vc, 16, 2, 128, 128, False, "none", [5, 300], in_place=True, keep_meta=False)
    _rope_case(vc, 16, 2, 128, 64, True, "none", [5], in_place=True)


def test_rope_keys_only(vc):
    _rope_case(vc, 8, 2, 64, 32, False, "none", [4, 1], keys_only=True)


def test_rope_full_batch(vc):
    _rope_case(vc, 8, 8, 64, 64, False, "none", [1 + b % 3 for b in range(32)], pos0=77)


# ---- attention -----------------------------------------------------------------------------------
def _attn_case(vc, Hq, Hkv, d, ns, rows, P=None, scored=False, seed=0, spread=1.0, ws_fill=NAN, own_ws=None):
    """ns[b] own rows, rows[b] query rows, P prefix rows (None: no prefix)."""
    g = gen(seed)
    B = len(ns)
    arr, keep = (vc.vc_live_req * B)(), []
    for b in range(B):
        cap = max(1, ns[b] + 3 - b % 2)
        k, v, score, pos = cache(g, Hkv, d, ns[b], cap)
        q = randn(g, max(rows[b], 1), Hq, d) * spread
        o = torch.full((max(rows[b], 1) + 1, Hq, d), NAN, dtype=torch.bfloat16, device="cuda")
        arr[b] = vc.vc_live_req(q.data_ptr(), o.data_ptr(), rows[b], vc.live_kv(k, v, ns[b], score if scored else None))
        keep.append((q, k, v, score, o, score.clone()))
    shape = vc.vc_shape(B, Hq, Hkv, d)
    prefix = pk = pv = None
    if P is not None:
        pk, pv, _, _ = cache(g, Hkv, d, P, P + 2)
        prefix = vc.vc_kv_full(pk.data_ptr(), pv.data_ptr(), P, P + 2)
    R = max(max(rows), 1)
    size = vc.vc_scored_workspace_size(shape, R, max(ns)) if scored else vc.vc_prefix_workspace_size(shape, R)
    ws = torch.full(((size + 3) // 4,), ws_fill, device="cuda") if own_ws is None else own_ws
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if scored:
        vc.vc_scored_attn(shape, arr, ws, status)
    else:
        vc.vc_prefix_attn(shape, prefix, arr, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for b, (q, k, v, score, o, old) in enumerate(keep):
        n, r = ns[b], rows[b]
        assert torch.isnan(o[r:]).all()
        pre = None if P is None else (f64(pk[:, :P]), f64(pv[:, :P]))
        if r > 0:
            ref, w = O.live_attn(f64(q[:r]), f64(k[:, :n]), f64(v[:, :n]), pre)
            seen = [(P or 0) + max(0, n - r + i + 1) > 0 for i in range(r)]
            for i in range(r):
                if not seen[i]:
                    assert not o[i].any(), "a row that sees nothing"
            if any(seen):
                assert_attn_close(o[:r][torch.tensor(seen)], ref[np.array(seen)], f"request {b}")
        if scored:
            got, was = f64(score), f64(old)
            assert np.array_equal(bits(score[:, n:]), bits(old[:, n:]))
            if r > 0 and n > 0:
                G = Hq // Hkv
                qq = np.abs(f64(q[:r])).reshape(r, Hkv, G, d)
                mag = np.einsum("rhgd,htd->rhgt", qq, np.abs(f64(k[:, :n]))).max() / np.sqrt(d)
                lim = w * (2 * d * 2.0 ** -23 * mag + 2.0 ** -20) + 2.0 ** -23 * (was[:, :n] + w)
                err = np.abs(got[:, :n] - (was[:, :n] + w))
                assert np.all(err <= lim), (b, float((err / np.maximum(lim, 1e-300)).max()))
            else:
                assert np.array_equal(bits(score), bits(old))
    return keep


SHAPES = [(8, 2, 64), (32, 8, 128), (5, 1, 128), (4, 4, 64), (32, 2, 128), (40, 8, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("scored", [False, True])
def test_attn_one_token(vc, Hq, Hkv, d, scored):
    _attn_case(vc, Hq, Hkv, d, [1, 300, 127, 128, 129, 64], [1] * 6, P=None if scored else 260, scored=scored)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000])
@pytest.mark.parametrize("scored", [False, True])
def test_attn_lengths(vc, n, scored):
    _attn_case(vc, 8, 2, 64, [n], [1], P=None if scored else 5, scored=scored, seed=n)
    _attn_case(vc, 8, 2, 128, [n], [min(n, 7)], P=None if scored else n, scored=scored, seed=n + 1)


@pytest.mark.parametrize("scored", [False, True])
def test_attn_many_rows(vc, scored):
    """Several rows a request: causal among themselves, over tile edges; ragged, some requests idle."""
    _attn_case(vc, 8, 2, 64, [200, 64, 130, 7, 500], [64, 64, 3, 0, 33], P=None if scored else 300, scored=scored)
    _attn_case(vc, 16, 2, 128, [140, 33], [32, 17], P=None if scored else 129, scored=scored)


def test_prefix_rows_beyond_two_tiles(vc):
    """Query rows of all requests together fill one, two and many 128-row tiles of the prefix."""
    for rows in ([1] * 32, [16] * 2, [40, 25, 1, 64], [129, 3], [200]):
        _attn_case(vc, 8, 2, 64, [r + 11 * b for b, r in enumerate(rows)], rows, P=333)
    _attn_case(vc, 40, 8, 128, [300, 31], [25, 30], P=1000)


def test_prefix_empty_parts(vc):
    """No own rows, no prefix rows, neither; rows whose mask leaves nothing."""
    _attn_case(vc, 8, 2, 64, [0, 5, 0], [2, 1, 0], P=100)
    _attn_case(vc, 8, 2, 64, [50, 5], [2, 1], P=0)
    _attn_case(vc, 8, 2, 64, [50, 0, 2], [2, 1, 6])
    _attn_case(vc, 8, 2, 64, [0, 0], [3, 1])


def test_scored_empty_parts(vc):
    _attn_case(vc, 8, 2, 64, [0, 5, 3, 9], [2, 1, 6, 0], scored=True)


@pytest.mark.parametrize("scored", [False, True])
def test_attn_peaked_and_flat(vc, scored):
    """Scores with a spread of tens (one key takes the weight, the running maximum moves) and nearly none."""
    for spread in (6.0, 0.01):
        _attn_case(vc, 8, 2, 128, [900, 300], [2, 5], P=None if scored else 700, scored=scored, spread=spread)


@pytest.mark.parametrize("scored", [False, True])
def test_attn_long(vc, scored):
    _attn_case(vc, 16, 2, 128, [20000, 3333], [1, 2], P=None if scored else 30011, scored=scored)


@pytest.mark.parametrize("scored", [False, True])
def test_attn_full_batch(vc, scored):
    _attn_case(vc, 8, 2, 64, [1 + 37 * b for b in range(32)], [1 + b % 2 for b in range(32)], P=None if scored else 77,
               scored=scored)


@pytest.mark.parametrize("bad", [NAN, float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("scored", [False, True])
def test_attn_rows_not_seen_do_not_reach(vc, scored, bad):
    """K and V of the last new token are broken: the rows before it come out as without it."""
    g = gen(3)
    for d, Hq, Hkv, n, r in ((64, 8, 2, 150, 4), (128, 40, 8, 130, 30), (128, 4, 4, 128, 128)):
        P = 0 if scored else 70
        q, (k, v, score, _) = randn(g, r, Hq, d), cache(g, Hkv, d, n, n + 1)
        pk, pv, _, _ = cache(g, Hkv, d, P + 1, P + 1)
        outs = []
        for broken in (False, True):
            if broken:
                k[:, n - 1], v[:, n - 1] = bad, bad
            o, s = torch.zeros_like(q), score.clone()
            shape = vc.vc_shape(1, Hq, Hkv, d)
            arr = (vc.vc_live_req * 1)(vc.vc_live_req(q.data_ptr(), o.data_ptr(), r, vc.live_kv(k, v, n, s)))
            if scored:
                vc.vc_scored_attn(shape, arr, torch.empty(vc.vc_scored_workspace_size(shape, r, n), dtype=torch.uint8, device="cuda"))
            else:
                vc.vc_prefix_attn(shape, vc.vc_kv_full(pk.data_ptr(), pv.data_ptr(), P, P + 1), arr,
                                  torch.empty(vc.vc_prefix_workspace_size(shape, r), dtype=torch.uint8, device="cuda"))
            torch.cuda.synchronize()
            outs.append(o)
        assert torch.isfinite(outs[1][: r - 1]).all()
        # bf16 weights, summed the same or in another order: each output within two roundings of the other's
        assert torch.all((outs[0][: r - 1].float() - outs[1][: r - 1].float()).abs() <= 2.0 ** -6 * (outs[0][: r - 1].float().abs() + 1))
        assert not torch.isfinite(outs[1][r - 1]).all() or bad == 3e38


def test_scored_same_bits_twice(vc):
    a = _attn_case(vc, 32, 8, 128, [5000, 300], [2, 1], scored=True, seed=9)
    b = _attn_case(vc, 32, 8, 128, [5000, 300], [2, 1], scored=True, seed=9, ws_fill=1e30)
    for x, y in zip(a, b):
        assert np.array_equal(bits(x[3]), bits(y[3])) and np.array_equal(bits(x[4]), bits(y[4]))


def test_workspaces_are_large_enough_and_checked(vc):
    """The sizes that the library names suffice exactly (guard words behind them stay), and one byte
    less than a call needs is refused."""
    for scored in (False, True):
        shape = vc.vc_shape(3, 8, 2, 64)
        ns, rows = [500, 70, 300], [9, 9, 2]
        size = vc.vc_scored_workspace_size(shape, 9, 500) if scored else vc.vc_prefix_workspace_size(shape, 9)
        buf = torch.zeros(size + 256, dtype=torch.uint8, device="cuda")
        _attn_case(vc, 8, 2, 64, ns, rows, P=None if scored else 300, scored=scored, own_ws=buf[:size])
        assert not buf[size:].any()


# ---- eviction --------------------------------------------------------------------------------------
def _evict_case(vc, Hkv, d, ns, keeps, sink=0, recent=0, seed=0, kind="random", ws=None):
    g = gen(seed)
    B = len(ns)
    arr, state = (vc.vc_evict_req * B)(), []
    for b in range(B):
        n, cap = ns[b], ns[b] + 2
        k, v, score, _ = cache(g, Hkv, d, n, cap)
        if kind == "ties":
            score = torch.randint(0, 3, (Hkv, cap), generator=g, device="cuda").float()
            score[torch.rand((Hkv, cap), generator=g, device="cuda") < 0.3] = -0.0
        elif kind == "equal":
            score = torch.full((Hkv, cap), 0.25, device="cuda")
        elif kind == "odd":
            pick = torch.randint(0, 6, (Hkv, cap), generator=g, device="cuda")
            vals = torch.tensor([NAN, float("inf"), float("-inf"), 1e-40, -1.5, 2.0], device="cuda")
            score = vals[pick]
        elif kind == "ascending":
            score = torch.arange(cap, device="cuda").float().repeat(Hkv, 1)
        elif kind == "descending":
            score = -torch.arange(cap, device="cuda").float().repeat(Hkv, 1)
        pos = torch.rand((Hkv, cap), generator=g, device="cuda").argsort(1).int()
        rf = n - recent if recent else 2 ** 31 - 1
        arr[b] = vc.vc_evict_req(vc.live_kv(k, v, n, score, pos), keeps[b], sink, rf)
        state.append((k, v, score, pos, [t.clone() for t in (k, v, score, pos)], rf))
    shape = vc.vc_shape(B, Hkv * 2, Hkv, d)
    size = vc.vc_evict_workspace_size(shape, max(ns))
    buf = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc.vc_evict_kv(shape, arr, buf[:size], status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and bool((buf[size:] == 0x5A).all())
    for b, (k, v, score, pos, old, rf) in enumerate(state):
        for h in range(Hkv):
            holes, moves = O.evict(old[2][h, : ns[b]].cpu().numpy(), old[3][h, : ns[b]].cpu().numpy(), keeps[b], sink, rf)
            for got, was in zip((k, v, score, pos), old):
                want = was[h].clone()
                want[holes] = was[h][moves]
                assert np.array_equal(bits(got[h]), bits(want)), (b, h, got.dtype)


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd", "ascending", "descending"])
@pytest.mark.parametrize("n,keep", [(2, 1), (33, 32), (100, 1), (100, 99), (777, 300), (5000, 4095)])
def test_evict(vc, kind, n, keep):
    _evict_case(vc, 2, 64, [n], [keep], kind=kind, seed=n)
    _evict_case(vc, 3, 128, [n, n // 2 + 1], [keep, keep], sink=2, recent=n // 4, kind=kind, seed=n + 1)


def test_evict_guards_beyond_the_budget(vc):
    """More guarded rows than the budget holds: the lowest of them stay. Every row guarded, none guarded."""
    _evict_case(vc, 2, 64, [300], [100], sink=50, recent=200)
    _evict_case(vc, 2, 64, [300], [100], sink=2 ** 31 - 1)
    _evict_case(vc, 2, 64, [300], [100], sink=-5)


def test_evict_batch_and_long(vc):
    _evict_case(vc, 2, 64, [50 + 31 * b for b in range(32)], [60] * 32, sink=4, recent=16, kind="ties")
    _evict_case(vc, 2, 128, [70001, 200, 40000], [20000, 300, 39999], sink=4, recent=500)


@pytest.mark.parametrize("kind", ["random", "ties"])
@pytest.mark.parametrize("n", [2047, 2048, 2100, 4095, 4096, 8191, 8192, 9000, 40960, 81920, 81921])
def test_evict_at_the_edges_of_the_cluster_sizes(vc, n, kind):
    _evict_case(vc, 1, 64, [n, 1500], [n - n // 3, 700], sink=3, recent=100, kind=kind, seed=n)


def test_evict_more_rows_than_the_ranks_held(vc):
    """Beyond 8 x 40960 rows the select kernel takes the ranks from memory again in every pass."""
    _evict_case(vc, 1, 64, [327681, 1000], [200000, 999], sink=4, recent=700)
    _evict_case(vc, 1, 64, [400000], [399990], kind="ties")


# ---- together ----------------------------------------------------------------------------------------
def _table(vc, d):
    return vc.vc_rope_init(vc.VC_ROPE_BANDS, d, vc.VC_ROPE_HALF, 500000.0, **ROPE["bands"])


def test_live_batch_decodes_within_its_budget(vc):
    """Three requests, a prompt chunk then single tokens: append, attend, evict, each against the oracle
    applied to the state the call found; the caches never exceed budget + slack after a step."""
    from lossless_compressed_kv_vc_gb300 import engine
    Hq, Hkv, d, B, R, budget, slack, recent = 8, 2, 64, 3, 12, 40, 3, 8
    g = gen(5)
    lb = engine.LiveBatch(Hq, Hkv, d, B, 64, _table(vc, d), max_rows=R, budget=budget, slack=slack, sink=2, recent=recent)
    freqs = O.rope_freqs("bands", d, 500000.0, **ROPE["bands"])
    evictions = 0
    for step in range(45):
        rows = [R, 5, 0] if step == 0 else [1, 1, 1] if step != 20 else [7, 0, 12]
        x = randn(g, B, R, (Hq + 2 * Hkv) * d)
        q, k, v = (t.unflatten(2, (-1, d)) for t in x.split([Hq * d, Hkv * d, Hkv * d], 2))
        o = torch.zeros((B, R, Hq, d), dtype=torch.bfloat16, device="cuda")
        first, p0 = list(lb.n), list(lb.next_pos)
        lb.append(q, k, v, rows)
        torch.cuda.synchronize()
        for b in range(B):
            at = p0[b] + np.arange(rows[b])
            ref = O.rope(f64(q[b, : rows[b]]), at, freqs, False)
            assert np.all(np.abs(f64(lb.q_rot[b, : rows[b]]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18)
            assert lb.n[b] == first[b] + rows[b] and lb.next_pos[b] == p0[b] + rows[b]
            assert np.array_equal(lb.pos[b, :, first[b] : lb.n[b]].cpu().numpy(), np.tile(at, (Hkv, 1)))
        was = lb.score.clone()
        lb.attend(o, rows)
        torch.cuda.synchronize()
        for b in range(B):
            if rows[b] == 0:
                assert torch.equal(lb.score[b], was[b])
                continue
            ref, w = O.live_attn(f64(lb.q_rot[b, : rows[b]]), f64(lb.k[b, :, : lb.n[b]]), f64(lb.v[b, :, : lb.n[b]]))
            assert_attn_close(o[b, : rows[b]], ref, f"step {step} request {b}")
            got = f64(lb.score[b, :, : lb.n[b]]) - f64(was[b, :, : lb.n[b]])
            # weights as derived at the top, with at most 16 for sum|q k| / sqrt(d); scores of at most 50
            assert np.all(np.abs(got - w) <= w * (2 * d * 2.0 ** -23 * 16 + 2.0 ** -20) + 2.0 ** -23 * 50)
        old = [t.clone() for t in (lb.k, lb.v, lb.score, lb.pos)]
        n = list(lb.n)
        lb.evict()
        torch.cuda.synchronize()
        for b in range(B):
            over = n[b] > budget + slack
            evictions += over
            assert lb.n[b] == (budget if over else n[b])
            for h in range(Hkv):
                holes, moves = O.evict(old[2][b, h, : n[b]].cpu().numpy(), old[3][b, h, : n[b]].cpu().numpy(), budget, 2,
                                       lb.next_pos[b] - recent) if over else ([], [])
                for got, t in zip((lb.k, lb.v, lb.score, lb.pos), old):
                    want = t[b, h].clone()
                    want[holes] = t[b, h][moves]
                    assert np.array_equal(bits(got[b, h]), bits(want))
            kept = lb.pos[b, 0, : lb.n[b]].tolist()
            assert len(set(kept)) == len(kept) and set(range(lb.next_pos[b] - min(recent, lb.next_pos[b]), lb.next_pos[b])) <= set(kept)
    assert evictions == 10 and int(lb.dev_status.item()) == 0  # 62, 48 and 55 tokens: every fourth row beyond 40


def test_live_batch_over_a_shared_prefix(vc):
    """Decode steps over a prefix equal the same requests with the prefix in their own caches."""
    from lossless_compressed_kv_vc_gb300 import engine
    Hq, Hkv, d, B, P = 16, 4, 128, 4, 150
    g = gen(6)
    pk, pv, _, _ = cache(g, Hkv, d, P, P + 9)
    shared = engine.LiveBatch(Hq, Hkv, d, B, 40, _table(vc, d), prefix=(pk, pv, P))
    whole = engine.LiveBatch(Hq, Hkv, d, B, 40 + P, _table(vc, d))
    whole.k[:, :, :P], whole.v[:, :, :P] = pk[:, :P], pv[:, :P]
    whole.n, whole.next_pos = [P] * B, [P] * B
    for step in range(30):
        q, k, v = randn(g, B, 1, Hq, d), randn(g, B, 1, Hkv, d), randn(g, B, 1, Hkv, d)
        rows = [int((b + step) % 4 != 3) for b in range(B)]
        a, c = torch.zeros_like(q), torch.zeros_like(q)
        shared.step(q, k, v, a, rows)
        whole.step(q, k, v, c, rows)
        torch.cuda.synchronize()
        assert shared.next_pos == whole.next_pos
        for b in range(B):
            if rows[b]:
                assert_attn_close(a[b], f64(c[b]), f"step {step} request {b}")
    assert int(shared.dev_status.item()) == 0 and int(whole.dev_status.item()) == 0


def test_live_batch_refusals(vc):
    from lossless_compressed_kv_vc_gb300 import engine
    t = _table(vc, 64)
    with pytest.raises(ValueError):
        engine.LiveBatch(8, 2, 64, 1, 10, t, budget=10)          # no room for the next row
    with pytest.raises(ValueError):
        engine.LiveBatch(8, 2, 64, 1, 10, t, budget=4, prefix=(None, None, 0))
    with pytest.raises(ValueError):
        engine.LiveBatch(8, 2, 64, 1, 100, t, max_rows=65)       # more rows than a scored call takes
    lb = engine.LiveBatch(8, 2, 64, 2, 10, t)
    x = lambda h, dt=torch.bfloat16: torch.zeros((2, 1, h, 64), dtype=dt, device="cuda")
    for q, k, rows in ((x(8), x(3), [1, 1]), (x(8, torch.float32), x(2), [1, 1]), (x(8), x(2), [1]), (x(8), x(2), [2, 1]),
                       (x(8), x(2), [-1, 1]), (x(8).expand(2, 1, 8, 64)[..., ::2], x(2), [1, 1])):
        with pytest.raises(ValueError):
            lb.append(q, k, x(2), rows)
    with pytest.raises(ValueError):
        lb.attend(x(8, torch.float32), [1, 1])
    for rows in ([2, 1], [1], [-1, 1]):                          # more rows than the batch holds queries for
        with pytest.raises(ValueError):
            lb.attend(x(8), rows)
    pk = torch.zeros((2, 20, 64), dtype=torch.bfloat16, device="cuda")
    for prefix in ((pk, pk[:1], 5), (pk, pk, 21), (pk, pk, -1), (pk.float(), pk.float(), 5), (pk[:, ::2], pk[:, ::2], 5)):
        with pytest.raises(ValueError):
            engine.LiveBatch(8, 2, 64, 1, 10, t, prefix=prefix)
    lb.n = [10, 0]
    with pytest.raises(vc.VCError):                               # full: the call is refused, nothing moves on
        lb.append(x(8), x(2), x(2), [1, 1])
    assert lb.n == [10, 0] and lb.next_pos == [0, 0]


def test_captured_step_replays(vc):
    """append + attend + evict of one step as a CUDA graph: replays on new inputs equal eager steps from
    the same state."""
    from lossless_compressed_kv_vc_gb300 import engine
    Hq, Hkv, d, B = 8, 2, 64, 2
    g = gen(8)
    make = lambda: engine.LiveBatch(Hq, Hkv, d, B, 160, _table(vc, d), budget=128, slack=0, recent=4)
    eager, graph = make(), make()
    for lb in (eager, graph):
        g2 = gen(9)
        lb.k.copy_(randn(g2, *lb.k.shape))
        lb.v.copy_(randn(g2, *lb.v.shape))
        lb.score.copy_(torch.rand(lb.score.shape, generator=g2, device="cuda"))
        lb.pos.copy_(torch.arange(160, device="cuda").int().expand_as(lb.pos))
        lb.n, lb.next_pos = [128, 128], [128, 128]
    q, k, v = randn(g, B, 1, Hq, d), randn(g, B, 1, Hkv, d), randn(g, B, 1, Hkv, d)
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        graph.step(q, k, v, o2)
    for _ in range(3):
        q.copy_(randn(g, *q.shape))
        k.copy_(randn(g, *k.shape))
        eager.n, eager.next_pos = [128, 128], [128, 128]  # the graph's step holds these
        eager.step(q, k, v, o1)
        cg.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, o2) and torch.equal(eager.score, graph.score) and torch.equal(eager.pos, graph.pos)
        assert torch.equal(eager.k, graph.k) and torch.equal(eager.v, graph.v)


def test_two_streams_with_a_workspace_each(vc):
    from lossless_compressed_kv_vc_gb300 import engine
    Hq, Hkv, d, B = 32, 8, 128, 4
    g = gen(10)
    q, k, v = randn(g, B, 1, Hq, d), randn(g, B, 1, Hkv, d), randn(g, B, 1, Hkv, d)

    def make():
        lb = engine.LiveBatch(Hq, Hkv, d, B, 3000, _table(vc, d), budget=2500, recent=100)
        g2 = gen(11)
        lb.k.copy_(randn(g2, *lb.k.shape))
        lb.v.copy_(randn(g2, *lb.v.shape))
        lb.pos.copy_(torch.arange(3000, device="cuda").int().expand_as(lb.pos))
        lb.n, lb.next_pos = [2490] * B, [2490] * B
        return lb

    alone, one, two = make(), make(), make()
    outs = [torch.zeros_like(q) for _ in range(3)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(30):
        alone.step(q, k, v, outs[0])
        one.step(q, k, v, outs[1], stream=s1)
        with torch.cuda.stream(s2):
            two.step(q, k, v, outs[2])
    torch.cuda.synchronize()
    for lb, o in ((one, outs[1]), (two, outs[2])):
        assert torch.equal(o, outs[0]) and torch.equal(lb.score, alone.score) and torch.equal(lb.pos, alone.pos)
        assert torch.equal(lb.k, alone.k) and torch.equal(lb.v, alone.v)


def test_draft_after_rope_reads_the_new_queries(vc):
    """vc_draft_attn may start reading before the kernel ahead of it ends, but not its queries while
    vc_rope_append writes them: the draft of freshly rotated queries equals the draft of settled ones."""
    from lossless_compressed_kv_vc_gb300 import engine
    from workloads import configs
    from tests.util import make_batch
    w = configs.scaled(configs.llama8b_drop(), ctx_div=16, batch=8, L=1)
    bt = make_batch(w, list(range(8)))
    bt.compress()
    lb = engine.LiveBatch(w.Hq, w.Hkv, w.d, 8, 64, _table(vc, w.d))
    g = gen(12)
    k, v = randn(g, 8, 1, w.Hkv, w.d), randn(g, 8, 1, w.Hkv, w.d)
    for b, r in enumerate(bt.reqs):
        r.q = lb.q_rot[b]
    for _ in range(20):
        q = randn(g, 8, 1, w.Hq, w.d)
        torch.cuda.synchronize()
        lb.append(q, k, v, [1] * 8)
        bt.draft_step(0)
        got = [r.o_draft.clone() for r in bt.reqs]
        torch.cuda.synchronize()
        bt.reset_window()
        bt.draft_step(0)
        torch.cuda.synchronize()
        for a, r in zip(got, bt.reqs):
            assert torch.equal(a, r.o_draft)
        bt.reset_window()


def test_offsets_beyond_32_bits(vc):
    """Caches whose second head starts beyond 2^31 elements (2^32 bytes): append, both attentions, eviction."""
    Hq, Hkv, d, n, cap = 4, 2, 128, 300, (1 << 24) + 5
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 20 GB")
    g = gen(21)
    k, v = (torch.empty((Hkv, cap, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    score = torch.empty((Hkv, cap), device="cuda")
    pos = torch.empty((Hkv, cap), dtype=torch.int32, device="cuda")
    k[:, :n], v[:, :n] = randn(g, Hkv, n, d), randn(g, Hkv, n, d)
    k[:, n : n + 200], v[:, n : n + 200] = NAN, NAN
    score[:, :n] = torch.rand((Hkv, n), generator=g, device="cuda")
    pos[:, :n] = torch.arange(n, device="cuda").int()
    q, kn, vn = randn(g, 3, Hq, d), randn(g, 3, Hkv, d), randn(g, 3, Hkv, d)
    q_rot, o = torch.empty_like(q), torch.empty_like(q)
    table = _table(vc, d)
    shape = vc.vc_shape(1, Hq, Hkv, d)
    e = vc.vc_rope_req(q=q.data_ptr(), k=kn.data_ptr(), v=vn.data_ptr(), pos0=n, n_rows=3, q_out=q_rot.data_ptr(),
                       kv=vc.live_kv(k, v, n, score, pos))
    vc.vc_rope_append(shape, table, (vc.vc_rope_req * 1)(e))
    n += 3
    torch.cuda.synchronize()
    freqs = O.rope_freqs("bands", d, 500000.0, **ROPE["bands"])
    ref = O.rope(f64(kn), n - 3 + np.arange(3), freqs, False)
    assert np.all(np.abs(f64(k[:, n - 3 : n].transpose(0, 1)) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18)
    assert torch.equal(v[:, n - 3 : n], vn.transpose(0, 1)) and not score[:, n - 3 : n].any()
    assert torch.isnan(k[:, n : n + 197]).all()
    was = score[:, :n].clone()
    live = (vc.vc_live_req * 1)(vc.vc_live_req(q_rot.data_ptr(), o.data_ptr(), 3, vc.live_kv(k, v, n, score)))
    ref, w = O.live_attn(f64(q_rot), f64(k[:, :n]), f64(v[:, :n]))
    ws = torch.empty(max(vc.vc_scored_workspace_size(shape, 3, n), vc.vc_prefix_workspace_size(shape, 3),
                         vc.vc_evict_workspace_size(shape, n)), dtype=torch.uint8, device="cuda")
    vc.vc_scored_attn(shape, live, ws)
    torch.cuda.synchronize()
    assert_attn_close(o, ref, "scored")
    # as derived at the top of the file, with at most 16 for sum|q k| / sqrt(d)
    assert np.all(np.abs(f64(score[:, :n]) - f64(was) - w) <= w * (2 * d * 2.0 ** -23 * 16 + 2.0 ** -20) + 2.0 ** -22)
    o.zero_()
    vc.vc_prefix_attn(shape, vc.vc_kv_full(k.data_ptr(), v.data_ptr(), n - 100, cap), live, ws)
    torch.cuda.synchronize()
    both, _ = O.live_attn(f64(q_rot), f64(k[:, :n]), f64(v[:, :n]), (f64(k[:, : n - 100]), f64(v[:, : n - 100])))
    assert_attn_close(o, both, "prefix")
    old = [t[:, :n].clone() for t in (k, v, score, pos)]
    vc.vc_evict_kv(shape, (vc.vc_evict_req * 1)(vc.vc_evict_req(vc.live_kv(k, v, n, score, pos), 120, 4, n - 10)), ws)
    torch.cuda.synchronize()
    for h in range(Hkv):
        holes, moves = O.evict(old[2][h].cpu().numpy(), old[3][h].cpu().numpy(), 120, 4, n - 10)
        for t, was in zip((k, v, score, pos), old):
            want = was[h].clone()
            want[holes] = was[h][moves]
            assert np.array_equal(bits(t[h, :n]), bits(want))


def test_prefix_requests_may_share_an_own_cache(vc):
    """vc_prefix_attn only reads caches: two requests over one, each with its own rows."""
    g = gen(22)
    Hq, Hkv, d, n = 8, 2, 64, 90
    k, v, _, _ = cache(g, Hkv, d, n, n + 4)
    qs = [randn(g, r, Hq, d) for r in (1, 3)]
    os_ = [torch.zeros_like(q) for q in qs]
    shape = vc.vc_shape(2, Hq, Hkv, d)
    arr = (vc.vc_live_req * 2)(*[vc.vc_live_req(q.data_ptr(), o.data_ptr(), q.shape[0], vc.live_kv(k, v, n)) for q, o in zip(qs, os_)])
    vc.vc_prefix_attn(shape, None, arr, torch.empty(vc.vc_prefix_workspace_size(shape, 3), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for q, o in zip(qs, os_):
        assert_attn_close(o, O.live_attn(f64(q), f64(k[:, :n]), f64(v[:, :n]))[0])


@pytest.mark.parametrize("Hq,Hkv,d", [(64, 64, 64), (48, 1, 128), (96, 2, 64), (300, 1, 64)])
def test_prefix_uncommon_head_counts(vc, Hq, Hkv, d):
    """A query head per KV head, many heads on one, groups that do not divide a tile, more than a unit of them."""
    _attn_case(vc, Hq, Hkv, d, [70, 200, 5], [3, 1, 5], P=150)


@pytest.mark.parametrize("Hq,Hkv,d", [(64, 64, 64), (48, 1, 128), (96, 2, 64), (256, 1, 64)])
def test_scored_uncommon_head_counts(vc, Hq, Hkv, d):
    _attn_case(vc, Hq, Hkv, d, [70, 200, 1], [1, 256 // (Hq // Hkv) if Hq // Hkv > 1 else 7, 1], scored=True)


def test_draft_after_eviction_and_accept(vc):
    """A draft's compact rows shrunk in place by vc_evict_kv, then vc_accept, then two draft steps, none waited
    for on the host: accept lets its followers start before it ends, and the drafts must not read rows that are
    still being moved. Equal to the same drafts on settled rows."""
    Hq, Hkv, d, n, keep, L = 32, 8, 128, 40000, 20000, 2
    g = gen(30)
    k0, v0 = randn(g, Hkv, n, d), randn(g, Hkv, n, d)
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(Hkv, n).contiguous()
    kw, vw = (torch.zeros((Hkv, 4, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, kn, vn = randn(g, L, Hq, d), randn(g, Hkv, d), randn(g, Hkv, d)
    shape = vc.vc_shape(1, Hq, Hkv, d)
    ws = torch.zeros(vc.vc_workspace_size(vc.VC_CALL_DRAFT, shape, 0), dtype=torch.uint8, device="cuda")
    ws_e = torch.empty(vc.vc_evict_workspace_size(shape, n), dtype=torch.uint8, device="cuda")
    logits = torch.randn((1, 2, 512), generator=g, device="cuda")
    tok = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens, out_tok = torch.ones(1, dtype=torch.int32, device="cuda"), torch.empty((1, 2), dtype=torch.int32, device="cuda")
    n_acc = torch.empty(1, dtype=torch.int32, device="cuda")
    for _ in range(10):
        k, v, p = k0.clone(), v0.clone(), pos.clone()
        score = torch.rand((Hkv, n), generator=g, device="cuda")
        comp = vc.vc_kv_comp(mode=vc.VC_TOKEN_DROP, keep=keep, compact=1, k_rows=k.data_ptr(), v_rows=v.data_ptr(),
                             rows_cap=n, k_win=kw.data_ptr(), v_win=vw.data_ptr(), win_cap=4)

        def drafts():
            o = torch.empty((L, Hq, d), dtype=torch.bfloat16, device="cuda")
            for step in range(L):
                comp.n_win = step
                req = (vc.vc_draft_req * 1)(vc.vc_draft_req(q=q[step].data_ptr(), k_new=kn.data_ptr(),
                                                            v_new=vn.data_ptr(), o=o[step].data_ptr(), comp=comp))
                vc.vc_draft_attn(shape, req, ws)
            return o

        evict = (vc.vc_evict_req * 1)(vc.vc_evict_req(vc.live_kv(k, v, n, score, p), keep, 4, n - 10))
        torch.cuda.synchronize()
        vc.vc_evict_kv(shape, evict, ws_e)
        vc.vc_accept(1, 1, 512, logits, tok, lens, out_tok, n_acc)
        got = drafts()
        torch.cuda.synchronize()
        assert torch.equal(got, drafts())


@pytest.mark.parametrize("rows", [1, 3, 8, 64])
def test_scored_around_the_score_blocks(vc, rows):
    """Lengths around the blocks of keys that scores are added up in, with few rows and with many."""
    _attn_case(vc, 8, 2, 64, [255, 256, 257, 511, 513, 1023, 1025, 2049], [rows] * 8, scored=True)


def test_scored_many_rows_of_long_caches(vc):
    """128 query rows a head over keys of many CTAs: more partials a row than a warp's lanes."""
    _attn_case(vc, 32, 2, 128, [14419, 9000], [8, 8], scored=True)


def test_live_batch_refuses_host_tensors(vc):
    """A tensor in host memory is turned down before its address reaches a kernel."""
    from lossless_compressed_kv_vc_gb300 import engine
    t = _table(vc, 64)
    z = lambda h, dev: torch.zeros((1, 1, h, 64), dtype=torch.bfloat16, device=dev)
    lb = engine.LiveBatch(8, 2, 64, 1, 10, t)
    for args in ((z(8, "cpu"), z(2, "cuda"), z(2, "cuda")), (z(8, "cuda"), z(2, "cpu"), z(2, "cuda")),
                 (z(8, "cuda"), z(2, "cuda"), z(2, "cpu"))):
        with pytest.raises(ValueError):
            lb.append(*args, [1])
    with pytest.raises(ValueError):
        lb.attend(z(8, "cpu"), [1])
    pk = torch.zeros((2, 20, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        engine.LiveBatch(8, 2, 64, 1, 10, t, prefix=(pk, pk, 5))
    assert lb.n == [0] and lb.next_pos == [0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [None, 70, 1000])
def test_prefix_many_rows_of_few_keys(vc, d, P):
    """More rows than a wave of warps, each with a few partials: rows that see nothing, empty own caches, several
    units a head."""
    _attn_case(vc, 32, 2, d, [66, 300, 20, 0, 41], [40, 41, 39, 40, 1], P=P)
