"""Live caches without a GPU: the oracle's pins, the rotary table, and every refusal of the C ABI and
the engine (validation runs before any CUDA call; the pointers are fake and never dereferenced)."""
import ctypes
import math

import numpy as np
import pytest

import oracle as O


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


# ---- oracle pins ---------------------------------------------------------------------------------
def test_rope_is_a_rotation_by_position():
    """A pair at position p has turned by p theta; scores depend on the distance of positions alone."""
    f = O.rope_freqs("none", 16, 100.0)
    assert f[0] == 1.0 and math.isclose(f[4], 0.1)
    x = np.zeros((1, 1, 20))
    x[..., 0] = 1.0
    y = O.rope(x, [3], f, interleaved=False)
    assert math.isclose(y[0, 0, 0], math.cos(3)) and math.isclose(y[0, 0, 8], math.sin(3)) and not y[0, 0, 16:].any()
    y = O.rope(x, [3], f, interleaved=True)
    assert math.isclose(y[0, 0, 0], math.cos(3)) and math.isclose(y[0, 0, 1], math.sin(3))
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 16))
    dots = [float((O.rope(q, [p + 5], f, False) * O.rope(k, [p], f, False)).sum()) for p in (0, 7, 1000)]
    assert np.allclose(dots, dots[0])


def test_rope_bands_edges():
    f0 = O.rope_freqs("none", 128, 500000.0)
    f = O.rope_freqs("bands", 128, 500000.0, 8.0, 8192, 1.0, 4.0)
    turns = 8192 * f0 / (2 * math.pi)
    assert np.allclose(f[turns > 4], f0[turns > 4]) and np.allclose(f[turns < 1], f0[turns < 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all(f[mid] < f0[mid]) and np.all(f[mid] > f0[mid] / 8)


def test_live_attn_against_the_other_oracle_and_closed_forms():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    o, w = O.live_attn(q, k, v)
    ref = O.verify_attn(q, k[:, :6], v[:, :6], k[:, 6:], v[:, 6:])
    assert np.allclose(o, ref)
    assert math.isclose(w.sum(), 3 * 4)  # every row and head spreads a weight of one
    # a prefix is as good as rows in front of the own ones
    o2, w2 = O.live_attn(q, k[:, 5:], v[:, 5:], (k[:, :5], v[:, :5]))
    assert np.allclose(o2, o) and np.allclose(w2, w[:, 5:])
    # a row with nothing to see
    o3, _ = O.live_attn(q, k[:, :2], v[:, :2])
    assert not o3[0].any() and np.allclose(o3[1], np.repeat(v[:, 0], 2, 0))


def test_evict_oracle():
    s = np.array([5, 1, 3, np.nan, 0.0, -0.0, 2, 9], np.float32)
    p = np.arange(8) + 10
    assert O.evict(s, p, 8, 0, 100) == ([], [])
    assert O.evict(s, p, 4, 0, 100) == ([1, 3], [6, 7])
    assert O.evict(s, p, 6, 0, 100) == ([3, 5], [6, 7])      # the tie of zeros keeps the lower row
    assert O.evict(s, p, 3, 11, 15) == ([1, 2], [5, 6])      # rows 0 (sink), 5, 6, 7 (recent) guarded: three lowest stay


# ---- the rotary table ------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,kw", [("none", {}), ("linear", {"factor": 4.0}), ("ntk", {"factor": 8.0}),
                                     ("bands", {"factor": 8.0, "orig_ctx": 8192, "low": 1.0, "high": 4.0})])
@pytest.mark.parametrize("rot", [16, 32, 96, 128])
def test_rope_init(vc, kind, kw, rot):
    code = {"none": vc.VC_ROPE_NONE, "linear": vc.VC_ROPE_LINEAR, "ntk": vc.VC_ROPE_NTK, "bands": vc.VC_ROPE_BANDS}
    t = vc.vc_rope_init(code[kind], rot, vc.VC_ROPE_HALF, 500000.0, **kw)
    assert t.rot_dim == rot and t.amp == 1.0
    # pow and a handful of operations in 64 bits on both sides
    assert np.allclose(list(t.freq)[: rot // 2], O.rope_freqs(kind, rot, 500000.0, **kw), rtol=1e-13, atol=0)


def test_rope_init_refusals(vc):
    bad = [dict(kind=9, rot_dim=64), dict(kind=0, rot_dim=64, layout=2), dict(kind=0, rot_dim=64, base=0.0),
           dict(kind=0, rot_dim=64, base=math.inf), dict(kind=0, rot_dim=64, base=math.nan),
           dict(kind=0, rot_dim=64, amp=math.nan), dict(kind=1, rot_dim=64, factor=0.0),
           dict(kind=2, rot_dim=64, factor=-1.0), dict(kind=3, rot_dim=64, factor=8.0, orig_ctx=0),
           dict(kind=3, rot_dim=64, factor=8.0, orig_ctx=10, low=4.0, high=4.0),
           dict(kind=3, rot_dim=64, factor=8.0, orig_ctx=10, low=-1.0)]
    for kw in bad:
        with pytest.raises(vc.VCError) as e:
            vc.vc_rope_init(**kw)
        assert e.value.status == vc.VC_ERR_INVALID, kw
    for rot in (0, 8, 24, 100, 144, -16):
        with pytest.raises(vc.VCError) as e:
            vc.vc_rope_init(vc.VC_ROPE_NONE, rot)
        assert e.value.status == vc.VC_ERR_UNSUPPORTED


# ---- refusals ------------------------------------------------------------------------------------
A = 1 << 12  # an aligned fake address


def _kv(vc, n=100, cap=128, **kw):
    f = dict(k=A, v=2 * A, score=3 * A, pos=4 * A, n=n, cap=cap)
    f.update(kw)
    return vc.vc_live_kv(**f)


def _rope(vc, shape=None, rope="ok", **kw):
    shape = shape or vc.vc_shape(1, 8, 2, 64)
    arr = (vc.vc_rope_req * shape.B)()
    kvkw = kw.pop("kv", {})
    for b in range(shape.B):
        f = dict(q=5 * A, k=6 * A, v=7 * A, q_stride=0, k_stride=0, v_stride=0, pos=None, pos0=0, n_rows=1, q_out=8 * A)
        f.update(kw)
        arr[b] = vc.vc_rope_req(kv=_kv(vc, **kvkw), **f)
    if rope == "ok":
        rope = vc.vc_rope_init(vc.VC_ROPE_NONE, 64)
    return vc.vc_rope_append(shape, rope, arr, stream=0, raise_on_error=False)


SHAPES = [((0, 8, 2, 64), "INVALID"), ((33, 8, 2, 64), "INVALID"), ((1, 8, 3, 64), "INVALID"), ((1, 2, 4, 64), "INVALID"),
          ((1, 8, 0, 64), "INVALID"), ((1, 8, 2, 96), "UNSUPPORTED")]


@pytest.mark.parametrize("dims,err", SHAPES)
def test_shapes_refused(vc, dims, err):
    s = vc.vc_shape(*dims)
    want = getattr(vc, "VC_ERR_" + err)
    one = (vc.vc_live_req * 1)()
    assert vc.vc_rope_append(s, vc.vc_rope_init(0, 64), (vc.vc_rope_req * 1)(), stream=0, raise_on_error=False) == want
    assert vc.vc_prefix_attn(s, None, one, stream=0, raise_on_error=False) == want
    assert vc.vc_scored_attn(s, one, stream=0, raise_on_error=False) == want
    assert vc.vc_evict_kv(s, (vc.vc_evict_req * 1)(), stream=0, raise_on_error=False) == want
    assert vc.vc_prefix_workspace_size(s, 1) == 0
    assert vc.vc_scored_workspace_size(s, 1, 10) == 0
    assert vc.vc_evict_workspace_size(s, 10) == 0


def test_rope_append_refusals(vc):
    ok, inv, uns = vc.VC_OK, vc.VC_ERR_INVALID, vc.VC_ERR_UNSUPPORTED
    assert _rope(vc, n_rows=0) == ok                       # nothing to do: nothing launched
    assert _rope(vc, n_rows=-1) == inv
    assert _rope(vc, n_rows=29) == inv                     # 100 + 29 rows do not fit 128
    assert _rope(vc, kv=dict(n=129)) == inv
    assert _rope(vc, kv=dict(n=-1)) == inv
    assert _rope(vc, kv=dict(cap=0, n=0), n_rows=0) == inv
    for f in ("q", "k", "v", "q_out"):
        assert _rope(vc, **{f: A + 8}) == inv
    assert _rope(vc, k=None) == inv
    assert _rope(vc, q=None) == inv and _rope(vc, q_out=None) == inv
    for f in ("k", "v"):
        assert _rope(vc, kv={f: A + 2}) == inv
    for f in ("score", "pos"):
        assert _rope(vc, kv={f: A + 2}) == inv
    assert _rope(vc, pos=A + 2) == inv
    assert _rope(vc, pos0=2 ** 31 - 1, n_rows=2) == inv
    assert _rope(vc, q_stride=8 * 64 - 8) == inv           # tokens would overlap
    assert _rope(vc, k_stride=2 * 64 + 4) == inv           # a token would start off a 16-byte boundary
    assert _rope(vc, q_out=5 * A, q_stride=1024) == inv    # in place needs packed rows
    assert _rope(vc, rope=None) == inv
    assert _rope(vc, rope=vc.vc_rope_init(0, 128)) == uns  # more rotated channels than d
    t = vc.vc_rope_init(0, 64)
    t.freq[3] = math.nan
    assert _rope(vc, rope=t) == inv
    t = vc.vc_rope_init(0, 64)
    t.layout = 5
    assert _rope(vc, rope=t) == inv


def _attn(vc, scored, shape=None, ws=None, n_rows=1, q=5 * A, o=6 * A, prefix=None, **kv):
    shape = shape or vc.vc_shape(1, 8, 2, 64)
    arr = (vc.vc_live_req * shape.B)()
    for b in range(shape.B):
        arr[b] = vc.vc_live_req(q, o, n_rows, _kv(vc, **kv))
    if scored:
        return vc.vc_scored_attn(shape, arr, ws, stream=0, raise_on_error=False)
    return vc.vc_prefix_attn(shape, prefix, arr, ws, stream=0, raise_on_error=False)


@pytest.mark.parametrize("scored", [False, True])
def test_attention_refusals(vc, scored):
    inv = vc.VC_ERR_INVALID
    assert _attn(vc, scored, n_rows=0) == vc.VC_OK
    assert _attn(vc, scored, n_rows=-1) == inv
    assert _attn(vc, scored, q=A + 8) == inv and _attn(vc, scored, o=A + 8) == inv
    assert _attn(vc, scored, q=None) == inv and _attn(vc, scored, o=None) == inv
    for f in ("k", "v"):
        assert _attn(vc, scored, **{f: None}) == inv and _attn(vc, scored, **{f: A + 8}) == inv
    assert _attn(vc, scored, n=129) == inv and _attn(vc, scored, n=-1) == inv and _attn(vc, scored, n=0, cap=0) == inv
    assert _attn(vc, scored, n=2 ** 30 + 1, cap=2 ** 31 - 1) == vc.VC_ERR_UNSUPPORTED
    fn = vc.vc_scored_attn if scored else (lambda s, r, **kw: vc.vc_prefix_attn(s, None, r, **kw))
    assert fn(vc.vc_shape(1, 8, 2, 64), None, stream=0, raise_on_error=False) == inv


def test_scored_attn_refusals(vc):
    assert _attn(vc, True, score=None) == vc.VC_ERR_INVALID
    assert _attn(vc, True, score=A + 2) == vc.VC_ERR_INVALID
    assert _attn(vc, True, n_rows=65) == vc.VC_ERR_UNSUPPORTED       # 65 x 4 heads of a group > 256
    assert vc.vc_scored_workspace_size(vc.vc_shape(1, 8, 2, 64), 65, 100) == 0
    assert vc.vc_scored_workspace_size(vc.vc_shape(1, 8, 2, 64), 64, 100) > 0
    assert _attn(vc, True) == vc.VC_ERR_WORKSPACE                    # no workspace


def test_prefix_attn_refusals(vc):
    P = lambda **kw: vc.vc_kv_full(**{**dict(k=A, v=2 * A, ctx=64, cap=64), **kw})
    for kw in (dict(k=None), dict(v=A + 8), dict(ctx=-1), dict(ctx=65)):
        assert _attn(vc, False, prefix=P(**kw)) == vc.VC_ERR_INVALID
    assert _attn(vc, False, prefix=P(k=None, v=None, ctx=0, cap=0), n_rows=0) == vc.VC_OK  # an empty prefix is none


def _evict(vc, ws=None, keep=50, sink=0, recent_from=2 ** 31 - 1, **kv):
    arr = (vc.vc_evict_req * 1)()
    arr[0] = vc.vc_evict_req(_kv(vc, **kv), keep, sink, recent_from)
    return vc.vc_evict_kv(vc.vc_shape(1, 8, 2, 64), arr, ws, stream=0, raise_on_error=False)


def test_evict_refusals(vc):
    inv = vc.VC_ERR_INVALID
    for f in ("k", "v", "score", "pos"):
        assert _evict(vc, **{f: None}) == inv
    assert _evict(vc, score=A + 2) == inv and _evict(vc, pos=A + 1) == inv
    assert _evict(vc, keep=0) == inv and _evict(vc, keep=-1) == inv
    assert _evict(vc, n=129) == inv
    assert _evict(vc, keep=100) == vc.VC_OK and _evict(vc, keep=1000) == vc.VC_OK  # nothing to evict
    assert _evict(vc) == vc.VC_ERR_WORKSPACE
    assert _evict(vc, n=2 ** 30 + 1, cap=2 ** 31 - 1) == vc.VC_ERR_UNSUPPORTED
    assert vc.vc_evict_workspace_size(vc.vc_shape(1, 8, 2, 64), -1) == 0


def test_descriptors_have_the_headers_sizes(vc):
    """The binding's structs against the C compiler's, through nvcc's host compiler."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ["vc_live_kv", "vc_rope_config", "vc_rope", "vc_rope_req", "vc_live_req", "vc_evict_req"]
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "s.cpp")
        with open(src, "w") as f:
            f.write('#include <stdio.h>\n#include "vc.h"\nint main() {\n' +
                    "".join('printf("%%zu\\n", sizeof(%s));\n' % n for n in names) + "}\n")
        cc = ["g++", "-I", os.path.join(root, "include"), "-I", "/usr/local/cuda/include", src, "-o", os.path.join(d, "s")]
        subprocess.run(cc, check=True)
        out = subprocess.run([os.path.join(d, "s")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(getattr(vc, n)) for n in names]


def test_live_kv_refuses_strided_tensors(vc):
    import torch
    k = torch.zeros((2, 8, 64), dtype=torch.bfloat16)
    assert vc.live_kv(k, k, 3).cap == 8
    with pytest.raises(ValueError):
        vc.live_kv(k[:, ::2], k, 3)


def test_sizes_beyond_the_kernels_counts_are_refused(vc):
    uns = vc.VC_ERR_UNSUPPORTED
    big = vc.vc_shape(1, 65536, 65536, 64)
    for scored in (False, True):
        assert _attn(vc, scored, shape=big) == uns
        assert _attn(vc, scored, shape=vc.vc_shape(1, 256, 256, 64), n=2 ** 30, cap=2 ** 30) == uns  # 2^31 tiles
    assert _rope(vc, shape=big) == uns
    assert vc.vc_evict_workspace_size(big, 10) == vc.vc_prefix_workspace_size(big, 1) == 0
    t = vc.vc_rope_init(0, 64)
    t.amp = 1e300                                                    # finite, but not in fp32
    assert _rope(vc, rope=t) == vc.VC_ERR_INVALID
    with pytest.raises(vc.VCError):
        vc.vc_rope_init(0, 64, amp=1e300)
