"""Sizes of the live-cache calls beyond what their kernels count, refused before anything is launched (the pointers
are fake and never dereferenced)."""
import pytest

A = 1 << 12  # an aligned fake address


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


@pytest.mark.parametrize("Hq,d", [(1 << 28, 64), ((1 << 27) + 1, 64), (1 << 27, 128), (2 ** 31 - 1, 128)])
@pytest.mark.parametrize("keys_only", [False, True])
def test_rope_tokens_of_too_many_channels_are_refused(vc, Hq, d, keys_only):
    """A token's 16-byte pieces are numbered in 32 bits: 2^28 heads of 64 channels have 2^31 of them."""
    kv = vc.vc_live_kv(k=A, v=2 * A, score=None, pos=None, n=0, cap=1)
    q, q_out = (None, None) if keys_only else (5 * A, 8 * A)
    req = (vc.vc_rope_req * 1)(vc.vc_rope_req(q=q, k=6 * A, v=7 * A, n_rows=1, q_out=q_out, kv=kv))
    got = vc.vc_rope_append(vc.vc_shape(1, Hq, 1, d), vc.vc_rope_init(vc.VC_ROPE_NONE, 64), req, stream=0, raise_on_error=False)
    assert got == vc.VC_ERR_UNSUPPORTED
