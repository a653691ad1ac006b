"""engine.LiveBatch's host side on the CPU: what it hands to the library, and what it turns down before. The library
call is replaced by a recorder, so nothing is launched and no address is read."""
import contextlib

import pytest
import torch

Hq, Hkv, D = 8, 2, 64


class _Event:
    def record(self, *_):
        pass


class _Calls(list):
    """The descriptors of each call, by name: (name, shape, [descriptor ...])."""

    def recorder(self, name, at):
        def call(shape, *args, **kw):
            arr = args[at]
            self.append((name, shape, [type(e).from_buffer_copy(e) for e in arr]))
            return 0
        return call


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__ as g
    g.build()
    import lossless_compressed_kv_vc_gb300 as m
    return m


@pytest.fixture
def calls(vc, monkeypatch):
    from lossless_compressed_kv_vc_gb300 import engine
    made = _Calls()
    monkeypatch.setattr(torch.cuda, "Event", _Event)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)  # no streams to put in order
    for name, at in (("vc_rope_append", 1), ("vc_prefix_attn", 1), ("vc_scored_attn", 0), ("vc_evict_kv", 0)):
        monkeypatch.setattr(engine, name, made.recorder(name, at))
    return made


def live(vc, B=2, cap=64, **kw):
    from lossless_compressed_kv_vc_gb300 import engine
    return engine.LiveBatch(Hq, Hkv, D, B, cap, vc.vc_rope_init(vc.VC_ROPE_NONE, D), device="cpu", **kw)


def new(heads, B=2, R=1):
    return torch.zeros((B, R, heads, D), dtype=torch.bfloat16)


def test_strides_of_a_fused_projection_are_passed_on(vc, calls):
    lb = live(vc, max_rows=4)
    x = torch.zeros((2, 4, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16)
    q, k, v = (t.unflatten(2, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 2))
    lb.append(q, k, v, [4, 2])
    name, _, arr = calls[0]
    assert name == "vc_rope_append" and [e.n_rows for e in arr] == [4, 2]
    for b, e in enumerate(arr):
        assert (e.q_stride, e.k_stride, e.v_stride) == ((Hq + 2 * Hkv) * D,) * 3
        assert (e.q, e.k, e.v) == (q[b].data_ptr(), k[b].data_ptr(), v[b].data_ptr())
    assert lb.n == [4, 2] and lb.next_pos == [4, 2]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_tokens_that_overlap_are_refused(vc, calls, which):
    """A tensor expanded over its tokens has stride 0 between them, which the library takes as packed tokens: it
    would read the memory behind the only one. Nothing is called and nothing moves on."""
    lb = live(vc, max_rows=4)
    for make in (lambda h: new(h).expand(2, 4, h, D), lambda h: new(h, R=4).as_strided((2, 4, h, D), (h * D, D, D, 1))):
        qkv = [new(Hq, R=4), new(Hkv, R=4), new(Hkv, R=4)]
        qkv[which] = make((Hq, Hkv, Hkv)[which])
        with pytest.raises(ValueError):
            lb.append(*qkv, [4, 1])
        assert not calls and lb.n == [0, 0] and lb.next_pos == [0, 0]
    qkv[which] = new((Hq, Hkv, Hkv)[which]).expand(2, 4, -1, D)
    lb.append(*qkv, [1, 1])  # no second token is read
    assert len(calls) == 1 and lb.n == [1, 1]


def test_a_single_token_has_no_stride(vc, calls):
    """[B][heads][1][d] transposed to [B][1][heads][d], the layout of a projection split by heads: the stride of its
    dimension of size one is d, less than a token, and says nothing."""
    lb = live(vc)
    q, k, v = (torch.zeros((2, h, 1, D), dtype=torch.bfloat16).transpose(1, 2) for h in (Hq, Hkv, Hkv))
    assert q.stride(1) == D
    lb.append(q, k, v, [1, 1])
    for b, e in enumerate(calls[0][2]):
        assert (e.q_stride, e.k_stride, e.v_stride) == (0, 0, 0)
        assert (e.q, e.k, e.v) == (q[b].data_ptr(), k[b].data_ptr(), v[b].data_ptr())
    x = torch.zeros((2, 3, Hq + 2 * Hkv, D), dtype=torch.bfloat16)  # the last of three tokens: strides of a longer tensor
    lb.append(x[:, 2:, :Hq], x[:, 2:, Hq : Hq + Hkv], x[:, 2:, Hq + Hkv :], [1, 0])
    assert [e.q for e in calls[1][2]] == [x[b, 2].data_ptr() for b in range(2)]


def test_a_budget_holds_the_rows_that_always_stay(vc, calls):
    """With more sink and recent rows than the budget, eviction would keep the lower of them and drop the newest."""
    for kw in (dict(sink=4, recent=128), dict(sink=129, recent=0), dict(sink=0, recent=129)):
        with pytest.raises(ValueError):
            live(vc, cap=200, budget=128, **kw)
    live(vc, cap=200, sink=4, recent=10 ** 6)  # no budget: nothing goes
    lb = live(vc, B=1, cap=200, budget=128, sink=4, recent=124)
    lb.n, lb.next_pos = [140], [140]
    lb.evict()
    name, shape, (e,) = calls[0]
    assert (name, shape.B, e.kv.n, e.keep, e.sink, e.recent_from) == ("vc_evict_kv", 1, 140, 128, 4, 16)
    assert lb.n == [128]


class _On0(torch.Tensor):
    """A host tensor that says it is on the first GPU."""
    device = torch.device("cuda", 0)


class _On1(torch.Tensor):
    device = torch.device("cuda", 1)


def test_tensors_of_another_gpu_are_refused(vc, calls, monkeypatch):
    """The batch lives on the device that was current when it was made; a tensor of another one of the same kind is
    turned down before its address is passed on."""
    for name in ("zeros", "empty"):
        real = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, device, real=real, **kw: real(*a, **kw).as_subclass(_On0))
    from lossless_compressed_kv_vc_gb300 import engine
    table = vc.vc_rope_init(vc.VC_ROPE_NONE, D)
    lb = engine.LiveBatch(Hq, Hkv, D, 2, 64, table, device="cuda")
    assert lb.device == torch.device("cuda", 0)
    make = lambda h, on: torch.ones((2, 1, h, D), dtype=torch.bfloat16).as_subclass(on)
    for which in range(3):
        on = [_On0] * 3
        on[which] = _On1
        with pytest.raises(ValueError):
            lb.append(make(Hq, on[0]), make(Hkv, on[1]), make(Hkv, on[2]), [1, 1])
    with pytest.raises(ValueError):
        lb.attend(make(Hq, _On1), [1, 1])
    pk, pv = (torch.ones((Hkv, 20, D), dtype=torch.bfloat16).as_subclass(c) for c in (_On0, _On1))
    for prefix in ((pk, pv, 5), (pv, pk, 5)):
        with pytest.raises(ValueError):
            engine.LiveBatch(Hq, Hkv, D, 2, 64, table, prefix=prefix, device="cuda")
    assert not calls and lb.n == [0, 0]
    lb.append(make(Hq, _On0), make(Hkv, _On0), make(Hkv, _On0), [1, 1])
    lb.attend(make(Hq, _On0), [1, 1])
    engine.LiveBatch(Hq, Hkv, D, 2, 64, table, prefix=(pk, pk, 5), device="cuda")
    assert [c[0] for c in calls] == ["vc_rope_append", "vc_scored_attn"]


def test_outputs_that_overlap_are_refused(vc, calls):
    """An output expanded over the batch would take every request's rows in one place."""
    lb = live(vc, max_rows=3)
    one = new(Hq, B=1, R=3)
    for o in (one.expand(2, 3, Hq, D), new(Hq, R=3).as_strided((2, 3, Hq, D), (2 * Hq * D, Hq * D, D, 1))):
        with pytest.raises(ValueError):
            lb.attend(o, [3, 1])
    assert not calls
    lb.attend(one.expand(2, 3, Hq, D), [0, 3])
    o = torch.zeros((2, 5, Hq, D), dtype=torch.bfloat16)[:, :3]
    lb.attend(o, [3, 2])
    assert [e.o for e in calls[1][2]] == [o[b].data_ptr() for b in range(2)]


def test_a_step_with_a_bad_output_moves_nothing(vc, calls):
    """step looks at its output before it appends: the caller can give the same tokens again."""
    lb = live(vc)
    q, k, v = new(Hq), new(Hkv), new(Hkv)
    odd = torch.zeros(2 * Hq * D + 4, dtype=torch.bfloat16)[4:].view(2, 1, Hq, D)
    for o in (new(Hq).float(), new(Hkv), new(Hq, B=1), new(Hq, B=1).expand(2, 1, Hq, D), odd):
        with pytest.raises(ValueError):
            lb.step(q, k, v, o)
        assert not calls and lb.n == [0, 0] and lb.next_pos == [0, 0]
    lb.step(q, k, v, new(Hq))
    assert [c[0] for c in calls] == ["vc_rope_append", "vc_scored_attn"] and lb.n == [1, 1]


def test_positions_stay_within_int32(vc, calls):
    """A descriptor's int32 would take 2^31 as a position before the first."""
    lb = live(vc, cap=200, budget=128)
    lb.next_pos = [2 ** 31 - 2, 7]
    x = [new(h) for h in (Hq, Hkv, Hkv)]
    lb.append(*x, [1, 1])
    assert [e.pos0 for e in calls[0][2]] == [2 ** 31 - 2, 7]
    with pytest.raises(ValueError):
        lb.append(*x, [1, 1])
    assert len(calls) == 1 and lb.n == [1, 1] and lb.next_pos == [2 ** 31 - 1, 8]
    lb.append(*x, [0, 1])
