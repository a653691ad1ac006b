"""Cases of the operators that serve a cache which grows, is shared and shrinks while requests decode:

  rope    rotary positions of new tokens: q rotated, k rotated and written to the cache with v
  prefix  attention of a batch over one shared prefix and each request's own cache
  scored  attention over a cache that adds every cached row's softmax weight to its score
  evict   the rows of highest accumulated weight kept, in place

Layouts are those of include/vc.h: q and o bf16 [rows][Hq][d] per request, caches bf16 [Hkv][cap][d], scores fp32 and
positions int32 [Hkv][cap]. run() makes the framework's calls when `own` is true and computes the plain form in fp32
(angles in fp64) otherwise. exact() restates each operator in fp64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
#: (query heads, KV heads, head dim): the shapes of workloads/configs.py, then one head per KV head and sixteen.
HEADS = ((8, 2, 64), (32, 8, 128), (40, 8, 128), (64, 8, 128), (16, 16, 128), (32, 2, 128))


def listed():
    t, a, q, b = HEADS[:4]
    h = lambda s: {"Hq": s[0], "Hkv": s[1], "d": s[2]}
    return [
        # one token of one small request: the call's latency
        {"name": "rope one token", "op": "rope", **h(t), "B": 1, "rows": 1, "n": 1024, "rot": 64, "inter": False,
         "kind": "none", "pos": 1024, "listed_pos": False, "fused": False},
        # the drafted tokens of a batch, half of each head rotated, positions of a drafting tree
        {"name": "rope drafts", "op": "rope", **h(q), "B": 16, "rows": 25, "n": 500, "rot": 64, "inter": True,
         "kind": "linear", "pos": 65536, "listed_pos": True, "fused": True},
        # prompt chunks of a long context, frequencies scaled by bands, straight from a fused projection
        {"name": "rope prompt chunks", "op": "rope", **h(b), "B": 4, "rows": 2047, "n": 1, "rot": 128, "inter": False,
         "kind": "bands", "pos": 129000, "listed_pos": False, "fused": True},
        # a few short requests under a short system prompt, one token each
        {"name": "prefix one token", "op": "prefix", **h(t), "B": 4, "rows": 1, "P": 1000, "n": 100, "ragged": True},
        # a full batch decoding under a long shared document
        {"name": "prefix decode", "op": "prefix", **h(a), "B": 32, "rows": 1, "P": 32768, "n": 2000, "ragged": True},
        # drafts of a batch checked against a shared document and each request's own turns
        {"name": "prefix drafts", "op": "prefix", **h(q), "B": 16, "rows": 25, "P": 65536, "n": 4100, "ragged": True},
        # one small request, one token
        {"name": "scored one token", "op": "scored", **h(t), "B": 1, "rows": 1, "n": 1024, "ragged": False},
        # a batch at a budget of 8192 rows, one token each
        {"name": "scored decode", "op": "scored", **h(a), "B": 8, "rows": 1, "n": 8200, "ragged": True},
        # long caches, one token each
        {"name": "scored long", "op": "scored", **h(b), "B": 4, "rows": 1, "n": 131072, "ragged": True},
        # one small request, one row over its budget
        {"name": "evict one row", "op": "evict", **h(t), "B": 1, "n": 1025, "keep": 1024, "sink": 4, "recent": 64},
        # a batch after a round of drafts
        {"name": "evict drafts", "op": "evict", **h(a), "B": 8, "n": 8224, "keep": 8192, "sink": 4, "recent": 512},
        # long prompts shrunk fourfold
        {"name": "evict prompts", "op": "evict", **h(b), "B": 4, "n": 131072, "keep": 32768, "sink": 4, "recent": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "prefix", "scored", "evict"))
    Hq, Hkv, d = rng.choice(HEADS)
    c = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": d}
    if op == "rope":
        B = _log(rng, 1, 32)
        c.update(B=B, rows=_log(rng, 1, max(1, 8188 // B)), n=_log(rng, 1, 2000),
                 rot=rng.choice((d, d, d // 2, d // 4)), inter=rng.random() < 0.5,
                 kind=rng.choice(("none", "linear", "ntk", "bands")), pos=_log(rng, 1, 1000000),
                 listed_pos=rng.random() < 0.5, fused=rng.random() < 0.5)
    elif op == "prefix":
        P = _log(rng, 64, 65536)
        most = max(1, 16 * 25 * 40 * 65536 // (Hq * P))  # query rows that cost no more than the largest listed case
        B = _log(rng, 1, 32)
        rows = min(_log(rng, 1, 64), max(1, most // B))
        c.update(B=B, rows=rows, P=P, n=rows + _log(rng, 1, 4000), ragged=rng.random() < 0.7)
    elif op == "scored":
        B = _log(rng, 1, 32)
        rows = min(rng.choice((1, 1, 1, 2, 5, 8)), 256 // (Hq // Hkv))
        c.update(B=B, rows=rows, n=rows + _log(rng, 16, max(32, 4 * 131000 // (B * rows))), ragged=rng.random() < 0.7)
    else:
        B = _log(rng, 1, 32)
        n = _log(rng, 64, max(128, 4 * 131072 // B))
        keep = n - 1 if rng.random() < 0.25 else max(1, int(n * rng.uniform(0.1, 0.99)))
        c.update(B=B, n=n, keep=keep, sink=rng.choice((0, 4)), recent=min(rng.choice((0, 32, 500)), keep // 2))
    return c


def _lengths(c):
    """Rows that each request's cache holds: all n, or down to three quarters of it."""
    n, B = c["n"], c["B"]
    if not c.get("ragged"):
        return [n] * B
    return [max(c["rows"], n - (b * 977) % (n // 4 + 1)) for b in range(B)]


def _row_counts(c):
    """Query rows of each request: every third one of a ragged batch has fewer."""
    r = c["rows"]
    return [r if not c.get("ragged") or b % 3 != 1 else (r + 1) // 2 for b in range(c["B"])]


_BANDS = {"factor": 8.0, "orig": 8192, "low": 1.0, "high": 4.0}
_BASE = 500000.0


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    B, Hq, Hkv, d, op = c["B"], c["Hq"], c["Hkv"], c["d"], c["op"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)

    s = {"case": c}
    if op == "rope":
        rows, n = c["rows"], c["n"]
        cap = n + rows + 3
        if c["fused"]:  # one projection's output, token by token: q heads, k heads, v heads
            x = randn(B, rows, (Hq + 2 * Hkv) * d)
            q, k, v = x.split([Hq * d, Hkv * d, Hkv * d], dim=2)
        else:
            q, k, v = randn(B, rows, Hq * d), randn(B, rows, Hkv * d), randn(B, rows, Hkv * d)
        s.update(q=q, k=k, v=v, q_out=torch.zeros((B, rows, Hq, d), dtype=torch.bfloat16, device=DEV),
                 kc=randn(B, Hkv, cap, d), vc=randn(B, Hkv, cap, d))
        s["score"] = torch.rand((B, Hkv, cap), generator=g, device=DEV)
        s["pos"] = torch.full((B, Hkv, cap), -1, dtype=torch.int32, device=DEV)
        first = torch.arange(B, device=DEV)[:, None] * 17 + c["pos"]
        if c["listed_pos"]:  # tokens of a tree share positions
            step = torch.randint(0, 2, (B, rows), generator=g, device=DEV)
            s["at"] = (first + step.cumsum(1)).to(torch.int32).contiguous()
        else:
            s["at"] = (first + torch.arange(rows, device=DEV)[None]).to(torch.int32).contiguous()
    elif op in ("prefix", "scored"):
        cap = c["n"] + 5
        s.update(q=randn(B, c["rows"], Hq, d), kc=randn(B, Hkv, cap, d), vc=randn(B, Hkv, cap, d),
                 o=torch.zeros((B, c["rows"], Hq, d), dtype=torch.bfloat16, device=DEV))
        if op == "prefix":
            s.update(pk=randn(Hkv, c["P"] + 3, d), pv=randn(Hkv, c["P"] + 3, d))
        else:
            s["score"] = torch.rand((B, Hkv, cap), generator=g, device=DEV)
    else:
        n, cap = c["n"], c["n"] + 5
        # accumulated weights: a few large, most small, some rows with none at all (ties)
        score = torch.rand((B, Hkv, cap), generator=g, device=DEV).log().neg().pow(3)
        score *= torch.rand((B, Hkv, cap), generator=g, device=DEV) > 0.05
        # positions with gaps, in any order of rows, as earlier evictions leave them; the newest stand in order behind
        pos = torch.randint(1, 4, (B, Hkv, n), generator=g, device=DEV).cumsum(2)
        old = n - c["recent"]
        perm = torch.rand((B, Hkv, old), generator=g, device=DEV).argsort(2)
        pos[:, :, :old] = pos[:, :, :old].gather(2, perm)
        pos = torch.nn.functional.pad(pos - pos.amax(2, keepdim=True) + 2 * n, (0, cap - n)).to(torch.int32).contiguous()
        s.update(kc=randn(B, Hkv, cap, d), vc=randn(B, Hkv, cap, d), score=score.clone(), pos=pos.clone(),
                 score_in=score, pos_in=pos)
        s["recent_from"] = 2 * n - c["recent"] + 1
    if own:
        _prepare_own(s)
    return s


# ---- the framework's calls ------------------------------------------------------------------------
def _prepare_own(s):
    """What a serving loop keeps between steps: descriptors of its caches, a workspace, the rotary table."""
    import lossless_compressed_kv_vc_gb300 as vc
    c = s["case"]
    B, Hq, Hkv, d, op = c["B"], c["Hq"], c["Hkv"], c["d"], c["op"]
    shape = vc.vc_shape(B, Hq, Hkv, d)
    lengths = _lengths(c) if op in ("prefix", "scored") else [c["n"]] * B
    rows = _row_counts(c) if op in ("prefix", "scored") else [c.get("rows", 0)] * B
    arr = ({"rope": vc.vc_rope_req, "evict": vc.vc_evict_req}.get(op, vc.vc_live_req) * B)()
    for b in range(B):
        r = arr[b]
        r.kv = vc.live_kv(s["kc"][b], s["vc"][b], lengths[b], s["score"][b] if "score" in s else None,
                          s["pos"][b] if "pos" in s else None)
        if op == "rope":
            r.q, r.k, r.v = s["q"][b].data_ptr(), s["k"][b].data_ptr(), s["v"][b].data_ptr()
            r.q_stride, r.k_stride, r.v_stride = s["q"].stride(1), s["k"].stride(1), s["v"].stride(1)
            r.q_out, r.n_rows, r.pos0 = s["q_out"][b].data_ptr(), rows[b], c["pos"] + 17 * b
            r.pos = s["at"][b].data_ptr() if c["listed_pos"] else None
        elif op == "evict":
            r.keep, r.sink, r.recent_from = c["keep"], c["sink"], s["recent_from"]
        else:
            r.q, r.o, r.n_rows = s["q"][b].data_ptr(), s["o"][b].data_ptr(), rows[b]
    s.update(vc=s["vc"], lib=vc, shape=shape, arr=arr, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if op == "rope":
        kind = {"none": vc.VC_ROPE_NONE, "linear": vc.VC_ROPE_LINEAR, "ntk": vc.VC_ROPE_NTK, "bands": vc.VC_ROPE_BANDS}
        layout = vc.VC_ROPE_INTERLEAVED if c["inter"] else vc.VC_ROPE_HALF
        s["table"] = vc.vc_rope_init(kind[c["kind"]], c["rot"], layout, _BASE, factor=_BANDS["factor"],
                                     orig_ctx=_BANDS["orig"], low=_BANDS["low"], high=_BANDS["high"])
        return
    if op == "prefix":
        s["prefix"] = vc.vc_kv_full(s["pk"].data_ptr(), s["pv"].data_ptr(), c["P"], s["pk"].shape[1])
        size = vc.vc_prefix_workspace_size(shape, c["rows"])
    elif op == "scored":
        size = vc.vc_scored_workspace_size(shape, c["rows"], c["n"])
    else:
        size = vc.vc_evict_workspace_size(shape, c["n"])
    s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)


def _run_own(s):
    c, vc = s["case"], s["lib"]
    if c["op"] == "rope":
        vc.vc_rope_append(s["shape"], s["table"], s["arr"])
    elif c["op"] == "prefix":
        vc.vc_prefix_attn(s["shape"], s["prefix"], s["arr"], s["ws"], s["status"])
    elif c["op"] == "scored":
        vc.vc_scored_attn(s["shape"], s["arr"], s["ws"], s["status"])
    else:
        vc.vc_evict_kv(s["shape"], s["arr"], s["ws"], s["status"])


# ---- the plain forms ------------------------------------------------------------------------------
def _freqs(c):
    """Radians a position of each pair of channels."""
    j = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    f, base, kind = _BANDS["factor"], _BASE, c["kind"]
    if kind == "ntk":
        base = base * f ** (c["rot"] / (c["rot"] - 2))
    w = base ** (-2 * j / c["rot"])
    if kind == "linear":
        return w / f
    if kind == "bands":
        turns = _BANDS["orig"] * w / (2 * math.pi)  # turns over the original context
        keep = ((turns - _BANDS["low"]) / (_BANDS["high"] - _BANDS["low"])).clamp(0, 1)
        return w * keep + w / f * (1 - keep)
    return w


def _rotate(c, x, cos, sin):
    """x fp32 [B][rows][heads][d]; cos, sin [B][rows][1][rot / 2]."""
    r = c["rot"]
    if c["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., r:]), -1)


def _run_rope(s):
    c = s["case"]
    B, rows, n, Hq, Hkv, d = c["B"], c["rows"], c["n"], c["Hq"], c["Hkv"], c["d"]
    a = s["at"].double()[..., None, None] * _freqs(c)
    cos, sin = a.cos().float(), a.sin().float()
    s["q_out"][:] = _rotate(c, s["q"].reshape(B, rows, Hq, d).float(), cos, sin).bfloat16()
    k = _rotate(c, s["k"].reshape(B, rows, Hkv, d).float(), cos, sin).bfloat16()
    s["kc"][:, :, n : n + rows] = k.transpose(1, 2)
    s["vc"][:, :, n : n + rows] = s["v"].reshape(B, rows, Hkv, d).transpose(1, 2)
    s["score"][:, :, n : n + rows] = 0.0
    s["pos"][:, :, n : n + rows] = s["at"][:, None]


def _run_attention(s):
    c = s["case"]
    B, R, Hq, Hkv, d, cap = c["B"], c["rows"], c["Hq"], c["Hkv"], c["d"], s["kc"].shape[2]
    G, P = Hq // Hkv, c.get("P", 0)
    n = torch.tensor(_lengths(c), device=DEV)[:, None, None]
    rows = torch.tensor(_row_counts(c), device=DEV)[:, None, None]
    i = torch.arange(R, device=DEV)[None, :, None]
    t = torch.arange(cap, device=DEV)[None, None, :]
    seen = (t <= n - rows + i) & (i < rows)  # [B][R][cap]
    seen = seen[:, None, :, None, :].expand(B, Hkv, R, G, cap).reshape(B, Hkv, R * G, cap)
    q = s["q"].float().reshape(B, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, d) / math.sqrt(d)
    so = (q @ s["kc"].float().transpose(2, 3)).masked_fill_(~seen, -math.inf)
    m = so.amax(3, keepdim=True)
    if P:
        qp = q.transpose(0, 1).reshape(Hkv, B * R * G, d)  # every request's rows against the one prefix
        sp = qp @ s["pk"][:, :P].float().transpose(1, 2)
        m = torch.maximum(m, sp.amax(2).view(Hkv, B, R * G, 1).transpose(0, 1))
    m = torch.where(m == -math.inf, 0.0, m)
    po = so.sub_(m).exp_()
    total = po.sum(3, keepdim=True)
    live = (t[0] < n[:, 0])[:, None, :, None]
    o = po @ torch.where(live, s["vc"].float(), 0.0)
    if P:
        pp = sp.sub_(m.transpose(0, 1).reshape(Hkv, B * R * G, 1)).exp_()
        total = total + pp.sum(2).view(Hkv, B, R * G, 1).transpose(0, 1)
        o = o + (pp @ s["pv"][:, :P].float()).view(Hkv, B, R * G, d).transpose(0, 1)
    inv = torch.where(total > 0, 1 / total, 0.0)
    o = (o * inv).view(B, Hkv, R, G, d).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d).bfloat16()
    s["o"][:] = torch.where((i < rows)[..., None], o, s["o"])
    if c["op"] == "scored":
        live_rows = (i < rows)[:, None, :, :].expand(B, 1, R, G).reshape(B, 1, R * G, 1)
        s["score"] += torch.where(live_rows, po * inv, 0.0).sum(2)


def _run_evict(s):
    c = s["case"]
    n, keep = c["n"], c["keep"]
    score, pos = s["score"][:, :, :n], s["pos"][:, :, :n]
    rank = torch.where(score.isnan(), -math.inf, score)
    guarded = (pos < c["sink"]) | (pos >= s["recent_from"])
    rank = torch.where(guarded, math.inf, rank)
    kept = torch.zeros_like(guarded)
    kept.scatter_(2, rank.sort(dim=2, descending=True, stable=True)[1][:, :, :keep], True)
    b, h, hole = (~kept[:, :, :keep]).nonzero(as_tuple=True)  # holes in ascending order, head by head,
    _, _, row = kept[:, :, keep:].nonzero(as_tuple=True)      # and as many survivors behind them
    row = row + keep
    for name in ("kc", "vc", "score", "pos"):
        s[name][b, h, hole] = s[name][b, h, row]


def run(s):
    op = s["case"]["op"]
    if op == "evict":  # rows that stay behind are never written, so with these two put back every pass is the same
        s["score"].copy_(s["score_in"])
        s["pos"].copy_(s["pos_in"])
    if own:
        _run_own(s)
    elif op == "rope":
        _run_rope(s)
    elif op == "evict":
        _run_evict(s)
    else:
        _run_attention(s)
    if op == "rope":
        return {"q": s["q_out"], "k": s["kc"], "v": s["vc"], "score": s["score"], "pos": s["pos"]}
    if op == "evict":
        return {"k": s["kc"], "v": s["vc"], "score": s["score"], "pos": s["pos"]}
    return {"o": s["o"], "score": s["score"]} if op == "scored" else {"o": s["o"]}


# ---- what a pass cannot do without ---------------------------------------------------------------------
def work(c):
    B, Hq, Hkv, d, op = c["B"], c["Hq"], c["Hkv"], c["d"], c["op"]
    if op == "rope":  # q, k, v read and written; position and zero score of every cached row written
        t = B * c["rows"]
        return {"bytes": t * ((Hq + 2 * Hkv) * d * 4 + Hkv * 8), "flops": t * (Hq + Hkv) * c["rot"] * 3}
    if op == "evict":
        # scores and positions read; the survivors behind the budget read and written with their score and position:
        # about the newest rows, which are always kept, and the kept share of the others
        n, keep = c["n"], c["keep"]
        newest = min(c["recent"] / 2, n - keep)
        moved = newest + (n - keep - newest) * max(0, keep - c["recent"] / 2) / (n - c["recent"] / 2)
        return {"bytes": B * Hkv * (n * 8 + moved * (d * 4 + 8) * 2), "flops": 0}
    n, rows, G, P = _lengths(c), _row_counts(c), Hq // Hkv, c.get("P", 0)
    pairs = sum(r * P + sum(max(0, m - r + i + 1) for i in range(r)) for m, r in zip(n, rows))
    by = sum(n) * Hkv * d * 4 + P * Hkv * d * 4 + sum(rows) * Hq * d * 4
    if op == "scored":
        by += sum(n) * Hkv * 8
    return {"bytes": by, "flops": 4 * pairs * Hkv * G * d}


# ---- the definitions in 64 bits ---------------------------------------------------------------------
def _exact_rope(c, s):
    B, rows, n, Hq, Hkv, d, rot = c["B"], c["rows"], c["n"], c["Hq"], c["Hkv"], c["d"], c["rot"]
    f = _BANDS["factor"]
    base = _BASE * (f ** (rot / (rot - 2)) if c["kind"] == "ntk" else 1.0)
    w = np.power(base, -np.arange(0, rot, 2, dtype=np.float64) / rot)
    if c["kind"] == "linear":
        w = w / f
    if c["kind"] == "bands":
        length = 2 * np.pi / w
        far, near = _BANDS["orig"] / _BANDS["low"], _BANDS["orig"] / _BANDS["high"]
        mix = (_BANDS["orig"] / length - _BANDS["low"]) / (_BANDS["high"] - _BANDS["low"])
        w = np.where(length > far, w / f, np.where(length < near, w, (1 - mix) * w / f + mix * w))
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                    s["at"].double()[:, :, None, None] * torch.from_numpy(w).to(DEV))

    def turned(x, heads):
        x = x.reshape(B, rows, heads, d).double()
        y = x.clone()
        first = slice(0, rot, 2) if c["inter"] else slice(0, rot // 2)
        second = slice(1, rot, 2) if c["inter"] else slice(rot // 2, rot)
        v = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = v.real, v.imag
        return y

    k, v, score, pos = s["kc"].double(), s["vc"].double(), s["score"].double(), s["pos"].clone()
    for b in range(B):
        k[b, :, n : n + rows] = turned(s["k"], Hkv)[b].movedim(0, 1)
        v[b, :, n : n + rows] = s["v"][b].reshape(rows, Hkv, d).double().movedim(0, 1)
        score[b, :, n : n + rows] = 0
        pos[b, :, n : n + rows] = s["at"][b]
    return {"q": turned(s["q"], Hq), "k": k, "v": v, "score": score, "pos": pos}


def _exact_attention(c, s):
    Hkv, G, P = c["Hkv"], c["Hq"] // c["Hkv"], c.get("P", 0)
    o = s["o"].double()
    score = s["score"].double() if c["op"] == "scored" else None
    for b, (n, rows) in enumerate(zip(_lengths(c), _row_counts(c))):
        for h in range(Hkv):
            k, v = s["kc"][b, h, :n], s["vc"][b, h, :n]
            if P:
                k, v = torch.cat((s["pk"][h, :P], k)), torch.cat((s["pv"][h, :P], v))
            q = s["q"][b, :rows, h * G : (h + 1) * G].double()
            z = torch.einsum("rgd,td->rgt", q, k.double()) * c["d"] ** -0.5
            for r in range(rows):  # row r does not see the rows that come after its own
                z[r, :, P + n - rows + r + 1 :] = -math.inf
            w = torch.softmax(z, -1)
            o[b, :rows, h * G : (h + 1) * G] = torch.einsum("rgt,td->rgd", w, v.double())
            if score is not None:
                score[b, h, :n] += w.sum((0, 1))
    return {"o": o} if score is None else {"o": o, "score": score}


def _exact_evict(c, s):
    n, keep = c["n"], c["keep"]
    k, v, score, pos = (s[x].cpu().clone() for x in ("kc", "vc", "score_in", "pos_in"))
    for b in range(c["B"]):
        for h in range(c["Hkv"]):
            p, w = pos[b, h, :n].numpy(), score[b, h, :n].numpy().astype(np.float64)
            plain = ~((p < c["sink"]) | (p >= s["recent_from"]))
            order = np.lexsort((np.arange(n), np.where(plain, -w, 0.0), plain))
            best = np.sort(order[:keep])
            src = torch.from_numpy(best[best >= keep].copy())
            dst = torch.from_numpy(np.setdiff1d(np.arange(keep), best))
            for x in (k, v, score, pos):
                x[b, h, dst] = x[b, h, src]
    return {"k": k, "v": v, "score": score.double(), "pos": pos}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s)
    return _exact_evict(c, s) if c["op"] == "evict" else _exact_attention(c, s)
