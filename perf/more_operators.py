"""Cases of the operators that decode drafted trees over a cache of pages:

  append   rotary positions of several axes: q rotated, k rotated and written with v behind a sequence's rows in its pages
  tree     attention of a tree of drafted tokens (or a chain, or one token) over a sequence's pages
  fork     sequences dropped, winners forked (pages shared), and pages made ready for what comes next
  compact  the pages in use moved to the front of the pool, tables rewritten
  turn     the end of a turn: ancestor masks and depths of the trees, append, greedy acceptance along each tree, and the
           accepted path's rows moved together

Layouts are those of include/vc.h: q and o bf16 [rows][Hq][d] per request, pools bf16 [pages][Hkv][page][d], page tables
int32 [sequences][most pages]. run() makes the framework's calls when `own` is true and computes the plain form in fp32
(angles in fp64) otherwise. exact() restates each operator in fp64 and in Python's whole numbers.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
#: (query heads, KV heads, head dim): the shapes of workloads/configs.py, then one head per KV head and sixteen.
HEADS = ((8, 2, 64), (32, 8, 128), (40, 8, 128), (64, 8, 128), (16, 16, 128), (32, 2, 128))
_BASE = 500000.0


def listed():
    t, a, q, b = HEADS[:4]
    h = lambda s: {"Hq": s[0], "Hkv": s[1], "d": s[2]}
    return [
        # one token of one small request: the call's latency
        {"name": "append one token", "op": "append", **h(t), "B": 1, "rows": 1, "n": 1000, "page": 16, "axes": 1,
         "dealt": False, "rot": 64, "inter": False, "pos": 1000, "fused": False},
        # frames of a video and their text in front of a long context, straight from a fused projection
        {"name": "append video", "op": "append", **h(b), "B": 4, "rows": 2047, "n": 700, "page": 64, "axes": 3,
         "dealt": True, "rot": 128, "inter": False, "pos": 129000, "fused": True},
        # one small request, one token
        {"name": "tree one token", "op": "tree", **h(t), "B": 1, "rows": 1, "n": 1000, "page": 16, "kind": "chain",
         "ragged": False},
        # a full batch decoding one token each from small pages
        {"name": "tree decode", "op": "tree", **h(a), "B": 32, "rows": 1, "n": 8200, "page": 16, "kind": "chain",
         "ragged": True},
        # the drafts of a batch, a narrow tree each
        {"name": "tree drafts", "op": "tree", **h(q), "B": 16, "rows": 25, "n": 16300, "page": 32, "kind": "tree",
         "ragged": True},
        # wide trees over long contexts
        {"name": "tree wide", "op": "tree", **h(b), "B": 8, "rows": 64, "n": 32768, "page": 64, "kind": "tree",
         "ragged": False},
        # two candidates from one small sequence
        {"name": "fork two", "op": "fork", **h(t), "parents": 1, "kids": 2, "rows": 1, "n": 1000, "page": 16},
        # a batch of searches, seven candidates each, room for the next drafts
        {"name": "fork beams", "op": "fork", **h(a), "parents": 4, "kids": 28, "rows": 25, "n": 8100, "page": 128},
        # a small pool after a few requests have left
        {"name": "compact small", "op": "compact", **h(t), "seqs": 3, "pages": 64, "used": 0.5, "page": 16},
        # a large pool half of which is free
        {"name": "compact pool", "op": "compact", **h(b), "seqs": 24, "pages": 16384, "used": 0.5, "page": 16},
        # a few drafts of one small request
        {"name": "turn small", "op": "turn", **h(t), "B": 1, "rows": 5, "n": 1000, "page": 16, "V": 1000, "ragged": False},
        # the trees of a batch, the vocabulary of a large model
        {"name": "turn batch", "op": "turn", **h(a), "B": 16, "rows": 32, "n": 4000, "page": 32, "V": 128256, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "tree", "tree", "fork", "compact", "turn"))
    Hq, Hkv, d = rng.choice(HEADS)
    c = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": d, "page": rng.choice((16, 32, 64, 128))}
    if op == "append":
        B = _log(rng, 1, 32)
        rot = rng.choice((d, d, d // 2))
        c.update(B=B, rows=_log(rng, 1, max(1, 8188 // B)), n=_log(rng, 1, 2000), axes=rng.choice((1, 2, 3, 3)),
                 dealt=rng.random() < 0.5, rot=rot, inter=rng.random() < 0.5, pos=_log(rng, 1, 1000000),
                 fused=rng.random() < 0.5)
    elif op == "tree":
        kind = rng.choice(("chain", "tree"))
        B = _log(rng, 1, 32)
        n = _log(rng, 1, max(2, min(131072, 8 * 32768 * 8 * 128 // (B * Hkv * d))))  # no more bytes than the largest listed case
        most = max(1, 8 * 64 * 64 * 32768 // (B * Hq * n))  # nor more products
        c.update(B=B, rows=min(_log(rng, 1, 512 if kind == "chain" else 96), most), n=n, kind=kind,
                 ragged=rng.random() < 0.7)
    elif op == "fork":
        parents = _log(rng, 1, 8)
        c.update(parents=parents, kids=parents * rng.randint(1, 32 // parents), rows=_log(rng, 1, 64), n=_log(rng, 1, 16000))
    elif op == "compact":
        row = Hkv * d * 4  # bytes of a token
        pages = _log(rng, 32, max(64, 16384 * 16 * 4096 // (c["page"] * row)))
        c.update(seqs=rng.randint(1, 24), pages=pages, used=round(rng.uniform(0.1, 0.95), 3))
    else:
        B = _log(rng, 1, 16)
        V = rng.choice((1000, 32000, 50257, 128256))
        c.update(B=B, rows=_log(rng, 1, max(2, min(64, 16 * 32 * 128256 // (B * V)))), n=_log(rng, 1, 4000), V=V,
                 ragged=rng.random() < 0.7)
    return c


def _lengths(c):
    """Rows each sequence holds before the new ones: all n, or down to three quarters of it."""
    n, B = c["n"], c.get("B") or c["parents"]
    if not c.get("ragged", c["op"] == "fork"):
        return [n] * B
    return [n - (b * 977) % (n // 4 + 1) for b in range(B)]


def _row_counts(c):
    """New rows of each request: every third one of a ragged batch has fewer."""
    r = c["rows"]
    return [r if not c.get("ragged") or b % 3 != 1 else (r + 1) // 2 for b in range(c["B"])]


def _sections(c):
    """Pairs of channels that each axis turns: time takes what height and width leave."""
    pairs = c["rot"] // 2
    if c["axes"] == 1:
        return [pairs]
    side = pairs * 5 // 16 if c["axes"] == 3 else pairs // 2
    return [pairs - side * (c["axes"] - 1)] + [side] * (c["axes"] - 1)


def _parents(B, N, g):
    """Trees of drafts: node 0 is the root (the last accepted token), half of the others continue the node before them."""
    j = torch.arange(N, device=DEV)
    back = torch.rand((B, N), generator=g, device=DEV) < 0.5
    any_ = (torch.rand((B, N), generator=g, device=DEV) * j).long().clamp_(max=N - 1)
    p = torch.where(back, j - 1, torch.minimum(any_, (j - 1).clamp(min=0)))
    p[:, 0] = -1
    return p


def _seen_nodes(parent):
    """[B][N][N]: node i sees node j, itself or an ancestor."""
    B, N = parent.shape
    see = torch.eye(N, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
    at = torch.arange(B, device=DEV)
    for j in range(1, N):
        see[:, j] |= see[at, parent[:, j].clamp(min=0).long()]
    return see


def _pack(see, words):
    """Bits 32 w .. 32 w + 31 of each row as the int32 word w."""
    see = torch.nn.functional.pad(see, (0, 32 * words - see.shape[-1])).unflatten(-1, (words, 32))
    x = (see.long() << torch.arange(32, device=DEV)).sum(-1)
    return torch.where(x >= 2 ** 31, x - 2 ** 32, x).to(torch.int32)


def _pool(s, held, n_seq, n_pages, most, g, lens, pos=None):
    """The state of a pool of pages: each sequence's pages anywhere in it, the rest on the stack of free ones.

    One int32 buffer holds all of it, so that a pass that moves it on can put it back in one copy."""
    c = s["case"]
    sizes = {"len": n_seq, "next": n_seq, "held": n_seq, "n_free": 1, "table": n_seq * most, "refs": n_pages, "free": n_pages + 1}
    pad = lambda n: (n + 3) // 4 * 4
    ints = torch.zeros(sum(pad(n) for n in sizes.values()), dtype=torch.int32, device=DEV)
    at = 0
    for name, n in sizes.items():
        s[name] = ints[at : at + n]
        at += pad(n)
    s["table"] = s["table"].view(n_seq, most)
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    used = 0
    for i, h in enumerate(held):
        s["table"][i, :h] = perm[used : used + h]
        used += h
    s["refs"][perm[:used].long()] = 1
    s["free"][: n_pages - used] = perm[used:]
    s["n_free"][0] = n_pages - used
    s["held"][: len(held)] = torch.tensor(held, dtype=torch.int32, device=DEV)
    s["len"][: len(held)] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["next"][: len(held)] = s["len"][: len(held)] if pos is None else torch.tensor(pos, dtype=torch.int32, device=DEV)
    s["ints"] = ints
    shape = (n_pages, c["Hkv"], c["page"], c["d"])
    s["k"], s["v"] = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    Hq, Hkv, d, op, page = c["Hq"], c["Hkv"], c["d"], c["op"], c["page"]
    up = lambda n: -(-n // page)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)

    s = {"case": c}
    if op in ("append", "tree", "turn"):
        B, rows, lens = c["B"], c["rows"], _lengths(c)
        held = [up(n + rows) for n in lens]
        pos = [c["pos"] + 17 * b for b in range(B)] if op == "append" else None
        _pool(s, held, B, sum(held) + 3, max(held) + 1, g, lens, pos)
    if op in ("append", "turn"):
        if c.get("fused"):  # one projection's output, token by token: q heads, k heads, v heads
            x = randn(B, rows, (Hq + 2 * Hkv) * d)
            s["q"], s["k_new"], s["v_new"] = x.split([Hq * d, Hkv * d, Hkv * d], dim=2)
        else:
            s["q"], s["k_new"], s["v_new"] = randn(B, rows, Hq * d), randn(B, rows, Hkv * d), randn(B, rows, Hkv * d)
        s["q_out"] = torch.zeros((B, rows, Hq, d), dtype=torch.bfloat16, device=DEV)
    if op == "append":
        i = torch.arange(rows, device=DEV, dtype=torch.int32)
        side = max(1, int(math.sqrt(rows / 4)))  # about four frames of side x side patches, row by row
        off = (i // (side * side), i // side % side, i % side)[: c["axes"]] if c["axes"] > 1 else (i,)
        s["off"] = torch.stack(off).contiguous()
    elif op == "tree":
        s["q"] = randn(B, rows, Hq, d)
        s["o"] = torch.zeros((B, rows, Hq, d), dtype=torch.bfloat16, device=DEV)
        s["mask"] = _pack(_seen_nodes(_parents(B, rows, g)), -(-rows // 32)) if c["kind"] == "tree" else None
    elif op == "turn":
        V, words = c["V"], -(-rows // 32)
        counts = torch.tensor(_row_counts(c), dtype=torch.int32, device=DEV)
        s["n_nodes"] = counts
        s["logits"] = torch.randn((B, rows, V), generator=g, device=DEV)
        p = _parents(B, rows, g)
        s["parent"] = p.to(torch.int32)
        best = s["logits"].argmax(2)
        token = torch.randint(0, V, (B, rows), generator=g, device=DEV)
        hit = torch.rand((B, rows), generator=g, device=DEV) < 0.6  # drafts that the full pass agrees with
        s["token"] = torch.where(hit, best.gather(1, p.clamp(min=0)), token).to(torch.int32)
        new = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=DEV)
        s.update(mask=new(B, rows, words), depth=new(B, rows), out=new(B, rows), path=new(B, rows), n_acc=new(B))
    elif op == "fork":
        lens, kids, rows = _lengths(c), c["kids"], c["rows"]
        held = [up(n) for n in lens]
        each = kids // c["parents"]
        more = sum(1 + up(lens[i // each] + rows) - held[i // each] for i in range(kids))
        _pool(s, held, c["parents"] + kids, sum(held) + more + 5, max(held) + up(rows) + 1, g, lens)
    elif op == "compact":
        n_pages, seqs = c["pages"], c["seqs"]
        used = max(seqs, int(n_pages * c["used"]))
        held = [used // seqs + (i < used % seqs) for i in range(seqs)]
        _pool(s, held, seqs, n_pages, max(held) + 2, g, [h * page - 3 for h in held])
        for i in range(1, seqs, 3):  # every third sequence is a fork of the first one's beginning
            shared = min(held[0], held[i]) // 3
            gone = s["table"][i, :shared].long()
            s["refs"][gone] = 0
            s["refs"][s["table"][0, :shared].long()] += 1
            s["table"][i, :shared] = s["table"][0, :shared]
            s["free"][s["n_free"].long() + torch.arange(shared, device=DEV)] = gone.to(torch.int32)
            s["n_free"] += shared
    if op in ("compact", "turn"):
        s["saved"] = s["ints"].clone()
    if own:
        _prepare_own(s)
    return s


# ---- the framework's calls ------------------------------------------------------------------------
def _prepare_own(s):
    """What a serving loop keeps between steps: the pool's descriptor, the requests' and a workspace."""
    import lossless_compressed_kv_vc_gb300 as vc
    c = s["case"]
    Hq, Hkv, d, op = c["Hq"], c["Hkv"], c["d"], c["op"]
    kv = vc.paged_kv(s["k"], s["v"], s["refs"], s["free"], s["n_free"], s["table"], s["len"], s["held"], s["next"])
    s.update(lib=vc, kv=kv, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    size = 0
    if op in ("append", "tree", "turn"):
        B, counts = c["B"], _row_counts(c)
        s["shape"] = vc.vc_shape(B, Hq, Hkv, d)
    if op in ("append", "turn"):
        layout = vc.VC_ROPE_INTERLEAVED if c.get("inter") else vc.VC_ROPE_HALF
        rope = vc.vc_rope_init(vc.VC_ROPE_NONE, c.get("rot", d), layout, _BASE)
        s["axes"] = vc.vc_rope_axes_init(rope, _sections(c) if op == "append" else [d // 2], c.get("dealt", False))
        s["rope_req"] = (vc.vc_rope_page_req * B)()
        for b, r in enumerate(s["rope_req"]):
            r.q, r.k, r.v = s["q"][b].data_ptr(), s["k_new"][b].data_ptr(), s["v_new"][b].data_ptr()
            r.q_stride, r.k_stride, r.v_stride = s["q"].stride(1), s["k_new"].stride(1), s["v_new"].stride(1)
            r.q_out, r.seq, r.n_rows = s["q_out"][b].data_ptr(), b, counts[b]
            r.off, r.off_stride = (s["off"] if op == "append" else s["depth"][b]).data_ptr(), c["rows"] if op == "append" else 0
    if op == "tree":
        s["req"] = (vc.vc_tree_req * B)()
        for b, r in enumerate(s["req"]):
            r.q, r.o, r.seq, r.n_rows = s["q"][b].data_ptr(), s["o"][b].data_ptr(), b, counts[b]
            if s["mask"] is not None:
                r.mask, r.mask_words = s["mask"][b].data_ptr(), s["mask"].shape[2]
        size = vc.vc_tree_workspace_size(s["shape"], c["rows"])
    elif op == "turn":
        s["req"] = (vc.vc_commit_req * B)()
        for b, r in enumerate(s["req"]):
            r.path, r.n_acc, r.seq, r.n_rows, r.advance = s["path"][b].data_ptr(), s["n_acc"][b:].data_ptr(), b, counts[b], -1
    elif op == "fork":
        kids, each, first = c["kids"], c["kids"] // c["parents"], c["parents"]
        s["shape"] = vc.vc_shape(kids, Hq, Hkv, d)
        # the last one first: the pages then lie on the stack as they were taken
        s["drop"] = (vc.vc_trim_req * kids)(*[vc.vc_trim_req(first + kids - 1 - i, 0, 0) for i in range(kids)])
        s["fork"] = (vc.vc_fork_req * kids)(*[vc.vc_fork_req(i // each, first + i) for i in range(kids)])
        s["room"] = (vc.vc_reserve_req * kids)(*[vc.vc_reserve_req(first + i, c["rows"]) for i in range(kids)])
        size = vc.vc_pages_workspace_size(s["shape"], kv)
    elif op == "compact":
        s["shape"] = vc.vc_shape(1, Hq, Hkv, d)
        size = vc.vc_pages_workspace_size(s["shape"], kv)
    s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)


def _run_own(s):
    c, vc, kv, st = s["case"], s["lib"], s["kv"], s["status"]
    op = c["op"]
    if op == "append":
        vc.vc_rope_pages(s["shape"], s["axes"], kv, s["rope_req"], st)
    elif op == "tree":
        vc.vc_tree_attn(s["shape"], kv, s["req"], s["ws"], st)
    elif op == "fork":
        vc.vc_pages_trim(s["shape"], kv, s["drop"], st)
        vc.vc_pages_fork(s["shape"], kv, s["fork"], st)
        vc.vc_pages_reserve(s["shape"], kv, s["room"], s["ws"], st)
    elif op == "compact":
        vc.vc_pages_compact(s["shape"], kv, s["ws"], st)
    else:
        B, N = c["B"], c["rows"]
        vc.vc_tree_mask(B, N, s["parent"], s["n_nodes"], s["mask"], s["depth"])
        vc.vc_rope_pages(s["shape"], s["axes"], kv, s["rope_req"], st)
        vc.vc_tree_accept(B, N, c["V"], s["logits"], s["token"], s["parent"], s["n_nodes"], s["out"], s["path"], s["n_acc"])
        vc.vc_tree_commit(s["shape"], kv, s["req"], st)


# ---- the plain forms ------------------------------------------------------------------------------
def _axis_of(c):
    """Axis of each pair: one after the other, or dealt round the axes that have pairs left."""
    left = _sections(c)
    if not c["dealt"]:
        return [a for a, n in enumerate(left) for _ in range(n)]
    out, a = [], 0
    while len(out) < c["rot"] // 2:
        if left[a]:
            left[a] -= 1
            out.append(a)
        a = (a + 1) % len(left)
    return out


def _rotate(c, x, cos, sin):
    """x fp32 [B][rows][heads][d]; cos, sin [B][rows][1][rot / 2]."""
    r = 2 * cos.shape[-1]
    if c.get("inter"):
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., r:]), -1)


def _run_append(s, pos):
    """pos int64 [B][rows][pairs]: each pair's position."""
    c = s["case"]
    B, R, Hq, Hkv, d, page = c["B"], c["rows"], c["Hq"], c["Hkv"], c["d"], c["page"]
    pairs = pos.shape[2]
    w = _BASE ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
    a = (pos.double() * w)[:, :, None]
    cos, sin = a.cos().float(), a.sin().float()
    live = torch.arange(R, device=DEV) < torch.tensor(_row_counts(c), device=DEV)[:, None]
    q = _rotate(c, s["q"].reshape(B, R, Hq, d).float(), cos, sin).bfloat16()
    s["q_out"][:] = torch.where(live[..., None, None], q, s["q_out"])
    k = _rotate(c, s["k_new"].reshape(B, R, Hkv, d).float(), cos, sin).bfloat16()
    row = s["len"][:, None].long() + torch.arange(R, device=DEV)
    pg, at = s["table"].long().gather(1, row // page), row % page
    s["k"][pg, :, at] = torch.where(live[..., None, None], k, s["k"][pg, :, at])
    s["v"][pg, :, at] = torch.where(live[..., None, None], s["v_new"].reshape(B, R, Hkv, d), s["v"][pg, :, at])


def _run_tree(s):
    c = s["case"]
    B, R, Hq, Hkv, d, page = c["B"], c["rows"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G = Hq // Hkv
    used = max(-(-(n + r) // page) for n, r in zip(_lengths(c), _row_counts(c)))
    cap = used * page
    counts = torch.tensor(_row_counts(c), device=DEV)[:, None]
    node = torch.arange(cap, device=DEV)[None] - s["len"][:, None]  # node that each row of the cache is, < 0: context
    if s["mask"] is None:
        see = torch.ones((R, R), dtype=torch.bool, device=DEV).tril()[None].expand(B, R, R)
    else:
        bit = (s["mask"][..., None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        see = bit.flatten(2)[:, :, :R].bool()
    seen = see.gather(2, node.clamp(0, R - 1).long()[:, None].expand(B, R, cap))
    seen = torch.where((node < 0)[:, None], True, seen & (node < counts)[:, None])
    i = torch.arange(R, device=DEV)[None, :, None]
    seen = seen & (i < counts[..., None])
    table = s["table"][:, :used].long().clamp(0, s["k"].shape[0] - 1)
    rows = lambda x: x[table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, cap, d).float()
    q = s["q"].float().reshape(B, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, d) / math.sqrt(d)
    x = (q @ rows(s["k"]).transpose(2, 3)).view(B, Hkv, R, G, cap)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(4, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = x.sum(4, keepdim=True).view(B, Hkv, R * G, 1)
    v = torch.where((node < counts)[:, None, :, None], rows(s["v"]), 0.0)
    o = (x.view(B, Hkv, R * G, cap) @ v) * torch.where(total > 0, 1 / total, 0.0)
    o = o.view(B, Hkv, R, G, d).permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d).bfloat16()
    s["o"][:] = torch.where((i < counts[..., None])[..., None], o, s["o"])


def _run_trim(s, seqs):
    """All pages of the sequences given back, one sequence after the other, its last page first."""
    i = torch.arange(s["table"].shape[1], device=DEV)
    for q in seqs:
        mine = i < s["held"][q]
        row = s["table"][q].long().clamp(min=0)
        s["refs"].index_add_(0, row, -mine.to(torch.int32))
        gone = mine & (s["refs"][row] == 0)
        order = gone.flip(0).cumsum(0).flip(0)  # 1 for the last one given back
        at = torch.where(gone, s["n_free"] + order - 1, s["free"].shape[0] - 1)
        s["free"].scatter_(0, at.long(), s["table"][q])
        s["n_free"] += gone.sum().to(torch.int32)
        s["held"][q], s["len"][q], s["next"][q] = 0, 0, 0


def _run_fork(s):
    c = s["case"]
    kids, first, page, rows = c["kids"], c["parents"], c["page"], c["rows"]
    each = kids // first
    _run_trim(s, [first + i for i in reversed(range(kids))])
    i = torch.arange(s["table"].shape[1], device=DEV)
    one = torch.ones((), dtype=torch.int32, device=DEV)
    for kid in range(kids):
        a, b = kid // each, first + kid
        n = (s["len"][a] + page - 1) // page
        s["table"][b] = torch.where(i < n, s["table"][a], s["table"][b])
        s["refs"].index_add_(0, s["table"][a].long().clamp(min=0), (i < n).to(torch.int32))
        s["held"][b], s["len"][b], s["next"][b] = n, s["len"][a], s["next"][a]
    in_page = torch.arange(page, device=DEV)[None, :, None]
    for kid in range(kids):
        b = first + kid
        n, held = s["len"][b], s["held"][b]
        tail = (n // page).long().clamp(max=i.numel() - 1)
        old = s["table"][b].gather(0, tail[None]).long().clamp(min=0)
        copy = ((n % page != 0) & (s["refs"][old] > 1)).to(torch.int32)  # a last page that others hold too
        more = ((n + rows + page - 1) // page - held).clamp(min=0)
        new = lambda k: s["free"].gather(0, (s["n_free"] - 1 - k).long().clamp(min=0))  # k-th page from the stack
        dst = torch.where(copy > 0, new(0 * one), old.to(torch.int32)).long()
        s["refs"].index_add_(0, old, -copy)
        for pool in ("k", "v"):
            s[pool][dst] = torch.where(in_page < n % page, s[pool][old], s[pool][dst])
        fresh = (i >= held) & (i < held + more)
        got = new(copy + (i - held).clamp(min=0).to(torch.int32))
        row = torch.where(fresh, got, s["table"][b])
        s["table"][b] = torch.where((i == tail) & (copy > 0), dst.to(torch.int32), row)
        s["refs"].index_add_(0, dst, copy)
        s["refs"].index_add_(0, got.long(), fresh.to(torch.int32))
        s["held"][b] += more
        s["n_free"] -= copy + more


def _run_compact(s):
    n_pages = s["refs"].numel()
    i = torch.arange(n_pages, device=DEV)
    used = s["refs"] > 0
    U = used.sum()
    move = (used & (i >= U)).nonzero()[:, 0]  # pages behind the others go into the free ones before them, both in order
    hole = (~used & (i < U)).nonzero()[:, 0]
    to = i.clone()
    to[move] = hole
    for pool in ("k", "v"):
        s[pool][hole] = s[pool][move]
    s["refs"][hole] = s["refs"][move]
    s["refs"][move] = 0
    mine = torch.arange(s["table"].shape[1], device=DEV) < s["held"][:, None]
    s["table"][:] = torch.where(mine, to[s["table"].long()].to(torch.int32), s["table"])
    free = s["free"][:n_pages]
    free[:] = torch.where(i < n_pages - U, (n_pages - 1 - i).to(torch.int32), free)
    s["n_free"][0] = n_pages - U


def _run_turn(s):
    c = s["case"]
    B, N, page = c["B"], c["rows"], c["page"]
    i, at = torch.arange(N, device=DEV), torch.arange(B, device=DEV)
    live = i < s["n_nodes"][:, None]
    see = _seen_nodes(s["parent"]) & live[..., None]
    s["mask"][:] = _pack(see, s["mask"].shape[2])
    s["depth"][:] = torch.where(live, see.sum(2) - 1, 0)
    _run_append(s, (s["next"][:, None] + s["depth"]).long()[..., None].expand(B, N, c["d"] // 2))
    # the full pass's token behind each node, the first of equal ones
    V = c["V"]
    top = s["logits"].amax(2, keepdim=True)
    pick = torch.where(s["logits"] == top, torch.arange(V, device=DEV, dtype=torch.int32), V).amin(2)
    cur, on = torch.zeros(B, dtype=torch.long, device=DEV), s["n_nodes"] > 0
    s["out"].fill_(-1)
    s["path"].fill_(-1)
    s["n_acc"].zero_()
    for step in range(N):
        t = pick[at, cur]
        s["path"][:, step] = torch.where(on, cur.to(torch.int32), -1)
        s["out"][:, step] = torch.where(on, t.to(torch.int32), -1)
        s["n_acc"] += on.to(torch.int32)
        fits = live & (s["parent"] == cur[:, None]) & (s["token"] == t[:, None]) & (i > cur[:, None])
        child = torch.where(fits, i, N).amin(1)
        on = on & (child < N)
        cur = torch.where(on, child, cur)
    # the accepted path's rows together
    taken = i < s["n_acc"][:, None]
    row = s["len"][:, None].long() + torch.where(taken, s["path"], i).long()
    dst = s["len"][:, None].long() + i
    table = s["table"].long()
    a, b = table.gather(1, row // page), table.gather(1, dst // page)
    for pool in ("k", "v"):
        s[pool][b, :, dst % page] = s[pool][a, :, row % page]
    s["len"] += s["n_acc"]
    s["next"] += s["n_acc"]


def run(s):
    c = s["case"]
    op = c["op"]
    if op in ("compact", "turn"):  # rows and pages that were moved are still there, so with this put back every pass is the same
        s["ints"].copy_(s["saved"])
    if own:
        _run_own(s)
    elif op == "append":
        axis = torch.tensor(_axis_of(c), device=DEV)
        _run_append(s, s["next"][:, None, None].long() + s["off"].long()[axis].t()[None])
    else:
        {"tree": _run_tree, "fork": _run_fork, "compact": _run_compact, "turn": _run_turn}[op](s)
    pool = {"k": s["k"], "v": s["v"]}
    state = {x: s[x] for x in ("len", "next", "held", "n_free", "table", "refs")}
    if op == "append":
        return {"q": s["q_out"], **pool}
    if op == "tree":
        return {"o": s["o"]}
    if op == "turn":
        return {"q": s["q_out"], **pool, **{x: s[x] for x in ("mask", "depth", "out", "path", "n_acc", "len", "next")}}
    return {**pool, **state, "free": s["free"][: s["refs"].numel()]}


# ---- what a pass cannot do without ---------------------------------------------------------------------
def work(c):
    Hq, Hkv, d, op, page = c["Hq"], c["Hkv"], c["d"], c["op"], c["page"]
    row = Hkv * d * 4  # bytes of a token's keys and values
    if op in ("append", "turn"):
        t = sum(_row_counts(c))
        by, fl = t * (Hq + 2 * Hkv) * d * 4, t * (Hq + Hkv) * c.get("rot", d) * 3
        if op == "append":
            return {"bytes": by, "flops": fl}
        # logits read; masks, depths, tokens and paths written; about a third of the trees' rows moved
        return {"bytes": by + t * c["V"] * 4 + t * 4 * (6 + -(-c["rows"] // 32)), "flops": fl + t * c["V"]}
    if op == "tree":
        n, r = _lengths(c), _row_counts(c)
        pairs = sum(a * m + a * (a + 1) // 2 for m, a in zip(n, r))
        tokens = sum(m + a for m, a in zip(n, r))
        return {"bytes": tokens * row + tokens // page * 4 + sum(r) * Hq * d * 4, "flops": 4 * pairs * Hq * d}
    if op == "fork":  # tables written, last pages' rows read and written, the children's counts up and down
        each = c["kids"] // c["parents"]
        lens = [_lengths(c)[i // each] for i in range(c["kids"])]
        return {"bytes": sum(-(-n // page) * 16 + n % page * row * 2 for n in lens), "flops": 0}
    # compact: counts read, pages behind the used ones' number read and written, tables rewritten
    share = c["used"] * (1 - 0.1)
    moved = c["pages"] * share * (1 - share)
    return {"bytes": int(moved * page * row * 2 + c["pages"] * (8 + 8 * share)), "flops": 0}


# ---- the definitions in 64 bits, and in Python's whole numbers ----------------------------------------------
def _exact_append(c, s, pos):
    """pos(b, t, j): position of pair j of token t of request b, or None for tokens that are not there."""
    B, R, Hq, Hkv, d, page = c["B"], c["rows"], c["Hq"], c["Hkv"], c["d"], c["page"]
    rot = c.get("rot", d)
    angle = np.zeros((B, R, rot // 2))
    for b, r in enumerate(_row_counts(c)):
        for t in range(r):
            for j in range(rot // 2):
                angle[b, t, j] = pos(b, t, j) * math.pow(_BASE, -2.0 * j / rot)
    z = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.from_numpy(angle).to(DEV))[:, :, None]
    first = slice(0, rot, 2) if c.get("inter") else slice(0, rot // 2)
    second = slice(1, rot, 2) if c.get("inter") else slice(rot // 2, rot)

    def turned(x, heads):
        x = x.reshape(B, R, heads, d).double()
        y = x.clone()
        w = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        return y

    q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
    qn, kn, vn = turned(s["q"], Hq), turned(s["k_new"], Hkv), s["v_new"].reshape(B, R, Hkv, d).double()
    table, lens = s["table"].tolist(), s["len"].tolist()
    for b, r in enumerate(_row_counts(c)):
        q[b, :r] = qn[b, :r]
        for lo in range(lens[b] // page * page, lens[b] + r, page):  # page by page
            t0, t1 = max(0, lo - lens[b]), min(r, lo + page - lens[b])
            at = slice(lens[b] + t0 - lo, lens[b] + t1 - lo)
            k[table[b][lo // page], :, at] = kn[b, t0:t1].transpose(0, 1)
            v[table[b][lo // page], :, at] = vn[b, t0:t1].transpose(0, 1)
    return {"q": q, "k": k, "v": v}


def _exact_tree(c, s):
    Hkv, G, page, d = c["Hkv"], c["Hq"] // c["Hkv"], c["page"], c["d"]
    o = s["o"].double()
    mask = None if s["mask"] is None else s["mask"].cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    for b, (n, r) in enumerate(zip(_lengths(c), _row_counts(c))):
        pages = s["table"][b, : -(-(n + r) // page)].long()
        blind, j = np.zeros((r, n + r), dtype=bool), np.arange(r)  # keys that a row does not see
        blind[:, n:] = j[None] > j[:, None] if mask is None else (mask[b, :r, j // 32].T >> (j % 32)) & 1 == 0
        blind = torch.from_numpy(blind).to(DEV)[:, None]
        for h in range(Hkv):
            k, v = (x[pages, h].reshape(-1, d)[: n + r].double() for x in (s["k"], s["v"]))
            for i0 in range(0, r, 64):
                q = s["q"][b, i0 : min(r, i0 + 64), h * G : (h + 1) * G].double()
                z = torch.einsum("rgd,td->rgt", q, k) * d ** -0.5
                w = torch.softmax(z.masked_fill(blind[i0 : i0 + 64], -math.inf), -1)
                o[b, i0 : i0 + q.shape[0], h * G : (h + 1) * G] = torch.einsum("rgt,td->rgd", w, v)
    return {"o": o}


def _exact_fork(c, s):
    page, first, kids, rows = c["page"], c["parents"], c["kids"], c["rows"]
    each, n_pages = kids // first, s["refs"].numel()
    x = {name: s[name].cpu().numpy().copy() for name in ("len", "next", "held", "table", "refs", "free")}
    top = int(s["n_free"][0])
    k, v = s["k"].double(), s["v"].double()
    for i in range(kids):  # the children are empty before the first pass, so dropping them changes nothing
        a, b = i // each, first + i
        n = int(x["len"][a])
        x["len"][b], x["next"][b], x["held"][b] = n, x["next"][a], -(-n // page)
        for j in range(-(-n // page)):
            x["table"][b, j] = x["table"][a, j]
            x["refs"][x["table"][a, j]] += 1
    for b in range(first, first + kids):
        n, tail = int(x["len"][b]), int(x["len"][b]) // page
        if n % page and x["refs"][x["table"][b, tail]] > 1:
            top -= 1
            old, new = int(x["table"][b, tail]), int(x["free"][top])
            x["refs"][old] -= 1
            x["refs"][new] = 1
            x["table"][b, tail] = new
            k[new, :, : n % page], v[new, :, : n % page] = k[old, :, : n % page].clone(), v[old, :, : n % page].clone()
        while x["held"][b] * page < n + rows:
            top -= 1
            x["table"][b, x["held"][b]] = x["free"][top]
            x["refs"][x["free"][top]] = 1
            x["held"][b] += 1
    out = {name: torch.from_numpy(a) for name, a in x.items()}
    out["free"] = out["free"][:n_pages]
    return {"k": k, "v": v, **out, "n_free": torch.tensor([top], dtype=torch.int32)}


def _exact_compact(c, s):
    refs, held, table, free = (s[x].cpu().numpy().copy() for x in ("refs", "held", "table", "free"))
    n_pages = len(refs)
    U = int((refs > 0).sum())
    to, hole = {}, 0
    for p in range(U, n_pages):
        if refs[p] > 0:
            while refs[hole] > 0:
                hole += 1
            to[p], refs[hole], refs[p] = hole, refs[p], 0
    k, v = s["k"].clone(), s["v"].clone()
    if to:
        src, dst = (torch.tensor(list(x), device=DEV) for x in (to.keys(), to.values()))
        k[dst], v[dst] = k[src], v[src]
    for q in range(len(held)):
        for j in range(held[q]):
            table[q, j] = to.get(int(table[q, j]), table[q, j])
    free[: n_pages - U] = np.arange(n_pages - 1, U - 1, -1)
    new = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32))
    return {"k": k, "v": v, "len": s["len"], "next": s["next"], "held": s["held"], "n_free": new([n_pages - U]),
            "table": new(table), "refs": new(refs), "free": new(free[:n_pages])}


def _exact_turn(c, s):
    B, N, page = c["B"], c["rows"], c["page"]
    words = s["mask"].shape[2]
    parent, token, counts = s["parent"].tolist(), s["token"].tolist(), s["n_nodes"].tolist()
    mask, depth = np.zeros((B, N, words), dtype=np.uint32), np.zeros((B, N), dtype=np.int32)
    out, path = np.full((B, N), -1, dtype=np.int32), np.full((B, N), -1, dtype=np.int32)
    n_acc = np.zeros(B, dtype=np.int32)
    for b in range(B):
        for i in range(counts[b]):
            j = i
            while j >= 0:
                mask[b, i, j // 32] |= np.uint32(1 << (j % 32))
                j = parent[b][j]
                depth[b, i] += j >= 0
    nxt, lens = s["next"].tolist(), s["len"].tolist()
    moved = _exact_append(c, s, lambda b, t, j: nxt[b] + int(depth[b, t]))
    table = s["table"].tolist()
    for b in range(B):
        cur = 0 if counts[b] else None
        while cur is not None:
            t = int(np.argmax(s["logits"][b, cur].cpu().numpy()))  # the first of equal ones
            path[b, n_acc[b]], out[b, n_acc[b]] = cur, t
            n_acc[b] += 1
            cur = next((j for j in range(cur + 1, counts[b]) if parent[b][j] == cur and token[b][j] == t), None)
        for i in range(n_acc[b]):
            x, y = lens[b] + int(path[b, i]), lens[b] + i
            for pool in ("k", "v"):
                moved[pool][table[b][y // page], :, y % page] = moved[pool][table[b][x // page], :, x % page].clone()
    new = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32))
    return {**moved, "mask": new(mask), "depth": new(depth), "out": new(out), "path": new(path), "n_acc": new(n_acc),
            "len": new(np.array(lens) + n_acc), "next": new(np.array(nxt) + n_acc)}


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "append":
        axis, off, nxt = _axis_of(c), s["off"].tolist(), s["next"].tolist()
        return _exact_append(c, s, lambda b, t, j: nxt[b] + off[axis[j]][t])
    return {"tree": _exact_tree, "fork": _exact_fork, "compact": _exact_compact, "turn": _exact_turn}[op](c, s)
