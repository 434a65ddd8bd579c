"""Workloads of the paged cache and of drafted tokens: rotary positions with
several axes (and their gradient), appending by such positions, attention for a
tree of drafted tokens over a cache, acceptance of a path of the tree, and the
cache's pages taken, shared and compacted.

Each case runs either in its plain form (elementary torch operations in 32
bits) or, with ``own`` set, through attention_fa2_fwd_sm_gb300.  Layouts are
the library's: caches [B, Hkv, slots, d] or pools of pages [pages, Hkv, page,
d] with a table [B, pages a sequence], bf16.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # A prompt of 8K tokens of text and video: time, height and width have pairs of their own.
        dict(name="axes prompt 8K", op="axes", B=1, Hq=64, Hkv=8, N=8192, d=128, rot=128, A=3, cycled=False, inter=False,
             inverse=False, packed=False),
        # Gradients of a training step through the rotation, taken from a fused projection's layout, pairs dealt out to
        # the axes in turn, an odd length.
        dict(name="axes gradients", op="axes", B=2, Hq=32, Hkv=32, N=4097, d=64, rot=64, A=2, cycled=True, inter=True,
             inverse=True, packed=True),
        # A serving step of 32 users: masks and positions of the drafted trees, then the drafted tokens into the pages.
        dict(name="append trees", op="draft", B=32, Hq=64, Hkv=8, T=16, w=2, S=8192, d=128, rot=128, page=64),
        # A chunk of four users' prompts with images, of unequal lengths, into small pages.
        dict(name="append images", op="append", B=4, Hq=64, Hkv=8, T=2000, S=8192, d=128, rot=64, A=3, cycled=True,
             inter=True, page=16),
        # One user, a few drafted tokens behind a short context in a contiguous cache: latency.
        dict(name="tree small", op="tree", B=1, Hq=8, Hkv=2, T=5, w=2, S=500, d=64, page=0),
        # A serving batch, 16 drafted tokens each.
        dict(name="tree batch", op="tree", B=32, Hq=64, Hkv=8, T=16, w=2, S=8192, d=128, page=64),
        # The largest: wide trees over long contexts, 512 query rows to every key.
        dict(name="tree wide", op="tree", B=16, Hq=64, Hkv=8, T=64, w=4, S=32768, d=128, page=128),
        # No drafting: one token of 64 users over small pages.
        dict(name="tree token", op="tree", B=64, Hq=64, Hkv=8, T=1, w=1, S=16001, d=128, page=16),
        # One model layer, a few users, contiguous caches: latency.
        dict(name="accept few", op="accept", B=4, Hkv=2, T=8, w=2, S=512, d=64, page=0, layers=1),
        # All layers of a model at once, 64 users.
        dict(name="accept layers", op="accept", B=64, Hkv=8, T=64, w=4, S=2048, d=128, page=16, layers=8),
        # A beam search's step: beams continue as others, share their pages, and get room for a token each.
        dict(name="pages beams", op="beams", B=64, Hkv=8, S=4096, d=128, page=64, layers=2),
        # A pool half of whose pages have been freed, moved together in all layers.
        dict(name="pages compact", op="compact", B=32, Hkv=8, S=8192, d=128, page=64, layers=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["axes", "draft", "append", "tree", "tree", "tree", "tree", "accept", "beams", "compact"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8, 16])
    T = rng.choice([1, _log(rng, 2, 64), _log(rng, 2, 64)])
    page = rng.choice([0, 16, 32, 64, 128, 256])
    c = dict(op=op, B=_log(rng, 1, 32), Hkv=Hkv, d=d)
    if op in ("axes", "append"):
        c.update(rot=rng.choice([d, d // 2]), A=rng.choice([1, 2, 3, 4]), cycled=rng.random() < 0.5, inter=rng.random() < 0.5)
    if op == "axes":
        c.update(B=_log(rng, 1, 8), Hq=Hkv * G, N=max(1, _log(rng, 1, 65536) // (8 * G)), inverse=rng.random() < 0.5,
                 packed=rng.random() < 0.5)
    elif op == "append":
        T = _log(rng, 1, 2048)
        c.update(B=_log(rng, 1, 8), Hq=Hkv * G, T=T, S=T + _log(rng, 16, 4096), page=page)
    elif op == "draft":
        c.update(Hq=Hkv * G, T=T, w=rng.choice([1, 2, 4, 7]), S=T + _log(rng, 16, 8192), rot=d, page=page)
    elif op == "tree":
        c.update(Hq=Hkv * G, T=T, w=rng.choice([1, 2, 4, 7]), S=T + _log(rng, 16, 32768 // c["B"] + 4096), page=page)
    elif op == "accept":
        c.update(T=T, w=rng.choice([1, 2, 4, 7]), S=T + _log(rng, 16, 1024), page=page, layers=rng.choice([1, 2, 4, 8]))
    else:
        c.update(S=_log(rng, 64, 8192), page=rng.choice([16, 32, 64, 128]), layers=rng.choice([1, 2, 4]))
    return c


def _mean(S, T):
    """Mean number of cached keys: spread evenly over the upper half of what fits before T more."""
    return max(0, (S - T) - (S - T) // 4)


def _drafted(T):
    return T - T // 4 if T > 1 else 1


def _path(c):
    """Nodes on the accepted path: three quarters of the tree's levels."""
    return (-(-c["T"] // c["w"]) * 3 - 1) // 4 + 1


def _beams_page(c):
    return -(-c["S"] // c["page"]) + 1


def work(c):
    op, B, d = c["op"], c["B"], c["d"]
    if op == "axes":
        n = B * (c["Hq"] + c["Hkv"]) * c["N"]
        return {"bytes": 4 * n * d + 4 * c["A"] * B * c["N"] + 6 * c["rot"], "flops": 3 * n * c["rot"]}
    if op in ("append", "draft"):
        T = c["T"]
        n = B * (c["Hq"] + 2 * c["Hkv"]) * T
        if op == "append":
            n = n * 3 // 4
        words = -(-T // 64)
        small = B * T * (8 * words + 8) if op == "draft" else 4 * c["A"] * B * T
        return {"bytes": 4 * n * d + small + 12 * B + 6 * c["rot"], "flops": 3 * n * c["rot"]}
    if op == "tree":
        rows, keys = c["Hq"] * _drafted(c["T"]), _mean(c["S"], c["T"])
        per = keys + _drafted(c["T"])
        return {"bytes": B * (4 * d * c["Hkv"] * per + c["Hq"] * c["T"] * (4 * d + 4) + 8 * c["T"] * -(-c["T"] // 64)),
                "flops": 4 * d * B * rows * (keys + (_path(c) + 1) // 2)}
    if op == "accept":
        moved = _path(c) if c["w"] > 1 else 0
        return {"bytes": 8 * d * B * c["Hkv"] * c["layers"] * moved + 20 * B, "flops": B * c["T"]}
    per = _beams_page(c)
    entries = B * per
    if op == "beams":
        # about every other beam has to copy the keys of a page that it shares
        copied = B // 2 * (c["page"] // 2)
        return {"bytes": 16 * entries + 8 * copied * c["Hkv"] * d * c["layers"], "flops": entries}
    moved = entries // 2 * c["page"]  # of twice as many pages half are in use, half of those in the upper half
    return {"bytes": 8 * moved * c["Hkv"] * d * c["layers"] + 8 * entries + 16 * entries, "flops": 2 * entries}


# ------------------------------------------------------------------ inputs
def _normal(shape, g, std=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    return x.mul_(std) if std != 1.0 else x


def _ints(lo, hi, shape, g):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _tokens(B, H, N, d, g, packed):
    return _normal((B, N, H, d), g).transpose(1, 2) if packed else _normal((B, H, N, d), g)


def _sections(pairs, A, cycled):
    """Axis of every pair: runs of unequal length, or dealt out in turn."""
    if cycled:
        return torch.arange(pairs, dtype=torch.int32, device=DEV) % A
    cut = [pairs * (i + 1) * (i + 2) // (A * (A + 1)) for i in range(A)]
    return torch.tensor([sum(i >= n for n in cut) for i in range(pairs)], dtype=torch.int32, device=DEV).clamp(max=A - 1)


def _positions(A, B, N, g):
    """A stretch of text, then frames: the first axis goes on, the others run over a grid."""
    n = torch.arange(N, device=DEV)
    start = _ints(0, 100000, (B, 1), g).long()
    rows = [start + (n if a == 0 else (n // 3 ** (3 - a)) % (7 + 5 * a)) for a in range(A)]
    return torch.stack(rows).to(torch.int32).contiguous()


def _tree(B, T, w, g):
    """Levels of w nodes, a node's parent anywhere in the level above; -1 behind the cache's last key."""
    t = torch.arange(T, device=DEV)
    pick = torch.randint(0, w, (B, T), generator=g, device=DEV)
    return torch.where(t < w, torch.full_like(pick, -1), (t // w - 1) * w + pick).to(torch.int32)


def _ancestors(parents):
    """[B, T, T]: whether node t has u on its way from the root, itself included."""
    B, T = parents.shape
    up = parents.long()
    seen = torch.eye(T, device=DEV, dtype=torch.bool).expand(B, T, T).clone()
    step = 1
    while step < T:
        at = up.clamp(min=0)
        there = (up >= 0)[..., None]
        seen |= seen.gather(1, at[..., None].expand(B, T, T)) & there
        up = torch.where(up >= 0, up.gather(1, at), up)
        step *= 2
    return seen


def _bits(seen):
    """[B, T, T] truth values -> [B, T, words] int64."""
    B, T, U = seen.shape
    words = -(-U // 64)
    x = torch.zeros((B, T, words * 64), device=DEV, dtype=torch.int64)
    x[..., :U] = seen.long()
    return (x.view(B, T, words, 64) << torch.arange(64, device=DEV)).sum(-1)


def _pool(c, g, layers=None):
    """(keys, values, table): contiguous caches without a table where page is 0, else pages in any order."""
    lead = () if layers is None else (layers,)
    if c["page"] == 0:
        shape, table = lead + (c["B"], c["Hkv"], c["S"], c["d"]), None
    else:
        per = -(-c["S"] // c["page"])
        n = c["B"] * per + 3
        order = torch.rand(n, generator=g, device=DEV).argsort()
        table = order[: c["B"] * per].view(c["B"], per).to(torch.int32).contiguous()
        shape = lead + (n, c["Hkv"], c["page"], c["d"])
    return _normal(shape, g), _normal(shape, g), table


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, B, d, Hkv = c["op"], c["B"], c["d"], c["Hkv"]
    s = dict(c)
    if op in ("axes", "append", "draft"):
        pairs = c["rot"] // 2
        s["freqs"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
        s["axes"] = None if op == "draft" else _sections(pairs, c["A"], c["cycled"])
    if op == "axes":
        s["q"], s["k"] = _tokens(B, c["Hq"], c["N"], d, g, c["packed"]), _tokens(B, Hkv, c["N"], d, g, c["packed"])
        s["pos"] = _positions(c["A"], B, c["N"], g)
        return s
    if op in ("append", "draft"):
        T = c["T"]
        s["q"], s["k"], s["v"] = _normal((B, T, c["Hq"] + 2 * Hkv, d), g).transpose(1, 2).split([c["Hq"], Hkv, Hkv], 1)
        s["kc"], s["vc"], s["table"] = _pool(c, g)
        s["lens"] = _ints(0, c["S"] - T, (B,), g)
    if op == "append":
        s["new"], s["pos"] = _ints(T // 2, T, (B,), g), _positions(c["A"], B, T, g)
    if op in ("draft", "tree", "accept"):
        s["parents"] = _tree(B, c["T"], c["w"], g)
    if op == "draft":
        s["inter"] = False
    if op == "tree":
        T = c["T"]
        s["q"] = _normal((B, c["Hq"], T, d), g, std=2.0)
        s["kc"], s["vc"], s["table"] = _pool(c, g)
        room = c["S"] - T
        s["lens"] = _ints((room + 1) // 2, room, (B,), g)
        s["lens"][0] = room
        s["drafted"] = _ints((T + 1) // 2, T, (B,), g)
        s["mask"] = _bits(_ancestors(s["parents"]))
    if op == "accept":
        s["kc"], s["vc"], s["table"] = _pool(c, g, c["layers"])
        s["lens"] = _ints(0, c["S"] - c["T"], (B,), g)
        s["mask"] = _bits(_ancestors(s["parents"]))
        level = _path(c) - 1
        s["last"] = (level * c["w"] + _ints(0, c["w"] - 1, (B,), g)).clamp(max=c["T"] - 1).to(torch.int32)
    if op in ("beams", "compact"):
        per = _beams_page(c)
        n = 2 * B * per + 8
        shape = (c["layers"], n, Hkv, c["page"], d)
        s["kp"], s["vp"] = _normal(shape, g), _normal(shape, g)
        order = torch.rand(n, generator=g, device=DEV).argsort()
        s["lens"] = _ints(max(1, c["S"] // 2), c["S"], (B,), g)
        held = torch.arange(per, device=DEV) < (-(-s["lens"] // c["page"]))[:, None]
        s["table0"] = torch.where(held, order[: B * per].view(B, per), -1).to(torch.int32)
        s["refs0"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        s["refs0"][s["table0"][held].long()] = 1
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
        s["table2"], s["lens2"] = torch.empty_like(s["table"]), torch.empty_like(s["lens"])
    if op == "beams":
        # half of the beams go on as others
        b = torch.arange(B, device=DEV)
        s["parent"] = torch.where(torch.rand(B, generator=g, device=DEV) < 0.5, b,
                                  torch.randint(0, B, (B,), generator=g, device=DEV)).to(torch.int32)
    return s


# ------------------------------------------------------- the library's calls
def _run_own(s):
    import attention_fa2_fwd_sm_gb300 as attn
    op = s["op"]
    if op == "axes":
        call = attn.rope_axes_backward if s["inverse"] else attn.rope_axes
        return call(s["q"], s["k"], s["freqs"], s["axes"], s["pos"], interleaved=s["inter"])
    if op == "append":
        q, lens = attn.rope_axes_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["lens"], s["freqs"], s["axes"], s["pos"],
                                        page_table=s["table"], new_lens=s["new"], interleaved=s["inter"])
        return q, s["kc"], s["vc"], lens
    if op == "draft":
        mask, pos = attn.tree_mask(s["parents"], s["lens"])
        q, lens = attn.rope_axes_append(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["lens"], s["freqs"], None, pos,
                                        page_table=s["table"])
        return mask, pos, q, s["kc"], s["vc"], lens
    if op == "tree":
        o, lse, s["ws"] = attn.decode_tree(s["q"], s["kc"], s["vc"], s["lens"], s["mask"], draft_lens=s["drafted"],
                                           page_table=s["table"], workspace=s.get("ws"))
        return o, lse
    if op == "accept":
        lens = attn.tree_accept(s["kc"], s["vc"], s["lens"], s["mask"], s["last"], page_table=s["table"])
        return s["kc"], s["vc"], lens
    # Both start from the same tables every time.
    s["refs"].copy_(s["refs0"])
    if op == "beams":
        attn.pages_fork(s["table0"], s["refs"], s["lens"], s["parent"], s["page"], page_table_out=s["table2"],
                        seqlens_out=s["lens2"])
        info, s["ws"] = attn.pages_extend(s["table2"], s["refs"], s["lens2"], 1, s["kp"], s["vp"], workspace=s.get("ws"))
        return s["table2"], s["refs"], s["lens2"], info, s["kp"], s["vp"]
    s["table"].copy_(s["table0"])
    info, s["ws"] = attn.pages_compact(s["table"], s["refs"], s["kp"], s["vp"], workspace=s.get("ws"))
    return s["table"], s["refs"], info, s["kp"], s["vp"]


# ---------------------------------------------------------------- plain form
def _rotate(x, pos, freqs, axes, inter, sign):
    """x [B, H, N, d]; pos [axes, B, N]."""
    r = 2 * freqs.numel()
    p = pos[axes.long()].permute(1, 2, 0) if axes is not None else pos[..., None]
    a = (p.double() * freqs)[:, None]  # angles of far positions need 64 bits
    c, n = torch.cos(a).float(), sign * torch.sin(a).float()
    y = x.float()
    u, v = (y[..., 0:r:2], y[..., 1:r:2]) if inter else (y[..., : r // 2], y[..., r // 2: r])
    u, v = u * c - v * n, v * c + u * n
    head = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((head, y[..., r:]), -1).to(x.dtype)


def _place(s, b, row):
    """Where rows `row` of sequences `b` are: (cache entry or page, row in it)."""
    if s["table"] is None:
        return b, row
    return s["table"][b, row // s["page"]].long(), row % s["page"]


def _append(s, pos, new):
    B, _, T, _ = s["q"].shape
    q, k = (_rotate(x, pos, s["freqs"], s["axes"], s["inter"], 1.0) for x in (s["q"], s["k"]))
    t = torch.arange(T, device=DEV)
    row = (s["lens"][:, None] + t).long()
    b, t = ((t < new[:, None]) & (row < s["S"])).nonzero(as_tuple=True)
    page, at = _place(s, b, row[b, t])
    s["kc"][page, :, at] = k[b, :, t]
    s["vc"][page, :, at] = s["v"][b, :, t]
    return q, (s["lens"] + new).clamp(max=s["S"])


def _keys(s, x, b):
    """One sequence's rows [Hkv, slots, d]."""
    if s["table"] is None:
        return x[b]
    return x[s["table"][b].long()].transpose(0, 1).flatten(1, 2)


def _attend(s):
    q = s["q"]
    B, Hq, T, d = q.shape
    Hkv = s["Hkv"]
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, T), device=DEV)
    u = torch.arange(T, device=DEV)
    for b in range(B):
        k, v = _keys(s, s["kc"], b), _keys(s, s["vc"], b)
        j = torch.arange(k.shape[1], device=DEV)
        draft = j - s["lens"][b]
        at = draft.clamp(0, T - 1)
        bit = (s["mask"][b][:, at // 64] >> (at % 64)) & 1
        sees = (draft < 0) | ((bit == 1) & (draft < s["drafted"][b]))
        sees &= (u < s["drafted"][b])[:, None]
        x = q[b].view(Hkv, -1, T, d).float().flatten(1, 2) @ k.float().transpose(1, 2) * d ** -0.5
        x = x.view(Hkv, -1, T, x.shape[-1]).masked_fill(~sees, -math.inf)
        top = x.amax(-1, keepdim=True)
        p = (x - top.clamp(min=-1e30)).exp()
        total = p.sum(-1, keepdim=True)
        out = p.flatten(1, 2) @ v.float().masked_fill((draft >= s["drafted"][b])[:, None], 0.0)
        out = out.view(Hkv, -1, T, d) / total.clamp(min=1e-30)
        o[b] = out.flatten(0, 1).to(q.dtype)
        lse[b] = (top + total.log()).view(Hq, T)
    return o, lse


def _accept(s):
    T = s["T"]
    row = s["mask"].gather(1, s["last"].long()[:, None, None].expand(-1, 1, s["mask"].shape[-1]))[:, 0]
    u = torch.arange(T, device=DEV)
    on = ((row[:, u // 64] >> (u % 64)) & 1).bool()
    to = on.cumsum(1) - 1
    b, src = on.nonzero(as_tuple=True)
    page, at = _place(s, b, s["lens"][b].long() + src)
    page2, at2 = _place(s, b, s["lens"][b].long() + to[b, src])
    for x in (s["kc"], s["vc"]):
        x[:, page2, :, at2] = x[:, page, :, at]
    return s["kc"], s["vc"], (s["lens"] + on.sum(1)).to(torch.int32)


def _beams(s):
    ps = s["page"]
    B, per = s["table"].shape
    slot = torch.arange(per, device=DEV)
    b = torch.arange(B, device=DEV)
    refs, table = s["refs"], s["table0"]
    one = torch.ones((), dtype=torch.int32, device=DEV)
    # continue as the parent
    p = s["parent"].long()
    lens = s["lens"][p]
    new = torch.where((slot < (-(-lens // ps))[:, None]) | (p == b)[:, None], table[p], -1)
    refs.index_add_(0, table[table >= 0].long(), -one.expand(int((table >= 0).sum())))
    refs.index_add_(0, new[new >= 0].long(), one.expand(int((new >= 0).sum())))
    # room for one more key: a missing page is taken, a shared one copied
    lo = lens // ps
    last = (slot == lo[:, None]) & (slot < per)
    at = new.clamp(min=0).long()
    shared = last & (new >= 0) & (refs[at] > 1)
    writers = torch.zeros_like(refs).index_add_(0, at[shared], one.expand(int(shared.sum())))
    latest = torch.full_like(refs, -1).scatter_reduce_(0, at[shared], b[:, None].expand(B, per)[shared].int(), "amax")
    keep = shared & (writers[at] == refs[at]) & (latest[at] == b[:, None])
    fresh = last & ((new < 0) | (shared & ~keep))
    free = (refs == 0).nonzero().flatten()
    fb, fs = fresh.nonzero(as_tuple=True)
    pages = free[: fb.numel()]
    old = new[fb, fs]
    new[fb, fs] = pages.int()
    refs[pages] = 1
    copied = old >= 0
    refs.index_add_(0, old[copied].long(), -one.expand(int(copied.sum())))
    src, dst = old[copied].long(), pages[copied]
    live = (torch.arange(ps, device=DEV) < (lens % ps)[fb[copied]][:, None])[None, :, None, :, None]
    for x in (s["kp"], s["vp"]):
        x[:, dst] = torch.where(live, x[:, src], x[:, dst])
    s["table2"].copy_(new)
    s["lens2"].copy_(lens)
    info = torch.stack((fresh.sum(), torch.zeros((), dtype=torch.int64, device=DEV))).to(torch.int32)
    return s["table2"], refs, s["lens2"], info, s["kp"], s["vp"]


def _compact(s):
    refs, table = s["refs"], s["table"]
    used = refs > 0
    n = int(used.sum())
    holes = (~used[:n]).nonzero().flatten()
    movers = used[n:].nonzero().flatten() + n
    for x in (s["kp"], s["vp"]):
        for layer in x:
            layer[holes] = layer[movers]
    to = torch.arange(refs.numel(), device=DEV, dtype=torch.int32)
    to[movers] = holes.int()
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    info = torch.tensor([n, holes.numel()], dtype=torch.int32, device=DEV)
    return table, refs, info, s["kp"], s["vp"]


def _run_plain(s):
    op = s["op"]
    if op == "axes":
        sign = -1.0 if s["inverse"] else 1.0
        return tuple(_rotate(x, s["pos"], s["freqs"], s["axes"], s["inter"], sign) for x in (s["q"], s["k"]))
    if op == "append":
        q, lens = _append(s, s["pos"], s["new"])
        return q, s["kc"], s["vc"], lens
    if op == "draft":
        seen = _ancestors(s["parents"])
        mask = _bits(seen)
        pos = (s["lens"][:, None] + seen.sum(-1) - 1).to(torch.int32)
        q, lens = _append(s, pos, torch.full_like(s["lens"], s["T"]))
        return mask, pos, q, s["kc"], s["vc"], lens
    if op == "tree":
        return _attend(s)
    if op == "accept":
        return _accept(s)
    s["refs"].copy_(s["refs0"])
    if op == "beams":
        return _beams(s)
    s["table"].copy_(s["table0"])
    return _compact(s)


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------- 64-bit definition
def _turned(x, pos, freqs, axes, inter, sign):
    """The rotation as a product of complex numbers; pos [axes, B, N]."""
    r = 2 * freqs.numel()
    which = [0] * (r // 2) if axes is None else axes.tolist()
    a = torch.stack([pos[w].double() * f for w, f in zip(which, freqs)], -1)
    z = torch.polar(torch.ones_like(a), sign * a)[:, None]
    y = x.double()
    if inter:
        w = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * z
        head = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., : r // 2].contiguous(), y[..., r // 2: r].contiguous()) * z
        head = torch.cat((w.real, w.imag), -1)
    return torch.cat((head, y[..., r:]), -1)


def _walk(parents):
    """Depth of every node, its ancestors in a list (one sequence)."""
    seen = []
    for t, p in enumerate(parents):
        seen.append(([] if p < 0 else seen[p]) + [t])
    return seen


def exact(c, seed):
    op = c["op"]
    if op in ("accept", "beams", "compact"):
        return None  # nothing is computed: rows and numbers are moved
    s = prepare(c, seed)
    if op == "axes":
        sign = -1.0 if c["inverse"] else 1.0
        return tuple(_turned(x, s["pos"], s["freqs"], s["axes"], c["inter"], sign) for x in (s["q"], s["k"]))
    B, T, lens = c["B"], c["T"], s["lens"].tolist()
    if op in ("append", "draft"):
        new = s["new"].tolist() if op == "append" else [T] * B
        if op == "draft":
            depth = [[len(x) - 1 for x in _walk(p)] for p in s["parents"].tolist()]
            s["pos"] = (torch.tensor(depth, device=DEV) + s["lens"][:, None])[None]
        q, k = (_turned(x, s["pos"], s["freqs"], s["axes"], s["inter"], 1.0) for x in (s["q"], s["k"]))
        kc, vc = s["kc"].double(), s["vc"].double()
        table = None if s["table"] is None else s["table"].tolist()
        for b in range(B):
            for t in range(min(new[b], c["S"] - lens[b])):
                at = lens[b] + t
                e, r = (b, at) if table is None else (table[b][at // c["page"]], at % c["page"])
                kc[e, :, r], vc[e, :, r] = k[b, :, t], s["v"][b, :, t].double()
        return (q, kc, vc, None) if op == "append" else (None, None, q, kc, vc, None)
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    o = torch.zeros((B, Hq, T, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    for b, drafted in enumerate(s["drafted"].tolist()):
        n = lens[b] + drafted
        k, v = (_keys(s, x, b)[:, :n].double() for x in (s["kc"], s["vc"]))
        hide = torch.zeros((drafted, n), dtype=torch.float64, device=DEV)
        for t, path in enumerate(_walk(s["parents"][b, :drafted].tolist())):
            hide[t, lens[b]:] = -math.inf
            hide[t, [lens[b] + u for u in path]] = 0.0
        for h in range(Hkv):
            G = Hq // Hkv
            x = s["q"][b, h * G: (h + 1) * G, :drafted].double() @ k[h].T / math.sqrt(d) + hide
            o[b, h * G: (h + 1) * G, :drafted] = torch.softmax(x, -1) @ v[h]
            lse[b, h * G: (h + 1) * G, :drafted] = torch.logsumexp(x, -1)
    return o, lse
