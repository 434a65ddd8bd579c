"""Workloads of the decode-cache operators: rotary positions (training and
prefill, and appending to a cache), decode over a prefix that the whole batch
shares, decode that accumulates every cached key's attention weight, and
eviction from the cache by that weight.

Each case runs either in its plain form (elementary torch operations in 32
bits) or, with ``own`` set, through attention_fa2_fwd_sm_gb300.  Layouts are
the library's: caches [B, Hkv, slots, d], a prefix [Hkv, P, d], bf16.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One prompt of 8K tokens before prefill: q and k as [B, H, N, d], whole head rotated.
        dict(name="rope prompt 8K", op="rope", B=1, Hq=64, Hkv=8, N=8192, d=128, rot=128, inter=False, inverse=False,
             packed=False, far=0, factor=1.0),
        # Gradients of a training step through the rotation, taken from a fused projection's layout
        # [B, N, H, d], interleaved pairs, an odd length.
        dict(name="rope gradients", op="rope", B=2, Hq=32, Hkv=32, N=4097, d=64, rot=64, inter=True, inverse=True,
             packed=True, far=0, factor=1.0),
        # One short prompt: latency.  Part of the head, frequencies stretched for a long context, far positions.
        dict(name="rope short", op="rope", B=1, Hq=16, Hkv=2, N=33, d=128, rot=32, inter=False, inverse=False,
             packed=True, far=1000000, factor=8.0),
        # One decode step of 32 users: a token each into their caches.
        dict(name="append token", op="append", B=32, Hq=64, Hkv=8, T=1, S=8192, d=128, rot=128, inter=False, far=0,
             factor=1.0, ragged=False),
        # A chunk of a long prompt of four users, of unequal lengths, into their caches.
        dict(name="append chunk", op="append", B=4, Hq=64, Hkv=8, T=2000, S=8192, d=128, rot=64, inter=True,
             far=100000, factor=4.0, ragged=True),
        # A few users, a short system prompt: latency.
        dict(name="prefix small", op="prefix", B=4, Hq=8, Hkv=2, P=500, S=64, d=64),
        # A serving batch behind a common 8K document.
        dict(name="prefix 8K", op="prefix", B=32, Hq=64, Hkv=8, P=8192, S=512, d=128),
        # The largest: 128 users behind a common 32K context, each with its own turns.
        dict(name="prefix 32K", op="prefix", B=128, Hq=64, Hkv=8, P=32768, S=1024, d=128),
        # One user's decode step that keeps count of what each key receives.
        dict(name="weights one user", op="weigh", B=1, Hq=64, Hkv=8, S=8192, d=128),
        # A batch's decode step over long caches, counted.
        dict(name="weights batch", op="weigh", B=32, Hq=64, Hkv=8, S=16001, d=128),
        # Steady state of a bounded cache: a token comes in, the lightest key goes out.
        dict(name="evict step", op="step", B=32, Hq=64, Hkv=8, keep=4096, recent=256, S=4104, d=128, rot=128,
             inter=False),
        # After a long prompt: its 32K keys compacted into a decode cache of 8K.
        dict(name="evict prompt", op="evict", B=4, Hkv=8, n=32768, keep=8000, recent=512, S=8192, d=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefix", "prefix", "weigh", "weigh", "step", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 5, 8])
    c = dict(op=op, B=_log(rng, 1, 16), d=d)
    if op in ("rope", "append", "step"):
        c.update(rot=rng.choice([d, d // 2, d // 4]), inter=rng.random() < 0.5)
    if op == "rope":
        c.update(Hq=Hkv * G, Hkv=Hkv, N=max(1, _log(rng, 1, 65536) // (c["B"] * G)), inverse=rng.random() < 0.5,
                 packed=rng.random() < 0.5, far=rng.choice([0, 1000, 1000000]), factor=rng.choice([1.0, 4.0, 8.0]))
    elif op == "append":
        T = rng.choice([1, _log(rng, 2, 2048)])
        c.update(Hq=Hkv * G, Hkv=Hkv, T=T, S=T + _log(rng, 16, 4096), far=rng.choice([0, 1000, 1000000]),
                 factor=rng.choice([1.0, 4.0, 8.0]), ragged=T > 1)
    elif op == "prefix":
        c.update(B=_log(rng, 1, 128), Hq=Hkv * G, Hkv=Hkv, P=_log(rng, 1, 32768), S=_log(rng, 1, 1024))
    elif op == "weigh":
        c.update(Hq=Hkv * G, Hkv=Hkv, S=_log(rng, 16, 16384))
    elif op == "step":
        keep = _log(rng, 64, 8192)
        c.update(Hq=Hkv * G, Hkv=Hkv, keep=keep, recent=keep // rng.choice([4, 8, 16]), S=keep + rng.randint(1, 32))
    else:
        keep = _log(rng, 64, 8192)
        c.update(B=_log(rng, 1, 4), Hkv=Hkv, n=keep + _log(rng, 1, 24000), keep=keep, recent=keep // rng.choice([4, 8]),
                 S=keep + rng.randint(0, 64))
    return c


def work(c):
    op, B, d = c["op"], c["B"], c["d"]
    if op == "rope":
        n = B * (c["Hq"] + c["Hkv"]) * c["N"]
        return {"bytes": 4 * n * d + 4 * B * c["N"] + 4 * c["rot"], "flops": 3 * n * c["rot"]}
    if op in ("append", "step"):
        T = c.get("T", 1)
        n = B * (c["Hq"] + 2 * c["Hkv"]) * T
        if c.get("ragged"):
            n = n * 3 // 4
        w = {"bytes": 4 * n * d + 12 * B + 8 * B * c["Hkv"] * T + 4 * c["rot"], "flops": 3 * n * c["rot"]}
        if op == "append":
            return w
        rows = B * c["Hkv"]
        # Every weight and position is looked at, and one key's row moves in about every head.
        return {"bytes": w["bytes"] + 8 * rows * (c["keep"] + 1) + 8 * rows * d, "flops": w["flops"] + rows * c["keep"]}
    if op == "prefix":
        keys = c["P"] + B * _mean_len(c["S"])
        return {"bytes": 4 * d * c["Hkv"] * keys + 4 * B * c["Hq"] * d + 4 * B * c["Hq"],
                "flops": 4 * d * c["Hq"] * B * (c["P"] + _mean_len(c["S"]))}
    if op == "weigh":
        keys = B * _mean_len(c["S"])
        return {"bytes": (4 * d + 8) * c["Hkv"] * keys + 4 * B * c["Hq"] * d + 4 * B * c["Hq"],
                "flops": 4 * d * c["Hq"] * keys}
    rows = B * c["Hkv"]
    return {"bytes": 8 * rows * c["n"] + rows * c["keep"] * (8 * d + 8), "flops": rows * c["n"]}


# ------------------------------------------------------------------ inputs
def _mean_len(S):
    return max(1, S - S // 4)  # lengths are spread evenly over the upper half of the cache


def _lens(B, S, g):
    """Lengths in [ceil(S / 2), S], the first one full."""
    lo = (S + 1) // 2
    n = torch.randint(lo, S + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    n[0] = S
    return n


def _normal(shape, g, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _frequencies(rot, factor):
    """Radians a position, 64 bits: base 10000, slow pairs stretched by `factor` (linear in the number of turns that a
    pair makes over 8192 positions, between 1 and 4)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    keep = ((8192 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
    return (f * (keep + (1.0 - keep) / factor)).to(DEV)


def _tokens(B, H, N, d, g, packed):
    """[B, H, N, d], as a view of [B, N, H, d] where packed."""
    return _normal((B, N, H, d), g).transpose(1, 2) if packed else _normal((B, H, N, d), g)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, B, d = c["op"], c["B"], c["d"]
    s = dict(c)
    if op == "rope":
        s["freqs"] = _frequencies(c["rot"], c["factor"])
        s["q"] = _tokens(B, c["Hq"], c["N"], d, g, c["packed"])
        s["k"] = _tokens(B, c["Hkv"], c["N"], d, g, c["packed"])
        start = c["far"] + torch.randint(0, 64, (B, 1), generator=g, device=DEV)
        s["pos"] = (start + torch.arange(c["N"], device=DEV)).to(torch.int32)
    if op in ("append", "step"):
        T = c.get("T", 1)
        # one projection's output: [B, T, Hq + 2 Hkv, d]
        qkv = _normal((B, T, c["Hq"] + 2 * c["Hkv"], d), g).transpose(1, 2)
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s["freqs"] = _frequencies(c["rot"], c.get("factor", 1.0))
    if op == "append":
        s["kcache"], s["vcache"] = _normal((B, c["Hkv"], c["S"], d), g), _normal((B, c["Hkv"], c["S"], d), g)
        s["lens"] = torch.randint(0, c["S"] - T + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["pos"] = s["lens"] + c["far"]
        s["new"] = torch.randint(T // 2, T + 1, (B,), generator=g, device=DEV, dtype=torch.int32) if c["ragged"] else None
    if op == "prefix":
        s["kp"], s["vp"] = _normal((c["Hkv"], c["P"], d), g), _normal((c["Hkv"], c["P"], d), g)
    if op in ("prefix", "weigh"):
        s["q"] = _normal((B, c["Hq"], d), g, std=2.0)
        s["kcache"], s["vcache"] = _normal((B, c["Hkv"], c["S"], d), g), _normal((B, c["Hkv"], c["S"], d), g)
        s["lens"] = _lens(B, c["S"], g)
    if op == "weigh":
        s["weights"] = torch.rand((B, c["Hkv"], c["S"]), generator=g, device=DEV) ** 4
    if op in ("step", "evict"):
        n = c["n"] if op == "evict" else c["S"]
        s["kcache"], s["vcache"] = _normal((B, c["Hkv"], n, d), g), _normal((B, c["Hkv"], n, d), g)
        # most keys have received little, a few much; some nothing at all
        w = torch.rand((B, c["Hkv"], n), generator=g, device=DEV)
        s["weights"] = torch.where(w < 0.05, torch.zeros_like(w), w ** 8 * 4)
    if op == "step":
        # slots in the order that earlier evictions left; positions up to 4 times the cache's size
        mixed = torch.rand((B, c["Hkv"], 4 * c["keep"]), generator=g, device=DEV).argsort(-1)[..., : c["S"]]
        s["pos"] = mixed.to(torch.int32).contiguous()
        s["lens"] = torch.full((B,), c["keep"], dtype=torch.int32, device=DEV)
        s["lens2"] = torch.empty_like(s["lens"])
        s["cur"] = torch.full((B,), 4 * c["keep"] - 1, dtype=torch.int32, device=DEV)
    if op == "evict":
        s["lens"] = torch.full((B,), c["n"], dtype=torch.int32, device=DEV)
        s["out"] = dict(kcache=torch.zeros((B, c["Hkv"], c["S"], d), dtype=torch.bfloat16, device=DEV),
                        vcache=torch.zeros((B, c["Hkv"], c["S"], d), dtype=torch.bfloat16, device=DEV),
                        weights=torch.zeros((B, c["Hkv"], c["S"]), device=DEV),
                        cache_pos=torch.zeros((B, c["Hkv"], c["S"]), dtype=torch.int32, device=DEV),
                        seqlens=torch.zeros((B,), dtype=torch.int32, device=DEV))
    return s


# ------------------------------------------------------- the library's calls
def _run_own(s):
    import attention_fa2_fwd_sm_gb300 as attn
    op = s["op"]
    if op == "rope":
        call = attn.rope_backward if s["inverse"] else attn.rope
        return call(s["q"], s["k"], s["freqs"], positions=s["pos"], interleaved=s["inter"])
    if op == "append":
        q, lens = attn.rope_append(s["q"], s["k"], s["v"], s["kcache"], s["vcache"], s["lens"], s["freqs"],
                                   start_pos=s["pos"], new_lens=s["new"], interleaved=s["inter"])
        return q, s["kcache"], s["vcache"], lens
    if op == "prefix":
        o, lse, s["ws"] = attn.decode_prefix(s["q"], s["kp"], s["vp"], s["kcache"], s["vcache"], s["lens"],
                                             workspace=s.get("ws"))
        return o, lse
    if op == "weigh":
        o, lse, s["ws"] = attn.decode_weighted(s["q"], s["kcache"], s["vcache"], s["lens"], s["weights"],
                                               workspace=s.get("ws"))
        return o, lse, s["weights"]
    if op == "step":
        s["cur"] += 1
        q, _ = attn.rope_append(s["q"], s["k"], s["v"], s["kcache"], s["vcache"], s["lens"], s["freqs"],
                                start_pos=s["cur"], interleaved=s["inter"], cache_pos=s["pos"], weights=s["weights"],
                                seqlens_out=s["lens2"])
        s["ews"] = attn.cache_evict(s["kcache"], s["vcache"], s["weights"], s["lens2"], s["keep"], s["recent"],
                                    cache_pos=s["pos"], cur_pos=s["cur"], seqlens_out=s["lens"],
                                    workspace=s.get("ews"))[-1]
        return q, s["kcache"], s["vcache"], s["weights"], s["pos"], s["lens"]
    o = s["out"]
    s["ews"] = attn.cache_evict(s["kcache"], s["vcache"], s["weights"], s["lens"], s["keep"], s["recent"],
                                out=o, workspace=s.get("ews"))[-1]
    return o["kcache"], o["vcache"], o["weights"], o["cache_pos"], o["seqlens"]


# ---------------------------------------------------------------- plain form
def _rotate(x, pos, freqs, inter, sign):
    """x [B, H, N, d]; pos [B, N]."""
    r = 2 * freqs.numel()
    a = (pos.double()[..., None] * freqs)[:, None]  # angles of far positions need 64 bits
    c, n = torch.cos(a).float(), sign * torch.sin(a).float()
    y = x.float()
    u, v = (y[..., 0:r:2], y[..., 1:r:2]) if inter else (y[..., : r // 2], y[..., r // 2: r])
    u, v = u * c - v * n, v * c + u * n
    head = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((head, y[..., r:]), -1).to(x.dtype)


def _append(s, pos):
    """Rotates the new tokens, puts keys and values behind each sequence's last; the rotated queries and new lengths."""
    B, _, T, _ = s["q"].shape
    t = torch.arange(T, device=DEV)
    at = pos[:, None] + t
    q, k = (_rotate(x, at, s["freqs"], s["inter"], 1.0) for x in (s["q"], s["k"]))
    new = s.get("new")
    new = torch.full_like(s["lens"], T) if new is None else new
    slot = (s["lens"][:, None] + t).long()
    live = (t < new[:, None]) & (slot < s["S"])
    b, t = live.nonzero(as_tuple=True)
    slot = slot[b, t]
    s["kcache"][b, :, slot] = k[b, :, t]
    s["vcache"][b, :, slot] = s["v"][b, :, t]
    if "cur" in s:
        s["pos"][b, :, slot] = at[b, t][:, None].expand(-1, s["Hkv"]).int()
        s["weights"][b, :, slot] = 0.0
    return q, (s["lens"] + new).clamp(max=s["S"])


def _decode(s):
    """Softmax over the prefix's keys and the sequence's own; (o, lse, weight of each own key)."""
    q = s["q"]
    B, Hq, d = q.shape
    Hkv = s["Hkv"]
    q = q.float().view(B, Hkv, Hq // Hkv, d) * d ** -0.5
    x = q @ s["kcache"].float().transpose(2, 3)
    gone = (torch.arange(s["S"], device=DEV) >= s["lens"][:, None])[:, None, None]
    x = x.masked_fill(gone, -math.inf)
    top = x.amax(-1, keepdim=True)
    if "kp" in s:
        y = torch.einsum("bghd,gpd->bghp", q, s["kp"].float())
        top = torch.maximum(top, y.amax(-1, keepdim=True))
        y = (y - top).exp()
    x = (x - top).exp()
    total = x.sum(-1, keepdim=True)
    o = x @ s["vcache"].float()
    if "kp" in s:
        total = total + y.sum(-1, keepdim=True)
        o = o + torch.einsum("bghp,gpd->bghd", y, s["vp"].float())
    return ((o / total).view(B, Hq, d).to(s["q"].dtype), (top + total.log()).view(B, Hq), (x / total).sum(2))


def _evict(kcache, vcache, weights, pos, lens, keep, recent, cur, out):
    """Keeps `keep` keys of every head: the latest `recent`, then the heaviest, the lowest slot first among equals.
    Kept slots below `keep` stay; the others fill the gaps in order."""
    n = weights.shape[-1]
    slot = torch.arange(n, device=DEV)
    live = slot < lens[:, None, None]
    rank = weights.masked_fill(pos > (cur - recent)[:, None, None], math.inf).masked_fill(~live, -math.inf)
    first = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.zeros_like(live.expand_as(rank)).scatter_(-1, first, True) & live
    gap = (live & ~kept)[..., :keep]
    filler = kept & (slot >= keep)
    far = torch.where(filler, slot, n).sort(-1).values[..., :keep]
    at = gap.cumsum(-1) - 1
    src = torch.where(gap, far.gather(-1, at.clamp(min=0)), slot[:keep].expand_as(at))
    mine = (slot[:keep] < lens[:, None, None]).expand_as(src)
    rows = src[..., None].expand(-1, -1, -1, kcache.shape[-1])
    for name, x in (("kcache", kcache), ("vcache", vcache)):
        old = out[name][:, :, :keep]
        out[name][:, :, :keep] = torch.where(mine[..., None], x.gather(2, rows), old)
    for name, x in (("weights", weights), ("cache_pos", pos)):
        out[name][..., :keep] = torch.where(mine, x.gather(-1, src), out[name][..., :keep])
    out["seqlens"].copy_(lens.clamp(max=keep))


def _run_plain(s):
    op = s["op"]
    if op == "rope":
        sign = -1.0 if s["inverse"] else 1.0
        return tuple(_rotate(x, s["pos"], s["freqs"], s["inter"], sign) for x in (s["q"], s["k"]))
    if op == "append":
        q, lens = _append(s, s["pos"])
        return q, s["kcache"], s["vcache"], lens
    if op == "prefix":
        return _decode(s)[:2]
    if op == "weigh":
        o, lse, w = _decode(s)
        s["weights"] += w
        return o, lse, s["weights"]
    if op == "step":
        s["cur"] += 1
        q, s["lens2"] = _append(s, s["cur"])
        _evict(s["kcache"], s["vcache"], s["weights"], s["pos"], s["lens2"], s["keep"], s["recent"], s["cur"],
               dict(kcache=s["kcache"], vcache=s["vcache"], weights=s["weights"], cache_pos=s["pos"], seqlens=s["lens"]))
        return q, s["kcache"], s["vcache"], s["weights"], s["pos"], s["lens"]
    o = s["out"]
    pos = torch.arange(s["n"], device=DEV, dtype=torch.int32).expand(s["B"], s["Hkv"], -1)
    _evict(s["kcache"], s["vcache"], s["weights"], pos, s["lens"], s["keep"], s["recent"], s["lens"] - 1, o)
    return o["kcache"], o["vcache"], o["weights"], o["cache_pos"], o["seqlens"]


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------- 64-bit definition
def _turned(x, pos, freqs, inter, sign):
    """The rotation as a product of complex numbers."""
    r = 2 * freqs.numel()
    y = x.double()
    z = torch.polar(torch.ones_like(pos.double())[..., None].expand(*pos.shape, r // 2).contiguous(),
                    sign * pos.double()[..., None] * freqs)[:, None]
    if inter:
        w = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * z
        head = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., : r // 2].contiguous(), y[..., r // 2: r].contiguous()) * z
        head = torch.cat((w.real, w.imag), -1)
    return torch.cat((head, y[..., r:]), -1)


def _put(s, pos):
    """exact()'s append, one sequence after another: (queries, key cache, value cache, lengths)."""
    T = s["q"].shape[2]
    at = pos.long()[:, None] + torch.arange(T, device=DEV)
    q, k = (_turned(x, at, s["freqs"], s["inter"], 1.0) for x in (s["q"], s["k"]))
    kc, vc, lens = s["kcache"].double(), s["vcache"].double(), s["lens"].tolist()
    new = [T] * s["B"] if s.get("new") is None else s["new"].tolist()
    for b in range(s["B"]):
        m = min(new[b], s["S"] - lens[b])
        kc[b, :, lens[b]: lens[b] + m] = k[b, :, :m]
        vc[b, :, lens[b]: lens[b] + m] = s["v"][b, :, :m].double()
        lens[b] += m
    return q, kc, vc, lens


def _chosen(weights, pos, n, keep, recent, cur):
    """Slots that hold the kept keys of one head, by slot of the result (numpy)."""
    w = weights[:n].astype(np.float64)
    w[pos[:n] > cur - recent] = np.inf
    kept = np.sort(np.lexsort((np.arange(n), -w))[:keep])
    src = np.arange(min(keep, n))
    src[~np.isin(src, kept)] = kept[kept >= keep]
    return src


def _kept(s, kc, vc, weights, pos, lens, cur, out):
    W, Q = weights.cpu().numpy(), pos.cpu().numpy()
    ok, ov, ow = (x.double() for x in (out["kcache"], out["vcache"], out["weights"]))
    for b in range(s["B"]):
        for h in range(s["Hkv"]):
            src = torch.from_numpy(_chosen(W[b, h], Q[b, h], lens[b], s["keep"], s["recent"], int(cur[b]))).to(DEV)
            m = src.numel()
            ok[b, h, :m], ov[b, h, :m] = kc[b, h, src].double(), vc[b, h, src].double()
            ow[b, h, :m] = weights[b, h, src].double()
    return ok, ov, ow


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "rope":
        sign = -1.0 if c["inverse"] else 1.0
        return tuple(_turned(x, s["pos"].long(), s["freqs"], c["inter"], sign) for x in (s["q"], s["k"]))
    if op == "append":
        q, kc, vc, _ = _put(s, s["pos"])
        return q, kc, vc, None
    if op in ("prefix", "weigh"):
        B, Hkv, d = c["B"], c["Hkv"], c["d"]
        G = c["Hq"] // Hkv
        o = torch.zeros((B, Hkv, G, d), dtype=torch.float64, device=DEV)
        lse = torch.zeros((B, Hkv, G), dtype=torch.float64, device=DEV)
        w = s["weights"].double() if op == "weigh" else None
        q = s["q"].double().view(B, Hkv, G, d)
        for b, n in enumerate(s["lens"].tolist()):
            k, v = s["kcache"][b, :, :n].double(), s["vcache"][b, :, :n].double()
            if op == "prefix":
                k, v = torch.cat((s["kp"].double(), k), 1), torch.cat((s["vp"].double(), v), 1)
            x = (q[b] @ k.transpose(1, 2)) / math.sqrt(d)
            p = torch.softmax(x, -1)
            o[b], lse[b] = p @ v, torch.logsumexp(x, -1)
            if op == "weigh":
                w[b, :, :n] += p.sum(1)
        o, lse = o.view(B, -1, d), lse.view(B, -1)
        return (o, lse, w) if op == "weigh" else (o, lse)
    if op == "step":
        cur = (s["cur"] + 1).tolist()
        q, kc, vc, lens = _put(s, s["cur"] + 1)
        w, pos = s["weights"].clone(), s["pos"].clone()
        w[:, :, c["keep"]], pos[:, :, c["keep"]] = 0.0, (s["cur"] + 1)[:, None]
        ok, ov, ow = _kept(s, kc, vc, w, pos, lens, cur, dict(kcache=kc, vcache=vc, weights=w))
        return q, ok, ov, ow, None, None
    lens = s["lens"].tolist()
    pos = torch.arange(c["n"], device=DEV).expand(c["B"], c["Hkv"], -1)
    ok, ov, ow = _kept(s, s["kcache"], s["vcache"], s["weights"], pos, lens, [n - 1 for n in lens], s["out"])
    return ok, ov, ow, None, None
