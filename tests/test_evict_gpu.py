"""Eviction by weight against the definition: a stable sort of every head's keys on the host.
Nothing is computed, keys only move, so everything is compared bit for bit."""
import math

import numpy as np
import pytest
import torch

from synthetic_inputs import normal_bf16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


def sources(weights, pos, n, keep, recent, cur):
    """Slots whose keys end up in slots 0, 1, ... of one head."""
    if n <= keep:
        return np.arange(n)
    w = weights[:n].astype(np.float64)
    number = ~np.isnan(w)
    latest = pos[:n].astype(np.int64) > int(cur) - recent
    order = np.lexsort((np.arange(n), -np.where(number, w, 0.0), ~number & ~latest, ~latest))
    # among the latest the slot alone decides
    first = np.concatenate((np.flatnonzero(latest), order[latest.sum():]))[:keep]
    kept = np.zeros(n, bool)
    kept[first] = True
    src = np.arange(keep)
    src[~kept[:keep]] = np.flatnonzero(kept[keep:]) + keep
    return src


def same(a, b):
    view = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(view).cpu(), b.view(view).cpu())


def check(attn, w, lens, keep, recent, d=8, pos=None, cur=None, in_place=True, slack=0, scalars=True):
    B, H, S = w.shape
    kc, vc = normal_bf16((B, H, S, d), 1, DEV), normal_bf16((B, H, S, d), 2, DEV)
    k0, v0, w0 = kc.cpu(), vc.cpu(), w.clone()
    n = [min(max(x, 0), S) for x in lens]
    p0 = pos if pos is not None else torch.arange(S, dtype=torch.int32).expand(B, H, S).contiguous()
    c0 = cur if cur is not None else torch.tensor(n, dtype=torch.int32) - 1
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    args = dict(cache_pos=None if pos is None else pos.to(DEV), cur_pos=None if cur is None else cur.to(DEV))
    wd = w.to(DEV)
    if in_place:
        got, ws = attn.cache_evict(kc, vc, wd, seq, keep, recent, **args)
        ko, vo, wo, po = kc, vc, wd, args["cache_pos"]
        ek, ev, ew, ep = k0.clone(), v0.clone(), w0.clone(), p0.clone()
    else:
        ko, vo = normal_bf16((B, H, keep + slack, d), 3, DEV), normal_bf16((B, H, keep + slack, d), 4, DEV)
        wo = torch.full((B, H, keep + slack), -5.0, device=DEV) if scalars else None
        po = torch.full((B, H, keep + slack), -5, dtype=torch.int32, device=DEV) if scalars else None
        ek, ev = ko.cpu(), vo.cpu()
        ew, ep = (wo.cpu(), po.cpu()) if scalars else (None, None)
        out = dict(kcache=ko, vcache=vo, weights=wo, cache_pos=po)
        got, ws = attn.cache_evict(kc, vc, wd, seq, keep, recent, out=out, **args)
        assert same(kc, k0) and same(vc, v0) and same(wd, w0)
    torch.cuda.synchronize()
    assert got.tolist() == [min(x, keep) for x in n] and seq.tolist() == lens
    for b in range(B):
        for h in range(H):
            s = torch.from_numpy(sources(w0[b, h].numpy(), p0[b, h].numpy(), n[b], keep, recent, c0[b]))
            m = len(s)
            ek[b, h, :m], ev[b, h, :m] = k0[b, h, s], v0[b, h, s]
            if ew is not None:
                ew[b, h, :m], ep[b, h, :m] = w0[b, h, s], p0[b, h, s]
    assert same(ko, ek) and same(vo, ev)
    if wo is not None:
        assert same(wo, ew)
    if po is not None:
        assert same(po, ep)
    return ws


def weights_of(kind, shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(shape, generator=g)
    if kind == "few values":  # ties everywhere
        return (w * 4).floor() / 4
    if kind == "equal":
        return torch.full(shape, 0.25)
    if kind == "odd":
        w = (w - 0.5) * 1e3
        pick = torch.randint(0, 12, shape, generator=g)
        for i, x in enumerate((math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45)):
            w[pick == i] = x
        return w
    return w ** 8


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["plain", "few values", "equal", "odd"])
@pytest.mark.parametrize("S,keep,recent", [(1, 1, 0), (2, 1, 1), (70, 64, 7), (200, 3, 0), (300, 100, 100), (1000, 999, 20),
                                           (1500, 700, 64), (4000, 33, 5)])
def test_against_the_definition(attn, S, keep, recent, kind, in_place):
    lens = [S, 0, keep, min(S, keep + 1), -4, S + 3, max(1, S - 1)]
    check(attn, weights_of(kind, (len(lens), 2, S)), lens, keep, recent, in_place=in_place, slack=3)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("d", [8, 56, 64, 128, 512])
def test_head_sizes(attn, d, in_place):
    for S, keep in ((90, 60), (400, 120)):
        check(attn, weights_of("plain", (3, 3, S), d), [S, S - 9, 61], keep, 10, d=d, in_place=in_place, scalars=d != 64)


@pytest.mark.parametrize("in_place", [True, False])
def test_positions(attn, in_place):
    """Slots out of order, as earlier evictions leave them; more recent keys than are kept; current positions at the ends of the
    int32 range; every key recent, none recent."""
    g = torch.Generator().manual_seed(3)
    B, H, S, keep = 6, 2, 500, 200
    pos = torch.stack([torch.stack([torch.randperm(4 * S, generator=g)[:S] for _ in range(H)]) for _ in range(B)])
    pos = pos.to(torch.int32)
    pos[1], pos[2] = 7, -2 ** 31
    cur = torch.tensor([4 * S - 1, 7, 2 ** 31 - 1, -2 ** 31, 100, 1000], dtype=torch.int32)
    check(attn, weights_of("few values", (B, H, S), 4), [S] * B, keep, 150, pos=pos, cur=cur, in_place=in_place)


@pytest.mark.parametrize("in_place,S,keep", [(True, 50001, 49990), (True, 60000, 20000), (False, 70000, 30001),
                                             (False, 43008, 100), (True, 43009, 43000), (True, 400001, 150000),
                                             (False, 350000, 349000)])
def test_long_rows(attn, in_place, S, keep):
    """Rows whose ranks fit in shared memory just so, and rows that do not."""
    check(attn, weights_of("plain", (1, 2, S)), [S], keep, 100, in_place=in_place)
    check(attn, weights_of("few values", (2, 1, S)), [S - 1, keep + 5], keep, 0, in_place=in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["plain", "few values", "equal", "odd"])
@pytest.mark.parametrize("B,H,S,keep", [(1, 2, 20001, 7000), (3, 8, 9000, 8000), (5, 9, 5000, 33), (1, 1, 17000, 16990)])
def test_rows_shared_by_several_ctas(attn, B, H, S, keep, kind, in_place):
    """Few long rows: a cluster of CTAs a row, one of whose ranges holds the last kept slot; lengths that leave
    some of them without a key."""
    lens = [S, keep + 1, S - 1, 40, (S + keep) // 2][:B]
    check(attn, weights_of(kind, (B, H, S), 7), lens, keep, 12, in_place=in_place, slack=1)


@pytest.mark.parametrize("kind", ["plain", "few values", "equal", "odd"])
@pytest.mark.parametrize("B,H,S,past", [(3, 2, 16384, 1), (2, 8, 9001, 4), (5, 1, 20000, 5), (4, 2, 33000, 64), (1, 1, 60001, 33),
                                        (2, 2, 180000, 3), (1, 2, 400000, 64)])
def test_few_keys_of_long_rows_go(attn, B, H, S, past, kind):
    """A bounded cache with few long rows, in place: the CTAs of a row select and move together.  From none to all of the
    keys past the bound go; the lengths leave some of the CTAs without one."""
    keep = S - past
    lens = [S, keep + min(past, 2), keep, S - past // 2, 50][:B]
    check(attn, weights_of(kind, (B, H, S), 11), lens, keep, 9, in_place=True)
    g = torch.Generator().manual_seed(12)
    pos = torch.stack([torch.randperm(2 * S, generator=g)[:S].to(torch.int32) for _ in range(B * H)]).view(B, H, S)
    check(attn, weights_of("few values", (B, H, S), 13), lens, keep, S // 2, pos=pos, cur=torch.full((B,), 2 * S, dtype=torch.int32))


def timed(attn, B, H, S, keep, n, d=64):
    """Milliseconds of 20 evictions in place of n - keep keys of every row (the weights decide, so each moves as many)."""
    kc, vc = normal_bf16((B, H, S, d), 70, DEV), normal_bf16((B, H, S, d), 71, DEV)
    w = weights_of("plain", (B, H, S), 14).to(DEV)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out, ws = attn.cache_evict(kc, vc, w, lens, keep, 8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(20):
            attn.cache_evict(kc, vc, w, lens, keep, 8, seqlens_out=out, workspace=ws)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(6)]
    ends[0].record()
    for e in ends[1:]:
        g.replay()
        e.record()
    torch.cuda.synchronize()
    return min(a.elapsed_time(b) for a, b in zip(ends, ends[1:]))


@pytest.mark.parametrize("fits,more", [(15, 16), (15, 19), (34, 38)])
def test_one_row_more_does_not_wait_for_the_others(attn, fits, more):
    """Clusters that do not all have SMs at once took a second wave: 16 rows of 64K keys 1.8 times as long as 15."""
    S = 1 << 16
    assert timed(attn, more, 1, S, S - 65, S) <= 1.4 * timed(attn, fits, 1, S, S - 65, S)


def test_few_keys_of_long_rows_take_no_longer_than_many(attn):
    """16 of 131072 keys of 8 rows go where the cache has 64 slots past the bound (one launch): with one CTA a row that
    took 6 times as long as with 65 slots, where a cluster selects and a second launch moves."""
    B, H, S, d = 1, 8, 1 << 17, 64
    kc, vc = normal_bf16((B, H, S, d), 70, DEV), normal_bf16((B, H, S, d), 71, DEV)
    w = weights_of("plain", (B, H, S), 14).to(DEV)
    us = []
    for past in (64, 65):
        lens = torch.full((B,), S - past + 16, dtype=torch.int32, device=DEV)
        out, ws = attn.cache_evict(kc, vc, w, lens, S - past, 8)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                attn.cache_evict(kc, vc, w, lens, S - past, 8, seqlens_out=out, workspace=ws)
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(6)]
        ends[0].record()
        for e in ends[1:]:
            g.replay()
            e.record()
        torch.cuda.synchronize()
        us.append(min(a.elapsed_time(b) for a, b in zip(ends, ends[1:])))
    assert us[0] <= 2 * us[1], us


def test_captured_loop_with_appends(attn):
    """A captured decode step on a bounded cache (append, evict), replayed: the lengths go round in device memory, positions
    advance, and every replay equals the eager step."""
    B, Hq, H, d, keep, S = 3, 4, 2, 64, 40, 44
    kc, vc = normal_bf16((B, H, S, d), 20, DEV), normal_bf16((B, H, S, d), 21, DEV)
    w = weights_of("plain", (B, H, S), 5).to(DEV)
    pos = torch.arange(S, dtype=torch.int32, device=DEV).expand(B, H, S).contiguous()
    lens = torch.tensor([40, 38, 10], dtype=torch.int32, device=DEV)
    lens2, cur = torch.empty_like(lens), lens - 1
    q, k, v = (normal_bf16((B, h, 1, d), 22 + h, DEV) for h in (Hq, H, H))
    f = attn.rope_freqs(d)
    state = [kc, vc, w, pos, lens, lens2, cur]

    def step(kc, vc, w, pos, lens, lens2, cur):
        cur += 1
        attn.rope_append(q, k, v, kc, vc, lens, f, start_pos=cur, cache_pos=pos, weights=w, seqlens_out=lens2)
        attn.cache_evict(kc, vc, w, lens2, keep, 5, cache_pos=pos, cur_pos=cur, seqlens_out=lens)

    step(*[t.clone() for t in state])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*state)
    eager = [t.clone() for t in state]
    for i in range(6):
        k.copy_(normal_bf16(k.shape, 30 + i, DEV))
        v.copy_(normal_bf16(v.shape, 40 + i, DEV))
        g.replay()
        step(*eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state, eager))
    assert lens.tolist() == [40, 40, 16] and cur.tolist() == [45, 43, 15]


def test_two_streams_and_equal_calls(attn):
    B, H, S, d, keep = 4, 2, 2000, 128, 500
    w = weights_of("few values", (B, H, S), 6).to(DEV)
    kc, vc = normal_bf16((B, H, S, d), 50, DEV), normal_bf16((B, H, S, d), 51, DEV)
    seq = torch.tensor([S, 600, 500, 1999], dtype=torch.int32, device=DEV)
    runs = []
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    copies = [(kc.clone(), vc.clone(), w.clone()) for _ in streams]
    torch.cuda.synchronize()
    for s, c in zip(streams, copies):
        runs.append(attn.cache_evict(*c, seq, keep, 50, stream=s)[0])
    torch.cuda.synchronize()
    for r, c in zip(runs[1:], copies[1:]):
        assert torch.equal(r, runs[0]) and all(torch.equal(a, b) for a, b in zip(c, copies[0]))


def test_caches_past_two_to_the_31_elements(attn):
    B, H, S, d, keep = 2, 3, 1 << 21, 256, 1000
    kc = torch.zeros((B, H, S, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    mark = normal_bf16((2, 400, d), 60, DEV)
    kc[1, 2, S - 400:], vc[1, 2, S - 400:] = mark[0], mark[1]
    w = torch.zeros((B, H, S), device=DEV)
    w[1, 2, S - 400: S - 300] = 2.0
    seq = torch.tensor([5, S], dtype=torch.int32, device=DEV)
    n, _ = attn.cache_evict(kc, vc, w, seq, keep, 100)
    assert n.tolist() == [5, keep]
    # 100 heavy keys and the 100 latest; among the rest (weight 0) the lowest slots stay
    at = list(range(keep - 200, keep))
    src = list(range(100)) + list(range(300, 400))
    assert torch.equal(kc[1, 2, at], mark[0][src]) and torch.equal(vc[1, 2, at], mark[1][src])
    assert not kc[1, 2, :keep - 200].any() and not kc[0].any()
    assert w[1, 2, keep - 200: keep - 100].eq(2).all() and not w[1, 2, keep - 100: keep].any()
    del kc, vc, w
    torch.cuda.empty_cache()


def test_helper_refusals(attn):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=DEV)
    kc, vc, w, n = z(2, 2, 300, 64), z(2, 2, 300, 64), z(2, 2, 300, dtype=torch.float32), z(2, dtype=torch.int32)
    o = dict(kcache=z(2, 2, 60, 64), vcache=z(2, 2, 60, 64))
    small = z(16)
    for call, code in [
        (lambda: attn.cache_evict(kc, vc, w.double(), n, 50), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc[:, :, :200], w, n, 50), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n.cpu(), 50), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 50, seqlens_out=n), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 0), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 301), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 50, 51), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 61, out=o), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 50, out=dict(o, vcache=o["kcache"])), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 50, out=dict(o, vcache=vc[:1, :, :120].reshape(2, 2, 60, 64))), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 50, out=dict(kcache=kc, vcache=o["vcache"])), attn.ATTN_ERR_ARG),
        (lambda: attn.cache_evict(kc, vc, w, n, 50, workspace=small), attn.ATTN_ERR_WORKSPACE),
    ]:
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == code
