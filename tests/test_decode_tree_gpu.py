"""Attention of drafted tokens over a cache, in pages or contiguous, against the
definition in 64 bits on the same bf16 inputs.

Tolerances, per element, as in test_decode_prefix_gpu.py: scores are fp32 sums of
d exact products, off by at most e = d 2^-24 scale sum_i |q_i k_i| (taken at its
largest over the row's keys); exp2, the logarithms and the merge add a few units of
2^-22 (|L| + 1), E = e + 2^-20 (|L| + 1) in all.  Then
    lse    E
    o      probabilities are rounded to bf16 for the product with V (half a
           step, 2^-8 of each), the result once more (2^-8 of it):
           (2^-8 + 2 E) sum_j p_j |v_j| + 2^-8 |o|."""
import math

import pytest
import torch

from synthetic_inputs import normal_bf16
from tests.test_tree_gpu import ancestors, bits_of, random_tree

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


def a_cache(B, Hkv, S, d, page, seed, spare=3):
    """(k, v, table): contiguous caches of S slots, or pages in any order for S slots rounded up."""
    if page == 0:
        shape, table = (B, Hkv, S, d), None
    else:
        per = -(-S // page)
        n = B * per + spare
        table = torch.randperm(n, generator=torch.Generator().manual_seed(seed))[: B * per].view(B, per).to(torch.int32)
        shape = (n, Hkv, page, d)
    return normal_bf16(shape, seed + 1, DEV), normal_bf16(shape, seed + 2, DEV), table


def rows_of(x, table, page, b):
    """Sequence b's rows [Hkv, slots, d], and which of them lie on a page."""
    if table is None:
        return x[b], torch.ones(x.shape[2], dtype=torch.bool, device=x.device)
    e = table[b].to(x.device).long()
    ok = (e >= 0) & (e < x.shape[0])
    return x[e.clamp(0, x.shape[0] - 1)].transpose(0, 1).flatten(1, 2), ok.repeat_interleave(page)


def reference(q, k, v, table, page, lens, sees, live, scale):
    """sees[b]: a set of drafted tokens for each token.  (o, lse, tolerances of both), on the GPU in 64 bits."""
    B, Hq, T, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    o, to = (torch.zeros(B, Hq, T, d, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
    tl = torch.zeros(B, Hq, T, dtype=torch.float64, device=DEV)
    for b in range(B):
        kb, ok = rows_of(k, table, page, b)
        vb, _ = rows_of(v, table, page, b)
        cap = kb.shape[1]
        n = min(max(lens[b], 0), cap)
        for t in range(min(max(live[b], 0), T)):
            at = [j for j in [n + u for u in sorted(sees[b][t]) if u < live[b]] if j < cap]
            idx = torch.cat((torch.arange(n, device=DEV), torch.tensor(at, dtype=torch.long, device=DEV)))
            idx = idx[ok[idx]]
            if idx.numel() == 0:
                continue
            for g in range(Hkv):
                rows = slice(g * G, (g + 1) * G)
                kk, vv, qq = kb[g, idx].double(), vb[g, idx].double(), q[b, rows, t].double()
                s = qq @ kk.T * scale
                L = torch.logsumexp(s, -1)
                p = torch.exp(s - L[:, None])
                E = (qq.abs() @ kk.T.abs()).amax(-1) * scale * d * 2.0 ** -24 + 2.0 ** -20 * (L.abs() + 1)
                o[b, rows, t], lse[b, rows, t], tl[b, rows, t] = p @ vv, L, E
                to[b, rows, t] = (STEP + 2 * E)[:, None] * (p @ vv.abs()) + STEP * o[b, rows, t].abs()
    return o, lse, to, tl


def run_and_check(attn, q, k, v, table, page, lens, parents=None, live=None, scale=None, sees=None, workspace=None):
    B, Hq, T, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    n_live = [T] * B if live is None else live
    mask = None
    if sees is not None:
        mask = torch.stack([bits_of(s, T) for s in sees]).to(DEV)
    elif parents is not None:
        sees = [ancestors(p, T) for p in parents.tolist()]
        mask, _ = attn.tree_mask(parents.to(DEV))
    else:
        sees = [[set(range(t + 1)) for t in range(T)]] * B
    i32 = dict(dtype=torch.int32, device=DEV)
    o, lse, ws = attn.decode_tree(q, k, v, torch.tensor(lens, **i32), mask, None if live is None else torch.tensor(live, **i32),
                                  None if table is None else table.to(DEV), scale=scale, workspace=workspace)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_OK
    ro, rl, to, tl = reference(q, k, v, table, page, lens, sees, n_live, scale)
    none = torch.isinf(rl)
    assert torch.equal(none, torch.isinf(lse)) and torch.all(lse[none] < 0) and torch.all(o[none] == 0)
    err = (o.double() - ro).abs()
    assert torch.all(err <= to), f"o off by {float((err / to.clamp(min=1e-300)).max()):.3g} of the bound"
    assert torch.all((lse.double() - rl)[~none].abs() <= tl[~none])
    return o, lse, ws


def some_lens(B, cap, T):
    edge = [cap - T, 0, 1, cap + 7, -2, cap // 2, 127, cap - 1]
    return [max(-2, x) for x in (edge + torch.randint(0, cap + 1, (max(B, 1),), generator=torch.Generator().manual_seed(B)).tolist())[:B]]


SHAPES = [
    # B, Hq, Hkv, T, S, d, page
    (1, 1, 1, 1, 1, 64, 0), (1, 8, 2, 5, 500, 64, 0), (2, 8, 1, 1, 130, 128, 0), (3, 6, 2, 7, 257, 128, 16),
    (8, 4, 4, 3, 300, 64, 32), (5, 10, 2, 33, 900, 128, 64), (4, 16, 1, 8, 640, 64, 128), (2, 32, 2, 9, 700, 128, 256),
    (9, 16, 2, 16, 1000, 128, 16), (2, 8, 1, 64, 1500, 128, 64), (1, 16, 1, 100, 400, 64, 16), (2, 16, 1, 256, 700, 128, 32),
    (3, 3, 3, 129, 500, 64, 64), (1, 5, 1, 26, 20000, 128, 64), (40, 8, 8, 2, 200, 64, 16), (1, 2, 2, 256, 256, 128, 0),
    (2, 11, 1, 65, 3000, 64, 1024),
]


@pytest.mark.parametrize("B,Hq,Hkv,T,S,d,page", SHAPES)
def test_trees(attn, B, Hq, Hkv, T, S, d, page):
    k, v, table = a_cache(B, Hkv, S, d, page, 100)
    cap = S if page == 0 else table.shape[1] * page
    q = (normal_bf16((B, Hq, T, d), 99).float() * 2).bfloat16().to(DEV)
    live = [T, T, max(1, T // 2), 0, T + 5, -1, 1][:B] + [T] * max(0, B - 7)
    run_and_check(attn, q, k, v, table, page, some_lens(B, cap, T), parents=random_tree(B, T, S), live=live)


@pytest.mark.parametrize("B,Hq,Hkv,T,S,d,page", [s for s in SHAPES if s[3] <= 64])
def test_chains(attn, B, Hq, Hkv, T, S, d, page):
    k, v, table = a_cache(B, Hkv, S, d, page, 200)
    cap = S if page == 0 else table.shape[1] * page
    q = normal_bf16((B, Hq, T, d), 199, DEV)
    run_and_check(attn, q, k, v, table, page, some_lens(B, cap, T))


@pytest.mark.parametrize("offset", list(range(0, 140, 9)) + [120, 127, 128])
def test_where_the_draft_begins(attn, offset):
    """Drafted keys at every place of a block, over the end of one and of a page."""
    T, page = 37, 16
    k, v, table = a_cache(2, 1, 320, 64, page, 300 + offset)
    q = normal_bf16((2, 8, T, 64), 301, DEV)
    run_and_check(attn, q, k, v, table, page, [offset, 140 - offset], parents=random_tree(2, T, offset, offset % 2 == 0))


def test_any_pattern(attn):
    """Masks that are no trees: tokens that attend nothing, not even themselves, or later ones; bits past the drafted
    tokens; and no cached keys at all."""
    B, T = 3, 70
    g = torch.Generator().manual_seed(4)
    sees = [[set(torch.nonzero(torch.rand(128, generator=g) < 0.2).flatten().tolist()) & set(range(T)) for _ in range(T)] for _ in range(B)]
    sees[1][5] = set()
    sees[0][0] = {T - 1}
    for d, Hq in ((64, 4), (128, 1)):
        k, v, table = a_cache(B, 1, 160, d, 16, 400)
        q = normal_bf16((B, Hq, T, d), 401, DEV)
        run_and_check(attn, q, k, v, table, 16, [0, 0, 77], sees=sees, live=[T, 40, 69])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 512])
@pytest.mark.parametrize("Hq,T", [(8, 4), (8, 40)])
def test_holes(attn, page, Hq, T):
    """Entries that are no page: their keys do not exist, drafted ones among them; whole blocks and sequences without a key."""
    B, S, d = 4, 1024, 64
    k, v, table = a_cache(B, 2, S, d, page, 500)
    g = torch.Generator().manual_seed(page)
    gone = torch.rand(table.shape, generator=g) < 0.4
    gone[1] = True
    gone[2, : max(1, 300 // page)] = True
    table = torch.where(gone, torch.tensor([-1, 10 ** 9, k.shape[0], -2 ** 31])[torch.randint(0, 4, table.shape, generator=g)].int(), table)
    q = normal_bf16((B, Hq, T, d), 501, DEV)
    run_and_check(attn, q, k, v, table, page, [900, 500, 700, 0], parents=random_tree(B, T, 1))


@pytest.mark.parametrize("Hq,T,d", [(8, 6, 128), (8, 40, 64)])
def test_peaked_and_huge_scores(attn, Hq, T, d):
    k, v, table = a_cache(2, 1, 600, d, 64, 600)
    q = (normal_bf16((2, Hq, T, d), 601).float() * 30).bfloat16().to(DEV)
    k[:, :, ::37] *= 8
    run_and_check(attn, q, k, v, table, 64, [500, 333], parents=random_tree(2, T, 2))


@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("Hq,T,d", [(8, 6, 128), (16, 40, 64)])
def test_what_no_token_attends_does_not_matter(attn, Hq, T, d, page):
    """NaN and infinities behind the last key, in pages that nobody uses, in drafted rows past draft_lens, and in drafted
    rows for the tokens that do not attend them."""
    B, S = 3, 600
    lens, live = [301, 0, 130], [T, T - 2, 3]
    k, v, table = a_cache(B, 2, S, d, page, 700)
    q = normal_bf16((B, Hq, T, d), 701, DEV)
    parents = random_tree(B, T, 3)
    want = run_and_check(attn, q, k, v, table, page, lens, parents=parents, live=live)[:2]
    cap = S if page == 0 else table.shape[1] * page
    for b in range(B):
        for r in range(lens[b] + live[b], cap):
            e, i = (b, r) if table is None else (int(table[b, r // page]), r % page)
            k[e, :, i] = float("nan")
            v[e, :, i] = float("inf") if r % 2 else float("nan")
    if table is not None:
        unused = sorted(set(range(k.shape[0])) - set(table.flatten().tolist()))
        k[unused], v[unused] = float("nan"), float("nan")
    got = run_and_check(attn, q, k, v, table, page, lens, parents=parents, live=live)[:2]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # one drafted row of sequence 0 and one of sequence 2
    sees = [ancestors(p, T) for p in parents.tolist()]
    touched = torch.zeros((B, T), dtype=torch.bool)
    for b, u, bad in ((0, 1, float("inf")), (0, T - 1, float("nan")), (2, 0, -float("inf"))):
        e, i = (b, lens[b] + u) if table is None else (int(table[b, (lens[b] + u) // page]), (lens[b] + u) % page)
        v[e, :, i, 3] = bad
        if u == T - 1:
            k[e, :, i, 0] = float("nan")
        touched[b] |= torch.tensor([u in sees[b][t] and t < live[b] for t in range(T)])
    i32 = dict(dtype=torch.int32, device=DEV)
    mask, _ = attn.tree_mask(parents.to(DEV))
    o, lse, _ = attn.decode_tree(q, k, v, torch.tensor(lens, **i32), mask, torch.tensor(live, **i32),
                                 None if table is None else table.to(DEV))
    torch.cuda.synchronize()
    hit = touched[:, None].expand(B, Hq, T).to(DEV)
    assert torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    assert not torch.isfinite(o[hit][:, 3]).any()
    only_v = hit.clone()
    only_v[0, :, T - 1] = False  # (its K is NaN too)
    keep = [c for c in range(d) if c != 3]
    # the zeroed element changes no sum but its own column's
    assert torch.equal(o[only_v][:, keep], want[0][only_v][:, keep]) and torch.equal(lse[only_v], want[1][only_v])
    assert torch.all(o[2][hit[2]][:, 3] == -float("inf"))


def test_scores_of_minus_infinity(attn):
    """Keys whose score is -inf count for nothing; tokens that attend only such keys get zeros."""
    B, T, d, S = 2, 5, 64, 200
    k, v, table = a_cache(B, 1, S, d, 16, 800)
    q = torch.ones((B, 4, T, d), dtype=torch.bfloat16, device=DEV)
    k[...] = -float("inf")
    o, lse, _ = attn.decode_tree(q, k, v, torch.tensor([100, 0], dtype=torch.int32, device=DEV), None, None, table.to(DEV))
    torch.cuda.synchronize()
    assert torch.all(o == 0) and torch.all(lse == -float("inf"))
    e = int(table[0, 2])
    k[e, :, 7] = 0.5
    o, lse, _ = attn.decode_tree(q, k, v, torch.tensor([100, 0], dtype=torch.int32, device=DEV), None, None, table.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(o[0], v[e, 0, 7].expand(4, T, d)) and torch.all((lse[0] - 0.5 * d * d ** -0.5).abs() < 1e-5)
    assert torch.all(o[1] == 0)


def test_agrees_with_decode(attn):
    """One token per sequence, the step behind attn_decode: draft_lens 1, the token's key already cached."""
    B, Hq, Hkv, d, S = 6, 16, 4, 128, 2000
    k, v, _ = a_cache(B, Hkv, S, d, 0, 900)
    q = normal_bf16((B, Hq, 1, d), 901, DEV)
    n = torch.tensor([2000, 1, 700, 64, 1999, 130], dtype=torch.int32, device=DEV)
    o, _, _ = attn.decode_tree(q, k, v, n - 1)
    ref, _, _ = attn.decode(q[:, :, 0].contiguous(), k, v, n)
    # both are within the tolerance of the definition; apart by at most twice it
    _, _, to, _ = reference(q, k, v, None, 0, (n - 1).tolist(), [[{0}]] * B, [1] * B, d ** -0.5)
    assert torch.all((o - ref[:, :, None]).double().abs() <= 2 * to)


@pytest.mark.parametrize("Hq,T", [(8, 4), (8, 40), (16, 200)])
def test_equal_calls_give_equal_bits_and_graphs_share_a_workspace(attn, Hq, T):
    B, d, page, S = 5, 128, 32, 1500
    k, v, table = a_cache(B, 1, S, d, page, 1000)
    q1, q2 = normal_bf16((B, Hq, T, d), 1001, DEV), normal_bf16((B, Hq, T, d), 1002, DEV)
    lens = torch.tensor([1200, 3, 800, 0, 555], dtype=torch.int32, device=DEV)
    mask, _ = attn.tree_mask(random_tree(B, T, 5).to(DEV))
    t = table.to(DEV)
    w1 = attn.decode_tree(q1, k, v, lens, mask, page_table=t)
    w2 = attn.decode_tree(q2, k, v, lens, mask, page_table=t)
    ws, n = w1[2], torch.zeros_like(lens)
    graphs, outs = [], []
    for q in (q1, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attn.decode_tree(q, k, v, n, mask, page_table=t, workspace=ws)[:2])
        graphs.append(g)
    n.copy_(lens)  # a replay takes the lengths as they are then
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for out, want in zip(outs, (w1, w2)):
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_streams_at_once(attn):
    B, Hq, Hkv, T, d, page, S = 4, 16, 2, 9, 128, 64, 3000
    k, v, table = a_cache(B, Hkv, S, d, page, 1100)
    t = table.to(DEV)
    lens = torch.tensor([2900, 100, 2000, 1], dtype=torch.int32, device=DEV)
    qs = [normal_bf16((B, Hq, T, d), 1101 + i, DEV) for i in range(2)]
    want = [attn.decode_tree(q, k, v, lens, page_table=t)[:2] for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            got[i] = attn.decode_tree(qs[i], k, v, lens, page_table=t, stream=s)[:2]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_pages_past_two_to_the_31_elements(attn):
    """A pool of more than 2^31 elements, the sequence's pages at its end."""
    Hkv, page, d, T = 8, 256, 128, 3
    n = (1 << 31) // (Hkv * page * d) + 20
    k = torch.zeros((n, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    table = torch.arange(n - 1, n - 5, -1, dtype=torch.int32)[None]
    k[n - 8:], v[n - 8:] = normal_bf16((8, Hkv, page, d), 1200, DEV), normal_bf16((8, Hkv, page, d), 1201, DEV)
    q = normal_bf16((1, 16, T, d), 1202, DEV)
    run_and_check(attn, q, k, v, table, page, [900])


@pytest.mark.parametrize("Hq,T", [(8, 4), (8, 40)])
def test_a_launch_that_gave_up_stays_in_bounds(attn, Hq, T):
    """With no time to wait the kernel leaves early and says so; the next call is right."""
    B, d, page, S = 3, 128, 16, 1500
    k, v, table = a_cache(B, 2, S, d, page, 1300)
    q = normal_bf16((B, Hq, T, d), 1301, DEV)
    lens = [1400, 2, 700]
    ws = torch.full((attn.attn_decode_tree_workspace_bytes(B, Hq, 2, T, d, page, table.shape[1]),), 0x7f, dtype=torch.uint8, device=DEV)
    old = attn.attn_set_wait_timeout_ns(0)
    try:
        attn.decode_tree(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV), page_table=table.to(DEV), workspace=ws)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_TIMEOUT
    finally:
        attn.attn_set_wait_timeout_ns(old)
    run_and_check(attn, q, k, v, table, page, lens, workspace=ws)


def test_helper_refusals(attn):
    k, v, table = a_cache(2, 2, 64, 64, 16, 1400)
    q, n, t = normal_bf16((2, 4, 3, 64), 1401, DEV), torch.zeros(2, dtype=torch.int32, device=DEV), table.to(DEV)
    mask = torch.zeros((2, 3, 1), dtype=torch.int64, device=DEV)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :, ::2]), dict(q=q.transpose(1, 2)), dict(seqlens=n.long()), dict(seqlens=n[:1]),
                dict(mask=mask.int()), dict(mask=mask[:, :2]), dict(draft_lens=n.cpu()), dict(page_table=t[:1]),
                dict(page_table=None), dict(kcache=k[:, :1]), dict(vcache=None), dict(kcache=k.cpu()),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        a = dict(q=q, kcache=k, vcache=v, seqlens=n, mask=mask, draft_lens=None, page_table=t)
        a.update(bad)
        with pytest.raises(attn.AttnError):
            attn.decode_tree(**a)


@pytest.mark.parametrize("Hq,T,d", [(8, 6, 128), (8, 6, 64), (8, 40, 128), (8, 40, 64)])
def test_rising_scores_and_large_values(attn, Hq, T, d):
    """Every block's scores are above those of all before it, by up to 300 in all, and values are near 2^90: a reference
    that is kept too long makes sums that 32 bits do not hold, although the result is no larger than the values."""
    S = 900
    k, v, _ = a_cache(2, 1, S, d, 0, 700)
    base = normal_bf16((d,), 703, DEV).float()
    rise = torch.arange(S, device=DEV).float() / S * 300 * d ** 0.5 / (base @ base)
    k = (rise[None, None, :, None] * base + 0.1 * k.float()).bfloat16()
    v = (v.float() * 2.0 ** 90).bfloat16()
    q = (base + 0.1 * normal_bf16((2, Hq, T, d), 704, DEV).float()).bfloat16()
    o, _, _ = run_and_check(attn, q, k, v, None, 0, [800, 450], parents=random_tree(2, T, 3))
    assert torch.all(torch.isfinite(o))
