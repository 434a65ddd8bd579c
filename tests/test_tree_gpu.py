"""Trees of drafted tokens on the GPU: attn_tree_mask and attn_tree_accept
against their definitions.  Nothing is rounded, so everything is equal bit for bit."""
import pytest
import torch

from synthetic_inputs import normal_bf16
from tests.test_rope_axes_gpu import a_table, row_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


def random_tree(B, T, seed, deep=False):
    """Parents anywhere before the node (the node before it where deep), some roots."""
    g = torch.Generator().manual_seed(seed)
    r = torch.rand((B, T), generator=g)
    t = torch.arange(T)
    p = torch.where(r < 0.05, torch.tensor(-1), ((t - 1) if deep else (r * 0.999 * t).floor().long()).expand(B, T))
    return p.to(torch.int32)


def ancestors(parents, live):
    """Sets of nodes that each node sees (one sequence, lists)."""
    seen = []
    for t, p in enumerate(parents[:live]):
        seen.append({t} | (seen[p] if 0 <= p < t else set()))
    return seen + [set()] * (len(parents) - live)


def bits_of(sets, T):
    words = (T + 63) // 64
    out = torch.zeros((len(sets), words), dtype=torch.int64)
    for t, s in enumerate(sets):
        for u in s:
            v = 1 << (u % 64)
            out[t, u // 64] |= v - (1 << 64) if u % 64 == 63 else v
    return out


@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("T", [1, 2, 5, 31, 33, 64, 65, 130, 256])
def test_mask(attn, T, deep):
    B = 4
    parents = random_tree(B, T, T, deep)
    parents[0, 0] = 7                       # not before the node: a root
    if T > 4:
        parents[1, 3], parents[1, 2] = 3, -9
    lens = torch.tensor([0, 5, 100000, 2 ** 31 - 1], dtype=torch.int32)
    live = torch.tensor([T, T + 3, T // 2, -1], dtype=torch.int32)
    for cut in (None, live):
        mask, pos = attn.tree_mask(parents.to(DEV), lens.to(DEV), None if cut is None else cut.to(DEV))
        for b in range(B):
            n = T if cut is None else min(max(int(cut[b]), 0), T)
            sets = ancestors(parents[b].tolist(), n)
            assert torch.equal(mask[b].cpu(), bits_of(sets, T))
            want = [int(lens[b]) + max(len(s) - 1, 0) for s in sets]
            assert pos[b].tolist() == [(w + 2 ** 31) % 2 ** 32 - 2 ** 31 for w in want]
    mask2, none = attn.tree_mask(parents.to(DEV), with_positions=False)
    assert none is None and torch.equal(mask2, attn.tree_mask(parents.to(DEV), lens.to(DEV))[0])
    assert torch.equal(attn.tree_mask(parents.to(DEV))[1].cpu(), torch.tensor(
        [[len(s) - 1 for s in ancestors(p, T)] for p in parents.tolist()], dtype=torch.int32))


@pytest.mark.parametrize("layers", [0, 3])
@pytest.mark.parametrize("page", [0, 16, 32])
@pytest.mark.parametrize("T,Hkv,d", [(1, 2, 64), (7, 3, 64), (64, 2, 128), (100, 1, 8), (256, 2, 56), (20, 33, 128)])
def test_accept(attn, T, Hkv, d, page, layers):
    B, S = 6, 352
    per = 1 if page == 0 else S // page
    cap = S
    n = B if page == 0 else 2 * B * per
    table = None if page == 0 else a_table(B, per, n, 40)
    shape = (n, Hkv, S if page == 0 else page, d)
    lead = (layers,) if layers else ()
    kc, vc = normal_bf16(lead + shape, 41, DEV), normal_bf16(lead + shape, 42, DEV)
    parents = random_tree(B, T, 43 + T)
    sets = [ancestors(p, T) for p in parents.tolist()]
    mask, _ = attn.tree_mask(parents.to(DEV))
    if T % 64:
        mask[..., -1] |= -1 << (T % 64)  # bits past the last node count as 0
    lens = torch.tensor([0, 17, cap - 2, 30, 50, -3], dtype=torch.int32)
    last = torch.tensor([T - 1, T // 2, T - 1, -1, T, max(T - 2, 0)], dtype=torch.int32)
    if table is not None:
        table[1, min((17 + T - 1) // page, per - 1)] = -1
        table[5, 0] = n  # its first rows lie on no page
    want = [kc.cpu().clone(), vc.cpu().clone()]
    out_len = []
    for b in range(B):
        i = int(last[b])
        path = sorted(sets[b][i]) if 0 <= i < T else []
        n0 = max(int(lens[b]), 0)
        out_len.append(min(cap, n0 + len(path)))
        for w in want:
            for layer in (w if layers else [w]):
                rows = {}
                for r, u in enumerate(path):
                    if n0 + u < cap and all(page == 0 or 0 <= int(table[b, (n0 + x) // page]) < n for x in (u, r)):
                        rows[r] = row_of(layer, table, page, b, n0 + u).clone()
                for r, x in rows.items():
                    row_of(layer, table, page, b, n0 + r).copy_(x)
    got = attn.tree_accept(kc, vc, lens.to(DEV), mask, last.to(DEV), page_table=None if table is None else table.to(DEV))
    assert got.tolist() == out_len
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])
    # a chain's rows are in their places
    got = attn.tree_accept(kc, vc, lens.to(DEV), None, last.to(DEV), page_table=None if table is None else table.to(DEV))
    assert got.tolist() == [min(cap, max(int(a), 0) + (int(i) + 1 if 0 <= i < 256 else 0)) for a, i in zip(lens, last)]
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])
