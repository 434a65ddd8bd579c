"""The paged cache's operators together, as a serving loop with drafted tokens uses them: a prompt in chunks, samples that
fork it, then steps of room for the drafts, masks and positions of the drafted trees, their keys into the pages, attention,
acceptance and freed pages, with a compaction between; every stage against its definition, the attention against the whole
history of each sequence as it was put in, wherever its rows lie."""
import pytest
import torch

from synthetic_inputs import normal_bf16
from tests.test_decode_tree_gpu import reference, run_and_check
from tests.test_rope_axes_gpu import check, turned
from tests.test_rope_gpu import FP32, STEP, freqs
from tests.test_tree_gpu import ancestors, random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


@pytest.mark.parametrize("d,Hq,Hkv,page,T", [(64, 8, 2, 16, 5), (128, 16, 2, 32, 20)])
def test_drafted_decoding_over_shared_pages(attn, d, Hq, Hkv, page, T):
    B, per, layers = 4, 14, 2
    pages = B * per + 9
    i32 = dict(dtype=torch.int32, device=DEV)
    kp, vp = (torch.full((layers, pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table, refs = torch.full((B, per), -1, **i32), torch.zeros(pages, **i32)
    lens = torch.zeros(B, **i32)
    f = attn.rope_freqs(d, rule="linear", factor=2.0)
    ws = attn.pages_extend(table, refs, lens, 0, kp, vp)[1]
    history = [[] for _ in range(B)]  # of each sequence: (k, v) [layers, Hkv, d] of every key, as the cache holds them

    def tokens(seed, n):
        qkv = [normal_bf16((B, n, Hq + 2 * Hkv, d), seed + i, DEV).transpose(1, 2) for i in range(layers)]
        return [x.split([Hq, Hkv, Hkv], dim=1) for x in qkv]

    def row(x, b, r):
        return x[:, int(table[b, r // page]), :, r % page]

    def same_as_history():
        for b in range(B):
            for r, (k, v) in enumerate(history[b]):
                assert torch.equal(row(kp, b, r), k) and torch.equal(row(vp, b, r), v), (b, r)
        assert lens.tolist() == [len(h) for h in history]

    def append(qkv, pos, new):
        """Every layer's tokens behind the sequences' last; rotated keys checked, the rows kept as history's candidates."""
        out = []
        for l, (q, k, v) in enumerate(qkv):
            qr, n = attn.rope_axes_append(q, k, v, kp[l], vp[l], lens, f, None, pos, page_table=table, new_lens=new)
            check(qr, q, pos[None].cpu(), f.cpu(), [0] * (d // 2), False)
            out.append(qr)
        added = [q.shape[2]] * B if new is None else new.tolist()
        for b in range(B):
            for l, (q, k, v) in enumerate(qkv):
                want, size = turned(k, pos[None].cpu(), f.cpu(), [0] * (d // 2), False)
                for t in range(added[b]):
                    r = int(lens[b]) + t
                    got = kp[l, int(table[b, r // page]), :, r % page].double().cpu()
                    assert torch.all((got - want[b, :, t]).abs() <= STEP * want[b, :, t].abs() + FP32 * size[b, :, t])
                    assert torch.equal(vp[l, int(table[b, r // page]), :, r % page], v[b, :, t])
        return out, n

    # a prompt for sequence 0, in two chunks of a padded batch
    for chunk, n0 in ((0, 37), (1, 22)):
        new = torch.tensor([n0, 0, 0, 0], **i32)
        info, _ = attn.pages_extend(table, refs, lens, new, kp, vp, workspace=ws)
        assert info.tolist()[1] == 0
        qkv = tokens(10 + 10 * chunk, n0)
        pos = (lens[:, None] + torch.arange(n0, device=DEV, dtype=torch.int32)).contiguous()
        _, n = append(qkv, pos, new)
        history[0] += [(row(kp, 0, int(lens[0]) + t).clone(), row(vp, 0, int(lens[0]) + t).clone()) for t in range(n0)]
        lens = n
    same_as_history()

    # three samples go on from it; the last page is partly filled and shared until somebody writes
    table, lens = attn.pages_fork(table, refs, lens, torch.zeros(B, **i32), page)
    history = [list(history[0]) for _ in range(B)]
    same_as_history()
    assert int(refs.max()) == B

    for step in range(6):
        info, _ = attn.pages_extend(table, refs, lens, T, kp, vp, workspace=ws)
        assert info.tolist()[1] == 0
        same_as_history()
        parents = random_tree(B, T, 60 + step, step % 2 == 0)
        live = torch.tensor([T, max(1, T - 3), 1, T], **i32)
        mask, pos = attn.tree_mask(parents.to(DEV), lens, live)
        sets = [ancestors(p, int(n)) for p, n in zip(parents.tolist(), live)]
        qkv = tokens(100 + 10 * step, T)
        qr, _ = append(qkv, pos, live)
        for l in range(layers):
            o, lse, _ = attn.decode_tree(qr[l], kp[l], vp[l], lens, mask, live, table)
            torch.cuda.synchronize()
            ro, rl, to, tl = reference(qr[l], kp[l], vp[l], table.cpu(), page, lens.tolist(), sets, live.tolist(), d ** -0.5)
            none = torch.isinf(rl)
            assert torch.all((o.double() - ro).abs() <= to) and torch.equal(none, torch.isinf(lse))
            assert torch.all((lse.double() - rl)[~none].abs() <= tl[~none])
        # a path of each tree is accepted; sequence 2 accepts nothing in the first step
        g = torch.Generator().manual_seed(step)
        last = torch.tensor([int(torch.randint(0, int(n), (1,), generator=g)) for n in live], **i32)
        if step == 0:
            last[2] = -1
        for b in range(B):
            path = sorted(sets[b][int(last[b])]) if int(last[b]) >= 0 else []
            history[b] += [(row(kp, b, int(lens[b]) + u).clone(), row(vp, b, int(lens[b]) + u).clone()) for u in path]
        lens = attn.tree_accept(kp, vp, lens, mask, last, page_table=table)
        same_as_history()
        attn.pages_trim(table, refs, lens, lens, page)
        same_as_history()
        held = {int(e) for e in table.flatten() if e >= 0}
        assert [int(r) for r in refs] == [sum(int(e) == p for e in table.flatten()) for p in range(pages)]
        if step == 2:  # the second sequence ends, the fourth goes on as the first
            table, lens = attn.pages_fork(table, refs, lens, torch.tensor([0, -1, 2, 0], **i32), page)
            history = [list(history[i]) if i >= 0 else [] for i in (0, -1, 2, 0)]
            same_as_history()
        if step == 3:
            info, _ = attn.pages_compact(table, refs, kp, vp, workspace=ws)
            assert info.tolist()[0] == len({int(e) for e in table.flatten() if e >= 0})
            assert {int(e) for e in table.flatten() if e >= 0} == set(range(info.tolist()[0]))
            same_as_history()
    assert attn.attn_device_status() == attn.ATTN_OK and held


def test_a_contiguous_cache_takes_part(attn):
    """The caches of attn_rope_append and attn_decode are caches of one page a sequence: drafts appended behind what a
    decode loop has put there, and its next step on what was accepted."""
    B, Hq, Hkv, S, d, T = 3, 8, 2, 90, 64, 6
    f = attn.rope_freqs(d)
    kc, vc = (torch.zeros((B, Hkv, S, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    qkv = normal_bf16((B, 40, Hq + 2 * Hkv, d), 1, DEV).transpose(1, 2)
    _, lens = attn.rope_append(*qkv.split([Hq, Hkv, Hkv], dim=1), kc, vc, lens, f,
                               new_lens=torch.tensor([40, 11, 0], dtype=torch.int32, device=DEV))
    parents = random_tree(B, T, 2)
    mask, pos = attn.tree_mask(parents.to(DEV), lens)
    q, k, v = normal_bf16((B, T, Hq + 2 * Hkv, d), 3, DEV).transpose(1, 2).split([Hq, Hkv, Hkv], dim=1)
    qr, full = attn.rope_axes_append(q, k, v, kc, vc, lens, f, None, pos)
    assert full.tolist() == [46, 17, 6]
    run_and_check(attn, qr, kc, vc, None, 0, lens.tolist(), parents=parents)
    last = torch.tensor([T - 1, 0, 3], dtype=torch.int32, device=DEV)
    lens = attn.tree_accept(kc, vc, lens, mask, last)
    q1 = normal_bf16((B, Hq, d), 4, DEV)
    o, _, _ = attn.decode(q1, kc, vc, lens)
    # the same through decode_tree: the last accepted key as the drafted one
    o2, _, _ = attn.decode_tree(q1[:, :, None].contiguous(), kc, vc, lens - 1)
    _, _, to, _ = reference(q1[:, :, None], kc, vc, None, 0, (lens - 1).tolist(), [[{0}]] * B, [1] * B, d ** -0.5)
    assert torch.all((o[:, :, None] - o2).double().abs() <= 2 * to)


def test_inputs_let_go_of_while_another_stream_uses_them(attn):
    """Calls on a stream that is still busy, whose inputs are freed at once: what is allocated and filled meanwhile is
    other memory."""
    B, Hq, Hkv, T, d, page, per, n = 3, 8, 2, 40, 128, 16, 40, 140
    f, s = attn.rope_freqs(d), torch.cuda.Stream()
    i32 = dict(dtype=torch.int32, device=DEV)

    def pool(seed):
        return [normal_bf16((n, Hkv, page, d), seed + i, DEV) for i in range(2)]

    def a_table():
        return torch.randperm(n, generator=torch.Generator().manual_seed(9))[: B * per].view(B, per).to(**i32)

    def lens():
        return torch.tensor([500, 3, 222], **i32)

    def axes():
        q, k = normal_bf16((B, Hq, 300, d), 1, DEV), normal_bf16((B, Hkv, 300, d), 2, DEV)
        pos, ax = torch.arange(600, **i32).view(2, 300), attn.rope_sections((32, 32))
        return [q, k, pos, ax], lambda stream: attn.rope_axes(q, k, f, ax, pos, stream=stream)

    def append():
        q, k, v = (normal_bf16((B, h, T, d), 3 + i, DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
        (kp, vp), t, m = pool(6), a_table(), lens()
        return [q, k, v, kp, vp, t, m], lambda stream: attn.rope_axes_append(q, k, v, kp, vp, m, f, page_table=t, stream=stream) + (kp, vp)

    def mask():
        p, m = random_tree(B, T, 5).to(DEV), lens()
        return [p, m], lambda stream: attn.tree_mask(p, m, stream=stream)

    def decode():
        q, (kp, vp), t, m = normal_bf16((B, Hq, T, d), 8, DEV), pool(10), a_table(), lens()
        b = attn.tree_mask(random_tree(B, T, 5).to(DEV))[0]
        return [q, kp, vp, t, m, b], lambda stream: attn.decode_tree(q, kp, vp, m, b, page_table=t, stream=stream)[:2]

    def accept():
        (kp, vp), t, m, last = pool(12), a_table(), lens(), torch.tensor([39, 7, -1], **i32)
        b = attn.tree_mask(random_tree(B, T, 5).to(DEV))[0]
        return [kp, vp, t, m, last, b], lambda stream: (attn.tree_accept(kp, vp, m, b, last, page_table=t, stream=stream), kp, vp)

    def tables():
        t, m, refs = a_table(), lens(), torch.zeros(n, **i32)
        used = torch.arange(per, device=DEV) < ((m + page - 1) // page)[:, None]
        t = torch.where(used, t, -1).to(torch.int32)
        refs[t[used].long()] = 1
        return t, m, refs

    def extend():
        (kp, vp), (t, m, refs) = pool(14), tables()
        return [kp, vp, t, m, refs], lambda stream: (attn.pages_extend(t, refs, m, 33, kp, vp, stream=stream)[0], t, refs)

    def fork():
        (t, m, refs), parent = tables(), torch.tensor([0, 0, 1], **i32)
        return [t, m, refs, parent], lambda stream: attn.pages_fork(t, refs, m, parent, page, stream=stream) + (refs,)

    def trim():
        (t, m, refs), keep = tables(), torch.tensor([17, 0, 900], **i32)
        return [t, m, refs, keep], lambda stream: (attn.pages_trim(t, refs, m, keep, page, stream=stream), t, refs)

    def compact():
        (kp, vp), (t, m, refs) = pool(16), tables()
        return [kp, vp, t, m, refs], lambda stream: (attn.pages_compact(t, refs, kp, vp, stream=stream)[0], t, refs, kp, vp)

    for make in (axes, append, mask, decode, accept, extend, fork, trim, compact):
        want = make()[1](None)
        inputs, call = make()
        sizes = [(t.shape, t.dtype) for t in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(60_000_000)
        got = call(s)
        del inputs, call
        other = [torch.empty(shape, dtype=dtype, device=DEV) for shape, dtype in sizes * 2]
        for t in other:
            t.fill_(float("nan") if t.dtype.is_floating_point else -1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), make.__name__
