"""The pages of a cache on the GPU: attn_pages_extend, _fork, _trim and _compact
against the rules written out one sequence at a time.  Nothing is rounded: equal bit for bit."""
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


class Pool:
    """Tables and counts as lists, K and V as CPU tensors [layers, pages, Hkv, page, d]."""

    def __init__(self, B, per, pages, page, shape, seed):
        self.page, self.per, self.pages = page, per, pages
        self.table = [[-1] * per for _ in range(B)]
        self.refs, self.lens = [0] * pages, [0] * B
        layers, Hkv, d = shape
        self.k, self.v = (normal_bf16((layers, pages, Hkv, page, d), seed + i, "cpu") for i in range(2))

    def ok(self, e):
        return 0 <= e < self.pages

    def reach(self, b, new):
        n = min(max(self.lens[b], 0), self.per * self.page)
        end = min(n + max(new, 0), self.per * self.page)
        return (range(n // self.page, -(-end // self.page)) if end > n else range(0)), n

    def extend(self, new):
        writers = {}
        for b, x in enumerate(new):
            for s in self.reach(b, x)[0]:
                e = self.table[b][s]
                if self.ok(e) and self.refs[e] > 1:
                    writers.setdefault(e, []).append(b)
        needed = []
        for b, x in enumerate(new):
            for s in self.reach(b, x)[0]:
                e = self.table[b][s]
                if not self.ok(e) or (e in writers and not (len(writers[e]) == self.refs[e] and max(writers[e]) == b)):
                    needed.append((b, s))
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        if len(free) < len(needed):
            return [0, len(needed) - len(free)]
        for (b, s), p in zip(needed, free):
            e, n = self.table[b][s], self.reach(b, 0)[1]
            if self.ok(e):
                live = n - s * self.page
                for x in (self.k, self.v):
                    if live > 0:
                        x[:, p, :, :live] = x[:, e, :, :live]
                self.refs[e] -= 1
            self.table[b][s], self.refs[p] = p, 1
        return [len(needed), 0]

    def fork(self, parent):
        old = [row[:] for row in self.table]
        lens = self.lens[:]
        for b, p in enumerate(parent):
            if p == b:
                self.lens[b] = min(max(lens[b], 0), self.per * self.page)
                continue
            has = 0 <= p < len(old)
            n = min(max(lens[p], 0), self.per * self.page) if has else 0
            row = [(old[p][s] if has and s < -(-n // self.page) and self.ok(old[p][s]) else -1) for s in range(self.per)]
            for e in old[b]:
                if self.ok(e):
                    self.refs[e] -= 1
            for e in row:
                if self.ok(e):
                    self.refs[e] += 1
            self.table[b], self.lens[b] = row, n

    def trim(self, keep):
        for b, x in enumerate(keep):
            n = min(max(x, 0), self.per * self.page)
            for s in range(-(-n // self.page), self.per):
                if self.ok(self.table[b][s]):
                    self.refs[self.table[b][s]] -= 1
                self.table[b][s] = -1
            self.lens[b] = min(min(max(self.lens[b], 0), self.per * self.page), n)

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        movers = [p for p in range(n, self.pages) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            for x in (self.k, self.v):
                x[:, b] = x[:, a]
        self.table = [[to.get(e, e) for e in row] for row in self.table]
        return [n, len(holes)]


class Device:
    """The same through the library."""

    def __init__(self, attn, pool, flat):
        self.attn, self.page = attn, pool.page
        i32 = dict(dtype=torch.int32, device=DEV)
        self.table, self.refs, self.lens = (torch.tensor(x, **i32) for x in (pool.table, pool.refs, pool.lens))
        self.k, self.v = (x.to(DEV)[0] if flat else x.to(DEV) for x in (pool.k, pool.v))
        self.ws = None

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def extend(self, new):
        same = len(set(new)) == 1 and new[0] >= 0
        info, self.ws = self.attn.pages_extend(self.table, self.refs, self.lens, new[0] if same else self.ints(new), self.k,
                                               self.v, workspace=self.ws)
        return info.tolist()

    def fork(self, parent):
        self.table, self.lens = self.attn.pages_fork(self.table, self.refs, self.lens, self.ints(parent), self.page)

    def trim(self, keep):
        self.attn.pages_trim(self.table, self.refs, self.lens, self.ints(keep), self.page, seqlens_out=self.lens)

    def compact(self):
        info, self.ws = self.attn.pages_compact(self.table, self.refs, self.k, self.v, workspace=self.ws)
        return info.tolist()

    def same(self, pool):
        assert self.table.tolist() == pool.table
        assert self.refs.tolist() == pool.refs
        assert self.lens.tolist() == pool.lens
        flat = self.k.dim() == 4
        for got, want in ((self.k, pool.k), (self.v, pool.v)):
            assert torch.equal(got.cpu(), want[0] if flat else want)


@pytest.mark.parametrize("B,per,pages,page,shape,seed", [
    (1, 1, 1, 16, (1, 1, 8), 1), (3, 4, 20, 16, (1, 2, 64), 2), (9, 7, 60, 32, (3, 2, 128), 3), (40, 3, 150, 16, (2, 3, 56), 4),
    (5, 40, 260, 64, (1, 1, 128), 5), (300, 5, 1700, 16, (1, 1, 8), 6), (17, 9, 90, 128, (2, 1, 64), 7),
])
def test_a_life_of_a_pool(attn, B, per, pages, page, shape, seed):
    """Prompts come in, samples fork, tokens are appended, beams end, the pool is compacted; after each call tables,
    counts, lengths and every byte of the pool are as the rules say."""
    g = torch.Generator().manual_seed(seed)
    pool = Pool(B, per, pages, page, shape, 50 + seed)
    dev = Device(attn, pool, shape[0] == 1)

    def draw(lo, hi):
        return torch.randint(lo, hi + 1, (B,), generator=g).tolist()

    def both(call, *args):
        want, got = getattr(pool, call)(*args), getattr(dev, call)(*args)
        assert want == got, (call, want, got)
        dev.same(pool)
        return want

    for step in range(6):
        new = draw(0, page * per // 2) if step % 3 == 0 else [1 + step % 2] * B if step % 3 == 1 else draw(-3, 3)
        if both("extend", new)[1] == 0:
            lens = [min(max(n, 0) + max(x, 0), page * per) for n, x in zip(pool.lens, new)]
            pool.lens = lens
            dev.lens = dev.ints(lens)
        parent = list(range(B)) if step == 4 else draw(-1, B)
        both("fork", [p if torch.rand(1, generator=g) < 0.6 else b for b, p in enumerate(parent)])
        both("extend", [1] * B)
        if step % 2:
            both("trim", [n if torch.rand(1, generator=g) < 0.5 else n // 2 for n in pool.lens])
        else:
            both("compact")
    both("trim", [0] * B)
    assert both("compact")[0] == 0


def test_not_enough_pages_changes_nothing(attn):
    pool = Pool(3, 4, 5, 16, (1, 1, 8), 70)
    dev = Device(attn, pool, True)
    assert pool.extend([16, 17, 1]) == dev.extend([16, 17, 1]) == [4, 0]
    dev.same(pool)
    pool.lens = [16, 17, 1]
    dev.lens = dev.ints(pool.lens)
    pool.fork([0, 0, 2]), dev.fork([0, 0, 2])
    dev.same(pool)
    assert pool.extend([30, 30, 30]) == dev.extend([30, 30, 30])
    dev.same(pool)
    assert pool.extend([100, 100, 100])[1] > 0 and dev.extend([100, 100, 100])[1] > 0
    dev.same(pool)


def test_all_writers_of_a_shared_page(attn):
    """Four sequences share a page that is partly filled; all write: three copies, and the last keeps it.  Then two of
    three write: both copy."""
    for writers, taken in (([1, 1, 1, 1], 3), ([1, 0, 1, 1], 3), ([0, 0, 0, 5], 1)):
        pool = Pool(4, 2, 9, 16, (2, 2, 64), 71)
        dev = Device(attn, pool, False)
        assert pool.extend([5, 0, 0, 0]) == dev.extend([5, 0, 0, 0]) == [1, 0]
        pool.lens[0] = 5
        dev.lens = dev.ints(pool.lens)
        pool.fork([0] * 4), dev.fork([0] * 4)
        assert pool.extend(writers) == dev.extend(writers) == [taken, 0]
        dev.same(pool)
        assert len({row[0] for row in pool.table}) == taken + 1


def test_many_pages(attn):
    """More pages than a block looks at in one round, free ones far behind."""
    B, per, pages = 2, 8, 70001
    pool = Pool(B, per, pages, 16, (1, 1, 8), 72)
    pool.refs = [1] * pages
    for p in (3, 16383, 16384, 40000, 69999, 70000):
        pool.refs[p] = 0
    dev = Device(attn, pool, True)
    assert pool.extend([40, 33]) == dev.extend([40, 33]) == [6, 0]
    dev.same(pool)
    pool.lens = [40, 33]
    dev.lens = dev.ints(pool.lens)
    for x in (pool, dev):
        x.trim([0, 20])
    dev.same(pool)
    assert pool.compact() == dev.compact()
    dev.same(pool)


def test_in_a_graph_and_on_another_stream(attn):
    pool = Pool(4, 6, 30, 16, (2, 2, 64), 73)
    dev = Device(attn, pool, False)
    new, parent = dev.ints([20, 3, 0, 17]), dev.ints([0, 0, 3, 1])
    s = torch.cuda.Stream()
    ws = torch.empty(attn.attn_pages_workspace_bytes(4, 30), dtype=torch.uint8, device=DEV)
    lens = torch.zeros(4, dtype=torch.int32, device=DEV)
    out, olens = torch.empty_like(dev.table), torch.empty_like(lens)
    info = torch.empty(2, dtype=torch.int32, device=DEV)

    def step():
        attn.pages_extend(dev.table, dev.refs, lens, new, dev.k, dev.v, workspace=ws, info=info)
        lens.copy_(new)
        attn.pages_fork(dev.table, dev.refs, lens, parent, 16, page_table_out=out, seqlens_out=olens)
        attn.pages_extend(out, dev.refs, olens, 1, dev.k, dev.v, workspace=ws, info=info)
        attn.pages_compact(out, dev.refs, dev.k, dev.v, workspace=ws, info=info)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        step()
    g.replay()
    torch.cuda.synchronize()
    pool.extend([20, 3, 0, 17])
    pool.lens = [20, 3, 0, 17]
    pool.fork([0, 0, 3, 1])
    pool.extend([1] * 4)
    pool.compact()
    dev.table, dev.lens = out, olens
    dev.same(pool)


def test_a_page_twice_in_a_sequence(attn):
    """Entries count, not sequences: of two that hold a page and are both written to, the last keeps it; the
    others get pages of their own, with the keys in use."""
    page, pages, B = 16, 12, 2
    k, v = (normal_bf16((pages, 1, page, 64), 40 + i, "cpu") for i in range(2))
    table = torch.tensor([[5, 5, 3, -1], [3, 7, 7, 7]], dtype=torch.int32, device=DEV)
    refs = torch.tensor([0, 0, 0, 2, 0, 2, 0, 3, 0, 0, 0, 0], dtype=torch.int32, device=DEV)
    lens = torch.tensor([10, 20], dtype=torch.int32, device=DEV)
    kd, vd = k.to(DEV), v.to(DEV)
    # sequence 0 writes to slots 0 and 1 (both entries of page 5), sequence 1 to slots 1 and 2 (two of the three of page 7)
    info, _ = attn.pages_extend(table, refs, lens, torch.tensor([20, 20], dtype=torch.int32, device=DEV), kd, vd)
    assert info.tolist() == [3, 0]
    assert table.tolist() == [[0, 5, 3, -1], [3, 1, 2, 7]]
    assert refs.tolist() == [1, 1, 1, 2, 0, 1, 0, 1, 0, 0, 0, 0]
    for got, was in ((kd.cpu(), k), (vd.cpu(), v)):
        want = was.clone()
        want[0, :, :10] = was[5, :, :10]
        want[1, :, :4] = was[7, :, :4]
        assert torch.equal(got, want)
