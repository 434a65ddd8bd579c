"""Rotary positions with several axes on the GPU: attn_rope_axes and
attn_rope_axes_append against the rotation as a complex product in 64 bits.

The kernels do attn_rope's arithmetic with another position per pair, so the
tolerance of a rotated element is the one derived in test_rope_gpu.py: half a
bf16 step, 2^-8 of the value, and 2^-20 of |x| + |y| from the fp32 arithmetic
before it.  Copied columns and rows are equal bit for bit."""
import pytest
import torch

from synthetic_inputs import normal_bf16
from tests.test_rope_gpu import FP32, STEP, freqs, packed

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


def turned(x, pos, f, axes, inter, scale=1.0, inverse=False):
    """x [B, H, N, d], pos [A, B, N], axes a list -> (64-bit result, |x| + |y| of each element's pair)."""
    x = x.double().cpu()
    r = 2 * f.numel()
    a = torch.stack([pos[axes[i]].cpu().double() * f[i] for i in range(r // 2)], -1)[:, None]
    z = torch.complex(torch.cos(a), torch.sin(a) * (-1 if inverse else 1)) * scale
    u, v = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., : r // 2], x[..., r // 2: r])
    w = torch.complex(u, v) * z
    size = (u.abs() + v.abs()) * abs(scale)
    join = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if inter else (lambda p, q: torch.cat((p, q), -1))
    return torch.cat((join(w.real, w.imag), x[..., r:]), -1), join(size, size)


def check(got, x, pos, f, axes, inter, scale=1.0, inverse=False):
    want, size = turned(x, pos, f, axes, inter, scale, inverse)
    r = 2 * f.numel()
    got = got.cpu()
    bound = STEP * want[..., :r].abs() + FP32 * size
    assert torch.all((got.double() - want)[..., :r].abs() <= bound)
    assert torch.equal(got[..., r:], x.cpu()[..., r:])


def some_positions(A, B, N, seed):
    return torch.randint(-7, 100000, (A, B, N), generator=torch.Generator().manual_seed(seed)).to(torch.int32)


CASES = [
    # B, Hq, Hkv, N, d, sections, cycled
    (1, 1, 1, 1, 8, (1,), False), (2, 4, 2, 33, 64, (8, 12, 12), False), (1, 16, 2, 257, 128, (16, 24, 24), True),
    (3, 5, 5, 31, 56, (0, 20, 8), False), (1, 2, 1, 65, 128, (3, 4, 2, 1), True), (2, 2, 2, 7, 64, (1, 1, 1), False),
    (1, 1, 1, 3, 512, (64, 64, 64, 64), True), (17, 64, 8, 60, 128, (32,), False),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,sections,cycled", CASES)
def test_axes_against_the_definition(attn, B, Hq, Hkv, N, d, sections, cycled, inter, inverse):
    q, k = packed((B, Hq, N, d), 1, DEV), normal_bf16((B, Hkv, N, d), 2, DEV)
    axes = attn.rope_sections(sections, cycled)
    f = freqs(2 * sum(sections))
    pos = some_positions(len(sections), B, N, 3)
    call = attn.rope_axes_backward if inverse else attn.rope_axes
    qo, ko = call(q, k, f.to(DEV), axes, pos.to(DEV), interleaved=inter, out_scale=1.25)
    assert qo.is_contiguous() and ko.is_contiguous()
    check(qo, q, pos, f, axes.tolist(), inter, 1.25, inverse)
    check(ko, k, pos, f, axes.tolist(), inter, 1.25, inverse)


def test_forms(attn):
    """One row of positions for the batch; a single axis is attn_rope bit for bit; in place; no k; axes out of range."""
    B, H, N, d = 3, 4, 50, 64
    q, f = packed((B, H, N, d), 4, DEV), freqs(32)
    pos = some_positions(2, 1, N, 5)[:, 0]
    axes = attn.rope_sections((6, 10))
    a, none = attn.rope_axes(q, None, f.to(DEV), axes, pos.to(DEV))
    assert none is None
    check(a, q, pos[:, None].expand(2, B, N), f, axes.tolist(), False)
    b, _ = attn.rope_axes(q, None, f.to(DEV), axes, pos[:, None].expand(2, B, N).contiguous().to(DEV))
    assert torch.equal(a, b)
    one, _ = attn.rope_axes(q, None, f.to(DEV), None, pos[0].to(DEV))
    assert torch.equal(one, attn.rope(q, None, f.to(DEV), positions=pos[0].contiguous().to(DEV))[0])
    odd = torch.tensor([-5, 0, 1, 2] * 4, dtype=torch.int32, device=DEV)
    c, _ = attn.rope_axes(q, None, f.to(DEV), odd, pos.to(DEV))
    check(c, q, pos[:, None].expand(2, B, N), f, odd.clamp(0, 1).tolist(), False)
    behind = q._base if q._base is not None else q
    rest = behind.clone()
    attn.rope_axes(q, None, f.to(DEV), axes, pos.to(DEV), out=(q, None))
    assert torch.equal(q, a)
    assert torch.equal(behind[:, :, 0], rest[:, :, 0]) and torch.equal(behind[:, :, -1], rest[:, :, -1])


def test_the_gradient_against_differences(attn):
    """<dy, (f(x + h e) - f(x - h e)) / 2h> of the map in 64 bits against rope_axes_backward's element, one pair at a
    time: the map is linear, so the difference is exact but for 64-bit rounding and the bound above applies."""
    B, H, N, d, sections = 1, 2, 5, 16, (3, 3)
    f, axes = freqs(12), [0, 0, 0, 1, 1, 1]
    pos = some_positions(2, B, N, 8)
    dy = normal_bf16((B, H, N, d), 9, DEV)
    dx, _ = attn.rope_axes_backward(dy, None, f.to(DEV), attn.rope_sections(sections), pos.to(DEV))
    x = normal_bf16((B, H, N, d), 10, DEV).double().cpu()
    want = torch.zeros_like(x)
    for i in range(d):
        e = torch.zeros_like(x)
        e[..., i] = 0.5
        diff = turned(x + e, pos, f, axes, False)[0] - turned(x - e, pos, f, axes, False)[0]
        want[..., i] = (dy.double().cpu() * diff).sum(-1)
    size = turned(dy, pos, f, axes, False)[1]
    bound = STEP * want[..., :12].abs() + FP32 * size + 2.0 ** -40
    assert torch.all((dx.double().cpu() - want)[..., :12].abs() <= bound)
    assert torch.equal(dx[..., 12:], dy[..., 12:])


def a_table(B, per, pages, seed):
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    return order[: B * per].view(B, per).to(torch.int32)


def row_of(cache, table, page, b, r):
    """Row r of sequence b: [Hkv, d]."""
    return cache[b, :, r] if table is None else cache[int(table[b, r // page]), :, r % page]


@pytest.mark.parametrize("with_pos", [True, False])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("d,r,T,inter", [(64, 64, 1, False), (128, 32, 40, True), (56, 20, 7, False), (64, 0, 5, False)])
def test_append(attn, d, r, T, inter, page, with_pos):
    B, Hq, Hkv, per, A = 3, 6, 2, 5, 2
    S = 90 if page == 0 else page * per
    lens = torch.tensor([0, min(S - 3, 61), 13], dtype=torch.int32)
    new = torch.tensor([T, T, T // 2], dtype=torch.int32)
    q, k, v = normal_bf16((B, T, Hq + 2 * Hkv, d), 20, DEV).transpose(1, 2).split([Hq, Hkv, Hkv], dim=1)
    table = None if page == 0 else a_table(B, per, 2 * B * per, 21)
    shape = (B, Hkv, S, d) if page == 0 else (2 * B * per, Hkv, page, d)
    kc, vc = normal_bf16(shape, 22, DEV), normal_bf16(shape, 23, DEV)
    if table is not None:
        table[0, -1] = -1                      # nothing goes there
        table[2, 0 if page > 16 else 1] = 10 ** 6
    k0, v0 = kc.cpu().clone(), vc.cpu().clone()
    f = freqs(r) if r else None
    axes = [i % A for i in range(r // 2)]
    pos = some_positions(A, B, T, 24)
    qo, lo = attn.rope_axes_append(q, k, v, kc, vc, lens.to(DEV), None if f is None else f.to(DEV),
                                   torch.tensor(axes, dtype=torch.int32, device=DEV) if r else None,
                                   None if not with_pos else (pos if r else pos[0]).to(DEV).contiguous(),
                                   page_table=None if table is None else table.to(DEV), new_lens=new.to(DEV),
                                   interleaved=inter, out_scale=1.0)
    assert lo.tolist() == [min(S, int(a + b)) for a, b in zip(lens, new)]
    if not with_pos:
        pos = (lens[:, None] + torch.arange(T, dtype=torch.int32)).expand(A, B, T)
    if r:
        check(qo, q, pos, f, axes, inter)
        kr, size = turned(k, pos, f, axes, inter)
    else:
        assert torch.equal(qo, q.contiguous())
        kr, size = k.double().cpu(), torch.zeros(1)
    want_v = v0.clone()
    for b in range(B):
        for t in range(int(new[b])):
            at = int(lens[b]) + t
            if at >= S or (table is not None and not 0 <= int(table[b, at // page]) < shape[0]):
                continue
            got = row_of(kc, table, page, b, at).cpu()
            if r:
                assert torch.all((got.double() - kr[b, :, t]).abs()[:, :r] <= (STEP * kr[b, :, t].abs()[:, :r] + FP32 * size[b, :, t]))
                assert torch.equal(got[:, r:], k[b, :, t, r:].cpu())
            else:
                assert torch.equal(got, k[b, :, t].cpu())
            row_of(want_v, table, page, b, at).copy_(v[b, :, t].cpu())
            row_of(k0, table, page, b, at).copy_(got)
    assert torch.equal(vc.cpu(), want_v) and torch.equal(kc.cpu(), k0)  # and no other row


def test_append_on_another_stream_and_in_a_graph(attn):
    B, Hq, Hkv, T, d, page, per = 2, 4, 2, 3, 64, 16, 4
    q, k, v = (normal_bf16((B, h, T, d), 30 + i, DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
    table = a_table(B, per, 3 * B * per, 31).to(DEV)
    f, axes = freqs(d).to(DEV), attn.rope_sections((16, 16))
    pos = some_positions(2, B, T, 32).to(DEV)
    pools = [[torch.zeros((3 * B * per, Hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(3)]
    lens = torch.tensor([5, 30], dtype=torch.int32, device=DEV)
    want = attn.rope_axes_append(q, k, v, *pools[0], lens, f, axes, pos, page_table=table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = attn.rope_axes_append(q, k, v, *pools[1], lens, f, axes, pos, page_table=table, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*want, *pools[0]), (*got, *pools[1])))
    g = torch.cuda.CUDAGraph()
    lens2 = torch.zeros_like(lens)
    with torch.cuda.graph(g):
        out = attn.rope_axes_append(q, k, v, *pools[2], lens2, f, axes, pos, page_table=table)
    lens2.copy_(lens)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*want, *pools[0]), (*out, *pools[2])))
