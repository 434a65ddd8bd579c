"""Rotary positions on the GPU: attn_rope and attn_rope_append against the
rotation as a complex product in 64 bits.

Tolerance of a rotated element.  The kernel forms x c - y s in fp32 and rounds
once to bf16.  The rounding is off by at most half a step, 2^-8 of the value.
Before it: the angle is off by at most 2^-24 half turns (pi 2^-24 radians),
sine and cosine by two steps (2^-22), the products and the difference by three
half steps (3 * 2^-24), the factor out_scale by one more on each of the two:
together below 2^-20 of |x| + |y| (times out_scale).  Copied columns are
equal bit for bit."""
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from synthetic_inputs import normal_bf16

pytestmark = pytest.mark.gpu
STEP, FP32 = 2.0 ** -8, 2.0 ** -20


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


def freqs(r, base=10000.0):
    return torch.tensor([base ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64)


def rotated(x, pos, f, inter, scale=1.0, inverse=False):
    """x [B, H, N, d] -> (64-bit result, |x| + |y| of each element's pair)."""
    x = x.double().cpu()
    r = 2 * f.numel()
    a = pos.cpu().double()[:, None, :, None] * f
    z = torch.complex(torch.cos(a), torch.sin(a) * (-1 if inverse else 1)) * scale
    u, v = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., : r // 2], x[..., r // 2: r])
    w = torch.complex(u, v) * z
    size = (u.abs() + v.abs()) * abs(scale)
    join = (lambda p, q: torch.stack((p, q), -1).flatten(-2)) if inter else (lambda p, q: torch.cat((p, q), -1))
    return torch.cat((join(w.real, w.imag), x[..., r:]), -1), join(size, size)


def check_rotated(got, x, pos, f, inter, scale=1.0, inverse=False):
    want, size = rotated(x, pos, f, inter, scale, inverse)
    r = 2 * f.numel()
    got = got.cpu()
    err = (got.double() - want)[..., :r].abs()
    bound = STEP * want[..., :r].abs() + FP32 * size
    assert torch.all(err <= bound), f"off by {float((err / bound.clamp(min=1e-300)).max()):.3g} of the bound"
    assert torch.equal(got[..., r:], x.cpu()[..., r:])


def packed(shape, seed, dev):
    """[B, H, N, d] as a view of [B, N, H + 2, d]: what a fused projection gives."""
    B, H, N, d = shape
    return normal_bf16((B, N, H + 2, d), seed, dev).transpose(1, 2)[:, 1:H + 1]


CASES = [
    # B, Hq, Hkv, N, d, rotary_dim
    (1, 1, 1, 1, 8, 2), (1, 3, 1, 5, 8, 8), (2, 4, 2, 33, 64, 64), (1, 16, 2, 257, 128, 128), (3, 5, 5, 31, 56, 56),
    (2, 9, 3, 19, 128, 32), (1, 2, 1, 65, 128, 20), (2, 2, 2, 7, 64, 6), (1, 4, 4, 40, 256, 250), (1, 1, 1, 3, 512, 512),
    (17, 64, 8, 200, 128, 64),  # eight heads a thread
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,r", CASES)
def test_rope_against_the_definition(attn, B, Hq, Hkv, N, d, r, inter, inverse):
    dev = torch.device("cuda")
    q, k = packed((B, Hq, N, d), 1, dev), normal_bf16((B, Hkv, N, d), 2, dev)
    f = freqs(r)
    pos = torch.randint(-5, 100000, (B, N), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    call = attn.rope_backward if inverse else attn.rope
    qo, ko = call(q, k, f.to(dev), positions=pos.to(dev), interleaved=inter, out_scale=1.25)
    assert qo.is_contiguous() and ko.is_contiguous()
    check_rotated(qo, q, pos, f, inter, 1.25, inverse)
    check_rotated(ko, k, pos, f, inter, 1.25, inverse)


@pytest.mark.parametrize("inter", [False, True])
def test_positions_forms(attn, inter):
    """No positions are 0..N-1; one row serves every batch entry; only q; in place; a broadcast input."""
    dev = torch.device("cuda")
    B, H, N, d = 3, 4, 50, 64
    q = normal_bf16((B, H, N, d), 4, dev)
    f = freqs(32)
    line = torch.arange(N, dtype=torch.int32)
    a, none = attn.rope(q, None, f.to(dev), interleaved=inter)
    assert none is None
    check_rotated(a, q, line.expand(B, N), f, inter)
    b, _ = attn.rope(q, None, f.to(dev), positions=line.to(dev), interleaved=inter)
    assert torch.equal(a, b)
    one = q[:, :1].expand(B, H, N, d)
    c, _ = attn.rope(one, None, f.to(dev), interleaved=inter)
    check_rotated(c, one, line.expand(B, N), f, inter)
    view = packed((B, H, N, d), 5, dev)
    before = view.clone()
    behind = view._base if view._base is not None else view
    rest = behind.clone()
    out, _ = attn.rope(view, None, f.to(dev), interleaved=inter, out=(view, None))
    assert out is view
    check_rotated(view, before, line.expand(B, N), f, inter)
    assert torch.equal(behind[:, :, 0], rest[:, :, 0]) and torch.equal(behind[:, :, -1], rest[:, :, -1])


def test_far_positions_and_odd_frequencies(attn):
    """Angles near the end of the int32 range, where p f in 64 bits is itself off by 2^-22 radians: the reference takes the whole turns out in 60
    decimal digits.  Frequencies that mean nothing leave finite columns."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    dev = torch.device("cuda")
    f = [1.0, 0.7, 3.0e-5, 1e-300, 5e-324, 0.0, 123456.789, -0.3, 6.283185307179586, 2.0 ** 53]
    pos = [2 ** 31 - 1, -2 ** 31, 1234567890, 1, 0]
    x = torch.zeros((1, 1, len(pos), 24), dtype=torch.bfloat16)
    x[..., :len(f)] = 1.0
    out, _ = attn.rope(x.to(dev), None, torch.tensor(f, dtype=torch.float64, device=dev),
                       positions=torch.tensor(pos, dtype=torch.int32, device=dev))
    out = out.cpu().double().numpy()[0, 0]
    for n, p in enumerate(pos):
        for i, w in enumerate(f):
            t = Decimal(p) * Decimal(w) / two_pi
            a = float((t - t.to_integral_value()) * two_pi)
            # besides the bound above: 2^66 / 2 pi is rounded, which is w / 8 units of 2^-64 turns, and u cut to one
            # such unit; p of them add up
            slack = FP32 + abs(p) * (abs(w) / 8 + 1) * 2.0 ** -64 * 6.2832
            assert abs(out[n, i] - np.cos(a)) <= STEP * abs(np.cos(a)) + slack, (p, w)
            assert abs(out[n, len(f) + i] - np.sin(a)) <= STEP * abs(np.sin(a)) + slack, (p, w)
    bad = torch.tensor([float("inf"), float("nan"), 1e300, 1.0], dtype=torch.float64, device=dev)
    y, _ = attn.rope(normal_bf16((1, 2, 9, 8), 6, dev), None, bad)
    assert torch.isfinite(y.float()).all()


def test_high_frequencies_at_far_positions(attn):
    """Up to 2^54 radians a position: besides the bound at the top the phase is off by less than |p| 2^-64 turns, 2^-33 at the farthest
    position."""
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    dev = torch.device("cuda")
    f = [2.0 ** 53, 2.0 ** 53 - 1, -(2.0 ** 54 - 2), 1e15, 12345678901.25, 2.0 ** 40 + 1, -7.5e12, 1e8 / 3, 2.0 ** 30, 10.5, 2.0 / 3, 1e-8]
    pos = [2 ** 31 - 1, -2 ** 31, 1234567890, -77777, 4099, 1]
    x = torch.zeros((1, 1, len(pos), 2 * len(f)), dtype=torch.bfloat16)
    x[..., :len(f)] = 1.0
    out, _ = attn.rope(x.to(dev), None, torch.tensor(f, dtype=torch.float64, device=dev),
                       positions=torch.tensor(pos, dtype=torch.int32, device=dev))
    out = out.cpu().double().numpy()[0, 0]
    for n, p in enumerate(pos):
        for i, w in enumerate(f):
            t = Decimal(p) * Decimal(w) / two_pi
            a = float((t - t.to_integral_value()) * two_pi)
            slack = FP32 + abs(p) * 2.0 ** -64 * 6.2832
            assert slack < 2.0 ** -19
            assert abs(out[n, i] - np.cos(a)) <= STEP * abs(np.cos(a)) + slack, (p, w)
            assert abs(out[n, len(f) + i] - np.sin(a)) <= STEP * abs(np.sin(a)) + slack, (p, w)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("r", [16, 20])
def test_gradient_is_the_adjoint_and_matches_differences(attn, inter, r):
    """L(x) = <dy, rope(x)>.  The kernel's dx against the formula is part of the test above; here against L itself: rope is linear, so a step of
    h in one coordinate changes L by h dx exactly, up to the outputs' roundings: each of the two outputs of a pair
    is within STEP |out| + FP32 (|x| + |y|) of the exact one, before and after the step, and dx within the same of its own."""
    dev = torch.device("cuda")
    B, H, N, d = 1, 2, 3, 24
    x, dy = normal_bf16((B, H, N, d), 7, dev), normal_bf16((B, H, N, d), 8, dev)
    pos = torch.tensor([[0, 5, 100003]], dtype=torch.int32, device=dev)
    f = freqs(r).to(dev)
    dx, _ = attn.rope_backward(dy, None, f, positions=pos, interleaved=inter)

    def loss(t):
        y, _ = attn.rope(t, None, f, positions=pos, interleaved=inter)
        return float((y.double() * dy.double()).sum()), y.double()

    l0, y0 = loss(x)
    h = 4.0
    g = np.random.RandomState(1)
    for _ in range(24):
        at = tuple(int(g.randint(n)) for n in x.shape)
        step = x.clone()
        step[at] = float(x[at]) + h
        real = float(step[at].double() - x[at].double())  # x + h is rounded to bf16
        l1, y1 = loss(step)
        moved = (y1 != y0)
        room = (STEP * (y0.abs() + y1.abs()) + 2 * FP32 * (16 + h)) * dy.double().abs()
        tol = float(room[moved].sum()) + abs(real) * (STEP * abs(float(dx[at])) + FP32 * 16)
        assert abs((l1 - l0) - real * float(dx[at])) <= tol


def test_rule_frequencies_reach_the_kernel(attn):
    dev = torch.device("cuda")
    q = normal_bf16((1, 2, 64, 64), 9, dev)
    pos = (torch.arange(64, dtype=torch.int32) * 1000)[None]
    for rule in attn.ROPE_RULES:
        f = attn.rope_freqs(64, rule=rule, factor=8.0)
        out, _ = attn.rope(q, None, f, positions=pos.to(dev))
        check_rotated(out, q, pos, f.cpu(), False)


# ------------------------------------------------------------------ appending
def _append_case(B, Hq, Hkv, T, S, d, seed, dev):
    qkv = normal_bf16((B, T, Hq + 2 * Hkv, d), seed, dev).transpose(1, 2)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    return q, k, v, normal_bf16((B, Hkv, S, d), seed + 1, dev), normal_bf16((B, Hkv, S, d), seed + 2, dev)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,T,S,d,r", [
    (1, 1, 1, 1, 1, 8, 8), (5, 8, 2, 1, 70, 64, 64), (5, 12, 4, 1, 33, 128, 128), (6, 4, 2, 17, 40, 128, 32),
    (6, 3, 3, 9, 30, 56, 20), (4, 64, 8, 300, 500, 128, 64), (5, 2, 2, 4, 16, 64, 0)])
def test_append_against_the_definition(attn, B, Hq, Hkv, T, S, d, r, inter):
    """Lengths at both ends and past them, padded entries, rows past the cache's end; everything else in the caches, cache_pos
    and weights stays as it was."""
    dev = torch.device("cuda")
    q, k, v, kc, vc = _append_case(B, Hq, Hkv, T, S, d, 20, dev)
    lens = [0, S, S - 1, -3, S + 9, max(0, S - T)][:B]
    new = [T, T, T + 5, T, -1, (T + 1) // 2][:B]
    start = [7, 100000, 0, 3, 5, 12][:B]
    f = freqs(r) if r else torch.zeros(0, dtype=torch.float64)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    cp, w = ints([[[-7] * S] * Hkv] * B), torch.full((B, Hkv, S), 3.5, device=dev)
    k0, v0 = kc.clone(), vc.clone()
    qo, lo = attn.rope_append(q, k, v, kc, vc, ints(lens), f.to(dev) if r else None, start_pos=ints(start),
                              new_lens=ints(new), interleaved=inter, cache_pos=cp, weights=w)
    at = torch.tensor(start)[:, None] + torch.arange(T)
    check_rotated(qo, q, at, f, inter)
    kr, size = rotated(k, at, f, inter)
    kc, vc, k0, v0, cp, w = (t.cpu() for t in (kc, vc, k0, v0, cp, w))
    want_lens = []
    for b in range(B):
        n0 = min(max(lens[b], 0), S)
        m = min(max(new[b], 0), T)
        stored = min(m, S - n0)
        want_lens.append(n0 + stored)
        row = slice(n0, n0 + stored)
        err = (kc[b, :, row].double() - kr[b, :, :stored]).abs()
        assert torch.all(err[..., :r] <= STEP * kr[b, :, :stored, :r].abs() + FP32 * size[b, :, :stored])
        assert torch.equal(kc[b, :, row, r:], k[b, :, :stored, r:].cpu())
        assert torch.equal(vc[b, :, row], v[b, :, :stored].cpu())
        assert torch.equal(cp[b, :, row], at[b, :stored].int().expand(Hkv, -1)) and torch.all(w[b, :, row] == 0)
        for rest in (slice(0, n0), slice(n0 + stored, S)):
            assert torch.equal(kc[b, :, rest], k0[b, :, rest]) and torch.equal(vc[b, :, rest], v0[b, :, rest])
            assert torch.all(cp[b, :, rest] == -7) and torch.all(w[b, :, rest] == 3.5)
    assert lo.tolist() == want_lens


def test_append_defaults(attn):
    """Without start_pos a token's position is its row; without new_lens all T enter; q_out may be q."""
    dev = torch.device("cuda")
    B, Hq, Hkv, T, S, d = 2, 4, 2, 3, 20, 64
    q, k, v, kc, vc = _append_case(B, Hq, Hkv, T, S, d, 30, dev)
    lens = torch.tensor([0, 11], dtype=torch.int32, device=dev)
    f = freqs(d)
    q0 = q.clone()
    qo, lo = attn.rope_append(q, k, v, kc, vc, lens, f.to(dev), q_out=q)
    at = lens.cpu()[:, None] + torch.arange(T)
    check_rotated(qo, q0, at, f, False)
    for b in range(B):
        n = int(lens[b])
        check_rotated(kc[b:b + 1, :, n:n + T], k[b:b + 1], at[b:b + 1], f, False)
    assert lo.tolist() == [3, 14]


def test_captured_step_and_another_stream(attn):
    """A captured append replays with the lengths and tokens that the buffers hold then, and two calls on different
    streams at once give what they give one after the other."""
    dev = torch.device("cuda")
    B, Hq, Hkv, S, d = 4, 16, 2, 64, 128
    q, k, v, kc, vc = _append_case(B, Hq, Hkv, 1, S, d, 40, dev)
    f = freqs(d).to(dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    nxt, qo = torch.empty_like(lens), torch.empty((B, Hq, 1, d), dtype=torch.bfloat16, device=dev)

    def step():
        attn.rope_append(q, k, v, kc, vc, lens, f, q_out=qo, seqlens_out=nxt)
        lens.copy_(nxt)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens.copy_(torch.tensor([0, 5, 62, 64], dtype=torch.int32))
    ref_k, ref_v = kc.clone(), vc.clone()
    ref_l = lens.clone()
    for i in range(3):
        q.copy_(normal_bf16(q.shape, 50 + i, dev))
        k.copy_(normal_bf16(k.shape, 60 + i, dev))
        g.replay()
        eq, ref_l = attn.rope_append(q, k, v, ref_k, ref_v, ref_l, f)
        torch.cuda.synchronize()
        assert torch.equal(qo, eq) and torch.equal(kc, ref_k) and torch.equal(vc, ref_v)
    assert lens.tolist() == [3, 8, 64, 64]

    a, b = normal_bf16((2, 8, 500, 128), 70, dev), normal_bf16((2, 8, 500, 128), 71, dev)
    one, two = attn.rope(a, None, f)[0], attn.rope(b, None, f)[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    o1 = attn.rope(a, None, f, stream=s1)[0]
    o2 = attn.rope(b, None, f, stream=s2)[0]
    torch.cuda.synchronize()
    assert torch.equal(o1, one) and torch.equal(o2, two)


def test_rows_past_two_to_the_31_elements(attn):
    """A cache of more than 2^31 elements: the last rows of the last entry."""
    dev = torch.device("cuda")
    B, Hkv, S, d = 2, 8, 1 << 20, 160
    kc = torch.zeros((B, Hkv, S, d), dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    q, k, v = (normal_bf16((B, h, 2, d), 80 + h, dev) for h in (8, 8, 8))
    f = freqs(d)
    lens = torch.tensor([S - 2, S - 1], dtype=torch.int32, device=dev)
    _, lo = attn.rope_append(q, k, v, kc, vc, lens, f.to(dev))
    assert lo.tolist() == [S, S]
    at = lens.cpu()[:, None] + torch.arange(2)
    check_rotated(kc[:1, :, S - 2:], k[:1], at[:1], f, False)
    check_rotated(kc[1:, :, S - 1:], k[1:, :, :1], at[1:, :1], f, False)
    assert torch.equal(vc[1, :, S - 1], v[1, :, 0]) and not kc[1, :, :S - 1].any() and not kc[0, :, :S - 2].any()
    del kc, vc
    torch.cuda.empty_cache()


def test_views_that_interleave_do_not_overlap(attn):
    """In place through one fused projection, whose q, k and v lie between one another: rotation and appending give what they give on separate
    tensors, v stays; so do tensors in the two halves of one buffer's columns, and outputs behind inputs in one allocation."""
    dev = torch.device("cuda")
    B, Hq, Hkv, N, d = 3, 6, 2, 19, 64
    f = freqs(d).to(dev)
    qkv = normal_bf16((B, N, Hq + 2 * Hkv, d), 90, dev)
    q, k, v = qkv.transpose(1, 2).split([Hq, Hkv, Hkv], dim=1)
    want, kept = attn.rope(q, k, f), v.clone()
    lens = torch.tensor([0, 4, 30], dtype=torch.int32, device=dev)
    caches = [torch.zeros((B, Hkv, 40, d), dtype=torch.bfloat16, device=dev) for _ in range(4)]
    q1, _ = attn.rope_append(q.clone(), k.clone(), v.clone(), *caches[:2], lens, f)
    q2 = normal_bf16((B, N, Hq + 2 * Hkv, d), 90, dev)
    qs, ks, vs = q2.transpose(1, 2).split([Hq, Hkv, Hkv], dim=1)
    attn.rope_append(qs, ks, vs, *caches[2:], lens, f, q_out=qs)
    assert torch.equal(qs, q1) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    attn.rope(q, k, f, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)
    both = normal_bf16((B, Hq, N, 2 * d), 91, dev)
    a, b = both[..., :d], both[..., d:]
    want = attn.rope(a, None, f)[0]
    attn.rope(a, None, f, out=(b, None))
    assert torch.equal(b, want)
    pool = normal_bf16((2, B, Hq, N, d), 92, dev)
    want = attn.rope(pool[0], None, f)[0]
    attn.rope(pool[0], None, f, out=(pool[1], None))
    assert torch.equal(pool[1], want)
    # keys in every other token of a longer row of tokens, the outputs in those between them
    rows = normal_bf16((B, Hkv, 2 * N, d), 93, dev)
    want = attn.rope(q, rows[:, :, ::2], f)[1]
    attn.rope(q, rows[:, :, ::2], f, out=(want.new_empty(q.shape), rows[:, :, 1::2]))
    assert torch.equal(rows[:, :, 1::2], want)
