"""The decode-cache operators together, as a serving loop uses them: a prompt prefix that the batch shares, then steps of
append (rotary positions into the caches), decode over prefix and caches with the weights counted, and eviction; every
stage of every step against its definition on what the stage before left in device memory."""
import torch
import pytest

from synthetic_inputs import normal_bf16
from tests.test_decode_prefix_gpu import reference
from tests.test_evict_gpu import sources
from tests.test_rope_gpu import FP32, STEP, check_rotated, rotated

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


@pytest.mark.parametrize("d,Hq,Hkv,inter", [(128, 16, 2, False), (64, 12, 4, True)])
def test_bounded_cache_behind_a_shared_prefix(attn, d, Hq, Hkv, inter):
    B, P, keep, recent, S = 3, 333, 24, 6, 28
    f = attn.rope_freqs(d, rule="by_parts", factor=4.0)
    # the prefix: rotated once, positions 0 .. P - 1
    raw = normal_bf16((1, Hkv, P, d), 1, DEV)
    kp, _ = attn.rope(raw, None, f, interleaved=inter)
    check_rotated(kp, raw, torch.arange(P)[None], f.cpu(), inter)
    kp, vp = kp[0].contiguous(), normal_bf16((Hkv, P, d), 2, DEV)
    kc = torch.zeros((B, Hkv, S, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    pos = torch.full((B, Hkv, S), -1, dtype=torch.int32, device=DEV)
    w = torch.zeros((B, Hkv, S), device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    ws = None

    # a first turn of unequal length for every user, in one padded call, then decode steps of one token
    turns = [(11, torch.tensor([11, 7, 1], dtype=torch.int32, device=DEV))] + [(1, None)] * 30
    cur = torch.full((B,), P - 1, dtype=torch.int32, device=DEV)
    for step, (T, new) in enumerate(turns):
        qkv = normal_bf16((B, T, Hq + 2 * Hkv, d), 10 + step, DEV).transpose(1, 2)
        q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
        n0 = lens.clone()
        start = cur + 1
        qr, lens = attn.rope_append(q, k, v, kc, vc, lens, f, start_pos=start, new_lens=new, interleaved=inter,
                                    cache_pos=pos, weights=w)
        added = (torch.full_like(lens, T) if new is None else new).cpu()
        cur = cur + added.to(DEV)
        at = start.cpu().long()[:, None] + torch.arange(T)
        check_rotated(qr, q, at, f.cpu(), inter)
        kr, size = rotated(k, at, f.cpu(), inter)
        for b in range(B):
            m, row = int(added[b]), slice(int(n0[b]), int(n0[b] + added[b]))
            err = (kc[b, :, row].cpu().double() - kr[b, :, :m]).abs()
            assert torch.all(err <= STEP * kr[b, :, :m].abs() + FP32 * size[b, :, :m])
            assert torch.equal(vc[b, :, row], v[b, :, :m]) and torch.all(w[b, :, row] == 0)
            assert torch.equal(pos[b, :, row].cpu(), at[b, :m].int().expand(Hkv, -1))
        assert lens.tolist() == (n0.cpu() + added).tolist()

        # the last token of every user attends
        last = qr[torch.arange(B, device=DEV), :, (added - 1).to(DEV).long()].contiguous()
        before = w.clone()
        o, lse, ws = attn.decode_prefix(last, kp, vp, kc, vc, lens, weights=w, workspace=ws)
        ro, rl, rw, to, e, tw = reference(last, kp, vp, kc, vc, lens.tolist(), d ** -0.5)
        assert torch.all((o.double().cpu() - ro).abs() <= to)
        assert torch.all((lse.double().cpu() - rl).abs() <= e)
        want = before.double().cpu() + rw
        assert torch.all((w.double().cpu() - want).abs() <= tw + 2.0 ** -24 * want.abs())
        # all that the own keys of a KV head receive and the prefix's share make up its query heads
        assert torch.all((w - before).sum(-1) <= Hq // Hkv + 1e-3)

        kept = [t.cpu().clone() for t in (kc, vc, w, pos)]
        n = lens.tolist()
        lens, _ = attn.cache_evict(kc, vc, w, lens, keep, recent, cache_pos=pos, cur_pos=cur)
        torch.cuda.synchronize()
        for b in range(B):
            for h in range(Hkv):
                src = torch.from_numpy(sources(kept[2][b, h].numpy(), kept[3][b, h].numpy(), n[b], keep, recent, int(cur[b])))
                for t, was in zip((kc, vc, w, pos), kept):
                    assert torch.equal(t[b, h, :len(src)].cpu(), was[b, h, src])
                # the latest tokens are all there
                held = set(pos[b, h, :len(src)].tolist())
                assert held >= set(range(max(P, int(cur[b]) - recent + 1), int(cur[b]) + 1))
        assert lens.tolist() == [min(x, keep) for x in n]
    assert attn.attn_device_status() == attn.ATTN_OK


def test_training_through_the_rotation(attn):
    """Gradients of sum(dO * attention(rope(q), rope(k), v)) by rope, attn_fwd, attn_bwd and rope_backward, against the
    64-bit gradient of the same function.  The relative error adds up from the stages, each of which rounds its results to
    bf16 once (2^-8 at most, 2^-9.8 in the root mean square) and, in the attention, its probabilities and their gradients:
    the backward tests allow 1e-2, the two rotations of either gradient add 2 * 2^-8."""
    B, Hq, Hkv, N, d = 2, 4, 2, 150, 64
    q, k, v = (normal_bf16((B, h, N, d), 70 + i, DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
    do = normal_bf16((B, Hq, N, d), 75, DEV)
    f = attn.rope_freqs(32)
    qr, kr = attn.rope(q, k, f, interleaved=True)
    o, lse = attn.forward(qr, kr, v, causal=True)
    dqr, dkr, dv = attn.backward(qr, kr, v, o, lse, do, causal=True)
    dq, dk = attn.rope_backward(dqr, dkr, f, interleaved=True)

    q64, k64, v64 = (t.double().cpu().requires_grad_() for t in (q, k, v))
    a = torch.arange(N).double()[:, None] * f.cpu()
    z = torch.polar(torch.ones_like(a), a)

    def turned(x):
        head = torch.view_as_real(torch.view_as_complex(x[..., :32].unflatten(-1, (16, 2)).contiguous()) * z).flatten(-2)
        return torch.cat((head, x[..., 32:]), -1)

    kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in (turned(k64), v64))
    s = turned(q64) @ kk.transpose(2, 3) * d ** -0.5
    s = s.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf"))
    (torch.softmax(s, -1) @ vv * do.double().cpu()).sum().backward()
    for got, want in ((dq, q64.grad), (dk, k64.grad), (dv, v64.grad)):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        assert rel <= 1e-2 + 2 * 2.0 ** -8, rel


def test_inputs_let_go_of_while_another_stream_uses_them(attn):
    """Calls on a stream that is still busy, whose inputs are freed at once: what is allocated and filled with NaN meanwhile is other memory."""
    B, Hq, Hkv, N, P, S, d = 2, 16, 4, 700, 300, 1000, 128
    f, s = attn.rope_freqs(d), torch.cuda.Stream()

    def tokens(seed, n):
        return [normal_bf16((B, h, n, d), seed + i, DEV) for i, h in enumerate((Hq, Hkv, Hkv))]

    def caches(seed):
        w = torch.rand((B, Hkv, S), generator=torch.Generator().manual_seed(seed)).to(DEV)
        return [normal_bf16((B, Hkv, S, d), seed + i, DEV) for i in range(2)] + [w, torch.full((B,), S - N, dtype=torch.int32, device=DEV)]

    def rope():
        q, k, _ = tokens(1, N)
        return [q, k, f], lambda stream: attn.rope(q, k, f, stream=stream)

    def append():
        q, k, v = tokens(5, N)
        kc, vc, _, n = caches(10)
        return [q, k, v, kc, vc, n], lambda stream: attn.rope_append(q, k, v, kc, vc, n, f, stream=stream) + (kc, vc)

    def decode():
        q, kp, vp = (normal_bf16(x, 20 + i, DEV) for i, x in enumerate(((B, Hq, d), (Hkv, P, d), (Hkv, P, d))))
        kc, vc, w, n = caches(25)
        return [q, kp, vp, kc, vc, n], lambda stream: attn.decode_prefix(q, kp, vp, kc, vc, n, weights=w, stream=stream)[:2] + (w,)

    def evict():
        kc, vc, w, n = caches(30)
        out = dict(kcache=torch.zeros_like(kc), vcache=torch.zeros_like(vc))
        return [kc, vc, w, n], lambda stream: (attn.cache_evict(kc, vc, w, n, 100, 10, out=out, stream=stream)[0], *out.values())

    for make in (rope, append, decode, evict):
        want = make()[1](None)
        inputs, call = make()
        sizes = [(t.shape, t.dtype) for t in inputs if t is not f]
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
