"""Decode over a shared prefix, and the attention weights of the cached keys,
against the definition in 64 bits on the same bf16 inputs.

Tolerances, per element.  Scores are fp32 sums of d exact products: each is off
by at most e = d 2^-24 scale sum_i |q_i k_i| (taken at its largest over the
row's keys), to which exp2, the logarithms and the merge add a few units of
2^-22 (|L| + 1), E = e + 2^-20 (|L| + 1) in all.  Then
    lse    E
    weight 2 E p per head, one fp32 rounding of the running sum (2^-24)
    o      probabilities are rounded to bf16 for the product with V (half a
           step, 2^-8 of each), the result once more (2^-8 of it):
           (2^-8 + 2 E) sum_j p_j |v_j| + 2^-8 |o|."""
import math

import pytest
import torch

from synthetic_inputs import normal_bf16

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


def inputs(B, Hq, Hkv, P, S, d, seed, std=1.0):
    q = (normal_bf16((B, Hq, d), seed).float() * std).bfloat16().to(DEV)
    kp, vp = (normal_bf16((Hkv, P, d), seed + i, DEV) if P else None for i in (1, 2))
    kc, vc = (normal_bf16((B, Hkv, S, d), seed + i, DEV) if S else None for i in (3, 4))
    return q, kp, vp, kc, vc


def reference(q, kp, vp, kc, vc, lens, scale):
    """Per row: o, lse, weights of the own keys [B, Hkv, S], and the sizes that the tolerances need."""
    q = q.double().cpu()
    B, Hq, d = q.shape
    Hkv = (kp if kp is not None else kc).shape[0 if kp is not None else 1]
    G, S = Hq // Hkv, 0 if kc is None else kc.shape[2]
    o, av = torch.zeros(B, Hq, d, dtype=torch.float64), torch.zeros(B, Hq, d, dtype=torch.float64)
    lse, e = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    w, werr = torch.zeros(B, Hkv, S, dtype=torch.float64), torch.zeros(B, Hkv, S, dtype=torch.float64)
    wide = lambda t: t.double().cpu()
    kpw, vpw = (wide(kp), wide(vp)) if kp is not None else (None, None)
    for b in range(B):
        n = min(max(lens[b], 0), S) if S else 0
        for g in range(Hkv):
            k = [kpw[g]] if kp is not None else []
            v = [vpw[g]] if kp is not None else []
            if n:
                k.append(wide(kc[b, g, :n]))
                v.append(wide(vc[b, g, :n]))
            if not k:
                continue
            k, v = torch.cat(k), torch.cat(v)
            rows = slice(g * G, (g + 1) * G)
            s = q[b, rows] @ k.T * scale
            L = torch.logsumexp(s, -1)
            p = torch.exp(s - L[:, None])
            size = (q[b, rows].abs() @ k.T.abs()).amax(-1) * scale * d * 2.0 ** -24
            E = size + 2.0 ** -20 * (L.abs() + 1)
            o[b, rows], av[b, rows], lse[b, rows], e[b, rows] = p @ v, p @ v.abs(), L, E
            if n:
                w[b, g, :n] = p[:, -n:].sum(0)
                werr[b, g, :n] = (2 * E[:, None] * p[:, -n:]).sum(0)
    return o, lse, w, (STEP + 2 * e)[..., None] * av + STEP * o.abs(), e, werr


def run_and_check(attn, q, kp, vp, kc, vc, lens, scale=None, weighted=True, workspace=None):
    B, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    seq = None if kc is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    w = w0 = None
    if weighted and kc is not None:
        w0 = torch.rand((B, kc.shape[1], kc.shape[2]), generator=torch.Generator().manual_seed(5)) * 3
        w = w0.to(DEV)
    o, lse, ws = attn.decode_prefix(q, kp, vp, kc, vc, seq, scale=scale, weights=w, workspace=workspace)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_OK
    ro, rl, rw, to, e, tw = reference(q, kp, vp, kc, vc, lens, scale)
    err = (o.double().cpu() - ro).abs()
    assert torch.all(err <= to), f"o off by {float((err / to.clamp(min=1e-300)).max()):.3g} of the bound"
    lse = lse.double().cpu()
    none = torch.isinf(rl)
    assert torch.equal(none, torch.isinf(lse)) and torch.all(o.cpu()[none] == 0)
    assert torch.all((lse - rl)[~none].abs() <= e[~none])
    if w is not None:
        got, want = w.double().cpu(), w0.double() + rw
        assert torch.all((got - want).abs() <= tw + 2.0 ** -24 * want.abs())
        for b, n in enumerate(lens):  # entries behind the last key keep their bits
            n = min(max(n, 0), kc.shape[2])
            assert torch.equal(w[b, :, n:].cpu(), w0[b, :, n:])
    return o, lse, w, ws


def lens_for(B, S):
    edge = [S, 0, 1, S + 7, -2, max(1, S // 2), min(S, 65), max(0, S - 1)]
    g = torch.Generator().manual_seed(B + S)
    return (edge + torch.randint(0, S + 1, (B,), generator=g).tolist())[:B]


SHAPES = [
    # B, Hq, Hkv, P, S, d
    (1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 0, 128), (2, 2, 2, 0, 5, 64), (1, 8, 1, 127, 3, 128), (4, 8, 2, 128, 64, 64),
    (8, 8, 8, 129, 100, 128), (9, 10, 2, 700, 33, 64), (5, 28, 4, 1000, 257, 128), (3, 48, 3, 300, 1200, 128),
    (8, 32, 2, 0, 3000, 64), (8, 64, 8, 2500, 513, 128), (30, 40, 8, 333, 70, 128), (130, 10, 2, 400, 40, 64),
    (260, 16, 1, 515, 20, 128), (300, 4, 4, 200, 9, 64), (70, 12, 1, 140, 200, 128), (1, 64, 8, 0, 8000, 128),
    (2, 16, 2, 20000, 70, 64), (16, 64, 8, 6000, 90, 128), (3, 2, 1, 40001, 5, 128), (17, 8, 1, 25000, 300, 128),
]


@pytest.mark.parametrize("B,Hq,Hkv,P,S,d", SHAPES)
def test_against_the_definition(attn, B, Hq, Hkv, P, S, d):
    q, kp, vp, kc, vc = inputs(B, Hq, Hkv, P, S, d, 100)
    run_and_check(attn, q, kp, vp, kc, vc, lens_for(B, S))


def test_more_row_units_than_fit_side_by_side(attn):
    """So many rows that the work is cut unit by unit instead of in lockstep."""
    B, Hq, Hkv, P, S, d = 2000, 16, 1, 260, 2, 64
    q, kp, vp, kc, vc = inputs(B, Hq, Hkv, P, S, d, 110)
    run_and_check(attn, q, kp, vp, kc, vc, lens_for(B, S))


@pytest.mark.parametrize("d", [64, 128])
def test_peaked_scores(attn, d):
    """Scores of hundreds: the running maximum moves, most weights vanish, the largest are near 1."""
    q, kp, vp, kc, vc = inputs(6, 16, 2, 600, 300, d, 120, std=40.0)
    run_and_check(attn, q, kp, vp, kc, vc, lens_for(6, 300))


def test_scale_and_no_weights(attn):
    q, kp, vp, kc, vc = inputs(4, 8, 4, 200, 50, 64, 130)
    seq = torch.tensor([50, 3, 0, 20], dtype=torch.int32, device=DEV)
    o, lse, w, _ = run_and_check(attn, q, kp, vp, kc, vc, seq.tolist(), scale=0.31)
    o2, none, _ = attn.decode_prefix(q, kp, vp, kc, vc, seq, scale=0.31, with_lse=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("P", [0, 300])
def test_what_lies_behind_the_last_key_does_not_matter(attn, P):
    """NaN and infinities in the cache behind each sequence's last key, and a workspace full of NaN."""
    B, Hq, Hkv, S, d = 5, 8, 2, 200, 128
    q, kp, vp, kc, vc = inputs(B, Hq, Hkv, P, S, d, 140)
    lens = [0, 1, 63, 130, 200]
    for b, n in enumerate(lens):
        kc[b, :, n:] = math.nan
        vc[b, :, n:] = math.inf
    ws = torch.full((attn.attn_decode_prefix_workspace_bytes(B, Hq, Hkv, P, d, S, True) // 4,), math.nan, device=DEV)
    run_and_check(attn, q, kp, vp, kc, vc, lens, workspace=ws)


def test_agrees_with_decode_and_with_a_copied_prefix(attn):
    """Without a prefix: attn_decode's result.  With one: that of caches into which the prefix was copied."""
    B, Hq, Hkv, P, S, d = 6, 16, 4, 777, 100, 128
    q, kp, vp, kc, vc = inputs(B, Hq, Hkv, P, S, d, 150)
    lens = [100, 1, 50, 0, 99, 64]
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    whole_k = torch.cat((kp[None].expand(B, -1, -1, -1), kc), 2).contiguous()
    whole_v = torch.cat((vp[None].expand(B, -1, -1, -1), vc), 2).contiguous()
    o, _, _ = attn.decode_prefix(q, kp, vp, kc, vc, seq)
    o1, _, _ = attn.decode_prefix(q, None, None, whole_k, whole_v, seq + P)
    o2, _, _ = attn.decode(q, whole_k, whole_v, seq + P)
    _, _, _, tol, _, _ = reference(q, kp, vp, kc, vc, lens, d ** -0.5)
    for other in (o1, o2):
        assert torch.all((o.double() - other.double()).abs().cpu() <= 2 * tol)


def test_equal_calls_give_equal_bits_and_graphs_share_a_workspace(attn):
    """Two captured steps on one workspace, replayed in turn with the lengths and queries that the buffers hold then."""
    B, Hq, Hkv, P, S, d = 6, 16, 2, 500, 300, 128
    q, kp, vp, kc, vc = inputs(B, Hq, Hkv, P, S, d, 160)
    w = torch.zeros((B, Hkv, S), device=DEV)
    seq = torch.tensor(lens_for(B, S), dtype=torch.int32, device=DEV)
    n = max(attn.attn_decode_prefix_workspace_bytes(B, Hq, Hkv, p, d, S, True) for p in (0, P))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    steps = [lambda: attn.decode_prefix(q, kp, vp, kc, vc, seq, weights=w, workspace=ws)[:2],
             lambda: attn.decode_weighted(q, kc, vc, seq, w, workspace=ws)[:2]]
    for s in steps:
        s()
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s()
        graphs.append((g, out))
    gen = torch.Generator().manual_seed(6)
    for i in range(3):
        q.copy_(normal_bf16(q.shape, 170 + i, DEV))
        seq.copy_(torch.randint(0, S + 1, (B,), generator=gen).int())
        for (g, out), s in zip(graphs, steps):
            w.fill_(0.5)
            g.replay()
            torch.cuda.synchronize()
            kept, counted = [t.clone() for t in out], w.clone()
            w.fill_(0.5)
            o, lse = s()
            assert torch.equal(kept[0], o) and torch.equal(kept[1], lse) and torch.equal(counted, w)
    assert attn.attn_device_status() == attn.ATTN_OK


def test_two_streams_at_once(attn):
    B, Hq, Hkv, P, S, d = 8, 32, 4, 3000, 500, 128
    a, b = inputs(B, Hq, Hkv, P, S, d, 180), inputs(B, Hq, Hkv, P, S, d, 190)
    seq = torch.tensor(lens_for(B, S), dtype=torch.int32, device=DEV)
    want = [attn.decode_prefix(*x, seq)[0] for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[attn.decode_prefix(*x, seq, stream=s)[0] for x, s in zip((a, b), streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_caches_past_two_to_the_31_elements(attn):
    """The last entry of a cache of more than 2^31 elements, at its end, and its scores past 2^31 bytes."""
    B, Hq, Hkv, S, d = 3, 16, 1, 8 << 20, 128
    kc = torch.zeros((B, Hkv, S, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    q = normal_bf16((B, Hq, d), 200, DEV)
    kc[2, :, S - 300:] = normal_bf16((Hkv, 300, d), 201, DEV) * 4
    vc[2, :, S - 300:] = normal_bf16((Hkv, 300, d), 202, DEV)
    seq = torch.tensor([0, 1, S], dtype=torch.int32, device=DEV)
    w = torch.zeros((B, Hkv, S), device=DEV)
    o, lse, _ = attn.decode_weighted(q, kc, vc, seq, w)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_OK
    s = q[2].double() @ kc[2, 0, S - 300:].double().T * d ** -0.5
    L = torch.logsumexp(torch.cat((s, torch.tensor(float(S - 300)).log().double().to(DEV).expand(Hq, 1)), 1), -1)
    p = torch.exp(s - L[:, None])
    E = float((q[2].double().abs() @ kc[2, 0, S - 300:].double().abs().T).max()) * d ** -0.5 * d * 2.0 ** -24
    E += 2.0 ** -20 * (float(L.abs().max()) + 1) + 2.0 ** -24 * 1e3  # sums of up to 2^23 equal terms in chunks
    assert float((lse[2].double() - L).abs().max()) <= E
    v = vc[2, 0, S - 300:].double()
    tol = (STEP + 2 * E) * (p @ v.abs()) + STEP * (p @ v).abs()
    assert torch.all((o[2].double() - p @ v).abs() <= tol)
    assert torch.all((w[2, 0, S - 300:].double() - p.sum(0)).abs() <= 2 * E * p.sum(0) + 1e-30)
    assert float(w[1, 0, 0]) == pytest.approx(Hq, rel=1e-5) and not w[0].any() and not w[1, 0, 1:].any()
    del kc, vc, w
    torch.cuda.empty_cache()


def test_more_than_two_to_the_29_keys_in_the_caches(attn):
    """Lengths are then scanned in 64 bits; K and V are one tensor, and most of it is never read."""
    B, Hq, Hkv, S, d = 600, 2, 1, (1 << 29) // 600 + 1, 64
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    kc = torch.empty((B, Hkv, S, d), dtype=torch.bfloat16, device=DEV)
    kc[:, :, :512] = normal_bf16((B, Hkv, 512, d), 203, DEV)
    q = normal_bf16((B, Hq, d), 204, DEV)
    kp, vp = (normal_bf16((Hkv, 200, d), 205 + i, DEV) for i in range(2))
    lens = torch.randint(-3, 70, (B,), generator=torch.Generator().manual_seed(206)).tolist()
    lens[300], lens[-1] = 512, 511
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    w = torch.zeros((B, Hkv, S), device=DEV)
    o, lse, _ = attn.decode_prefix(q, kp, vp, kc, kc, seq, weights=w)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_OK
    near = kc[:, :, :512]
    ro, rl, rw, to, e, tw = reference(q, kp, vp, near, near, lens, d ** -0.5)
    assert torch.all((o.double().cpu() - ro).abs() <= to)
    assert torch.all((lse.double().cpu() - rl).abs() <= e)
    assert torch.all((w[:, :, :512].double().cpu() - rw).abs() <= tw + 2.0 ** -24 * rw)
    assert not w[:, :, 512:].any()
    del kc, near, w
    torch.cuda.empty_cache()


@pytest.mark.parametrize("G,d", [(1, 64), (4, 128), (8, 64), (16, 128)])
def test_scores_of_minus_infinity(attn, G, d):
    """Keys whose score is -inf add nothing; a sequence with no others gets o = 0, lse = -inf and no weight."""
    B, Hkv, S = 3, 2, 300
    q, _, _, kc, vc = inputs(B, G * Hkv, Hkv, 0, S, d, 230)
    q[..., 0] = 1
    gone = torch.zeros(B, S, dtype=torch.bool)
    gone[0] = True
    gone[1, torch.randperm(S, generator=torch.Generator().manual_seed(231))[:200]] = True
    kc[:, :, :, 0] = torch.where(gone.to(DEV)[:, None], -math.inf, kc[:, :, :, 0].float()).bfloat16()
    seq = torch.tensor([S, S, S], dtype=torch.int32, device=DEV)
    w = torch.ones((B, Hkv, S), device=DEV)
    o, lse, _ = attn.decode_weighted(q, kc, vc, seq, w)
    torch.cuda.synchronize()
    assert attn.attn_device_status() == attn.ATTN_OK
    assert torch.all(o[0] == 0) and torch.all(lse[0] == -math.inf)
    assert torch.all(w.cpu()[gone[:, None].expand(B, Hkv, S)] == 1)
    for b in (1, 2):
        left = (~gone[b]).nonzero()[:, 0].to(DEV)
        n = len(left)
        ro, rl, rw, to, e, tw = reference(q[b:b + 1], None, None, kc[b:b + 1, :, left], vc[b:b + 1, :, left], [n], d ** -0.5)
        assert torch.all((o[b].double().cpu() - ro[0]).abs() <= to[0])
        assert torch.all((lse[b].double().cpu() - rl[0]).abs() <= e[0])
        assert torch.all((w[b][:, left].double().cpu() - 1 - rw[0]).abs() <= tw[0] + 2.0 ** -24 * (1 + rw[0]))


def test_wait_limit_is_reported_and_recovered(attn):
    q, kp, vp, kc, vc = inputs(4, 16, 2, 3000, 1500, 128, 210)
    lens = [1500, 0, 17, 900]
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    old = attn.attn_set_wait_timeout_ns(0)
    try:
        attn.decode_prefix(q, kp, vp, kc, vc, seq)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_TIMEOUT
    finally:
        attn.attn_set_wait_timeout_ns(old)
    run_and_check(attn, q, kp, vp, kc, vc, lens)


@pytest.mark.parametrize("B,Hq,Hkv,P,S,d", [
    (4, 16, 2, 3000, 1500, 128), (300, 8, 1, 700, 20, 64), (2, 8, 2, 900, 0, 128), (3, 8, 8, 0, 700, 64), (64, 64, 8, 4000, 90, 128),
])
def test_a_launch_that_gave_up_stays_in_bounds(attn, B, Hq, Hkv, P, S, d):
    """With no time to wait the phases leave early.  What the merge and the weights
    read out of the workspace as numbers and positions is there all the same."""
    q, kp, vp, kc, vc = inputs(B, Hq, Hkv, P, S, d, 240)
    lens = lens_for(B, S) if S else []
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV) if S else None
    w = torch.zeros((B, Hkv, S), device=DEV) if S else None
    ws = torch.full((attn.attn_decode_prefix_workspace_bytes(B, Hq, Hkv, P, d, S, bool(S)),), 0x7f, dtype=torch.uint8, device=DEV)
    old = attn.attn_set_wait_timeout_ns(0)
    try:
        attn.decode_prefix(q, kp, vp, kc, vc, seq, weights=w, workspace=ws)
        torch.cuda.synchronize()
        assert attn.attn_device_status() == attn.ATTN_ERR_TIMEOUT
    finally:
        attn.attn_set_wait_timeout_ns(old)
    run_and_check(attn, q, kp, vp, kc, vc, lens, workspace=ws)


def test_helper_refusals(attn):
    q, kp, vp, kc, vc = inputs(2, 8, 2, 100, 16, 64, 220)
    seq = torch.tensor([1, 2], dtype=torch.int32, device=DEV)
    small = torch.empty(64, dtype=torch.uint8, device=DEV)
    for call, code in [
        (lambda: attn.decode_prefix(q, kp, vp, kc, vc, seq.long()), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, vp, kc.transpose(2, 3), vc, seq), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp[:, ::2], vp, kc, vc, seq), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp[:1], vp[:1], kc, vc, seq), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, vp, kc, vc, seq.cpu()), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q.half(), kp, vp, kc, vc, seq), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, vp, None, None, None, weights=kc), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, vp, kc, vc, seq, workspace=small), attn.ATTN_ERR_WORKSPACE),
        (lambda: attn.decode_prefix(q, kp, vp, kc, vc, seq, scale=-1.0), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, None, kc, vc, seq), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, vp, None, vc, seq), attn.ATTN_ERR_ARG),
        (lambda: attn.decode_prefix(q, kp, vp, kc, vc, None), attn.ATTN_ERR_ARG),
    ]:
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == code
