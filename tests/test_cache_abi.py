"""CPU-only checks of the decode-cache entry points (rotary positions,
shared-prefix decode, eviction): refusals come from the host before any CUDA
call, the host-side rules agree with their definitions, and the torch helpers
refuse tensors whose addresses alone would not tell.  No kernel runs."""
import ctypes
import math

import pytest
import torch

import attention_fa2_fwd_sm_gb300 as attn
from attention_fa2_fwd_sm_gb300 import _build

A16 = 0x10000  # a fake 16-byte-aligned address: never dereferenced by these calls
ARG, UNSUP, WS = attn.ATTN_ERR_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    attn.lib()


def strides(*v):
    return (ctypes.c_longlong * 12)(*v)


PACKED = (2 * 16 * 64, 16 * 64, 64)  # B = 3, H = 2, N = 16, d = 64


def _rope(**kw):
    a = dict(q=A16, q_out=A16 + 4096, k=A16 + 8192, k_out=A16 + 16384, pos=None, pos_stride=0, freqs=A16, B=3, Hq=2,
             Hkv=2, N=16, d=64, r=64, inter=0, scale=1.0, inverse=0, strides=None)
    a.update(kw)
    return attn.attn_rope(*a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(q=A16 + 8), ARG), (dict(q_out=None), ARG), (dict(k_out=None), ARG), (dict(k=None), ARG),
    (dict(k_out=A16 + 2), ARG), (dict(B=0), ARG), (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(N=-1), ARG),
    (dict(N=0), ARG), (dict(pos=A16 + 2), ARG), (dict(pos_stride=-1), ARG), (dict(freqs=None), ARG),
    (dict(freqs=A16 + 4), ARG), (dict(r=0), ARG), (dict(r=63), ARG), (dict(r=66), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(d=60, r=32), UNSUP), (dict(d=0), UNSUP),
    (dict(d=520, r=64), UNSUP),
    (dict(strides=strides(*PACKED, *PACKED, *PACKED, PACKED[0], PACKED[1], 60)), ARG),   # not a multiple of 8
    (dict(strides=strides(*PACKED, PACKED[0], PACKED[1], 0, *PACKED, *PACKED)), ARG),    # an output laid over itself
    (dict(strides=strides(-8, 64, 64, *PACKED, *PACKED, *PACKED)), ARG),
    (dict(strides=strides(1 << 40, 64, 64, *PACKED, *PACKED, *PACKED)), ARG),
    (dict(q_out=A16, strides=strides(*PACKED, 2 * PACKED[0], PACKED[1], 64, *PACKED, *PACKED)), ARG),  # in place, moved
    (dict(q_out=A16 + 8192), ARG), (dict(k_out=A16), ARG), (dict(k_out=A16 + 4096), ARG),     # one tensor laid over another
])
def test_rope_refusals(kw, code):
    assert _rope(**kw) == code


KC, VC = A16 + (1 << 20), A16 + (2 << 20)


def _append(**kw):
    a = dict(q=A16, q_out=A16 + 4096, k=A16 + 8192, v=A16 + 16384, kc=KC, vc=VC, lens=A16, start=None, new=None, out=A16 + 64,
             cache_pos=None, weights=None, freqs=A16, B=3, Hq=2, Hkv=2, T=1, d=64, r=64, inter=0, scale=1.0, S=16,
             strides=None)
    a.update(kw)
    return attn.attn_rope_append(*a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(k=A16 + 8), ARG), (dict(v=None), ARG), (dict(kc=None), ARG), (dict(vc=KC), ARG),
    (dict(vc=VC + 4), ARG), (dict(k=KC), ARG), (dict(v=KC), ARG), (dict(v=VC), ARG), (dict(q=KC), ARG), (dict(q_out=VC), ARG),
    (dict(q_out=A16 + 8192), ARG), (dict(q_out=A16 + 16384), ARG), (dict(lens=None), ARG), (dict(lens=A16 + 1), ARG), (dict(out=A16), ARG),
    (dict(out=A16 + 8), ARG), (dict(start=A16 + 64), ARG), (dict(new=A16 + 72), ARG), (dict(cache_pos=A16 + 2), ARG),
    (dict(weights=A16 + 3), ARG), (dict(S=0), ARG), (dict(T=0), ARG), (dict(Hkv=0), ARG), (dict(r=-2), ARG),
    (dict(r=64, freqs=None), ARG), (dict(r=130, d=128), ARG), (dict(d=12), UNSUP), (dict(scale=-float("inf")), ARG),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


@pytest.mark.parametrize("s", [
    (1024, 1024, 64), (1024, 64, 64), (64, 1024, 64), (1024, 64, 1024), (960, 2048, 64), (2048, 1000, 64), (1032, 512, 32)])
def test_outputs_laid_over_themselves_are_refused(s):
    """B = 3, H = 2, N = 16 (T = 16 with a cache of 40 rows), d = 64."""
    assert _rope(q_out=1 << 26, k=None, k_out=None, strides=strides(*PACKED, *s, *PACKED, *PACKED)) == ARG
    assert _rope(q_out=1 << 25, k_out=1 << 26, strides=strides(*PACKED, *PACKED, *PACKED, *s)) == ARG
    assert _append(q_out=1 << 26, T=16, S=40, kc=1 << 27, vc=1 << 28, v=A16 + (1 << 20), strides=strides(*PACKED, *s, *PACKED, *PACKED)) == ARG


CACHE_ROWS = (2 * 16 * 64, 16 * 64, 64)  # strides of a [3, 2, T, 64] view of a cache of 16 rows
NEW = (2 * 64, 64, 0)                    # those of [3, 2, 1, 64] tokens


@pytest.mark.parametrize("kw", [
    dict(q_out=A16 + 2048), dict(k_out=A16 + 128), dict(q_out=A16 + 8192 - 4096), dict(k_out=A16 + 12288 - 128),  # one row in the other
    # q_out in the rows of q one token further; k_out in a gap of k that is too narrow for it
    dict(q_out=A16 + 128, strides=strides(*PACKED, *PACKED, *PACKED, *PACKED)),
    dict(q=A16, q_out=1 << 24, k=A16 + 2048, k_out=A16 + 2048 + 64,
         strides=strides(4 * 64 * 16, 64, 4 * 64, *PACKED, 4 * 64 * 16, 64, 4 * 64, 4 * 64 * 16, 64, 4 * 64)),
])
def test_rope_refuses_partial_overlaps(kw):
    """[3, 2, 16, 64] tensors are 12288 bytes; these share some of their rows."""
    assert _rope(**dict(dict(q=A16, q_out=1 << 24, k=1 << 25, k_out=1 << 26), **kw)) == ARG


@pytest.mark.parametrize("kw", [
    # tokens that lie in a cache: its rows 3.., the last one's last element, the other cache
    dict(k=KC + 3 * 128, strides=strides(*NEW, *NEW, *CACHE_ROWS, *NEW)), dict(v=KC + 3 * 128, strides=strides(*NEW, *NEW, *NEW, *CACHE_ROWS)),
    dict(k=VC + 5 * 128, strides=strides(*NEW, *NEW, *CACHE_ROWS, *NEW)), dict(k=KC + 3 * 2 * 16 * 128 - 128), dict(q=VC - 640),
    dict(q_out=KC + 128), dict(vc=KC + 3 * 2 * 16 * 128 - 16), dict(kc=VC + 16),  # the caches in each other
    dict(q_out=A16 + 8192 + 128), dict(q_out=A16 + 16384 - 128), dict(q_out=A16 + 128),
])
def test_append_refuses_partial_overlaps(kw):
    """Caches [3, 2, 16, 64] are 12288 bytes, new tokens [3, 2, 1, 64] 768."""
    assert _append(**kw) == ARG


def test_frequency_rules():
    r, base, L = 64, 10000.0, 4096.0
    plain = [base ** (-2 * i / r) for i in range(r // 2)]
    close = lambda a, b: all(math.isclose(x, y, rel_tol=1e-14) for x, y in zip(a, b)) and len(a) == len(b)
    assert close(attn.attn_rope_freqs(r, base), plain)
    assert close(attn.attn_rope_freqs(r, base, 1, 8.0), [f / 8 for f in plain])
    stretched = attn.attn_rope_freqs(r, base, 2, 8.0)
    assert stretched[0] == 1.0 and math.isclose(stretched[-1], plain[-1] / 8, rel_tol=1e-12)
    parts = attn.attn_rope_freqs(r, base, 3, 8.0, 1.0, 4.0, L)
    want = []
    for f in plain:
        g = min(max((L * f / (2 * math.pi) - 1) / 3, 0.0), 1.0)
        want.append(f * (g + (1 - g) / 8))
    assert close(parts, want) and parts[0] == plain[0] and math.isclose(parts[-1], plain[-1] / 8, rel_tol=1e-14)


@pytest.mark.parametrize("args", [
    (0,), (7,), (64, 1.0), (64, float("nan")), (64, 1e4, 4), (64, 1e4, -1), (64, 1e4, 1, 0.0), (64, 1e4, 1, float("inf")),
    (2, 1e4, 2, 8.0), (64, 1e4, 3, 8.0, 4.0, 1.0), (64, 1e4, 3, 8.0, 1.0, 4.0, 0.0)])
def test_frequency_refusals(args):
    with pytest.raises(attn.AttnError) as e:
        attn.attn_rope_freqs(*args)
    assert e.value.code == ARG


def test_rope_helpers_refuse_what_an_address_does_not_tell():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    f = z(32, dtype=torch.float64)
    for call in (lambda: attn.rope(z(1, 2, 3, 64), None, f),                       # on the CPU
                 lambda: attn.rope(z(2, 3, 64), None, f),
                 lambda: attn.rope(z(1, 2, 3, 64, dtype=torch.float16), None, f),
                 lambda: attn.rope_append(z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 9, 64), z(1, 2, 9, 64),
                                          z(1, dtype=torch.int32), f),
                 lambda: attn.rope_append(z(1, 2, 64), None, None, z(1, 2, 9, 64), None, None)):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == ARG


# ------------------------------------------------------ shared-prefix decode
def _prefix(**kw):
    a = dict(q=A16, kp=A16, vp=A16, kc=A16, vc=A16, lens=A16, o=A16, lse=None, w=None, B=2, Hq=4, Hkv=2, P=100, d=64,
             scale=0.125, S=32, ws=A16, nbytes=1 << 40)
    a.update(kw)
    return attn.attn_decode_prefix(*a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(q=A16 + 8), ARG), (dict(o=None), ARG), (dict(kp=None), ARG), (dict(vp=A16 + 2), ARG),
    (dict(kc=None), ARG), (dict(vc=A16 + 8), ARG), (dict(lens=None), ARG), (dict(lens=A16 + 2), ARG),
    (dict(lse=A16 + 1), ARG), (dict(w=A16 + 2), ARG), (dict(w=A16, S=0), ARG), (dict(P=0, S=0), ARG), (dict(P=-1), ARG),
    (dict(S=-1), ARG), (dict(B=0), ARG), (dict(Hq=3), ARG), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(d=56), UNSUP), (dict(d=256), UNSUP), (dict(Hq=34, Hkv=2), UNSUP), (dict(ws=None), WS), (dict(ws=A16 + 8), WS),
    (dict(P=0, kp=None, vp=None, kc=None), ARG), (dict(S=0, kc=None, vc=None, lens=None, ws=None), WS),
    (dict(P=(1 << 30) + 1), ARG), (dict(S=(1 << 30) + 1), ARG), (dict(B=(1 << 28) + 1, Hq=4, Hkv=4), ARG),
])
def test_decode_prefix_refusals(kw, code):
    assert _prefix(**kw) == code


@pytest.mark.parametrize("sms", [152, 8, 1])
@pytest.mark.parametrize("S,keys", [(0, 0), (1000, 0), (1000, 1.0), (1000, 0.3), (50000, 1.0)])
@pytest.mark.parametrize("B,Hq,Hkv,P,d", [
    (1, 1, 1, 1, 64), (1, 8, 1, 129, 128), (4, 8, 2, 500, 64), (32, 64, 8, 8192, 128), (128, 64, 8, 32768, 128),
    (7, 40, 8, 5001, 128), (300, 16, 16, 1000, 64), (2000, 64, 4, 700, 64), (1000, 15, 1, 257, 128), (5000, 16, 1, 300, 128)])
def test_prefix_segments_cover_every_block_once(B, Hq, Hkv, P, d, S, keys, sms):
    """Whatever the own keys' number: every (KV head, unit, key block) belongs to one segment; a unit's partials are numbered
    without gaps up to the one that every segment names as the last; no two segments of a unit share a number."""
    G, nblk = Hq // Hkv, -(-P // 128)
    units = (-(-B // (128 // G)) + 1) // 2
    seen, numbers, last, load = {}, {}, {}, []
    cta = 0
    while True:
        mine, i = 0, 0
        try:
            while (s := attn.attn_decode_prefix_segment(B, Hq, Hkv, P, d, S, int(keys * B * S), sms, cta, i)) is not None:
                g, m, j0, n, part, end = s
                assert n > 0 and 0 <= g < Hkv and 0 <= m < units and j0 + n <= nblk
                for j in range(j0, j0 + n):
                    assert (g, m, j) not in seen
                    seen[g, m, j] = cta
                numbers.setdefault((g, m), []).append(part)
                assert last.setdefault((g, m), end) == end
                mine, i = mine + n, i + 1
        except attn.AttnError:
            break
        load.append(mine)
        cta += 1
    assert 0 < cta <= max(sms, units)
    assert len(seen) == Hkv * units * nblk
    for unit, parts in numbers.items():
        assert sorted(parts) == list(range(min(parts), last[unit] + 1))
    assert len({(p, u[1]) for u, parts in numbers.items() for p in parts}) == sum(map(len, numbers.values()))
    if S == 0:  # nothing beside it: equal shares
        assert max(load) <= -(-Hkv * units * nblk // max(1, int(0.9 * sms))) + units


def test_prefix_shares_leave_room_for_the_own_keys():
    """The more own keys, the less falls to the CTAs that start behind them; all CTAs at or above some number start behind them."""
    loads = []
    for own in (0, 20000, 60000, 100000, 10 ** 7):
        load = []
        for cta in range(152):
            n = i = 0
            while (s := attn.attn_decode_prefix_segment(128, 64, 8, 32768, 128, 1024, own, 152, cta, i)) is not None:
                n, i = n + s[3], i + 1
            load.append(n)
        loads.append(load)
    late = [sum(x[120:]) for x in loads]
    assert late == sorted(late, reverse=True) and late[0] > late[1] > 0 and late[-1] == 0
    assert len({n for n in loads[0][:148]}) == 1  # nothing own: equal shares (the last one takes the rest)
    assert all(sum(x) == 4 * 8 * 256 for x in loads)


OWN_US = {(128, False): (2.0, 0.0112), (128, True): (3.0, 0.0127), (64, False): (1.4, 0.0074), (64, True): (1.7, 0.0097)}


def test_own_keys_get_the_sms_that_they_need(tmp_path):
    """Beside a prefix the own keys' kernel gets its SMs from the sizes.  A group of one of its CTAs takes OWN_US (measured on
    its own) for a row and for each key of it; at caches three quarters full that must not outlast the
    prefix's work on the SMs that it starts on (which takes up to twice as long beside own keys at
    HBM's rate), however short the caches are and however the prefix's groups divide the GPU."""
    import os
    import subprocess
    src, exe = tmp_path / "sms.cpp", tmp_path / "sms"
    csrc = os.path.join(os.path.dirname(attn.__file__), "csrc")
    src.write_text('#include <cstdio>\n#include "prefix_order.cuh"\nint main() {\n    int B, G, H, P, d, S, most;\n'
                   '    while (scanf("%d%d%d%d%d%d%d", &B, &G, &H, &P, &d, &S, &most) == 7)\n'
                   '        printf("%d\\n", attn::prefix_own_sms(B, G, H, P, d, S, most, 152));\n}\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", csrc, str(src), "-o", str(exe)], check=True)
    cases = [(B, G, H, P, d, S) for B in (4, 16, 32, 64, 128, 300, 512, 1216, 2000) for G in (1, 8, 16) for H in (2, 8)
             for P in (8192, 16384, 32768) for d in (64, 128) for S in (1, 16, 32, 40, 45, 48, 64, 128, 256, 1024)]
    most = lambda B, G, H, S: min(152, -(-B * H * S // (32 * (2 if G > 8 else 3))))
    lines = [" ".join(map(str, (*c, most(c[0], c[1], c[2], c[5])))) for c in cases]
    out = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True, check=True).stdout.split()
    assert len(out) == len(cases)
    for (B, G, H, P, d, S), sms in zip(cases, map(int, out)):
        tiles = -(-B // (128 // G))
        mt = (tiles + 1) // 2
        row, key = OWN_US[d, G > 8]
        own = B * H * (row + key * 0.75 * S) / (2 if G > 8 else 3) / sms
        block = (1.37 if tiles > 1 else 1.0) if d == 64 else 1.55 if tiles > 1 else 1.2
        lockstep = 10 * (152 // mt) * mt >= 9 * 152 if mt <= 152 else False
        start = 152 - sms
        if lockstep and start // mt == 1 or start <= 1 or sms >= most(B, G, H, S):
            continue  # one group of the prefix is left, or every share of the own keys has a group
        prefix = H * mt * -(-P // 128) * block / (start // mt * mt if lockstep else start)
        assert own <= 2 * prefix, (B, G, H, P, d, S, sms, own, prefix)


def test_prefix_segment_refusals():
    ok = dict(B=2, Hq=4, Hkv=2, P=100, d=128, S=10, own=5, sms=152, cta=0, i=0)
    assert attn.attn_decode_prefix_segment(*ok.values()) == (0, 0, 0, 1, 0, 0)
    for kw in (dict(B=0), dict(P=0), dict(sms=0), dict(cta=-1), dict(cta=152), dict(i=-1), dict(own=-1), dict(d=96), dict(S=-1)):
        with pytest.raises(attn.AttnError):
            attn.attn_decode_prefix_segment(*dict(ok, **kw).values())


def test_decode_helpers_refuse_what_an_address_does_not_tell():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    n = z(1, dtype=torch.int32)
    for call in (lambda: attn.decode_prefix(z(1, 2, 64), z(2, 5, 64), z(2, 5, 64), z(1, 2, 9, 64), z(1, 2, 9, 64), n),
                 lambda: attn.decode_weighted(z(1, 2, 64), z(1, 2, 9, 64), z(1, 2, 9, 64), n, z(1, 2, 9))):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == ARG


# ----------------------------------------------------------------- eviction
def _evict(**kw):
    M = 1 << 24  # far apart: nothing overlaps
    a = dict(kc=M, vc=2 * M, w=3 * M, pos=4 * M, lens=A16, cur=None, ko=M, vo=2 * M, wo=3 * M, po=4 * M, lo=A16 + 64,
             B=2, Hkv=2, d=64, S=512, So=512, keep=100, recent=10, ws=A16, nbytes=1 << 30)
    a.update(kw)
    return attn.attn_cache_evict(*a.values(), stream=0)


OUT = dict(ko=5 << 24, vo=6 << 24, wo=7 << 24, po=8 << 24)


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), ARG), (dict(vc=8), ARG), (dict(w=None), ARG), (dict(lens=None), ARG), (dict(lens=A16 + 1), ARG),
    (dict(cur=A16 + 2), ARG), (dict(lo=A16), ARG), (dict(lo=A16 + 4), ARG), (dict(cur=A16 + 64), ARG), (dict(B=0), ARG),
    (dict(S=0), ARG), (dict(keep=0), ARG), (dict(keep=513), ARG), (dict(recent=101), ARG), (dict(recent=-1), ARG),
    (dict(d=60), UNSUP), (dict(d=520), UNSUP), (dict(So=600), ARG), (dict(vo=9 << 24), ARG), (dict(wo=None), ARG),
    (dict(po=None), ARG), (dict(S=(1 << 30) + 1, So=(1 << 30) + 1), ARG), (dict(ws=None), WS), (dict(ws=A16 + 8), WS),
    (dict(nbytes=64), WS),
    (dict(OUT, vo=5 << 24), ARG), (dict(OUT, ko=(1 << 24) + 4096), ARG), (dict(OUT, wo=3 << 24), ARG),
    (dict(OUT, po=(7 << 24) + 64), ARG), (dict(OUT, nbytes=64), WS),
])
def test_evict_refusals(kw, code):
    assert _evict(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(vc=(1 << 24) + 4096, vo=(1 << 24) + 4096), dict(vc=(1 << 24) - 262144 + 16, vo=(1 << 24) - 262144 + 16),
    dict(w=(1 << 24) + 64, wo=(1 << 24) + 64), dict(pos=(2 << 24) + 64, po=(2 << 24) + 64), dict(pos=(3 << 24) + 8188, po=(3 << 24) + 8188)])
def test_evict_refuses_partial_overlaps_in_place(kw):
    """Caches of [2, 2, 512, 64] are 262144 bytes, weights and positions 8192."""
    assert _evict(**kw) == ARG


def test_evict_workspace():
    ws = attn.attn_cache_evict_workspace_bytes
    assert ws(2, 2, 164, 100, True) == 0 and ws(2, 2, 165, 100, True) > 0  # few slots past the kept ones: one kernel
    assert ws(2, 2, 164, 100, False) >= 4 * 4 * (100 + 64)  # a source for every slot, and the fillers
    assert ws(0, 2, 300, 100, True) == ws(2, 0, 300, 100, True) == ws(2, 2, 0, 100, True) == ws(2, 2, 300, 0, True) == 0
    assert ws(2, 2, 80, 100, False) >= 4 * 4 * 80  # a cache below the bound is only copied
