"""CPU-only checks of the entry points of the paged cache and of drafted tokens:
refusals come from the host before any CUDA call, and the torch helpers refuse
tensors whose addresses alone would not tell.  No kernel runs."""
import ctypes

import pytest
import torch

import attention_fa2_fwd_sm_gb300 as attn
from attention_fa2_fwd_sm_gb300 import _build

A16 = 0x10000  # a fake 16-byte-aligned address: never dereferenced by these calls
ARG, UNSUP, WS = attn.ATTN_ERR_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_WORKSPACE
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    attn.lib()


def _axes(**kw):
    a = dict(q=A16, q_out=A16 + MB, k=A16 + 2 * MB, k_out=A16 + 3 * MB, pos=A16, axis_stride=48, pos_stride=16, A=2, freqs=A16,
             axes=A16, B=3, Hq=2, Hkv=2, N=16, d=64, r=64, inter=0, scale=1.0, inverse=0, strides=None)
    a.update(kw)
    return attn.attn_rope_axes(*a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ARG), (dict(q=A16 + 8), ARG), (dict(q_out=None), ARG), (dict(k_out=None), ARG), (dict(k=None), ARG),
    (dict(pos=None), ARG), (dict(pos=A16 + 2), ARG), (dict(axis_stride=-1), ARG), (dict(pos_stride=-1), ARG), (dict(A=0), ARG),
    (dict(A=5), ARG), (dict(axes=A16 + 1), ARG), (dict(freqs=None), ARG), (dict(freqs=A16 + 4), ARG), (dict(B=0), ARG),
    (dict(Hq=0), ARG), (dict(Hkv=0), ARG), (dict(N=0), ARG), (dict(r=0), ARG), (dict(r=63), ARG), (dict(r=66), ARG),
    (dict(scale=float("nan")), ARG), (dict(d=60, r=32), UNSUP), (dict(d=520), UNSUP), (dict(q_out=A16 + 2 * MB), ARG),
    (dict(k_out=A16 + MB), ARG),
    (dict(strides=(ctypes.c_longlong * 12)(2048, 1024, 64, 2048, 1024, 60, *(2048, 1024, 64) * 2)), ARG),
])
def test_rope_axes_refusals(kw, code):
    assert _axes(**kw) == code


KP, VP = A16 + 16 * MB, A16 + 64 * MB


def _append(**kw):
    a = dict(q=A16, q_out=A16 + MB, k=A16 + 2 * MB, v=A16 + 3 * MB, kp=KP, vp=VP, table=A16 + 4 * MB, lens=A16, pos=None,
             axis_stride=0, pos_stride=0, A=1, new=None, out=A16 + 64, freqs=A16, axes=None, B=3, Hq=2, Hkv=2, T=1, d=64, r=64,
             inter=0, scale=1.0, pages=20, page=16, per=4, strides=None)
    a.update(kw)
    return attn.attn_rope_axes_append(*a.values(), stream=0)


PAGED = [
    (dict(page=24), ARG), (dict(page=8), ARG), (dict(page=1 << 17), ARG), (dict(page=0), ARG), (dict(per=0), ARG),
    (dict(pages=0), ARG), (dict(per=1 << 27), ARG), (dict(pages=1 << 30), ARG), (dict(B=0), ARG),
    (dict(table=A16 + 4 * MB + 2), ARG), (dict(table=None), ARG), (dict(table=None, pages=3), ARG), (dict(table=None, per=1), ARG),
]


@pytest.mark.parametrize("kw,code", PAGED + [
    (dict(q=None), ARG), (dict(k=A16 + 8), ARG), (dict(v=None), ARG), (dict(kp=None), ARG), (dict(vp=KP), ARG),
    (dict(vp=VP + 4), ARG), (dict(k=KP), ARG), (dict(v=VP), ARG), (dict(q_out=KP + 16 * 64 * 2 * 2 * 19), ARG),
    (dict(lens=None), ARG), (dict(lens=A16 + 1), ARG), (dict(out=A16), ARG), (dict(out=A16 + 8), ARG),
    (dict(out=A16 + 4 * MB + 16), ARG), (dict(new=A16 + 72), ARG), (dict(pos=A16 + 2), ARG), (dict(A=5), ARG), (dict(A=0), ARG),
    (dict(T=0), ARG), (dict(r=64, freqs=None), ARG), (dict(d=12), UNSUP), (dict(scale=-float("inf")), ARG),
])
def test_append_refusals(kw, code):
    assert _append(**kw) == code


def test_sections():
    assert attn.rope_sections((2, 3), device="cpu").tolist() == [0, 0, 1, 1, 1]
    assert attn.rope_sections((2, 3, 1), cycled=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 1]
    for bad in ((), (1,) * 5, (0, 0), (3, -1)):
        with pytest.raises(attn.AttnError):
            attn.rope_sections(bad, device="cpu")


def test_helpers_refuse_cpu_tensors():
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    f, lens = torch.ones(32, dtype=torch.float64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: attn.rope_axes(x, x, f, None, torch.zeros(3, dtype=torch.int32)),
                 lambda: attn.rope_axes_append(x, x, x, x, x, lens, f)):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == ARG


def _mask(**kw):
    a = dict(parents=A16, lens=A16 + MB, live=None, mask=A16 + 2 * MB, pos=A16 + 3 * MB, B=3, T=70)
    a.update(kw)
    return attn.attn_tree_mask(*a.values(), stream=0)


@pytest.mark.parametrize("kw", [
    dict(parents=None), dict(parents=A16 + 2), dict(lens=A16 + 1), dict(live=A16 + 3), dict(mask=None), dict(mask=A16 + 4),
    dict(pos=A16 + 2), dict(B=0), dict(T=0), dict(T=257), dict(mask=A16), dict(pos=A16 + 3 * 70 * 4 - 4), dict(pos=A16 + MB),
    dict(mask=A16 + MB), dict(pos=A16 + 2 * MB + 3 * 70 * 16 - 4), dict(live=A16 + 2 * MB),
])
def test_mask_refusals(kw):
    assert _mask(**kw) == ARG


def _accept(**kw):
    a = dict(kp=KP, vp=VP, table=A16 + 4 * MB, lens=A16, mask=A16 + MB, last=A16 + 2 * MB, out=A16 + 3 * MB, layers=2, B=3,
             Hkv=2, T=70, d=64, pages=20, page=16, per=4)
    a.update(kw)
    return attn.attn_tree_accept(*a.values(), stream=0)


@pytest.mark.parametrize("kw,code", PAGED + [
    (dict(kp=None), ARG), (dict(vp=None), ARG), (dict(kp=KP + 8), ARG), (dict(vp=KP + 2 * 20 * 2 * 16 * 64 * 2 - 16), ARG),
    (dict(lens=None), ARG), (dict(last=None), ARG), (dict(lens=A16 + 2), ARG), (dict(last=A16 + 1), ARG), (dict(out=A16 + 3), ARG),
    (dict(mask=A16 + 4), ARG), (dict(T=0), ARG), (dict(T=257), ARG), (dict(layers=0), ARG), (dict(d=60), UNSUP), (dict(d=520), UNSUP),
    (dict(out=A16), ARG), (dict(out=A16 + 2 * MB + 8), ARG), (dict(out=A16 + MB), ARG), (dict(out=A16 + 4 * MB), ARG), (dict(out=KP), ARG),
    (dict(lens=KP), ARG), (dict(last=VP + 64), ARG), (dict(mask=KP), ARG), (dict(layers=1 << 27, pages=1, B=1, per=1), ARG),
])
def test_accept_refusals(kw, code):
    assert _accept(**kw) == code


def _extend(**kw):
    a = dict(table=A16, refs=A16 + MB, lens=A16 + 2 * MB, new=None, T=1, kp=KP, vp=VP, info=A16 + 3 * MB, layers=2, B=3, Hkv=2,
             d=64, pages=20, page=16, per=4, ws=A16 + 4 * MB, bytes=1 << 20)
    a.update(kw)
    return attn.attn_pages_extend(*a.values(), stream=0)


def _compact(**kw):
    a = dict(table=A16, refs=A16 + MB, kp=KP, vp=VP, info=A16 + 3 * MB, layers=2, B=3, Hkv=2, d=64, pages=20, page=16, per=4,
             ws=A16 + 4 * MB, bytes=1 << 20)
    a.update(kw)
    return attn.attn_pages_compact(*a.values(), stream=0)


def _fork(**kw):
    a = dict(table=A16, out=A16 + MB, refs=A16 + 2 * MB, lens=A16 + 3 * MB, lens_out=A16 + 4 * MB, parent=A16 + 5 * MB, B=3,
             pages=20, page=16, per=4)
    a.update(kw)
    return attn.attn_pages_fork(*a.values(), stream=0)


def _trim(**kw):
    a = dict(table=A16, refs=A16 + MB, lens=A16 + 2 * MB, lens_out=A16 + 3 * MB, keep=A16 + 4 * MB, B=3, pages=20, page=16, per=4)
    a.update(kw)
    return attn.attn_pages_trim(*a.values(), stream=0)


SIZES = [(kw, code) for kw, code in PAGED if "table" not in kw]


@pytest.mark.parametrize("call", [_extend, _compact, _fork, _trim])
@pytest.mark.parametrize("kw,code", SIZES + [(dict(table=None), ARG), (dict(table=A16 + 2), ARG), (dict(refs=None), ARG),
                                             (dict(refs=A16 + 1), ARG), (dict(refs=A16 + 44), ARG)])
def test_pages_sizes_and_tables(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("call", [_extend, _compact])
@pytest.mark.parametrize("kw,code", [
    (dict(kp=None), ARG), (dict(vp=VP + 8), ARG), (dict(vp=KP), ARG), (dict(info=None), ARG), (dict(info=A16 + 2), ARG),
    (dict(info=A16 + MB), ARG), (dict(info=A16 + 47), ARG), (dict(layers=0), ARG), (dict(Hkv=0), ARG), (dict(d=60), UNSUP),
    (dict(d=520), UNSUP), (dict(ws=None), WS), (dict(ws=A16 + 4 * MB + 8), WS), (dict(bytes=16), WS), (dict(ws=A16), ARG),
    (dict(ws=KP), ARG), (dict(table=KP), ARG), (dict(refs=VP), ARG),
])
def test_pages_move_refusals(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("call,kw", [
    (_extend, dict(lens=None)), (_extend, dict(lens=A16 + 2)), (_extend, dict(new=A16 + 1)), (_extend, dict(T=-1)),
    (_extend, dict(lens=A16)), (_extend, dict(new=A16 + MB)), (_extend, dict(new=KP)),
    (_fork, dict(out=None)), (_fork, dict(out=A16)), (_fork, dict(out=A16 + 44)), (_fork, dict(lens=None)),
    (_fork, dict(lens_out=None)), (_fork, dict(lens_out=A16 + 3 * MB)), (_fork, dict(parent=None)), (_fork, dict(parent=A16 + 2)),
    (_fork, dict(parent=A16 + 2 * MB)), (_fork, dict(lens=A16 + 3)),
    (_trim, dict(lens=None)), (_trim, dict(keep=None)), (_trim, dict(keep=A16)), (_trim, dict(lens_out=A16 + 4 * MB)),
    (_trim, dict(lens_out=A16 + MB)), (_trim, dict(keep=A16 + 4 * MB + 2)),
])
def test_pages_other_refusals(call, kw):
    assert call(**kw) == ARG


def test_pages_workspace():
    f = attn.attn_pages_workspace_bytes
    assert f(0, 5) == f(5, 0) == f(-1, 5) == f(1, (1 << 30) + 1) == 0
    assert f(1, 1) >= 16 and f(64, 1000) >= 4 * 4 * 1000 + 20 * 64


def test_page_helpers_refuse_cpu_tensors():
    t, r, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    k = torch.zeros((5, 1, 16, 8), dtype=torch.bfloat16)
    for call in (lambda: attn.tree_mask(t), lambda: attn.tree_accept(k, k, n, None, n, page_table=t),
                 lambda: attn.pages_extend(t, r, n, 1, k, k), lambda: attn.pages_fork(t, r, n, n, 16),
                 lambda: attn.pages_trim(t, r, n, n, 16), lambda: attn.pages_compact(t, r, k, k)):
        with pytest.raises(attn.AttnError) as e:
            call()
        assert e.value.code == ARG


def _tree(**kw):
    a = dict(q=A16, kp=KP, vp=VP, table=A16 + MB, lens=A16 + 2 * MB, mask=A16 + 3 * MB, live=None, o=A16 + 4 * MB, lse=A16 + 5 * MB,
             B=3, Hq=4, Hkv=2, T=70, d=64, scale=0.1, pages=20, page=16, per=4, ws=A16 + 128 * MB, bytes=1 << 30)
    a.update(kw)
    return attn.attn_decode_tree(*a.values(), stream=0)


@pytest.mark.parametrize("kw,code", [(kw, code) for kw, code in PAGED if kw != dict(table=A16 + 4 * MB + 2)] + [
    (dict(q=None), ARG), (dict(q=A16 + 8), ARG), (dict(kp=None), ARG), (dict(vp=VP + 8), ARG), (dict(o=None), ARG),
    (dict(o=A16 + 4), ARG), (dict(lens=None), ARG), (dict(lens=A16 + 1), ARG), (dict(mask=A16 + 4), ARG), (dict(live=A16 + 2), ARG),
    (dict(lse=A16 + 2), ARG), (dict(scale=0.0), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
    (dict(Hq=5), ARG), (dict(Hq=34), UNSUP), (dict(T=0), ARG), (dict(T=257), UNSUP), (dict(d=56), UNSUP), (dict(d=256), UNSUP),
    (dict(table=A16 + MB + 2), ARG), (dict(ws=None), WS), (dict(ws=A16 + 128 * MB + 8), WS),
    (dict(B=1 << 20, Hkv=64, Hq=64, per=1 << 20), ARG),
])
def test_decode_tree_refusals(kw, code):
    assert _tree(**kw) == code


def test_decode_tree_workspace():
    f = attn.attn_decode_tree_workspace_bytes
    for bad in ((0, 4, 2, 1, 64, 16, 4), (1, 5, 2, 1, 64, 16, 4), (1, 4, 2, 0, 64, 16, 4), (1, 4, 2, 257, 64, 16, 4),
                (1, 4, 2, 1, 56, 16, 4), (1, 4, 2, 1, 64, 0, 4), (1, 4, 2, 1, 64, 1 << 20, 1 << 20)):
        assert f(*bad) == 0


@pytest.mark.parametrize("call", [_extend, _compact])
def test_pages_whose_units_are_not_counted_in_32_bits(call):
    # 8192 heads x 65536 rows x 4 units of 16 bytes are 2^31
    assert call(pages=1, B=1, per=1, page=65536, Hkv=8192, d=32, layers=1, kp=1 << 40, vp=1 << 44) == ARG


@pytest.mark.parametrize("pos", [A16 + 64 - 4, A16 + 64 + 8, A16 + 64 - 100 * 4, A16 + 64 - 8 * 4])
def test_append_refuses_new_lengths_over_positions(pos):
    # two axes 100 apart, three entries 4 apart, one token: the last one is at 108
    assert _append(pos=pos, axis_stride=100, pos_stride=4, A=2) == ARG
