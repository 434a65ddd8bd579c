"""CPU-only: attn_rope_axes and attn_rope_axes_append refuse every output that is laid over an array that the call reads
or over another output.  The refusals come from the host before any CUDA call; addresses are made up, and each call here
is refused, or, where there is no GPU, ends for want of one."""
import ctypes

import pytest
import torch

import attention_fa2_fwd_sm_gb300 as attn
from attention_fa2_fwd_sm_gb300 import _build

MB = 1 << 20
Q, QO, K, V, KO = (16 * MB * (i + 1) for i in range(5))
KP, VP = 256 * MB, 512 * MB
TABLE, LENS, OUT, NEW, POS, FREQS, AXES = (1024 * MB + MB * i for i in range(7))
B, HQ, HKV, T, D, R, PAGES, PAGE, PER = 3, 4, 2, 5, 64, 64, 20, 16, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    attn.lib()


def append(**kw):
    a = dict(q=Q, q_out=QO, k=K, v=V, kp=KP, vp=VP, table=TABLE, lens=LENS, pos=POS, axis_stride=100, pos_stride=7, A=2,
             new=NEW, out=OUT, freqs=FREQS, axes=AXES, B=B, Hq=HQ, Hkv=HKV, T=T, d=D, r=R, inter=0, scale=1.0, pages=PAGES,
             page=PAGE, per=PER, strides=None)
    a.update(kw)
    return attn.attn_rope_axes_append(*a.values(), stream=0)


# Bytes of each array: the last position is at 100 + 2 x 7 + 4.
ARRAYS = dict(table=B * PER * 4, lens=B * 4, new=B * 4, pos=119 * 4, freqs=R // 2 * 8, axes=R // 2 * 4)
STEP = dict(freqs=8)
POOL = PAGES * HKV * PAGE * D * 2


@pytest.mark.parametrize("name", list(ARRAYS) + ["out"])
@pytest.mark.parametrize("to,bytes", [(QO, B * HQ * T * D * 2), (KP, POOL), (VP, POOL)])
def test_arrays_over_outputs(name, to, bytes):
    step, size = STEP.get(name, 4), ARRAYS.get(name, B * 4)
    for at in (to, to + bytes - step, to - size + step, to + bytes // 2 // 8 * 8):
        assert append(**{name: at}) == attn.ATTN_ERR_ARG


@pytest.mark.parametrize("name", list(ARRAYS))
def test_new_lengths_over_what_is_read(name):
    base, size = dict(table=TABLE, lens=LENS, new=NEW, pos=POS, freqs=FREQS, axes=AXES)[name], ARRAYS[name]
    for at in (base, base + size - 4, base - B * 4 + 4):
        assert append(out=at) == attn.ATTN_ERR_ARG


@pytest.mark.parametrize("name,heads", [("q", HQ), ("k", HKV), ("v", HKV)])
def test_new_lengths_over_the_tokens(name, heads):
    base = dict(q=Q, k=K, v=V)[name]
    for at in (base, base - 8, base + B * heads * T * D * 2 - 4):
        assert append(out=at) == attn.ATTN_ERR_ARG


def test_rows_of_a_strided_output():
    """Token rows of 128 bytes, 192 apart: an array that touches a row is refused, wherever in the tensor."""
    s = (ctypes.c_longlong * 12)(HQ * T * D, T * D, D, HQ * T * 96, T * 96, 96, *(HKV * T * D, T * D, D) * 2)
    for row in (0, 1, 7, T * HQ, B * T * HQ - 1):
        for at in (QO + row * 192, QO + row * 192 + 124, QO + row * 192 - 8):
            assert append(strides=s, lens=at) == attn.ATTN_ERR_ARG


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")


@no_gpu
def test_what_is_apart_is_not_refused():
    """Every array at either side of an output's rows, and between the rows of a strided one."""
    s = (ctypes.c_longlong * 12)(HQ * T * D, T * D, D, HQ * T * 96, T * 96, 96, *(HKV * T * D, T * D, D) * 2)
    assert append() == rope() == append(q_out=Q) == attn.ATTN_ERR_CUDA
    for name, size in (*ARRAYS.items(), ("out", B * 4)):
        for to, bytes in ((QO, B * HQ * T * D * 2), (KP, POOL), (VP, POOL)):
            for at in (to + bytes, to - (size + 7) // 8 * 8):
                assert append(**{name: at}) == attn.ATTN_ERR_CUDA
        if size <= 64:
            for row in (0, 1, B * T * HQ - 2):
                for at in (QO + row * 192 + 128, QO + row * 192 + 192 - (size + 7) // 8 * 8):
                    assert append(strides=s, **{name: at}) == attn.ATTN_ERR_CUDA


def rope(**kw):
    a = dict(q=Q, q_out=QO, k=K, k_out=KO, pos=POS, axis_stride=100, pos_stride=7, A=2, freqs=FREQS, axes=AXES, B=B, Hq=HQ,
             Hkv=HKV, N=T, d=D, r=R, inter=0, scale=1.0, inverse=0, strides=None)
    a.update(kw)
    return attn.attn_rope_axes(*a.values(), stream=0)


@pytest.mark.parametrize("name", ["pos", "freqs", "axes"])
@pytest.mark.parametrize("to,heads", [(QO, HQ), (KO, HKV)])
def test_rotation_over_what_it_reads(name, to, heads):
    step, bytes = STEP.get(name, 4), B * heads * T * D * 2
    for at in (to, to + bytes - step, to - ARRAYS[name] + step):
        assert rope(**{name: at}) == attn.ATTN_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=K + 8), dict(v=None), dict(kp=None), dict(vp=KP), dict(vp=VP + 4), dict(k=KP), dict(v=VP),
    dict(q_out=KP + POOL - 128), dict(lens=None), dict(lens=LENS + 1), dict(new=NEW + 2), dict(out=OUT + 1), dict(pos=POS + 2),
    dict(A=0), dict(A=5), dict(T=0), dict(freqs=None), dict(axes=AXES + 2), dict(scale=float("nan")), dict(page=24), dict(page=8),
    dict(per=0), dict(pages=0), dict(B=0), dict(table=TABLE + 2), dict(table=None), dict(r=63), dict(axis_stride=-1),
])
def test_other_refusals(kw):
    """One fault each, in a call whose arrays are all apart."""
    assert append(**kw) == attn.ATTN_ERR_ARG
