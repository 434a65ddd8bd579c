"""CPU-only: the largest page that attn_pages_extend and attn_pages_compact take.  Its 16-byte units are rounded up to whole
warps' work of 256 in 32 bits, so that those of K in a page are at most 2^31 - 256.  Addresses are made up."""
import pytest
import torch

import attention_fa2_fwd_sm_gb300 as attn
from attention_fa2_fwd_sm_gb300 import _build
from tests.test_paged_abi import _compact, _extend


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    attn.lib()


def call(f, Hkv, page, d):
    return f(pages=2, B=1, per=1, layers=1, kp=1 << 42, vp=1 << 44, Hkv=Hkv, page=page, d=d)


@pytest.mark.parametrize("f", [_extend, _compact])
@pytest.mark.parametrize("units,Hkv,page,d", [
    (2 ** 31 - 16, 19173961, 16, 56), (2 ** 31 - 32, 7 * 9586980 + 3, 32, 8), (2 ** 31 - 64, 33554431, 64, 8),
    (2 ** 31 - 240, 134217713, 16, 8), (2 ** 31, 8192, 65536, 32),
])
def test_too_large(f, units, Hkv, page, d):
    assert Hkv * page * (d // 8) == units
    assert call(f, Hkv, page, d) == attn.ATTN_ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
@pytest.mark.parametrize("f", [_extend, _compact])
@pytest.mark.parametrize("units,Hkv,page,d", [(2 ** 31 - 256, 134217712, 16, 8), (2 ** 30, 8192, 65536, 16)])
def test_largest(f, units, Hkv, page, d):
    assert Hkv * page * (d // 8) == units
    assert call(f, Hkv, page, d) == attn.ATTN_ERR_CUDA  # there is no GPU
