"""Acceptance of a chain of drafted tokens (no mask): lengths by attn.h's rule, `last` outside [0, T) accepts nothing."""
import pytest
import torch

from synthetic_inputs import normal_bf16
from tests.test_rope_axes_gpu import a_table

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("T", [1, 8, 65, 256])
def test_a_node_that_was_not_drafted_accepts_nothing(attn, T, page, side):
    B, S = 6, 320
    n, table = (B, None) if page == 0 else (2 * B * S // page, a_table(B, S // page, 2 * B * S // page, 50))
    kc = normal_bf16((n, 2, page or S, 64), 51, DEV)
    vc, was = kc.clone(), kc.clone()
    lens, last = torch.tensor([0, 17, 40, S - 2, 5, -3]), torch.tensor([T - 1, T, 2 ** 31 - 1, T - 1, -1, 0])
    dev = dict(dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    got = attn.tree_accept(kc, vc, lens.to(**dev), None, last.to(**dev), page_table=None if table is None else table.to(DEV),
                           stream=s, drafted=T)
    torch.cuda.synchronize()
    want = [min(S, max(a, 0) + (i + 1 if 0 <= i < T else 0)) for a, i in zip(lens.tolist(), last.tolist())]
    assert got.tolist() == want
    assert torch.equal(kc, was) and torch.equal(vc, was)


def test_refusals(attn):
    dev = dict(dtype=torch.int32, device=DEV)
    n, k = torch.zeros(2, **dev), torch.zeros((2, 1, 32, 8), dtype=torch.bfloat16, device=DEV)
    mask = torch.zeros((2, 7, 1), dtype=torch.int64, device=DEV)
    for bad in (dict(mask=None, drafted=0), dict(mask=None, drafted=257), dict(mask=mask, drafted=8), dict(mask=mask, drafted=6)):
        with pytest.raises(attn.AttnError) as e:
            attn.tree_accept(k, k.clone(), n, last=n, **bad)
        assert e.value.code == attn.ATTN_ERR_ARG
    assert attn.tree_accept(k, k.clone(), n, mask, n, drafted=7).tolist() == [0, 0]
