"""Attention of drafted tokens over a cache at the edges of its warps, against the definition in 64 bits (reference and
tolerances of test_decode_tree_gpu.py)."""
import pytest
import torch

from synthetic_inputs import normal_bf16
from tests.test_decode_tree_gpu import a_cache, run_and_check
from tests.test_tree_gpu import random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


@pytest.fixture(scope="module")
def attn():
    from attention_fa2_fwd_sm_gb300 import _build
    _build.build()
    import attention_fa2_fwd_sm_gb300 as A
    A.lib()
    return A


# Query heads (of one KV head) and tokens: 1 to 255 rows, the last warp of which holds 1 to 31, or a tile with idle warps.
ROWS = [(1, 1), (5, 1), (8, 1), (1, 31), (3, 11), (16, 3), (9, 7), (13, 5), (16, 7), (1, 127), (3, 43), (16, 11), (5, 51)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,T", ROWS)
def test_rows_that_do_not_fill_a_warp(attn, Hq, T, d):
    """All columns of all rows where some lanes of a warp have a row and others have none: pairs in one piece (short
    caches), cut into partials and shared by the two chains of a CTA (one user of many keys)."""
    k, v, table = a_cache(7, 1, 300, d, 16, 40)
    cap = table.shape[1] * 16
    q = normal_bf16((7, Hq, T, d), 41, DEV)
    run_and_check(attn, q, k, v, table, 16, [cap - T, 0, 1, 64, 127, 200, max(0, cap - 1)], parents=random_tree(7, T, 42))
    k, v, _ = a_cache(1, 1, 21000, d, 0, 43)
    run_and_check(attn, q[:1], k, v, None, 0, [20000 - T], parents=random_tree(1, T, 44))
