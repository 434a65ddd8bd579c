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


def guarded(shape, dtype, skip, seed):
    """A tensor `skip` bytes behind the start of an allocation, and all of that, filled with a pattern."""
    size = torch.empty(0, dtype=dtype).element_size()
    n = torch.Size(shape).numel()
    whole = torch.randint(0, 128, (skip + n * size + 256,), generator=torch.Generator().manual_seed(seed), dtype=torch.uint8).to(DEV)
    return whole[skip:skip + n * size].view(dtype).view(shape), whole


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,T,S,page", [
    (1, 8, 1, 9000, 0), (1, 8, 5, 9000, 16), (7, 8, 5, 300, 16), (2, 16, 8, 3000, 64), (1, 8, 33, 9000, 0), (3, 16, 20, 300, 16),
    (2, 16, 40, 3000, 64), (40, 8, 5, 500, 64),
])
def test_outputs_and_workspace_on_16_bytes(attn, B, Hq, T, S, page, d):
    """Outputs, queries and a workspace that are 16-byte aligned and no more: the bits of the call that has them on 256
    bytes, and not a byte around them changed.  Pairs in one piece, cut ones and those that a CTA's chains share."""
    k, v, table = a_cache(B, 2, S, d, page, 60)
    q = normal_bf16((B, Hq, T, d), 61, DEV)
    table = None if table is None else table.to(DEV)
    per = 1 if page == 0 else table.shape[1]
    lens = torch.randint(0, S, (B,), generator=torch.Generator().manual_seed(62)).to(torch.int32)
    lens[0] = S - T
    lens = lens.to(DEV)
    mask, _ = attn.tree_mask(random_tree(B, T, 63).to(DEV))
    want = attn.decode_tree(q, k, v, lens, mask, page_table=table)
    nbytes = attn.attn_decode_tree_workspace_bytes(B, Hq, 2, T, d, page or S, per)
    for q_at, o_at, ws_at in ((0, 16, 0), (0, 0, 16), (16, 16, 48)):
        o, o_all = guarded((B, Hq, T, d), torch.bfloat16, o_at, 64)
        lse, lse_all = guarded((B, Hq, T), torch.float32, 4, 65)
        ws, ws_all = guarded((nbytes,), torch.uint8, ws_at, 66)
        queries = guarded((B, Hq, T, d), torch.bfloat16, q_at, 67)[0]
        queries.copy_(q)
        was = [x.clone() for x in (o_all, lse_all, ws_all)]
        rc = attn.attn_decode_tree(queries, k, v, table, lens, mask, None, o, lse, B, Hq, 2, T, d, d ** -0.5, k.shape[0],
                                   page or S, per, ws, nbytes)
        torch.cuda.synchronize()
        assert rc == attn.ATTN_OK and attn.attn_device_status() == attn.ATTN_OK
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        for part, x, old in ((o, o_all, was[0]), (lse, lse_all, was[1]), (ws, ws_all, was[2])):
            at, n = part.data_ptr() - x.data_ptr(), part.numel() * part.element_size()
            assert torch.equal(x[:at], old[:at]) and torch.equal(x[at + n:], old[at + n:])


@pytest.mark.parametrize("Hq,T,d", [(8, 6, 64), (8, 6, 128), (8, 40, 64), (8, 40, 128)])
@pytest.mark.parametrize("S", [500, 5000])
def test_values_at_their_limit(attn, Hq, T, d, S):
    """Values of just below 2^111 over the number of keys, all of one sign, and weights that the reference of a row, which
    stays at its first block's, lets grow as far as it does: 11 log2(e) = 15.9 of 16 binary orders.  Sums before the
    division reach 2^15.9 2^111 = 2^126.9, just below what 32 bits hold."""
    k, v, _ = a_cache(2, 1, S, d, 0, 70)
    n = S - 9
    k[...] = 11 / d ** 0.5
    k[:, :, :128] = 0
    v = ((0.75 + 0.24 * torch.tanh(v.float())) * (2.0 ** 111 / S)).bfloat16()
    q = torch.ones((2, Hq, T, d), dtype=torch.bfloat16, device=DEV)
    o, _, _ = run_and_check(attn, q, k, v, None, 0, [n - T, n // 2], parents=random_tree(2, T, 71))
    assert torch.all(torch.isfinite(o)) and torch.all(o > 2.0 ** 110 / S)
