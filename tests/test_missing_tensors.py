"""The torch helpers of the paged cache, of drafted tokens and of the decode cache name a tensor that is missing, or a table of another shape,
in an AttnError, as they do a tensor of the wrong type."""
import pytest
import torch

import attention_fa2_fwd_sm_gb300 as attn
from attention_fa2_fwd_sm_gb300 import _build

HELPERS = {
    "rope_axes": ("q", "k", "inv_freq", "axes", "positions"),
    "rope_axes_append": ("q", "k", "v", "kcache", "vcache", "seqlens", "inv_freq", "axes", "positions", "page_table"),
    "decode_tree": ("q", "kcache", "vcache", "seqlens", "mask", "draft_lens", "page_table"),
    "tree_mask": ("parents", "seqlens", "draft_lens"),
    "tree_accept": ("kcache", "vcache", "seqlens", "mask", "last", "page_table"),
    "pages_extend": ("page_table", "refs", "seqlens", "new", "kpages", "vpages"),
    "pages_fork": ("page_table", "refs", "seqlens", "parent", "page_size"),
    "pages_trim": ("page_table", "refs", "seqlens", "keep", "page_size"),
    "pages_compact": ("page_table", "refs", "kpages", "vpages"),
    "rope": ("q", "k", "inv_freq"),
    "rope_append": ("q", "k", "v", "kcache", "vcache", "seqlens", "inv_freq"),
}
# What may be None (k: a single tensor is rotated; inv_freq of an append: nothing is).
FREE = {("rope_axes", "k"), ("rope_axes", "axes"), ("rope_axes_append", "inv_freq"), ("rope_axes_append", "axes"),
        ("rope_axes_append", "positions"), ("decode_tree", "mask"), ("decode_tree", "draft_lens"), ("tree_mask", "seqlens"),
        ("tree_mask", "draft_lens"), ("tree_accept", "mask"), ("rope", "k"),
        ("rope_append", "inv_freq")}


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    attn.lib()


def refused(name, args, text):
    with pytest.raises(attn.AttnError) as e:
        getattr(attn, name)(**args)
    assert e.value.code == attn.ATTN_ERR_ARG and text in str(e.value), str(e.value)


@pytest.mark.parametrize("name", list(HELPERS))
def test_the_first_tensor(name):
    refused(name, dict.fromkeys(HELPERS[name]), HELPERS[name][0])


def arguments(name):
    """Of a call that works: two sequences, three tokens, two pages of 16 each."""
    dev = dict(device="cuda")
    i32, bf16 = dict(dtype=torch.int32, **dev), dict(dtype=torch.bfloat16, **dev)
    table, lens, x = torch.arange(4, **i32).view(2, 2), torch.zeros(2, **i32), torch.zeros((2, 2, 3, 64), **bf16)
    refs, pool = torch.ones(4, **i32), [torch.zeros((4, 2, 16, 64), **bf16) for _ in range(2)]
    f = torch.ones(32, dtype=torch.float64, **dev)
    every = dict(q=x, k=x.clone(), v=x.clone(), inv_freq=f, axes=torch.zeros(32, **i32), positions=torch.zeros((1, 3), **i32),
                 kcache=pool[0], vcache=pool[1], kpages=pool[0], vpages=pool[1], seqlens=lens, page_table=table, refs=refs,
                 mask=torch.zeros((2, 3, 1), dtype=torch.int64, **dev), draft_lens=lens.clone(), parents=torch.zeros((2, 3), **i32),
                 last=lens.clone(), new=1, parent=lens.clone(), keep=lens.clone(), page_size=16)
    if name == "rope_append":
        every.update(kcache=pool[0][:2], vcache=pool[1][:2])
    return {k: every[k] for k in HELPERS[name]}


@pytest.mark.gpu
@pytest.mark.parametrize("name", HELPERS)
def test_every_tensor(name):
    getattr(attn, name)(**arguments(name))
    for arg in HELPERS[name]:
        if (name, arg) in FREE or arg == "page_size":
            continue
        if arg == "page_table" and not name.startswith("pages"):  # (without one the pools are caches, of which there are four)
            refused(name, {**arguments(name), arg: None}, "")
            for table in (torch.zeros((), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")):
                refused(name, {**arguments(name), arg: table}, "page_table")
        else:
            # (the caches' shapes are looked at together)
            refused(name, {**arguments(name), arg: None}, "the caches" if arg == "kcache" and name != "tree_accept" else arg)
