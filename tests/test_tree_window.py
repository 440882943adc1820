"""Sliding windows shorter than a tree of drafts: csa.tree_masks leaves out the ancestors that the window hides, so that
a chain of drafts is csa_paged_attn's causal attention with the same window."""
import pytest
import torch

from compressed_sparse_attention_indexer_gb300 import csa
from test_paged_attn import _exact as causal
from test_paged_attn import _check, _pool
from test_tree_attn import DEV, _gpu, _sees


def _parents(b, s, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.minimum((torch.rand(b, s, generator=g).sqrt() * (torch.arange(s) + 1)).long() - 1, torch.arange(s) - 1)


@pytest.mark.parametrize("s,win", [(1, 1), (9, 1), (9, 4), (70, 3), (70, 69), (70, 70), (130, 65), (130, 1000)])
def test_masks_leave_out_what_the_window_hides(s, win):
    parent = _parents(4, s, s + win)
    parent[1] = torch.arange(s) - 1
    got = _sees(csa.tree_masks(parent, win), s)
    want = torch.zeros_like(got)
    for i in range(4):
        for t in range(s):
            u = t
            for _ in range(win):                          # the draft itself and win - 1 tokens before it
                want[i, t, u] = True
                u = int(parent[i, u])
                if u < 0:
                    break
    assert torch.equal(got, want)
    if win >= s:
        assert torch.equal(csa.tree_masks(parent, win), csa.tree_masks(parent))


def test_refusal():
    with pytest.raises(csa.CsaError):
        csa.tree_masks(torch.tensor([[-1, 0]]), -1)


@pytest.mark.gpu
@pytest.mark.parametrize("s,h,hk,d,fp8", [(8, 8, 2, 128, False), (64, 8, 2, 128, False), (12, 8, 2, 128, True), (64, 8, 2, 128, True),
                                          (70, 8, 2, 64, False), (9, 4, 1, 256, False)])
@pytest.mark.parametrize("win", [1, 5, 40])
@pytest.mark.parametrize("max_len", [None, 1 << 20])
def test_a_chain_with_a_window_is_the_causal_attention(s, h, hk, d, fp8, win, max_len):
    _gpu()
    lens, block = [s, 300, 1111], 64
    pool, k, v = _pool(lens, hk, d, block, 4, fp8)
    q = torch.randn(3, s, h, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32)
    chain = csa.tree_masks((torch.arange(s) - 1).repeat(3, 1), win)
    pos = (n[:, None] - s + torch.arange(s)).int()
    kk, vv = pool.pop("k"), pool.pop("v")
    got = csa.TreeAttention(q.to(DEV), kk, vv, n.to(DEV), chain.to(DEV), pos=pos.to(DEV), win=win, max_len=max_len, **pool)()
    torch.cuda.synchronize()
    _check(got, causal(q, k, v, lens, pool["table"].cpu(), block, win, d ** -0.5))
