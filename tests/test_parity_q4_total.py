"""attn_fwd_varlen_paged_q4 past the page stream with a total_k that the lengths exceed (reported,
the keys that fit read back, nothing outside the workspace written) or stay far below, and the
read-back of more pages than its blocks take at once."""
import numpy as np
import pytest
import torch

import oracle
from attention_paged_kv_gqa_b200 import binding as A
from oracle import rope_q4 as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL_O, TOL_LSE = 2e-2, 1e-3              # the tensor-core forward's elsewhere (probabilities in bf16)


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert A.attn_check_device(0) == 0
    torch.cuda.set_device(0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


class Space:
    """A workspace of exactly the size that is asked for, between bytes that must stay."""

    def __init__(self, need):
        self.all = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        self.ws = self.all[4096:4096 + need]

    def untouched(self):
        return bool((self.all[:4096] == 0xA5).all()) and bool((self.all[4096 + self.ws.numel():] == 0xA5).all())


def test_sum_of_lengths_past_31_bits():
    """Lengths whose sum is past 2^31 are seen to exceed total_k; the rows' offsets stay within it."""
    B, Hq, Hkv, D, group, total_k, n = 5, 2, 1, 64, 32, 50, 70
    cache = R.fill((1, Hkv, 16, D // 2), group, 1)
    bt = torch.zeros(B, 1 << 25, dtype=torch.int32, device=DEV)          # (every page is page 0)
    q = randn((n + 4, Hq, D), 2)
    need = A.attn_fwd_q4_workspace_size(B, n, Hq, Hkv, D, total_k)
    space = Space(need)
    o, lse = A.attn_fwd_varlen_paged_q4(q.to(DEV), *(t.to(DEV) for t in cache), block_table=bt,
                                        cu_seqlens_q=i32([0, n, n + 1, n + 2, n + 3, n + 4]).to(DEV), max_seqlen_q=n,
                                        seqused_k=i32([1 << 29] * B).to(DEV), total_k=total_k, mask=A.MASK_NONE,
                                        workspace=space.ws)
    assert A.attn_device_error() == 531
    assert space.untouched()
    rows = 2 * total_k * Hkv * D * 2
    assert space.ws[rows:rows + 4 * (B + 1)].view(torch.int32).tolist() == [0] + [total_k] * B
    # the first sequence's keys that fit: tokens 0 .. 49; the others have none
    k, v = R.packed(*cache, torch.zeros(1, 4, dtype=torch.int32), [total_k])
    o_ref, lse_ref = oracle.attn_varlen(q[:n], k, v, cu_seqlens_q=[0, n], cu_seqlens_k=[0, total_k], num_heads_kv=Hkv,
                                        scale=D ** -0.5, mask=0)
    assert np.abs(o[:n].double().cpu().numpy() - o_ref).max() <= TOL_O
    assert np.abs(lse[:, :n].double().cpu().numpy() - lse_ref).max() <= TOL_LSE
    assert not o[n:].any() and bool(torch.isneginf(lse[:, n:]).all())


@pytest.mark.parametrize("total_k", [120, 100, 133])
def test_first_sequences_and_the_bytes_behind_the_workspace(total_k):
    Hq, Hkv, D, group, lens, qs = 4, 2, 64, 32, [100, 34], [10, 70]
    need = [(m + 15) // 16 for m in lens]
    bt = torch.full((2, max(need)), 1 << 29, dtype=torch.int32)
    bt[0, :need[0]], bt[1, :need[1]] = torch.arange(need[0]) + 1, torch.arange(need[1]) + 1 + need[0]
    cache = R.fill((sum(need) + 1, Hkv, 16, D // 2), group, 33)
    q = randn((80, Hq, D), 34)
    space = Space(A.attn_fwd_q4_workspace_size(2, 70, Hq, Hkv, D, total_k))
    o, lse = A.attn_fwd_varlen_paged_q4(q.to(DEV), *(t.to(DEV) for t in cache), block_table=bt.to(DEV),
                                        cu_seqlens_q=i32([0, 10, 80]).to(DEV), max_seqlen_q=70, seqused_k=i32(lens).to(DEV),
                                        total_k=total_k, mask=A.MASK_CAUSAL, workspace=space.ws)
    assert A.attn_device_error() == 531
    assert space.untouched()
    k, v = R.packed(*cache, bt, [100, total_k - 100])
    assert torch.equal(space.ws[:k.numel() * 2].view(torch.bfloat16).cpu(), k.flatten())
    assert torch.equal(space.ws[k.numel() * 2:k.numel() * 4].view(torch.bfloat16).cpu(), v.flatten())
    o_ref, lse_ref = oracle.attn_varlen(q[:10], k[:100], v[:100], cu_seqlens_q=[0, 10], cu_seqlens_k=[0, 100],
                                        num_heads_kv=Hkv, scale=D ** -0.5, mask=1)
    assert np.abs(o[:10].double().cpu().numpy() - o_ref).max() <= TOL_O
    assert np.abs(lse[:, :10].double().cpu().numpy() - lse_ref).max() <= TOL_LSE
    assert torch.isfinite(o).all()


def test_total_far_above_the_lengths():
    Hq, Hkv, D, group, lens = 4, 2, 64, 32, [100, 0, 34]
    n = [(m + 15) // 16 for m in lens]
    bt = torch.zeros(3, max(n), dtype=torch.int32)
    bt[0, :n[0]], bt[2, :n[2]] = torch.arange(n[0]) + 1, torch.arange(n[2]) + 1 + n[0]
    cache = [t.to(DEV) for t in R.fill((sum(n) + 1, Hkv, 16, D // 2), group, 35)]
    q, cu = randn((81, Hq, D), 36).to(DEV), i32([0, 10, 11, 81]).to(DEV)
    got = []
    for total_k in (134, 2_000_000):
        space = Space(A.attn_fwd_q4_workspace_size(3, 70, Hq, Hkv, D, total_k))
        got.append(A.attn_fwd_varlen_paged_q4(q, *cache, block_table=bt.to(DEV), cu_seqlens_q=cu, max_seqlen_q=70,
                                              seqused_k=i32(lens).to(DEV), total_k=total_k, mask=A.MASK_CAUSAL,
                                              workspace=space.ws))
        assert A.attn_device_error() == 0 and space.untouched()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("lens", [[40001], [700] * 64, [300] * 65, [0, 33, 20000, 1, 16, 19000]])
def test_read_back_of_many_pages(lens):
    Hkv, D, group = 8, 64, 32
    n = [(m + 15) // 16 for m in lens]
    order = torch.randperm(sum(n), generator=torch.Generator().manual_seed(37)).to(torch.int32)
    bt = torch.full((len(lens), max(n)), 1 << 29, dtype=torch.int32)
    for b, pages in enumerate(order.split(n)):
        bt[b, :n[b]] = pages
    cache = R.fill((sum(n), Hkv, 16, D // 2), group, 38)
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    gk, gv = A.attn_kv_gather_paged_q4(*(t.to(DEV) for t in cache), bt.to(DEV), cu.to(DEV), int(cu[-1]))
    assert A.attn_device_error() == 0
    k, v = R.packed(*cache, bt, lens)
    assert torch.equal(gk.cpu(), k) and torch.equal(gv.cpu(), v)
