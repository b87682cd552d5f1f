"""The 4-bit KV cache: append, read back and attention, against the fp64 oracle.

Codes and metas must be the oracle's exactly, and so must what is read back.  The
attention kernels read the same codes as the oracle, so no quantisation error enters
their tolerances:
  O    half a bf16 step of itself (2^-8), plus the f16 rounding of the weights
       p step (2^-11 relative) times a code of at most 15, averaged over p: 2^-11 *
       15 * the largest step, plus fp32 sums of up to D or 16 terms per page
       (2^-18 of the same)
  LSE  the fp32 sum of D products of magnitude |q| 15 step (truncating adds,
       2^-22 each at most of the running sum) plus 2^-18
The packed path past 128 query rows rounds its probabilities to bf16 (the library's
tensor-core forward): 2e-2 and 1e-3, its tolerances elsewhere.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from attention_paged_kv_gqa_b200 import binding as A
from oracle import rope_q4 as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOL_O_PACKED, TOL_LSE_PACKED = 2e-2, 1e-3


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert A.attn_check_device(0) == 0
    torch.cuda.set_device(0)


def randn(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def table_for(lens, extra=2, seed=0):
    """(block table, pages of the pool): shuffled pages, unused entries outside the cache."""
    need = [(n + 15) // 16 for n in lens]
    pool = sum(need) + extra
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    bt = torch.full((len(lens), max(max(need), 1)), 1 << 29, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    return bt, pool


def steps(meta):
    return (((meta.to(torch.int32) & 0xFFF0) << 16).view(torch.float32))


def tolerances(q, cache, scale):
    sk, sv = float(steps(cache[2]).nan_to_num().max()), float(steps(cache[3]).nan_to_num().max())
    D = q.shape[-1]
    w = 15 * sv
    tol_lse = 2.0 ** -22 * D * float(q.abs().float().sum(-1).max()) * 15 * sk * scale + 2.0 ** -18
    # an error of the scores moves p by its size, and O by that times the values
    return (2.0 ** -11 + 2.0 ** -18 + 2 * tol_lse) * w, tol_lse


def check(o, lse, o_ref, lse_ref, tol_o, tol_lse):
    o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(lse), np.isneginf(lse_ref))
    fin = np.isfinite(lse_ref)
    assert np.isfinite(o).all()
    err = np.abs(o - o_ref) - 2.0 ** -8 * np.abs(o_ref)
    assert err.max(initial=0.0) <= tol_o, (float(err.max()), tol_o)
    if fin.any():
        assert np.abs(lse[fin] - lse_ref[fin]).max() <= tol_lse, (float(np.abs(lse[fin] - lse_ref[fin]).max()), tol_lse)
    assert not o[np.moveaxis(~fin, 0, -1) if lse.shape != o.shape[:2] else ~fin].any()


def reference(q, cache, bt, lens, cu_q, scale, causal, window, softcap):
    """fp64 attention of packed q over the packed values of the cache."""
    k, v = R.packed(*cache, bt, lens)
    cu_k = i32(np.concatenate([[0], np.cumsum(lens)]))
    return oracle.attn_varlen(q, k if len(k) else torch.zeros(1, *k.shape[1:], dtype=k.dtype),
                              v if len(v) else torch.zeros(1, *v.shape[1:], dtype=v.dtype), cu_seqlens_q=cu_q,
                              cu_seqlens_k=cu_k, num_heads_kv=cache[0].shape[1], scale=scale, mask=1 if causal else 0,
                              window_left=window, softcap=softcap)


def same(a, b):
    return bool(torch.equal(a.cpu(), b.cpu()))


def dev(*ts):
    return [t.to(DEV) for t in ts]


# ---------------------------------------------------------------- append and read back
@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("rot,interleaved,axes", [(0, False, 1), (64, False, 1), (48, False, 1), (64, True, 3), (32, True, 1)])
def test_append_matches_oracle(D, group, rot, interleaved, axes):
    Hq, Hkv = 3, 3
    before, new = [0, 1, 15, 16, 7, 30], [3, 0, 1, 16, 23, 2]
    T = sum(new)
    qkv = randn((T, Hq + 2 * Hkv, D), 1)
    qkv[3] *= 1e-3
    qkv[5] = qkv[5].abs() + 4                    # one-sided groups
    qkv[6] = -qkv[5]
    qkv[7] = 0
    dq = qkv.to(DEV)
    q, k, v = dq[:, :Hq], dq[:, Hq:Hq + Hkv], dq[:, Hq + Hkv:]
    bt, pool = table_for([a + b for a, b in zip(before, new)], seed=2)
    cache = R.fill((pool, Hkv, 16, D // 2), group, 3)
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    kw = {}
    rq, rk = q, k
    if rot:
        pos = torch.cat([torch.arange(a, a + n, dtype=torch.int32) for a, n in zip(before, new)])
        kw = dict(cos_sin=R.table(64, rot).to(DEV), interleaved=interleaved)
        if axes > 1:
            pos = torch.stack([pos, pos // 3, pos % 5])
            kw.update(positions=pos.to(DEV), pair_axis=i32([i % 3 for i in range(rot // 2)]).to(DEV))
        rq, rk = A.attn_rope(q, k, **dict(kw, positions=pos.to(DEV)))
    want = R.append(*cache, rk.cpu(), v.cpu(), bt, cu, before, group)
    got = dev(*cache)
    yq, out = A.attn_kv_append_paged_q4(q, k, v, *got, bt.to(DEV), i32(before).to(DEV), cu_seqlens_new=cu.to(DEV), **kw)
    assert A.attn_device_error() == 0
    assert torch.equal(yq, rq)
    assert out.tolist() == [a + b for a, b in zip(before, new)]
    for g, w in zip(got, want):
        assert same(g, w)
    # read back: the new rows, and all of them
    gk, gv = A.attn_kv_gather_paged_q4(*got, bt.to(DEV), cu.to(DEV), T, starts=i32(before).to(DEV))
    wk, wv = R.packed(*want, bt, new, before)
    assert torch.equal(gk.cpu(), wk) and torch.equal(gv.cpu(), wv)
    ends = [a + b for a, b in zip(before, new)]
    cu_all = i32(np.concatenate([[0], np.cumsum(ends)]))
    gk, gv = A.attn_kv_gather_paged_q4(*got, bt.to(DEV), cu_all.to(DEV), int(cu_all[-1]))
    wk, wv = R.packed(*want, bt, ends)
    assert torch.equal(gk.cpu(), wk) and torch.equal(gv.cpu(), wv)
    assert A.attn_device_error() == 0


def test_append_every_ratio_of_a_value_to_a_step():
    """All bf16 significands against all steps: each code is the nearest one, ties to even."""
    D = group = 64
    rows = []
    for s in range(8, 16):                       # step s / 8: the range's ends are 7 and -8 steps
        for x in range(0, 256, 62):
            vals = [(128 + (x + i) % 128) / 128.0 * 2.0 ** ((x + i) // 128 + e) for i in range(62) for e in (0,)]
            for mul in (1.0, 0.25, 2.0):
                r = torch.tensor([7 * s / 8, -8 * s / 8] + [min(v * mul, 7 * s / 8) for v in vals])
                rows.append(r)
                rows.append(torch.cat([r[:2], -r[2:]]))
    x = torch.stack(rows).to(torch.bfloat16)
    T = x.shape[0]
    kv = x.view(T, 1, D)
    bt = torch.arange((T + 15) // 16, dtype=torch.int32).view(1, -1)
    cache = [torch.zeros((T + 15) // 16, 1, 16, 32, dtype=torch.uint8), torch.zeros((T + 15) // 16, 1, 16, 32, dtype=torch.uint8),
             torch.zeros((T + 15) // 16, 1, 16, 1, dtype=torch.int16), torch.zeros((T + 15) // 16, 1, 16, 1, dtype=torch.int16)]
    want = R.append(*cache, kv, kv, bt, [0, T], [0], group)
    got = dev(*cache)
    A.attn_kv_append_paged_q4(None, kv.to(DEV), kv.to(DEV), *got, bt.to(DEV), i32([0]).to(DEV), cu_seqlens_new=i32([0, T]).to(DEV))
    for g, w in zip(got, want):
        assert same(g, w)


def test_append_special_values_and_sizes():
    D, group = 128, 32
    k = randn((4, 1, D), 5)
    k[0, 0, 3] = float("inf")
    k[0, 0, 40] = float("nan")
    k[1] *= 2.0 ** 110
    k[2] *= 2.0 ** -100
    k[3] *= 2.0 ** -90
    v = k.flip(0).contiguous()
    bt = i32([[0]])
    cache = [torch.zeros(1, 1, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16, 64, dtype=torch.uint8),
             torch.zeros(1, 1, 16, 4, dtype=torch.int16), torch.zeros(1, 1, 16, 4, dtype=torch.int16)]
    got = dev(*cache)
    args = (bt.to(DEV), i32([0]).to(DEV))
    A.attn_kv_append_paged_q4(None, k.to(DEV), v.to(DEV), *got, *args, cu_seqlens_new=i32([0, 4]).to(DEV))
    gk, gv = A.attn_kv_gather_paged_q4(*got, bt.to(DEV), i32([0, 4]).to(DEV), 4)
    gk = gk.cpu().double()
    bad = torch.isnan(gk[0, 0])
    assert bad[:64].all() and not bad[64:].any()         # the two groups, and no other
    for r in range(1, 4):
        ref = R.values(*R.quantise(k[r], group))
        assert np.array_equal(gk[r].numpy(), ref)
    assert torch.equal(gv.flip(0).cpu().double().nan_to_num(), gk.nan_to_num())


def test_append_bad_pages_and_rows_behind():
    D, group, Hkv = 64, 64, 2
    cache = R.fill((6, Hkv, 16, 32), group, 7)
    k, v, q = randn((9, Hkv, D), 8), randn((9, Hkv, D), 9), randn((9, 4, D), 10)
    bt = i32([[0, 1], [2, 6], [-1, 3]])
    used, cu = [14, 15, 2], [1, 4, 6, 8]                  # rows 0 and 8 belong to no sequence
    got = dev(*cache)
    out_q = torch.full((9, 4, D), 9.0, dtype=torch.bfloat16, device=DEV)
    A.attn_kv_append_paged_q4(q.to(DEV), k.to(DEV), v.to(DEV), *got, bt.to(DEV), i32(used).to(DEV),
                              cu_seqlens_new=i32(cu).to(DEV), out_q=out_q)
    assert A.attn_device_error() == 502
    want = R.append(*cache, k[1:5], v[1:5], i32([[0, 1], [2, 0]]), [0, 3, 4], [14, 15], group)
    for g, w in zip(got, want):
        assert same(g, w)
    assert (out_q[0] == 9).all() and (out_q[8] == 9).all() and torch.equal(out_q[1:8].cpu(), q[1:8])
    # a position past the block table
    A.attn_kv_append_paged_q4(None, k[:3].to(DEV), v[:3].to(DEV), *got, i32([[0], [1], [2]]).to(DEV), i32([16, -1, 100]).to(DEV))
    assert A.attn_device_error() == 501
    for g, w in zip(got, want):
        assert same(g, w)


def test_gather_leaves_other_rows():
    D, group, Hkv = 128, 64, 1
    cache = R.fill((4, Hkv, 16, 64), group, 11)
    bt = i32([[2, 0, 1], [3, 3, 99]])
    out = [torch.full((40, Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    gk, gv = A.attn_kv_gather_paged_q4(*dev(*cache), bt.to(DEV), i32([3, 20, 27]).to(DEV), 40,
                                       starts=i32([9, 13]).to(DEV), out_k=out[0], out_v=out[1])
    assert A.attn_device_error() == 0
    wk, wv = R.packed(*cache, bt, [17, 7], [9, 13])
    assert torch.equal(gk[3:27].cpu(), wk) and torch.equal(gv[3:27].cpu(), wv)
    for t in (gk, gv):
        assert (t[:3] == 5).all() and (t[27:] == 5).all()
    # a page outside the cache: reported, page 0 in its place
    gk, _ = A.attn_kv_gather_paged_q4(*dev(*cache), bt.to(DEV), i32([0, 0, 3]).to(DEV), 3, starts=i32([0, 32]).to(DEV))
    assert A.attn_device_error() == 411
    assert torch.equal(gk.cpu(), R.packed(*cache, i32([[0]]), [3])[0])


# ---------------------------------------------------------------- decode
def run_decode(lens, Hq, Hkv, D, group, seed=0, window=-1, softcap=0.0, scale=None, qscale=1.0, cache=None):
    bt, pool = table_for(lens, seed=seed)
    cache = R.fill((pool, Hkv, 16, D // 2), group, seed + 1) if cache is None else cache(pool)
    q = randn((len(lens), Hq, D), seed + 2, qscale)
    o, lse = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), bt.to(DEV), i32(lens).to(DEV), scale=scale,
                                    window_left=window, softcap=softcap)
    assert A.attn_device_error() == 0
    s = scale or 1 / math.sqrt(D)
    o_ref, lse_ref = reference(q, cache, bt, lens, list(range(len(lens) + 1)), s, True, window, softcap)
    tol_o, tol_lse = tolerances(q, cache, s)
    check(o, lse, o_ref, lse_ref.T.copy(), tol_o, tol_lse)
    return q, cache, bt, o, lse


@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (16, 1), (9, 3), (32, 8)])
def test_decode_matches_oracle(D, group, Hq, Hkv):
    run_decode([0, 1, 2, 15, 16, 17, 33, 250, 0, 700], Hq, Hkv, D, group, seed=D + Hq)


@pytest.mark.parametrize("Hq,Hkv", [(16, 16), (24, 12), (11, 11), (34, 17), (7, 1), (40, 8), (20, 1), (25, 1), (64, 2), (64, 1)])
def test_decode_head_counts(Hq, Hkv):
    run_decode([5, 100, 0, 333], Hq, Hkv, 64, 32, seed=Hq)


@pytest.mark.parametrize("window", [0, 1, 15, 16, 100, 5000])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_decode_window_and_softcap(window, softcap):
    run_decode([1, 16, 17, 300, 0, 1000], 8, 2, 128, 64, seed=window, window=window, softcap=softcap)


def test_decode_many_and_long():
    run_decode([3] * 300 + [2000], 2, 1, 64, 64, seed=3)
    run_decode([9000], 4, 1, 128, 128, seed=4)


def test_decode_all_sequences_empty():
    run_decode([0, 0, 0], 8, 2, 128, 128, seed=5)


def test_decode_sharp_and_large_scores():
    run_decode([600, 40], 8, 2, 128, 64, seed=6, qscale=30.0)
    run_decode([600, 40], 8, 2, 128, 64, seed=7, qscale=1e-20)
    run_decode([90, 40], 4, 2, 64, 32, seed=8, scale=0.7)


def test_decode_steps_of_very_different_size():
    """Values that grow by 2^60 along the sequence, and shrink: the weights keep in range."""
    D, group, Hkv = 64, 32, 1
    lens = [200, 199]
    for order in (1, -1):
        bt, pool = table_for(lens, seed=9)
        cache = [torch.zeros(pool, Hkv, 16, D // 2, dtype=torch.uint8) for _ in range(2)] + \
                [torch.zeros(pool, Hkv, 16, D // group, dtype=torch.int16) for _ in range(2)]
        k, v = randn((399, Hkv, D), 10), randn((399, Hkv, D), 11)
        size = torch.cat([torch.linspace(-30, 30, n) for n in lens])[:, None, None] * order
        v = (v.float() * 2.0 ** size.round()).to(torch.bfloat16)
        got = dev(*cache)
        A.attn_kv_append_paged_q4(None, k.to(DEV), v.to(DEV), *got, bt.to(DEV), i32([0, 0]).to(DEV),
                                  cu_seqlens_new=i32([0, 200, 399]).to(DEV))
        cache = [t.cpu() for t in got]
        q = randn((2, 4, D), 12)
        o, lse = A.attn_decode_paged_q4(q.to(DEV), *got, bt.to(DEV), i32(lens).to(DEV))
        o_ref, lse_ref = reference(q, cache, bt, lens, [0, 1, 2], 1 / 8, True, -1, 0.0)
        tol_o, tol_lse = tolerances(q, cache, 1 / 8)
        check(o, lse, o_ref, lse_ref.T.copy(), tol_o, tol_lse)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_decode_zero_queries_of_a_tiny_scale(softcap):
    # the smallest unit of a score times the smallest scale is not a float
    Hq, Hkv, D, group, lens, scale = 4, 2, 64, 32, [37, 5], 1e-25
    bt, pool = table_for(lens)
    cache = R.fill((pool, Hkv, 16, D // 2), group, 5)
    q = randn((2, Hq, D), 6)
    q[:, ::2] = 0
    o, lse = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), bt.to(DEV), i32(lens).to(DEV), scale=scale, softcap=softcap)
    o_ref, lse_ref = reference(q, cache, bt, lens, i32([0, 1, 2]), scale, True, -1, softcap)
    check(o, lse, o_ref, lse_ref.T, *tolerances(q, cache, scale))


def test_decode_ignores_what_lies_behind_the_length():
    """NaN steps in the last page's free rows and in unused pages change nothing."""
    lens = [5, 18, 0]
    bt, pool = table_for(lens, seed=13)
    cache = R.fill((pool, 2, 16, 32), 32, 14)
    q = randn((3, 4, 64), 15)
    o, lse = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), bt.to(DEV), i32(lens).to(DEV))
    used = torch.zeros(pool, 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[bt[b, t // 16], t % 16] = True
    for m in cache[2:]:
        m.transpose(1, 2)[~used] = 0x7FC0
    o2, lse2 = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), bt.to(DEV), i32(lens).to(DEV))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    cache[2][bt[0, 0], 1, 3] = 0x7FC0                     # a NaN among the keys of head 1 of sequence 0
    cache[3][bt[1, 0], 0, 3] = 0x7FC0                     # among the values of head 0 of sequence 1
    o3, lse3 = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), bt.to(DEV), i32(lens).to(DEV))
    assert torch.isnan(o3[0, 2:]).all() and torch.isnan(lse3[0, 2:]).all() and torch.equal(o3[0, :2], o[0, :2])
    assert torch.isnan(o3[1, :2]).all() and torch.equal(lse3[1], lse[1]) and torch.equal(o3[1, 2:], o[1, 2:])
    assert torch.equal(o3[2], o[2])


def test_decode_reports_pages_outside():
    bt = i32([[0, 77, 1]])
    cache = R.fill((3, 1, 16, 64), 128, 16)
    q = randn((1, 4, 128), 17)
    o, lse = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), bt.to(DEV), i32([40]).to(DEV))
    assert A.attn_device_error() == 411
    o2, lse2 = A.attn_decode_paged_q4(q.to(DEV), *dev(*cache), i32([[0, 0, 1]]).to(DEV), i32([40]).to(DEV))
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and A.attn_device_error() == 0


def test_decode_is_the_same_every_time_and_in_graphs_that_share_nothing():
    lens = [700, 33, 1200, 5]
    q, cache, bt, o, lse = run_decode(lens, 8, 2, 128, 64, seed=18)
    dc, dbt, dl, dq = dev(*cache), bt.to(DEV), i32(lens).to(DEV), q.to(DEV)
    for _ in range(3):
        o2, lse2 = A.attn_decode_paged_q4(dq, *dc, dbt, dl)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        ws = torch.empty(A.attn_decode_q4_workspace_size(4, 8, 2, 128), dtype=torch.uint8, device=DEV)
        with torch.cuda.graph(g):
            outs.append(A.attn_decode_paged_q4(dq, *dc, dbt, dl, workspace=ws))
        graphs.append((g, ws))
    s = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        with torch.cuda.stream(s[i]):
            for _ in range(5):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for x in outs:
        assert torch.equal(x[0], o) and torch.equal(x[1], lse)


def test_decode_refuses_small_workspace_and_wrong_tensors():
    lens = [20]
    bt, pool = table_for(lens)
    cache = dev(*R.fill((pool, 1, 16, 32), 32, 19))
    q, dl = randn((1, 2, 64), 20).to(DEV), i32(lens).to(DEV)
    dbt = bt.to(DEV)
    with pytest.raises(A.AttnError) as e:
        A.attn_decode_paged_q4(q, *cache, dbt, dl, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == 5
    for bad in (dict(q=q.float()), dict(q=q.transpose(0, 1)), dict(dl=dl.long()), dict(dbt=dbt.cpu()),
                dict(dl=i32([20, 3]).to(DEV))):
        a = dict(q=q, dbt=dbt, dl=dl)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            A.attn_decode_paged_q4(a["q"], *cache, a["dbt"], a["dl"])
    for i in range(4):
        c = list(cache)
        c[i] = c[i][..., :-1]
        with pytest.raises((TypeError, ValueError)):
            A.attn_decode_paged_q4(q, *c, dbt, dl)


def test_decode_past_4_gib_and_without_lse():
    """Page offsets past 32 bits, in the append, the read back and the decode alike."""
    Hkv, D, group, pool = 8, 128, 128, 540_000                 # 4.4 GB of codes each
    big = [torch.empty(pool, Hkv, 16, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
          [torch.empty(pool, Hkv, 16, 1, dtype=torch.int16, device=DEV) for _ in range(2)]
    small = [torch.zeros(3, Hkv, 16, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
            [torch.zeros(3, Hkv, 16, 1, dtype=torch.int16, device=DEV) for _ in range(2)]
    far, near = i32([[pool - 1, 5, pool - 2]]).to(DEV), i32([[0, 1, 2]]).to(DEV)
    k, v, q = randn((45, Hkv, D), 70).to(DEV), randn((45, Hkv, D), 71).to(DEV), randn((1, 16, D), 72).to(DEV)
    cu, used = i32([0, 45]).to(DEV), i32([45]).to(DEV)
    got = []
    for cache, bt in ((big, far), (small, near)):
        A.attn_kv_append_paged_q4(None, k, v, *cache, bt, i32([0]).to(DEV), cu_seqlens_new=cu)
        o, none = A.attn_decode_paged_q4(q, *cache, bt, used, return_lse=False)
        assert none is None
        got.append((o, *A.attn_kv_gather_paged_q4(*cache, bt, cu, 45)))
    assert A.attn_device_error() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_decode_nan_query_stays_in_its_row():
    lens = [300, 20]
    bt, pool = table_for(lens, seed=73)
    cache = dev(*R.fill((pool, 2, 16, 32), 64, 74))
    q = randn((2, 8, 64), 75)
    want = A.attn_decode_paged_q4(q.to(DEV), *cache, bt.to(DEV), i32(lens).to(DEV))
    q[0, 3, 7] = float("nan")
    o, lse = A.attn_decode_paged_q4(q.to(DEV), *cache, bt.to(DEV), i32(lens).to(DEV))
    assert torch.isnan(o[0, 3]).all() and torch.isnan(lse[0, 3])
    keep = torch.ones(2, 8, dtype=torch.bool, device=DEV)
    keep[0, 3] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_calls_on_a_given_stream():
    lens = [500, 77]
    bt, pool = table_for(lens, seed=76)
    cache = dev(*R.fill((pool, 2, 16, 64), 64, 77))
    q, dbt, dl = randn((2, 8, 128), 78).to(DEV), bt.to(DEV), i32(lens).to(DEV)
    want = A.attn_decode_paged_q4(q, *cache, dbt, dl)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [A.attn_decode_paged_q4(q, *cache, dbt, dl, stream=s) for _ in range(8)]
    outs += [A.attn_fwd_varlen_paged_q4(q, *cache, block_table=dbt, cu_seqlens_q=i32([0, 1, 2]).to(DEV), max_seqlen_q=17,
                                        seqused_k=dl, total_k=577, mask=A.MASK_CAUSAL, stream=s)]
    s.synchronize()
    for o, lse in outs[:-1]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    # the packed path (its own rounding of the probabilities): its tolerances
    assert float((outs[-1][0].float() - want[0].float()).abs().max()) <= TOL_O_PACKED
    assert float((outs[-1][1] - want[1].t()).abs().max()) <= TOL_LSE_PACKED


def test_a_given_stream_takes_memory_of_its_own():
    """What the current stream may still read is not handed to a call on another stream."""
    lens = [64, 64]
    bt, pool = table_for(lens, seed=79)
    cache = dev(*R.fill((pool, 2, 16, 64), 64, 80))
    q, dbt, dl = randn((2, 8, 128), 81).to(DEV), bt.to(DEV), i32(lens).to(DEV)
    cu, cs = i32([0, 64, 128]).to(DEV), R.table(64, 128).to(DEV)
    pos, s = i32([3, 5]).to(DEV), torch.cuda.Stream()
    kv = randn((2, 2, 128), 82).to(DEV)
    calls = [lambda: A.attn_decode_paged_q4(q, *cache, dbt, dl, stream=s),
             lambda: A.attn_fwd_varlen_paged_q4(q, *cache, block_table=dbt, cu_seqlens_q=i32([0, 1, 2]).to(DEV),
                                                max_seqlen_q=1, seqused_k=dl, total_k=128, mask=1, stream=s),
             lambda: A.attn_rope(q, kv, cos_sin=cs, positions=pos, stream=s),
             lambda: A.attn_kv_append_paged_q4(q, kv, kv, *cache, dbt, dl - 1, cos_sin=cs, stream=s),
             lambda: A.attn_kv_gather_paged_q4(*cache, dbt, cu, 128, stream=s)]
    for call in calls:
        torch.cuda.synchronize()
        shapes = [(t.shape, t.dtype) for t in call()]
        torch.cuda.synchronize()
        olds = [torch.zeros(shape, dtype=dtype, device=DEV) for shape, dtype in shapes]
        places = {t.data_ptr() for t in olds}
        del olds
        assert not places & {t.data_ptr() for t in call()}
    torch.cuda.synchronize()
    assert A.attn_device_error() == 0


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (8, 2), (12, 12), (32, 8)])
def test_decode_many_short_sequences(D, group, Hq, Hkv):
    """Shares that hold many sequences, some without keys, and their joins."""
    g = torch.Generator().manual_seed(Hq)
    lens = [int(n) for n in torch.randint(0, 60, (170,), generator=g)]
    lens[5:9] = [0, 0, 0, 1]
    run_decode(lens, Hq, Hkv, D, group, seed=80 + Hq)


def test_decode_largest_batch():
    g = torch.Generator().manual_seed(3)
    lens = [int(n) for n in torch.randint(0, 40, (4096,), generator=g)]
    run_decode(lens, 4, 2, 64, 64, seed=91)
    with pytest.raises(A.AttnError):
        run_decode([1] * 4097, 4, 2, 64, 64, seed=92)


# ---------------------------------------------------------------- several queries
def run_fwd(lens, qs, Hq, Hkv, D, group, causal=True, window=-1, softcap=0.0, seed=0, total_k=None):
    bt, pool = table_for(lens, seed=seed)
    cache = R.fill((pool, Hkv, 16, D // 2), group, seed + 1)
    q = randn((sum(qs), Hq, D), seed + 2)
    cu_q = i32(np.concatenate([[0], np.cumsum(qs)]))
    total_k = sum(lens) if total_k is None else total_k
    o, lse = A.attn_fwd_varlen_paged_q4(q.to(DEV), *dev(*cache), block_table=bt.to(DEV), cu_seqlens_q=cu_q.to(DEV),
                                        max_seqlen_q=max(qs), seqused_k=i32(lens).to(DEV), total_k=total_k,
                                        mask=A.MASK_CAUSAL if causal else A.MASK_NONE, window_left=window, softcap=softcap)
    assert A.attn_device_error() == 0
    s = 1 / math.sqrt(D)
    o_ref, lse_ref = reference(q, cache, bt, lens, cu_q, s, causal, window, softcap)
    tol_o, tol_lse = tolerances(q, cache, s)
    if max(qs) * (Hq // Hkv) > 128:
        tol_o, tol_lse = TOL_O_PACKED, TOL_LSE_PACKED
    check(o, lse, o_ref, lse_ref, tol_o, tol_lse)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("qs", [[1, 1, 1, 1, 1], [2, 1, 0, 2, 2], [4, 3, 0, 1, 4], [5, 0, 6, 1, 2], [8, 5, 1, 1, 7], [11, 16, 0, 1, 13], [5, 40, 0, 1, 130]])
@pytest.mark.parametrize("causal", [True, False])
def test_fwd_matches_oracle(D, group, qs, causal):
    run_fwd([5, 64, 20, 1, 300], qs, 8, 2, D, group, causal=causal, seed=sum(qs))


@pytest.mark.parametrize("qs", [[3, 4, 2], [8, 7, 8], [20, 33, 17]])
@pytest.mark.parametrize("window,softcap", [(0, 0.0), (7, 15.0), (40, 0.0)])
def test_fwd_window_softcap(qs, window, softcap):
    run_fwd([100, 34, 17], qs, 4, 1, 128, 64, window=window, softcap=softcap, seed=window)


@pytest.mark.parametrize("qs", [[4, 4], [8, 7], [30, 20]])
def test_fwd_more_queries_than_keys(qs):
    run_fwd([2, 0], qs, 4, 1, 64, 64, seed=30)
    run_fwd([2, 0], qs, 4, 1, 64, 64, seed=31, causal=False)


@pytest.mark.parametrize("Hq,Hkv,qs", [(8, 2, [17, 32, 0, 1, 25]), (8, 8, [128, 9, 100, 0, 65]), (12, 3, [3, 24, 31, 2, 8]),
                                       (8, 1, [16, 2, 1, 9, 12]), (14, 2, [18, 5, 9, 1, 16]), (5, 5, [9, 16, 17, 33, 0])])
@pytest.mark.parametrize("D,group,causal", [(64, 64, True), (128, 32, True), (128, 128, False)])
def test_fwd_row_tiles(Hq, Hkv, qs, D, group, causal):
    # up to 128 query rows per KV head, in tiles that a sequence fills, half fills or leaves empty
    run_fwd([37, 500, 20, 0, 163], qs, Hq, Hkv, D, group, causal=causal, seed=Hq)


@pytest.mark.parametrize("B", [127, 128, 129, 300])
def test_fwd_many_short_sequences(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 70, (B,), generator=g).tolist()
    qs = torch.randint(0, 4, (B,), generator=g).tolist()
    run_fwd(lens, qs, 8, 2, 64, 32, seed=B)


@pytest.mark.parametrize("qs", [[3, 3, 2], [40, 50, 33]])
def test_fwd_ignores_its_neighbours_and_the_workspace(qs):
    """NaN and infinite values of one sequence, and a workspace full of NaN, reach no other sequence."""
    Hq, Hkv, D, group, lens = 8, 2, 128, 64, [70, 37, 0]
    bt, pool = table_for(lens, seed=60)
    cache = R.fill((pool, Hkv, 16, D // 2), group, 61)
    for meta in cache[2:]:                            # all of sequence 1 stands for NaN
        for page in bt[1, :3].tolist():
            meta[page] = 0x7fc0
    q = randn((sum(qs), Hq, D), 62)
    cu = np.concatenate([[0], np.cumsum(qs)])
    need = A.attn_fwd_q4_workspace_size(3, max(qs), Hq, Hkv, D, 500)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    o, lse = A.attn_fwd_varlen_paged_q4(q.to(DEV), *dev(*cache), block_table=bt.to(DEV), cu_seqlens_q=i32(cu).to(DEV),
                                        max_seqlen_q=max(qs), seqused_k=i32(lens).to(DEV), total_k=500, mask=1, workspace=ws)
    assert A.attn_device_error() == 0
    first = R.fill((pool, Hkv, 16, D // 2), group, 61)
    o_ref, lse_ref = reference(q[:qs[0]], first, bt[:1], lens[:1], [0, qs[0]], D ** -0.5, True, -1, 0.0)
    tol_o, tol_lse = tolerances(q, first, D ** -0.5)
    if max(qs) * 4 > 128:
        tol_o, tol_lse = TOL_O_PACKED, TOL_LSE_PACKED
    check(o[:qs[0]], lse[:, :qs[0]], o_ref, lse_ref, tol_o, tol_lse)
    assert o[cu[1]:cu[2]].isnan().any()
    assert not o[cu[2]:].any() and bool((lse[:, cu[2]:] == -math.inf).all())


def test_fwd_without_any_key_past_the_page_stream():
    run_fwd([0, 0], [40, 50], 8, 2, 64, 32, seed=63)
    run_fwd([2, 0, 1], [40, 50, 3], 8, 2, 128, 64, seed=64)


def test_fwd_total_k_past_the_page_stream():
    lens = [100, 34]
    bt, pool = table_for(lens)
    cache = dev(*R.fill((pool, 2, 16, 32), 32, 33))
    q = randn((80, 4, 64), 34).to(DEV)
    A.attn_fwd_varlen_paged_q4(q, *cache, block_table=bt.to(DEV), cu_seqlens_q=i32([0, 10, 80]).to(DEV), max_seqlen_q=70,
                               seqused_k=i32(lens).to(DEV), total_k=120, mask=A.MASK_CAUSAL)
    assert A.attn_device_error() == 531


def test_fwd_total_k():
    run_fwd([100, 34], [40, 20], 4, 2, 64, 32, seed=32, total_k=1000)
    # too small a total: reported, and nothing outside the workspace
    lens = [100, 34]
    bt, pool = table_for(lens)
    cache = dev(*R.fill((pool, 2, 16, 32), 32, 33))
    q = randn((40, 4, 64), 34).to(DEV)
    A.attn_fwd_varlen_paged_q4(q, *cache, block_table=bt.to(DEV), cu_seqlens_q=i32([0, 20, 40]).to(DEV), max_seqlen_q=40,
                               seqused_k=i32(lens).to(DEV), total_k=120, mask=A.MASK_CAUSAL)
    assert A.attn_device_error() == 531


def test_fwd_reports_queries_outside():
    # offsets past total_q, and more queries than max_seqlen_q: reported, the rows inside computed
    Hq, Hkv, D, group, lens = 4, 2, 64, 32, [40, 70]
    bt, pool = table_for(lens)
    cache = R.fill((pool, Hkv, 16, D // 2), group, 5)
    q = randn((5, Hq, D), 6)
    run = lambda cu, most: A.attn_fwd_varlen_paged_q4(
        q.to(DEV), *dev(*cache), block_table=bt.to(DEV), cu_seqlens_q=i32(cu).to(DEV), max_seqlen_q=most,
        seqused_k=i32(lens).to(DEV), total_k=sum(lens), mask=1)
    o, lse = run([0, 2, 9], 7)
    assert A.attn_device_error() == 532
    o_ref, lse_ref = reference(q, cache, bt, lens, i32([0, 2, 5]), 1 / math.sqrt(D), True, -1, 0.0)
    check(o, lse, o_ref, lse_ref, *tolerances(q, cache, 1 / math.sqrt(D)))
    run([0, 2, 5], 2)
    assert A.attn_device_error() == 532
    run([-1, 2, 5], 3)
    assert A.attn_device_error() == 532
    assert A.attn_device_error() == 0


def test_fwd_leaves_rows_behind_the_last_sequence():
    for qs, top in (([2, 3], 3), ([20, 3], 20), ([40, 3], 40)):
        lens = [50, 30]
        bt, pool = table_for(lens)
        cache = dev(*R.fill((pool, 2, 16, 32), 32, 35))
        n = sum(qs) + 6
        q = randn((n, 4, 64), 36).to(DEV)
        out = torch.full_like(q, 3.0)
        lse = torch.full((4, n), 3.0, device=DEV)
        A.attn_fwd_varlen_paged_q4(q, *cache, block_table=bt.to(DEV), cu_seqlens_q=i32(np.concatenate([[0], np.cumsum(qs)])).to(DEV),
                                   max_seqlen_q=top, seqused_k=i32(lens).to(DEV), total_k=80, mask=A.MASK_CAUSAL, out=out, lse=lse)
        assert A.attn_device_error() == 0
        assert (out[sum(qs):] == 3).all() and (lse[:, sum(qs):] == 3).all() and torch.isfinite(out[:sum(qs)]).all()


def test_nothing_to_do():
    cache = dev(*R.fill((2, 1, 16, 32), 32, 50))
    none, bt = i32([]).to(DEV), i32([[0], [1]]).to(DEV)
    used = i32([3, 4]).to(DEV)
    e = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    q, out = A.attn_kv_append_paged_q4(e, e, e, *cache, bt, used, cu_seqlens_new=i32([0, 0, 0]).to(DEV))
    assert q.shape == (0, 1, 64) and out.tolist() == [3, 4]
    assert A.attn_kv_gather_paged_q4(*cache, bt, i32([0, 0, 0]).to(DEV), 0)[0].shape == (0, 1, 64)
    assert A.attn_decode_paged_q4(e, *cache, torch.empty(0, 1, dtype=torch.int32, device=DEV), none)[0].shape == (0, 1, 64)
    o, lse = A.attn_fwd_varlen_paged_q4(e, *cache, block_table=bt, cu_seqlens_q=i32([0, 0, 0]).to(DEV), max_seqlen_q=0,
                                        seqused_k=used, total_k=7)
    assert o.shape == (0, 1, 64) and lse.shape == (1, 0)


# ---------------------------------------------------------------- together
def test_serving_run_prefill_decode_and_draft():
    """Prefill a prompt into 4-bit pages, decode tokens one by one, verify a draft: each
    step's attention is the oracle's over the cache as it then stands."""
    B, Hq, Hkv, D, group, rot = 3, 8, 2, 128, 64, 64
    prompt, made = [40, 7, 130], 4
    bt, pool = table_for([p + 32 for p in prompt], seed=40)
    cache = [torch.zeros(pool, Hkv, 16, D // 2, dtype=torch.uint8, device=DEV) for _ in range(2)] + \
            [torch.zeros(pool, Hkv, 16, D // group, dtype=torch.int16, device=DEV) for _ in range(2)]
    dbt = bt.to(DEV)
    cs = R.table(512, rot).to(DEV)
    s = 1 / math.sqrt(D)
    used = torch.zeros(B, dtype=torch.int32, device=DEV)
    seed = 41

    def step(new, used):
        nonlocal seed
        T = sum(new)
        q, k, v = (randn((T, h, D), seed + i).to(DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
        seed += 3
        cu = i32(np.concatenate([[0], np.cumsum(new)]))
        q, used = A.attn_kv_append_paged_q4(q, k, v, *cache, dbt, used, cos_sin=cs, cu_seqlens_new=cu.to(DEV))
        if max(new) == 1:
            o, lse = A.attn_decode_paged_q4(q, *cache, dbt, used)
            lse = lse.t()
        else:
            o, lse = A.attn_fwd_varlen_paged_q4(q, *cache, block_table=dbt, cu_seqlens_q=cu.to(DEV), max_seqlen_q=max(new),
                                                seqused_k=used, total_k=512, mask=A.MASK_CAUSAL)
        host = [c.cpu() for c in cache]
        o_ref, lse_ref = reference(q.cpu(), host, bt, used.tolist(), cu, s, True, -1, 0.0)
        tol = tolerances(q.cpu(), host, s) if max(new) * Hq // Hkv <= 64 else (TOL_O_PACKED, TOL_LSE_PACKED)
        check(o, lse, o_ref, lse_ref, *tol)
        return used

    used = step(prompt, used)
    for _ in range(made):
        used = step([1] * B, used)
    used = step([4, 3, 2], used)
    assert used.tolist() == [p + made + n for p, n in zip(prompt, (4, 3, 2))]
    assert A.attn_device_error() == 0


def test_training_run_rope_attention_and_its_gradient():
    """rope -> attention -> backward -> inverse rope: the gradient with respect to the
    unrotated q and k is that of the fp64 chain."""
    L, Hq, Hkv, D, rot = 70, 4, 2, 64, 32
    q, k, v, do = (randn((L, h, D), 60 + i) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    cs, pos = R.table(L, rot), torch.arange(L, dtype=torch.int32)
    dcs, dpos = cs.to(DEV), pos.to(DEV)
    rq, rk = A.attn_rope(q.to(DEV), k.to(DEV), cos_sin=dcs, positions=dpos)
    o, lse = A.attn_fwd_dense(rq[None], rk[None], v.to(DEV)[None], causal=True)
    dq, dk, dv = A.attn_bwd_dense(rq[None], rk[None], v.to(DEV)[None], o, do.to(DEV)[None], lse, causal=True)
    gq, gk = A.attn_rope(dq[0], dk[0], cos_sin=dcs, positions=dpos, inverse=True)
    rq64, rk64 = R.rope(q, cs, pos), R.rope(k, cs, pos)
    wq, wk, wv = oracle.attn_bwd_dense(torch.from_numpy(rq64)[None], torch.from_numpy(rk64)[None], v[None], do[None],
                                       scale=1 / math.sqrt(D), causal=True)
    for got, ref in ((gq, R.rope(torch.from_numpy(np.ascontiguousarray(wq[0])), cs, pos, inverse=True)),
                     (gk, R.rope(torch.from_numpy(np.ascontiguousarray(wk[0])), cs, pos, inverse=True))):
        err = float(np.abs(got.double().cpu().numpy() - ref).max())
        # the library's bound for its gradients (2e-2 of the largest plus 2e-3), twice for the
        # rounding of the rotated operands and of the gradient's own rotation
        assert err <= 2 * (2e-2 * float(np.abs(ref).max()) + 2e-3), err
