"""Rotary positions and the rotating append, against the fp64 oracle and bit for bit.

attn_rope's result is the fp64 rotation off by three roundings to fp32 of terms of at
most |x1| + |x2| and one to bf16 (half a step: 2^-8 relative).  The append must equal
attn_rope followed by the plain append bit for bit.
"""
import numpy as np
import pytest
import torch

from attention_paged_kv_gqa_b200 import binding as A
from oracle import rope_q4 as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert A.attn_check_device(0) == 0
    torch.cuda.set_device(0)


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def close(y, x, ref):
    y, x = y.double().cpu().numpy(), x.double().cpu().numpy()
    big = np.abs(x).max(-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(ref) + 4 * 2.0 ** -24 * 2 * big
    assert (np.abs(y - ref) <= tol).all(), float(np.abs(y - ref).max())


def axes_of(n_axes, total, rot, seed, top):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, top, (n_axes, total), generator=g, dtype=torch.int32)
    axis = torch.randint(0, n_axes, (rot // 2,), generator=g, dtype=torch.int32)
    return pos, axis


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 64), (128, 48), (128, 96), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hkv,T", [(1, 1, 1), (8, 2, 5), (5, 5, 67), (32, 8, 700)])
def test_rope_matches_oracle(D, rot, interleaved, Hq, Hkv, T):
    q, k = randn((T, Hq, D), 1), randn((T, Hkv, D), 2)
    cs = R.table(1000, rot)
    pos = torch.randint(0, 1000, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    for inverse in (False, True):
        yq, yk = A.attn_rope(q.to(DEV), k.to(DEV), cos_sin=cs.to(DEV), positions=pos.to(DEV), interleaved=interleaved,
                             inverse=inverse)
        close(yq, q, R.rope(q, cs, pos, None, interleaved, inverse))
        close(yk, k, R.rope(k, cs, pos, None, interleaved, inverse))
    assert A.attn_device_error() == 0


@pytest.mark.parametrize("n_axes", [2, 3, 4])
@pytest.mark.parametrize("sections", [False, True])
def test_rope_axes(n_axes, sections):
    T, H, D, rot = 33, 6, 128, 96
    q = randn((T, H, D), 4)
    pos, axis = axes_of(n_axes, T, rot, 5, 60)
    if sections:                                    # whole runs of eight pairs on one axis
        axis = i32([min(i // 16, n_axes - 1) for i in range(rot // 2)])
    cs = R.table(60, rot)
    for interleaved in (False, True):
        y, none = A.attn_rope(q.to(DEV), cos_sin=cs.to(DEV), positions=pos.to(DEV), pair_axis=axis.to(DEV),
                              interleaved=interleaved)
        assert none is None
        close(y, q, R.rope(q, cs, pos, axis, interleaved))


def test_rope_packed_views_in_place_and_rows_beside():
    T, Hq, Hkv, D = 19, 4, 2, 64
    x = randn((T, Hq + 2 * Hkv + 1, D), 6).to(DEV)
    before = x.clone()
    cs, pos = R.table(40, 32).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    want = A.attn_rope(q.contiguous(), k.contiguous(), cos_sin=cs, positions=pos)
    got = A.attn_rope(q, k, cos_sin=cs, positions=pos, out_q=q, out_k=k)
    assert got[0].data_ptr() == x.data_ptr()
    assert torch.equal(x[:, :Hq], want[0]) and torch.equal(x[:, Hq:Hq + Hkv], want[1])
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])


def test_rope_inverse_is_the_gradient():
    """<dy, J dx> by the forward on basis directions equals <inverse(dy), dx>, and the
    inverse's value is the formula's."""
    T, H, D, rot = 3, 2, 64, 64
    cs, pos = R.table(300, rot), i32([0, 17, 299])
    dy, dx = randn((T, H, D), 7), randn((T, H, D), 8)
    g, _ = A.attn_rope(dy.to(DEV), cos_sin=cs.to(DEV), positions=pos.to(DEV), inverse=True)
    close(g, dy, R.rope(dy, cs, pos, inverse=True))
    # differences of the (linear) forward: f(x + dx) - f(x) in fp64 by the oracle
    x = randn((T, H, D), 9).double()
    diff = R.rope(x + dx.double(), cs, pos) - R.rope(x, cs, pos)
    left = float((torch.from_numpy(diff) * dy.double()).sum())
    right = float((g.double().cpu() * dx.double()).sum())
    # each gradient element is off by 2^-8 of itself at most
    tol = 2.0 ** -8 * float((g.double().cpu().abs() * dx.double().abs()).sum()) + 1e-5
    assert abs(left - right) <= tol


def test_rope_reports_positions_and_axes_outside():
    T, D, rot = 4, 64, 32
    q = randn((T, 1, D), 10)
    cs = R.table(8, rot)
    y, _ = A.attn_rope(q.to(DEV), cos_sin=cs.to(DEV), positions=i32([0, 8, -3, 7]).to(DEV))
    assert A.attn_device_error() == 521
    close(y, q, R.rope(q, cs, i32([0, 7, 0, 7])))
    axis = torch.zeros(rot // 2, dtype=torch.int32)
    axis[5] = 2
    pos = i32([[1, 2, 3, 4], [0, 0, 0, 0]])
    y, _ = A.attn_rope(q.to(DEV), cos_sin=cs.to(DEV), positions=pos.to(DEV), pair_axis=axis.to(DEV))
    assert A.attn_device_error() == 522
    axis[5] = 0
    close(y, q, R.rope(q, cs, pos, axis))
    y, _ = A.attn_rope(q[:0].to(DEV), cos_sin=cs.to(DEV), positions=i32([]).to(DEV))
    assert y.shape == (0, 1, D) and A.attn_device_error() == 0


def test_rope_special_values_stay_in_their_pair():
    q = randn((2, 1, 64), 11)
    q[0, 0, 3] = float("inf")
    q[1, 0, 5] = float("nan")
    cs = R.table(9, 64).to(DEV)
    y, _ = A.attn_rope(q.to(DEV), cos_sin=cs, positions=i32([3, 4]).to(DEV))
    bad = (~torch.isfinite(y.cpu().float())).nonzero().tolist()
    assert {tuple(b) for b in bad} == {(0, 0, 3), (0, 0, 35), (1, 0, 5), (1, 0, 37)}


def appended(q, k, v, cache, bt, used, dtype, descale, **kw):
    """attn_rope, the cast and attn_kv_append_paged, one after the other."""
    rope = {n: kw.pop(n) for n in ("cos_sin", "positions", "pair_axis", "interleaved") if n in kw}
    cu = kw.get("cu_seqlens_new")
    if rope.get("cos_sin") is not None:
        if rope.get("positions") is None:
            c = cu.tolist() if cu is not None else list(range(len(used) + 1))
            rope["positions"] = torch.cat([torch.arange(int(used[b]), int(used[b]) + c[b + 1] - c[b], dtype=torch.int32)
                                           for b in range(len(used))]).to(DEV)
        q, k = A.attn_rope(q, k, **rope)
    x = []
    for t, d in zip((q, k, v), descale):
        t = t.contiguous()
        if dtype == torch.float8_e4m3fn:
            t = (t.float() * (1 / d)).clamp(-448, 448).to(dtype)
        x.append(t)
    kc, vc = (c.clone() for c in cache)
    out = A.attn_kv_append_paged(x[1], x[2], kc, vc, bt, used, cu_seqlens_new=cu)
    return x[0], kc, vc, out


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 96), (128, 0)])
@pytest.mark.parametrize("own_positions", [False, True])
def test_append_equals_rope_then_append(dtype, D, rot, own_positions):
    Hq, Hkv = 6, 3
    before, new = [0, 1, 15, 16, 17, 100, 255, 3], [3, 0, 1, 16, 40, 300, 1, 0]
    T, B = sum(new), len(new)
    qkv = randn((T, Hq + 2 * Hkv, D), 20).to(DEV) * 3
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cache = [randn((300, 16, Hkv, D), s).to(dtype).to(DEV) for s in (21, 22)]
    bt = torch.randperm(300, generator=torch.Generator().manual_seed(23))[:B * 30].reshape(B, 30).to(torch.int32).to(DEV)
    cu = i32(np.concatenate([[0], np.cumsum(new)])).to(DEV)
    used = i32(before).to(DEV)
    descale = [torch.tensor([d], device=DEV) for d in (0.013, 0.03, 0.007)]
    kw = dict(cu_seqlens_new=cu)
    if rot:
        kw.update(cos_sin=R.table(500, rot).to(DEV), interleaved=D == 64)
        if own_positions:
            pos, axis = axes_of(3, T, rot, 24, 500)
            kw.update(positions=pos.to(DEV), pair_axis=axis.to(DEV))
    want = appended(q, k, v, cache, bt, used, dtype, descale, **kw)
    kc, vc = (c.clone() for c in cache)
    if dtype == torch.float8_e4m3fn:
        kw.update(descale_q=descale[0], descale_k=descale[1], descale_v=descale[2])
    yq, out = A.attn_kv_append_rope_paged(q, k, v, kc, vc, bt, used, **kw)
    assert A.attn_device_error() == 0
    assert yq.dtype == dtype and torch.equal(bits(yq), bits(want[0]))
    assert torch.equal(bits(kc), bits(want[1])) and torch.equal(bits(vc), bits(want[2])) and torch.equal(out, want[3])
    # keys and values alone
    kc, vc = (c.clone() for c in cache)
    none, _ = A.attn_kv_append_rope_paged(None, k, v, kc, vc, bt, used, **kw)
    assert none is None and torch.equal(bits(kc), bits(want[1])) and torch.equal(bits(vc), bits(want[2]))


def test_append_one_token_per_sequence_and_bad_pages():
    B, Hq, Hkv, D = 9, 8, 2, 128
    q, k, v = (randn((B, h, D), s).to(DEV) for h, s in ((Hq, 30), (Hkv, 31), (Hkv, 32)))
    cache = [randn((40, 16, Hkv, D), s).to(DEV) for s in (33, 34)]
    used = i32([0, 5, 16, 31, 32, 33, 47, 48, 2]).to(DEV)          # the eighth: past its three pages
    bt = torch.arange(27, dtype=torch.int32).reshape(9, 3)
    bt[1, 0], bt[2, 1] = 40, -1                                      # outside the cache
    cs = R.table(64, D).to(DEV)
    kc, vc = (c.clone() for c in cache)
    yq, out = A.attn_kv_append_rope_paged(q, k, v, kc, vc, bt.to(DEV), used, cos_sin=cs)
    assert A.attn_device_error() in (501, 502)
    wq, wk = A.attn_rope(q, k, cos_sin=cs, positions=used)
    assert torch.equal(yq, wq) and torch.equal(out, used + 1)
    wkc, wvc = (c.clone() for c in cache)
    for b in (0, 3, 4, 5, 6, 8):
        p = int(used[b])
        wkc[bt[b, p // 16], p % 16], wvc[bt[b, p // 16], p % 16] = wk[b], v[b]
    assert torch.equal(kc, wkc) and torch.equal(vc, wvc)


def test_append_leaves_rows_behind_the_last_sequence():
    T, Hq, Hkv, D = 12, 2, 1, 64
    q, k, v = (randn((T, h, D), s).to(DEV) for h, s in ((Hq, 40), (Hkv, 41), (Hkv, 42)))
    cache = [torch.zeros(8, 16, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    bt = torch.arange(8, dtype=torch.int32, device=DEV).reshape(2, 4)
    out_q = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    A.attn_kv_append_rope_paged(q, k, v, *cache, bt, i32([0, 0]).to(DEV), cos_sin=R.table(16, 64).to(DEV),
                                cu_seqlens_new=i32([2, 5, 9]).to(DEV), out_q=out_q)
    assert A.attn_device_error() == 0
    assert (out_q[:2] == 7).all() and (out_q[9:] == 7).all() and not (out_q[2:9] == 7).all(-1).any()
    assert torch.equal(cache[1][0, :3], v[2:5]) and torch.equal(cache[1][4, :4], v[5:9])
    assert not cache[1][0, 3:].any() and not cache[1][1:4].any() and not cache[1][4, 4:].any()


def test_rope_on_another_stream_and_in_a_graph():
    T, Hq, Hkv, D = 40, 8, 2, 128
    q, k = randn((T, Hq, D), 50).to(DEV), randn((T, Hkv, D), 51).to(DEV)
    cs, pos = R.table(64, D).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    want = A.attn_rope(q, k, cos_sin=cs, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    oq, ok = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        A.attn_rope(q, k, cos_sin=cs, positions=pos, out_q=oq, out_k=ok)
        A.attn_rope(oq, ok, cos_sin=cs, positions=pos, out_q=oq, out_k=ok, inverse=True)
    q.copy_(randn((T, Hq, D), 52))
    graph.replay()
    torch.cuda.synchronize()
    # turned there and back: two roundings to bf16 of values of at most sqrt(2) the pair's size
    assert float((oq.float() - q.float()).abs().max()) <= 2 * 2.0 ** -8 * 1.5 * float(q.float().abs().max())
    got = A.attn_rope(q, k, cos_sin=cs, positions=pos, stream=s)
    s.synchronize()
    assert torch.equal(got[1], want[1])
