"""Attention over the 4-bit KV cache held to the size of its output, where the weights
p step differ widely, hardly at all, or belong to NaN.

The kernels read the same codes as the fp64 attention here.  Per query row and group g of
columns, with a_j the softmax weights, s_j the steps and v_j the values of the keys, the
error of O may be, as a root mean square over the group's columns:
  2^-8 rms(O)           the rounding to bf16: half a step, 2^-8 of each value
  2^-11 rms(O)          the f16 rounding of the weights, where all of them err alike
  4 * 2^-11 spread      the same where they err at random: n terms of at most 2^-11 a_j |v_j|
                        sum to an RMS of 2^-11 spread, spread^2 = sum a_j^2 v_j^2; four times that
  tol_s (rms(O) + 4 spread)   the error of the scores, which moves the a_j: in the same two ways
  2^-18 W               fp32 sums: W = sum a_j s_j 15 bounds sum a_j s_j c_j.  The accumulators take
                        16 truncating sums before they are centred, the i-th of at most i / 16 of
                        their keys' sum: 8.5 * 2^-23 of it for truncation to 24 bits; 2^-18 leaves
                        a factor of four for the alignment within an instruction and the joins
  2^-30 M               M = max a_j s_j 15, times the number of keys: weights below 2^-31 of the
                        row's and group's largest are lost (they are subnormal f16 numbers then)
The scores: with u the sum of |q| 15 s over the dims, eight truncating sums of at most 2^-23 of
it each, times two for alignment: tol_s = 2^-19 u scale, plus 2^-18 for exponentials, logarithm
and the running maximum in fp32.  tol_s bounds the error of the LSE as well.
"""
import math

import numpy as np
import pytest
import torch

from attention_paged_kv_gqa_b200 import binding as A
from oracle import rope_q4 as R

gpu = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert A.attn_check_device(0) == 0
    torch.cuda.set_device(0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def randn(shape, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(torch.bfloat16)


def pages_of(x, group, which):
    """(codes, metas) of the pages, in order, that hold the values x [tokens, Hkv, D]."""
    L, Hkv, D = x.shape
    n = -(-L // 16)
    full = torch.zeros(n * 16, Hkv, D, dtype=torch.bfloat16)
    full[:L] = x
    code, meta = R.quantise(full.view(n, 16, Hkv, D).transpose(1, 2), group)
    at = R._index(D, which).reshape(-1)
    nib = np.zeros((n, Hkv, 16 * D), np.uint8)
    nib[..., at] = code.reshape(n, Hkv, -1)
    return (torch.from_numpy((nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(n, Hkv, 16, D // 2)),
            torch.from_numpy(meta.view(np.int16).copy()))


def cache_of(k, v, group):
    """The cache (k, v, metas) of one sequence on pages 0, 1, .. in order."""
    (kc, km), (vc, vm) = pages_of(k, group, R.k_nibble), pages_of(v, group, R.v_nibble)
    return [kc, vc, km, vm]


def join(caches):
    """One cache of several sequences' pages, and its block table (unused entries outside)."""
    n = [c[0].shape[0] for c in caches]
    bt = torch.full((len(n), max(max(n), 1)), 1 << 29, dtype=torch.int32)
    at = 0
    for b, m in enumerate(n):
        bt[b, :m] = torch.arange(at, at + m)
        at += m
    return [torch.cat(x) for x in zip(*caches)], bt


def steps_of(meta):
    return ((meta.to(torch.int32) & 0xFFF0) << 16).view(torch.float32).double()


class Attention:
    """fp64 attention of q [n, Hq, D], the newest n of the cache's L tokens, with what its
    tolerances need: o, spread, W, M [n, Hq, D] and lse, tol_s [n, Hq]."""

    def __init__(self, q, cache, L, group, causal=True, window=-1, scale=None, skip=()):
        n, Hq, D = q.shape
        Hkv = cache[0].shape[1]
        G = Hq // Hkv
        pages = list(range(-(-L // 16)))
        k = torch.from_numpy(R.read(cache[0], cache[2], pages, True))[:L]
        v = torch.from_numpy(R.read(cache[1], cache[3], pages, False))[:L]
        ks, vs = (steps_of(m.transpose(1, 2).reshape(-1, Hkv, D // group))[:L].repeat_interleave(group, 2)
                  for m in cache[2:])
        scale = scale or 1 / math.sqrt(D)
        at = torch.arange(L - n, L)[:, None]
        j = torch.arange(L)[None]
        hidden = (j > at) | (j < at - window if window >= 0 else j < 0) if causal else torch.zeros(n, L, dtype=torch.bool)
        for first, last in skip:
            hidden = hidden | ((j >= first) & (j < last))
        self.n, self.group, self.keys = n, group, L
        self.o, self.spread, self.W, self.M = (torch.zeros(n, Hq, D, dtype=torch.float64) for _ in range(4))
        self.lse, self.tol_s = (torch.zeros(n, Hq, dtype=torch.float64) for _ in range(2))
        for h in range(Hkv):
            for g in range(h * G, (h + 1) * G):
                x = (q[:, g].double() @ k[:, h].T) * scale
                x[hidden] = -math.inf
                self.lse[:, g] = torch.logsumexp(x, -1)
                a = torch.exp(x - self.lse[:, g].clamp(min=-1e300)[:, None])
                a[hidden] = 0
                # a NaN reaches the rows that see its key, and no others
                for i in range(n):
                    see = ~hidden[i]
                    self.o[i, g] = a[i, see] @ v[see, h]
                    self.spread[i, g] = (a[i, see] ** 2 @ v[see, h] ** 2).sqrt()
                    self.W[i, g] = a[i, see] @ vs[see, h] * 15
                    if see.any():
                        self.M[i, g] = (a[i, see, None] * vs[see, h]).nan_to_num(0.0).amax(0) * 15
                u = (q[:, g].double().abs() @ ks[:, h].nan_to_num(0.0).T) * 15
                u[hidden] = 0
                self.tol_s[:, g] = 2.0 ** -19 * u.amax(-1) * scale + 2.0 ** -18

    def excess(self, o, lse):
        """The largest error of O as a share of its tolerance, and that of the LSE."""
        n, Hq, D = self.o.shape
        o, lse = o.double().cpu().view(n, Hq, D), lse.double().cpu().view(n, Hq)
        assert torch.equal(torch.isnan(o), torch.isnan(self.o))
        assert torch.equal(torch.isneginf(lse), torch.isneginf(self.lse))
        assert torch.equal(torch.isnan(lse), torch.isnan(self.lse))
        rms = lambda x: x.unflatten(-1, (-1, self.group)).square().mean(-1).sqrt()
        t = self.tol_s[..., None]
        tol = ((2.0 ** -8 + 2.0 ** -11 + t) * rms(self.o) + 4 * (2.0 ** -11 + t) * rms(self.spread)
               + 2.0 ** -18 * rms(self.W) + 2.0 ** -30 * self.keys * rms(self.M) + 1e-300)
        err = (rms(o - self.o) / tol).nan_to_num(0.0, posinf=math.inf)
        fin = torch.isfinite(self.lse)
        e = ((lse - self.lse).abs()[fin] / self.tol_s[fin])
        return float(err.max()), float(e.max()) if e.numel() else 0.0

    def check(self, o, lse):
        eo, el = self.excess(o, lse)
        assert eo <= 1 and el <= 1, "of the tolerance: O %.3g, LSE %.3g" % (eo, el)


def attend(q, caches, lens, group, causal=True, window=-1, softcap=0.0, max_q=None):
    """The library's attention of q (a list of [n, Hq, D]) -> lists of o and of lse [n, Hq]."""
    cache, bt = join(caches)
    ns = [len(x) for x in q]
    dc = [t.to(DEV) for t in cache]
    dq, dbt, dl = torch.cat(q).to(DEV), bt.to(DEV), i32(lens).to(DEV)
    if ns == [1] * len(ns) and max_q is None:
        o, lse = A.attn_decode_paged_q4(dq, *dc, dbt, dl, window_left=window, softcap=softcap)
    else:
        cu = i32(np.concatenate([[0], np.cumsum(ns)])).to(DEV)
        o, lse = A.attn_fwd_varlen_paged_q4(dq, *dc, block_table=dbt, cu_seqlens_q=cu, max_seqlen_q=max_q or max(ns),
                                            seqused_k=dl, total_k=sum(lens), mask=A.MASK_CAUSAL if causal else A.MASK_NONE,
                                            window_left=window, softcap=softcap)
        lse = lse.t()
    assert A.attn_device_error() == 0
    return o.split(ns), lse.split(ns)


def run(q, k, v, group, **kw):
    """One sequence: the library's attention against fp64."""
    L = k.shape[0]
    cache = cache_of(k, v, group)
    o, lse = attend([q], [cache], [L], group, **kw)
    kw.pop("max_q", None)
    Attention(q, cache, L, group, **kw).check(o[0], lse[0])


# ---------------------------------------------------------------- weights that hardly differ
@gpu
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("L,D,group", [(8000, 128, 128), (65000, 64, 32)])
@pytest.mark.parametrize("qscale", [0.0, 1e-4, 1e-2])
def test_nearly_flat_scores(device, n, L, D, group, qscale):
    """The weights of many keys are rounded alike: both sums that make up O have to see that."""
    run(randn((n, 4, D), 1, qscale), randn((L, 1, D), 2), randn((L, 1, D), 3), group)


@gpu
@pytest.mark.parametrize("n", [1, 4])
@pytest.mark.parametrize("offset", [0.37, 1.71, 3.13, 6.59])
@pytest.mark.parametrize("D,group", [(128, 128), (128, 32), (64, 64)])
def test_equal_scores_above_the_held_maximum(device, n, offset, D, group):
    """Repeated keys some log2 units above each share's first pages: p is one number above 1."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    low, share = 24, 48                      # pages: at least two for each warp of a CTA; a CTA's share
    L = (sms * share - 13) * 16              # (a sequence counts for 13 pages more)
    page = torch.arange(L // 16)
    high = ((page + 13) % share >= low).repeat_interleave(16)
    one = randn((1, 1, D), 4)
    q = randn((1, 1, D), 5)
    # k = t one: the quantised values scale with t where t is a power of two; q turned to fit offset
    kk = torch.from_numpy(R.values(*R.quantise(one, group)))[0, 0]
    s = float(q[0, 0].double() @ kk) / math.sqrt(D) / math.log(2)      # score of a key in log2 units
    q = (q.double() * (2 * offset / s)).to(torch.bfloat16)             # of a high key: 2 offset; of a low one: offset
    k = torch.where(high[:, None, None], one, one / 2)
    run(q.expand(n, 2, D).contiguous(), k, randn((L, 1, D), 6), group, causal=False if n > 1 else True)


@gpu
@pytest.mark.parametrize("n", [1, 3])
def test_strong_channel(device, n):
    v = randn((4000, 2, 128), 7)
    v[:, :, 5] *= 80
    run(randn((n, 8, 128), 8), randn((4000, 2, 128), 9), v, 64)
    one = randn((4000, 2, 128), 7)
    one[1234, 0, 5] *= 80
    run(randn((n, 8, 128), 8), randn((4000, 2, 128), 9), one, 128)


# ---------------------------------------------------------------- NaN
@gpu
@pytest.mark.parametrize("n", [1, 2, 5])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 64)])
@pytest.mark.parametrize("power", [-60, -20, 0, 8, 17, 60])
@pytest.mark.parametrize("at", [0, 700])
def test_nan_group_leaves_the_other_groups(device, n, D, group, power, at):
    """One group of one key stands for NaN: its columns are NaN, the others what they were."""
    L, Hkv = 900, 2
    cache = cache_of(randn((L, Hkv, D), 10), (randn((L, Hkv, D), 11).float() * 2.0 ** power).to(torch.bfloat16), group)
    cache[3][at // 16, 1, at % 16, 0] = 0x7FC0
    q = randn((n, 8, D), 12)
    o, lse = attend([q], [cache], [L], group)
    want = Attention(q, cache, L, group)
    assert torch.isnan(want.o[:, 4:, :group]).all() and int(torch.isnan(want.o).sum()) == n * 4 * group
    want.check(o[0], lse[0])


# ---------------------------------------------------------------- steps far apart
@gpu
@pytest.mark.parametrize("power", [20, 24, 30, 60, -60])
@pytest.mark.parametrize("n,window", [(1, 300), (1, 0), (3, 100)])
def test_hidden_key_of_another_size(device, power, n, window):
    """A key outside the window, on a page that the window's first keys share, changes nothing."""
    L, Hkv, D, group = 1000, 1, 128, 64
    k, v = randn((L, Hkv, D), 20), randn((L, Hkv, D), 21)
    first = L - n - window                               # the window's first key; its page holds earlier ones
    assert first % 16
    cache = cache_of(k, v, group)
    v[first - 1] = (v[first - 1].float() * 2.0 ** power).to(torch.bfloat16)
    big = cache_of(k, v, group)
    q = randn((n, 4, D), 22)
    o, lse = attend([q], [big], [L], group, window=window)
    want = Attention(q, cache, L, group, window=window)
    want.check(o[0], lse[0])


@gpu
@pytest.mark.parametrize("power", [24, 30, 60])
def test_key_that_causality_hides(device, power):
    """The newest key's values reach the newest query alone."""
    L, Hkv, D, group, n = 700, 1, 64, 32, 3
    k, v = randn((L, Hkv, D), 23), randn((L, Hkv, D), 24)
    v[-1] = (v[-1].float() * 2.0 ** power).to(torch.bfloat16)
    run(randn((n, 4, D), 25), k, v, group)


@gpu
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("power,below", [(20, 30), (24, 40), (30, 25), (30, 30), (30, 45), (60, 80), (60, 60), (100, 99)])
@pytest.mark.parametrize("at", [0, 555, 999])
def test_strong_key_of_little_weight(device, n, power, below, at):
    """Values 2^power times the others' on a key whose p is 2^-below of theirs."""
    L, Hkv, D, group = 1000, 1, 128, 32
    k, v = randn((L, Hkv, D), 26, 0.05), randn((L, Hkv, D), 27)
    q = randn((n, 2, D), 28)
    away = -q[0, 0].double()                             # every query shares head 0's direction
    q[:] = q[0, 0]
    t = below * math.log(2) * math.sqrt(D) / float(away @ away)
    k[at] = (away * t).to(torch.bfloat16)
    v[at] = (v[at].float() * 2.0 ** power).to(torch.bfloat16)
    run(q, k, v, group, causal=False if n > 1 else True)


@gpu
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("powers", [(0, 30, -30, 60), (40, 0, 0, -90), (-20, 17, 0, 8)])
def test_groups_of_different_size(device, n, powers):
    """Each group's columns are as exact as if the others were not there."""
    L, D, group = 600, 128, 32
    v = randn((L, 1, D), 29).float().unflatten(-1, (4, 32)) * torch.tensor([2.0 ** p for p in powers])[:, None]
    run(randn((n, 4, D), 30), randn((L, 1, D), 31), v.flatten(-2).to(torch.bfloat16), group)


@gpu
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("order", [1, -1])
def test_sizes_that_grow_along_the_sequence(device, n, order):
    L, D, group = 1500, 64, 32
    size = torch.linspace(-40, 40, L).round()[:, None, None] * order
    v = (randn((L, 1, D), 32).float() * 2.0 ** size).to(torch.bfloat16)
    run(randn((n, 4, D), 33), randn((L, 1, D), 34), v, group)


@gpu
@pytest.mark.parametrize("n", [1, 3])
def test_groups_of_zeros_and_a_sharp_key(device, n):
    """Values of zero everywhere but on keys of little weight, and a key that takes all of it."""
    L, D, group = 800, 64, 32
    v = torch.zeros(L, 1, D, dtype=torch.bfloat16)
    v[10] = randn((1, D), 35)
    v[500, 0, 32:] = randn((32,), 36, 2.0 ** -90)
    k = randn((L, 1, D), 37)
    q = randn((n, 2, D), 38)
    run(q, k, v, group)
    q[:] = q[0, 0]
    k[600] = (q[0, 0].float() * 1.5).to(torch.bfloat16)      # about 2^17 of the others; its values are zero
    run(q, k, v, group)
    k[600] = (q[0, 0].float() * 30).to(torch.bfloat16)       # past 2^-126: the others' p are zero
    cache = cache_of(k, v, group)
    o, _ = attend([q], [cache], [L], group)
    assert not o[0][-1].any()


@gpu
@pytest.mark.parametrize("n,window", [(1, 300), (1, 0), (3, 100)])
def test_nan_before_the_window(device, n, window):
    L, D, group = 1000, 64, 32
    first = L - n - window
    k, v = randn((L, 1, D), 40), randn((L, 1, D), 41)
    q = randn((n, 4, D), 42)
    cache = cache_of(k, v, group)
    want = Attention(q, cache, L, group, window=window)
    for m in cache[2:]:
        m[(first - 1) // 16, 0, (first - 1) % 16] = 0x7FC0
    o, lse = attend([q], [cache], [L], group, window=window)
    want.check(o[0], lse[0])


@gpu
@pytest.mark.parametrize("n", [2, 3, 8, 20])
def test_nan_that_causality_hides(device, n):
    """NaN values of a drafted token reach the queries from it on, and no earlier one."""
    L, D, group = 500, 64, 32
    cache = cache_of(randn((L, 2, D), 43), randn((L, 2, D), 44), group)
    q = randn((n, 4, D), 45)
    t = L - n + n // 2                                       # the token of query n // 2
    cache[3][t // 16, 0, t % 16, 1] = 0x7FC0                 # its values of head 0, second group
    cache[2][t // 16, 1, t % 16, 0] = 0x7FC0                 # its key of head 1
    o, lse = attend([q], [cache], [L], group)
    want = Attention(q, cache, L, group)
    assert int(torch.isnan(want.o[:, :2]).sum()) == (n - n // 2) * 2 * 32
    assert torch.isnan(want.o[n // 2:, 2:]).all() and not torch.isnan(want.o[:n // 2]).any()
    want.check(o[0], lse[0])


# ---------------------------------------------------------------- long sequences
LONG = [(9000, 4, 1, 128, 128), (30011, 2, 1, 128, 32), (65003, 2, 1, 64, 64), (4100, 8, 4, 128, 64)]


@gpu
@pytest.mark.parametrize("n", [1, 3, 20])
@pytest.mark.parametrize("L,Hq,Hkv,D,group", LONG)
def test_long_sequences(device, L, Hq, Hkv, D, group, n):
    run(randn((n, Hq, D), 50), randn((L, Hkv, D), 51), randn((L, Hkv, D), 52), group)


@pytest.mark.parametrize("L,Hq,Hkv,D,group", LONG)
@pytest.mark.parametrize("page", [0.0, 0.3, 1.0])
def test_a_page_left_out_would_be_seen(L, Hq, Hkv, D, group, page):
    """The tolerances refuse attention over all pages but one, in fp64, by its LSE and by its O."""
    q, k, v = randn((1, Hq, D), 50), randn((L, Hkv, D), 51), randn((L, Hkv, D), 52)
    cache = cache_of(k, v, group)
    want = Attention(q, cache, L, group)
    at = int(page * (-(-L // 16) - 1)) * 16
    less = Attention(q, cache, L, group, skip=[(at, at + 16)])
    eo, el = want.excess(less.o.to(torch.bfloat16), less.lse)
    assert el > 1, el
    assert eo > 1, eo
    assert max(want.excess(want.o.to(torch.bfloat16), want.lse)) <= 0.95


@gpu
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("L,Hkv,group", [(60000, 1, 64), (777, 2, 32)])
def test_every_page_counts(device, L, Hkv, group, n):
    """One page in turn holds the one key that matters: its values are the output."""
    D = 64
    k, v = randn((L, Hkv, D), 53), randn((L, Hkv, D), 54)
    q = randn((n, Hkv, D), 55)
    q[:] = q[0]
    cache = cache_of(k, v, group)
    strong = (q[0].float() * 6).to(torch.bfloat16)
    values = torch.from_numpy(R.read(cache[1], cache[3], list(range(-(-L // 16))), False))
    kc, km = pages_of(strong[None], group, R.k_nibble)
    pages = range(-(-L // 16)) if L < 1000 else range(0, L // 16, 97)
    dc, bt = [t.to(DEV) for t in cache], torch.arange(-(-L // 16), dtype=torch.int32)[None].to(DEV)
    dq, dl, cu = q.to(DEV), i32([L]).to(DEV), i32([0, n]).to(DEV)
    for p in pages:
        t = p * 16 + p % 16
        if t > L - n:
            continue
        keep = [dc[0][p].clone(), dc[2][p].clone()]
        dc[0][p, :, p % 16] = kc[0, :, 0].to(DEV)
        dc[2][p, :, p % 16] = km[0, :, 0].to(DEV)
        if n == 1:
            o, _ = A.attn_decode_paged_q4(dq, *dc, bt, dl)
        else:
            o, _ = A.attn_fwd_varlen_paged_q4(dq, *dc, block_table=bt, cu_seqlens_q=cu, max_seqlen_q=n, seqused_k=dl,
                                              total_k=L, mask=A.MASK_CAUSAL)
        dc[0][p], dc[2][p] = keep
        # 6 |q|^2 / 8 is 40 or more above the other scores (of deviation 1, or |q| = 8): they weigh
        # 60000 e^-30 at most
        o = o.double().cpu()
        err = (o - values[t]).abs() - 2.0 ** -8 * values[t].abs()
        assert float(err.max()) <= 2.0 ** -10 * float(values[t].abs().max()), (p, float(err.max()))
    assert A.attn_device_error() == 0
