"""Pins of the oracle of rotary positions and of the 4-bit cache format (CPU only)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import rope_q4 as R


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_quarter_turn_and_inverse(interleaved):
    rot, D = 16, 64
    cs = torch.zeros(1, rot)
    cs[:, rot // 2:] = 1.0                       # cos 0, sin 1: (x1, x2) -> (-x2, x1)
    x = torch.randn(3, 2, D, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    y = R.rope(x, cs, pos, interleaved=interleaved)
    a = x.double().numpy()
    for i in range(rot // 2):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        assert np.array_equal(y[..., p], -a[..., q]) and np.array_equal(y[..., q], a[..., p])
    assert np.array_equal(y[..., rot:], a[..., rot:])
    back = R.rope(torch.from_numpy(y), cs, pos, interleaved=interleaved, inverse=True)
    assert np.array_equal(back, a)


def test_rope_depends_on_the_difference_of_positions():
    D = rot = 64
    cs = R.table(200, rot)
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(1, 1, D, generator=g), torch.randn(1, 1, D, generator=g)

    def dot(p, s):
        return float((R.rope(q, cs, torch.tensor([p])) * R.rope(k, cs, torch.tensor([s]))).sum())

    # two fp32 table entries per pair: each product is off by at most 4 * 2^-24 |q| |k|
    tol = 8 * 2.0 ** -24 * float(q.norm() * k.norm())
    assert abs(dot(7, 3) - dot(104, 100)) <= tol


def test_rope_axes_take_their_own_positions():
    D = rot = 64
    cs = R.table(50, rot)
    x = torch.randn(4, 1, D, generator=torch.Generator().manual_seed(2))
    pos = torch.tensor([[0, 1, 2, 3], [5, 5, 6, 6], [7, 8, 9, 10]], dtype=torch.int32)
    axis = torch.tensor([i % 3 for i in range(rot // 2)], dtype=torch.int32)
    y = R.rope(x, cs, pos, axis)
    for i in range(rot // 2):
        one = R.rope(x, cs, pos[i % 3])
        assert np.array_equal(y[..., i], one[..., i]) and np.array_equal(y[..., i + 32], one[..., i + 32])


@pytest.mark.parametrize("D", [64, 128])
def test_nibble_orders_are_permutations(D):
    for which in (R.k_nibble, R.v_nibble):
        at = sorted(which(t, d, D) for t in range(16) for d in range(D))
        assert at == list(range(16 * D))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantise_by_fractions(group):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(6, 128, generator=g)
    x[1] *= 1e-3
    x[2] += 5.0                                  # one-sided: zero is the lowest code
    x[3] = -x[2]
    x[4] = 0.0
    x[5, :64] = 0.25                             # a constant group
    x = x.to(torch.bfloat16)
    code, meta = R.quantise(x, group)
    back = R.values(code, meta)
    for r in range(6):
        for j in range(128 // group):
            v = [Fraction(float(e)) for e in x[r, j * group:(j + 1) * group]]
            lo, hi = min(min(v), Fraction(0)), max(max(v), Fraction(0))
            width = (hi - lo) / 15
            m = int(meta[r, j])
            step = Fraction(float(np.uint32((m & 0xFFF0) << 16).view(np.float32)))
            if width == 0:
                assert m == 0 and not code[r, j * group:(j + 1) * group].any()
                continue
            assert width <= step < width * Fraction(9, 8) + Fraction(1, 10 ** 30)   # up to 4 significant bits
            for i, e in enumerate(v):
                assert abs(Fraction(float(back[r, j * group + i])) - e) <= step / 2
    assert torch.equal(torch.from_numpy(back).to(torch.bfloat16).double(), torch.from_numpy(back))


def test_quantise_loses_noise_and_keeps_zero():
    x = torch.randn(5, 64, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    once = R.values(*R.quantise(x, 32))
    assert np.abs(once - x.double().numpy()).max() > 0
    zero = R.values(*R.quantise(torch.zeros(1, 64, dtype=torch.bfloat16), 32))
    assert not zero.any()


@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 128)])
def test_append_and_read_round_trip(D, group):
    cache = R.fill((7, 2, 16, D // 2), group, 5)
    g = torch.Generator().manual_seed(6)
    k = torch.randn(22, 2, D, generator=g).to(torch.bfloat16)
    v = torch.randn(22, 2, D, generator=g).to(torch.bfloat16)
    bt = torch.tensor([[3, 0, 6], [2, 5, 1]], dtype=torch.int32)
    out = R.append(*cache, k, v, bt, [0, 20, 22], [5, 31], group)
    got_k, got_v = R.packed(*out, bt, [20, 2], [5, 31])
    assert np.array_equal(got_k.double().numpy(), R.values(*R.quantise(k, group)))
    assert np.array_equal(got_v.double().numpy(), R.values(*R.quantise(v, group)))
    before = R.packed(*cache, bt, [5, 31])
    after = R.packed(*out, bt, [5, 31])
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert torch.equal(out[0][4], cache[0][4]) and torch.equal(out[3][4], cache[3][4])   # a page of neither
