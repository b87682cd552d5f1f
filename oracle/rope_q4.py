"""fp64 oracle of the rotary positions and of the 4-bit cache format.

Plain definitions, one nibble and one pair at a time where that is cheap enough:
``rope`` turns the pairs of a head by table angles, ``quantise`` gives codes and
metas of the 4-bit form, ``write`` / ``read`` place and fetch single nibbles by
the format's index formulas.  Attention over a 4-bit cache is the other oracle's
attention over what ``read`` returns.
"""
from __future__ import annotations

import numpy as np
import torch

PAGE = 16


def table(n: int, rot: int, base: float = 10000.0) -> torch.Tensor:
    """fp32 [n, rot]: cosines, then sines, of place * base^(-2 i / rot) (angles in fp64)."""
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def rope(x, cos_sin, positions, pair_axis=None, interleaved=False, inverse=False) -> np.ndarray:
    """x [T, H, D] -> the rotated values in fp64.  positions [T] or [axes, T]."""
    y = x.double().numpy().copy()
    src = y.copy()
    cs = cos_sin.double().numpy()
    half = cs.shape[1] // 2
    pos = positions.numpy().reshape(-1, x.shape[0])
    for i in range(half):
        p = pos[0 if pair_axis is None else int(pair_axis[i])]
        c, s = cs[p, i][:, None], cs[p, half + i][:, None] * (-1.0 if inverse else 1.0)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = src[..., a] * c - src[..., b] * s
        y[..., b] = src[..., b] * c + src[..., a] * s
    return y


def quantise(x: torch.Tensor, group: int):
    """x [..., D] bf16 -> (codes uint8 [..., D], metas uint16 [..., D / group] as numpy)."""
    v = x.double().numpy()
    g = v.reshape(*v.shape[:-1], -1, group)
    lo = np.minimum(g.min(-1), 0.0)
    hi = np.maximum(g.max(-1), 0.0)
    part, power = np.frexp((hi - lo) / 15.0)
    step = np.ldexp(np.ceil(part * 16.0) / 16.0, power)
    step[step < 2.0 ** -100] = 0.0
    by = np.where(step > 0, step, 1.0)
    zero = np.where(step > 0, np.rint(-lo / by), 0.0)
    code = np.where(step[..., None] > 0, np.rint(g / by[..., None]), 0.0) + zero[..., None]
    code = np.clip(code, 0, 15).astype(np.uint8).reshape(v.shape)
    bits = step.astype(np.float32).view(np.uint32) >> 16
    assert not (bits & 15).any()
    return code, (bits + zero.astype(np.uint32)).astype(np.uint16)


def values(code: np.ndarray, meta: np.ndarray) -> np.ndarray:
    """What codes [..., D] with metas [..., D / group] stand for."""
    step = ((meta.astype(np.uint32) & 0xFFF0) << 16).view(np.float32).astype(np.float64)
    zero = (meta & 15).astype(np.float64)
    c = code.astype(np.float64).reshape(*code.shape[:-1], meta.shape[-1], -1)
    return ((c - zero[..., None]) * step[..., None]).reshape(code.shape)


def k_nibble(t: int, d: int, D: int) -> int:
    """Index of the nibble of token row t, dim d in a K tile."""
    w, c, e = d // 32, d % 32 // 8, d % 8
    return t * D + (c * (D // 32) + w) * 8 + e


def v_nibble(t: int, d: int, D: int) -> int:
    """Index of the nibble of token row t, dim d in a V tile."""
    a, c, h = t // 8, t % 8 // 2, t % 2
    u, j, r = d // 32, d % 32 // 8, d % 8
    return ((((a * 8 + r) * 4 + c) * (D // 32) + u) * 2 + h) * 4 + j


def _index(D: int, which) -> np.ndarray:
    return np.array([[which(t, d, D) for d in range(D)] for t in range(PAGE)])


def write(cache: torch.Tensor, page: int, head: int, row: int, code: np.ndarray, is_k: bool):
    """Puts the codes [D] of one token into its tile, nibble by nibble (in place)."""
    D = code.shape[0]
    tile = cache[page, head].view(-1).numpy()
    for d in range(D):
        n = (k_nibble if is_k else v_nibble)(row, d, D)
        shift = 4 * (n % 2)
        tile[n // 2] = (tile[n // 2] & (0xF0 >> shift)) | (int(code[d]) << shift)


def append(k_cache, v_cache, k_meta, v_meta, k_new, v_new, block_table, cu_new, seqused, group):
    """The cache tensors (CPU) with the new tokens' rows (bf16, already rotated) in them."""
    out = [t.clone() for t in (k_cache, v_cache, k_meta, v_meta)]
    kc, km = quantise(k_new, group)
    vc, vm = quantise(v_new, group)
    for b in range(len(cu_new) - 1):
        for i in range(int(cu_new[b + 1]) - int(cu_new[b])):
            t, p = int(cu_new[b]) + i, int(seqused[b]) + i
            page, row = int(block_table[b, p // PAGE]), p % PAGE
            for h in range(k_new.shape[1]):
                write(out[0], page, h, row, kc[t, h], True)
                write(out[1], page, h, row, vc[t, h], False)
                out[2][page, h, row] = torch.from_numpy(km[t, h].view(np.int16).copy())
                out[3][page, h, row] = torch.from_numpy(vm[t, h].view(np.int16).copy())
    return out


def read(cache: torch.Tensor, meta: torch.Tensor, pages, is_k: bool) -> np.ndarray:
    """fp64 [len(pages) * 16, Hkv, D]: the values of whole pages, in order."""
    n, Hkv, _, half = cache.shape
    D = 2 * half
    at = _index(D, k_nibble if is_k else v_nibble)
    tiles = cache[list(pages)].numpy().reshape(len(pages), Hkv, -1)
    code = (tiles[..., at // 2] >> (4 * (at % 2))) & 15                    # [pages, Hkv, 16, D]
    v = values(code, meta[list(pages)].numpy().view(np.uint16))
    return v.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)


def packed(k_cache, v_cache, k_meta, v_meta, block_table, lens, starts=None):
    """Packed bf16 K and V of tokens starts[b] .. starts[b] + lens[b] - 1 of each sequence."""
    ks, vs = [], []
    for b, n in enumerate(lens):
        s = 0 if starts is None else int(starts[b])
        pages = [int(p) for p in block_table[b, : (s + int(n) + PAGE - 1) // PAGE]]
        if n == 0:
            continue
        ks.append(read(k_cache, k_meta, pages, True)[s:s + int(n)])
        vs.append(read(v_cache, v_meta, pages, False)[s:s + int(n)])
    Hkv, D = k_cache.shape[1], 2 * k_cache.shape[3]
    out = []
    for x in (ks, vs):
        x = np.concatenate(x) if x else np.zeros((0, Hkv, D))
        y = torch.from_numpy(x).to(torch.bfloat16)
        assert np.array_equal(y.double().numpy(), x, equal_nan=True)      # the values are bf16 numbers
        out.append(y)
    return out


def fill(k_cache_shape, group, seed):
    """(k_cache, v_cache, k_meta, v_meta) whose pages hold quantised N(0, 1) values."""
    n, Hkv, page, half = k_cache_shape
    D = 2 * half
    g = torch.Generator().manual_seed(seed)
    out = []
    for which in (k_nibble, v_nibble):
        x = torch.randn(n, Hkv, page, D, generator=g).to(torch.bfloat16)
        code, meta = quantise(x, group)
        at = _index(D, which).reshape(-1)
        nib = np.zeros((n, Hkv, page * D), np.uint8)
        nib[..., at] = code.reshape(n, Hkv, -1)
        out.append(torch.from_numpy((nib[..., 0::2] | (nib[..., 1::2] << 4)).reshape(n, Hkv, page, half)))
        out.append(torch.from_numpy(meta.view(np.int16)))
    return out[0], out[2], out[1], out[3]
