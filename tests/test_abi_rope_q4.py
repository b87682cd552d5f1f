"""Argument checks of the rotary and 4-bit cache entry points, before any launch (CPU only)."""
import ctypes

import pytest
import torch

from attention_paged_kv_gqa_b200 import binding as A
from attention_paged_kv_gqa_b200 import build as B

P0 = 1 << 20
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    B.build()
    return A.lib()


def st(row=2048, head=128):
    return (ctypes.c_int64 * 2)(row, head)


def call(fn, base, **kw):
    a = dict(base)
    for k, v in kw.items():
        assert k in a, k
        a[k] = v
    return fn(*a.values())


def rope(L, **kw):
    base = dict(q=P0, q_out=P0, k=P0, k_out=P0, sq=st(), sqo=st(), sk=st(), sko=st(), total=4, Hq=8, Hkv=2, D=128,
                cos_sin=P0, max_position=16, rot_dim=64, positions=P0, n_axes=1, pair_axis=None, interleaved=0,
                inverse=0, stream=None)
    return call(L.attn_rope, base, **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID), (dict(sq=None), INVALID),
    (dict(k=None, k_out=None), INVALID),                      # Hkv without k
    (dict(total=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(cos_sin=None), INVALID), (dict(cos_sin=P0 + 4), INVALID), (dict(max_position=0), INVALID),
    (dict(rot_dim=0), INVALID), (dict(rot_dim=144), INVALID), (dict(rot_dim=24), UNSUPPORTED),
    (dict(positions=None), INVALID), (dict(n_axes=0), INVALID), (dict(n_axes=5, pair_axis=P0), UNSUPPORTED),
    (dict(n_axes=3), INVALID),                                # axes without pair_axis
    (dict(n_axes=3, pair_axis=P0 + 4), INVALID),
    (dict(q=P0 + 8), INVALID), (dict(k_out=P0 + 2), INVALID), (dict(sq=st(2048, 100)), INVALID),
    (dict(sko=st(2044, 128)), INVALID), (dict(sqo=st(0, 128)), INVALID), (dict(sko=st(2048, 64)), INVALID)])
def test_rope_refusals(L, kw, want):
    assert rope(L, **kw) == want


APPEND = dict(q=P0, q_out=P0, k_new=P0, v_new=P0, sq=st(), sk=st(), sv=st(), k_cache=P0, v_cache=P0)
PAGES = dict(block_table=P0, max_blocks=4, num_blocks=9, block_size=16)
NEW = dict(cu=P0, used=P0, used_out=P0 + 64, B=2, total=5, Hq=8, Hkv=2, D=128)
ROPE = dict(cos_sin=P0, max_position=64, rot_dim=128, positions=None, n_axes=1, pair_axis=None, interleaved=0)

APPEND_BAD = [
    (dict(k_new=None), INVALID), (dict(v_new=None), INVALID), (dict(sk=None), INVALID), (dict(sv=None), INVALID),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(sq=None), INVALID),
    (dict(q=None, q_out=None), INVALID),                      # Hq without q
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(block_table=None), INVALID),
    (dict(used=None), INVALID), (dict(B=-1), INVALID), (dict(total=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(D=80), UNSUPPORTED), (dict(block_size=32), UNSUPPORTED),
    (dict(num_blocks=0), INVALID), (dict(max_blocks=0), INVALID), (dict(num_blocks=1 << 28), UNSUPPORTED),
    (dict(max_blocks=1 << 27), UNSUPPORTED), (dict(cu=None), INVALID), (dict(used_out=P0), INVALID),
    (dict(k_new=P0 + 8), INVALID), (dict(k_cache=P0 + 8), INVALID), (dict(sk=st(2048, 4)), INVALID),
    (dict(rot_dim=40), UNSUPPORTED), (dict(rot_dim=256), INVALID), (dict(max_position=0), INVALID),
    (dict(n_axes=2, pair_axis=P0), INVALID)]                  # axes without positions


@pytest.mark.parametrize("kw,want", APPEND_BAD + [
    (dict(dtype=2), INVALID), (dict(dtype=1), INVALID), (dict(dtype=1, dk=P0, dv=P0), INVALID)])
def test_append_rope_refusals(L, kw, want):
    base = dict(APPEND, **PAGES, **NEW, **ROPE, dtype=0, dq=None, dk=None, dv=None, stream=None)
    assert call(L.attn_kv_append_rope_paged, base, **kw) == want


@pytest.mark.parametrize("kw,want", APPEND_BAD + [
    (dict(k_meta=None), INVALID), (dict(v_meta=P0 + 8), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(group=96), UNSUPPORTED), (dict(D=64, rot_dim=64, group=128), UNSUPPORTED), (dict(B=5000), UNSUPPORTED)])
def test_append_q4_refusals(L, kw, want):
    base = dict(APPEND, k_meta=P0, v_meta=P0, **PAGES, **NEW, group=64, **ROPE, stream=None)
    assert call(L.attn_kv_append_paged_q4, base, **kw) == want


CACHE = dict(k_cache=P0, v_cache=P0, k_meta=P0, v_meta=P0)
CACHE_BAD = [
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(k_meta=None), INVALID),
    (dict(v_meta=None), INVALID), (dict(block_table=None), INVALID), (dict(max_blocks=0), INVALID),
    (dict(num_blocks=0), INVALID), (dict(block_size=8), UNSUPPORTED), (dict(B=-1), INVALID), (dict(B=5000), UNSUPPORTED),
    (dict(Hkv=0), INVALID), (dict(D=96), UNSUPPORTED), (dict(group=48), UNSUPPORTED), (dict(v_cache=P0 + 4), INVALID),
    (dict(num_blocks=1 << 28), UNSUPPORTED), (dict(max_blocks=1 << 27), UNSUPPORTED),
    (dict(B=4096, max_blocks=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", CACHE_BAD + [
    (dict(cu=None), INVALID), (dict(k_out=None), INVALID), (dict(total=-1), INVALID), (dict(v_out=P0 + 8), INVALID)])
def test_gather_q4_refusals(L, kw, want):
    base = dict(CACHE, **PAGES, cu=P0, starts=None, B=2, total=5, Hkv=2, D=128, group=64, k_out=P0, v_out=P0, stream=None)
    assert call(L.attn_kv_gather_paged_q4, base, **kw) == want


SCORE_BAD = [(dict(q=None), INVALID), (dict(o=None), INVALID), (dict(used=None), INVALID), (dict(Hq=7), INVALID),
             (dict(Hq=0), INVALID), (dict(softcap=-1.0), INVALID), (dict(softcap=float("inf")), INVALID),
             (dict(softcap=float("nan")), INVALID), (dict(q=P0 + 8), INVALID), (dict(o=P0 + 2), INVALID)]


@pytest.mark.parametrize("kw,want", CACHE_BAD + SCORE_BAD + [(dict(Hq=130), UNSUPPORTED)])
def test_decode_q4_refusals(L, kw, want):
    base = dict(q=P0, **CACHE, **PAGES, used=P0, B=2, Hq=8, Hkv=2, D=128, group=64, scale=0.0, window=-1, softcap=0.0,
                o=P0, lse=None, ws=P0, ws_bytes=1 << 30, stream=None)
    assert call(L.attn_decode_paged_q4, base, **kw) == want


@pytest.mark.parametrize("kw,want", CACHE_BAD + SCORE_BAD + [
    (dict(cu=None), INVALID), (dict(mask=3), INVALID), (dict(mask=-1), INVALID), (dict(mask=2), UNSUPPORTED),
    (dict(mask=0, window=4), UNSUPPORTED), (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID),
    (dict(max_q=-1), INVALID)])
def test_fwd_q4_refusals(L, kw, want):
    base = dict(q=P0, **CACHE, **PAGES, cu=P0, used=P0, B=2, total_q=6, total_k=100, max_q=4, Hq=8, Hkv=2, D=128,
                group=64, scale=0.0, mask=1, window=-1, softcap=0.0, o=P0, lse=None, ws=P0, ws_bytes=1 << 30, stream=None)
    assert call(L.attn_fwd_varlen_paged_q4, base, **kw) == want


def test_workspace_sizes(L):
    assert L.attn_decode_q4_workspace_size(0, 8, 2, 128) == 0
    assert L.attn_decode_q4_workspace_size(2, 7, 2, 128) == 0
    assert L.attn_decode_q4_workspace_size(2, 130, 2, 128) == 0
    small, large = (L.attn_decode_q4_workspace_size(b, 32, 8, 128) for b in (1, 64))
    assert 0 < small < large
    # past 128 query rows per KV head the packed bf16 rows of K and V
    assert L.attn_fwd_q4_workspace_size(2, 33, 8, 2, 128, 100000) >= 2 * 100000 * 2 * 128 * 2
    assert L.attn_fwd_q4_workspace_size(2, 16, 8, 2, 128, 100000) < 2 * 100000 * 2 * 128 * 2
    assert L.attn_fwd_q4_workspace_size(2, -1, 8, 2, 128, 1000) == 0


def test_binding_refuses_wrong_tensors():
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_rope(q, cos_sin=torch.zeros(4, 64), positions=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_kv_append_paged_q4(None, q, q, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="three dimensions"):
        A.attn_decode_paged_q4(q[0], None, None, None, None, None, None)
    with pytest.raises(TypeError, match="tensor"):
        A.attn_fwd_varlen_paged_q4(None, None, None, None, None, block_table=None, cu_seqlens_q=None, max_seqlen_q=1,
                                   seqused_k=None, total_k=1)
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_kv_gather_paged_q4(None, None, None, None, None, torch.zeros(2, dtype=torch.int32), 4)
