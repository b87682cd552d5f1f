"""attn_rope refuses outputs whose rows share memory, before any launch (CPU only)."""
import ctypes

import pytest

from attention_paged_kv_gqa_b200 import binding as A
from attention_paged_kv_gqa_b200 import build as B

P0, P1 = 1 << 20, 1 << 24
INVALID = 1


@pytest.fixture(scope="module")
def L():
    B.build()
    return A.lib()


def st(row, head):
    return (ctypes.c_int64 * 2)(row, head)


def rope(L, sqo, sko=st(2048, 128), q_out=P1, k_out=P1 + (1 << 20), total=4, Hq=8, Hkv=2, sq=st(2048, 128)):
    return L.attn_rope(P0, q_out, P0 + (1 << 16), k_out, sq, sqo, st(2048, 128), sko, total, Hq, Hkv, 128, P0, 16, 64, P0, 1,
                       None, 0, 0, None)


@pytest.mark.parametrize("kw", [
    dict(sqo=st(128, 128)), dict(sqo=st(1016, 128)), dict(sqo=st(2048, 296)), dict(sqo=st(128, 504)),
    dict(sqo=st(1024, 128), sko=st(128, 128)), dict(sqo=st(1 << 62, 1 << 62)),
    dict(sqo=st(1024, 128), q_out=P0), dict(sqo=st(2048, 256), q_out=P0), dict(sqo=st(1024, 128), sko=st(1024, 128), k_out=P0 + (1 << 16))])
def test_outputs_that_overlap(L, kw):
    assert rope(L, **kw) == INVALID


@pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="the calls would run, on addresses that are none")
@pytest.mark.parametrize("kw", [
    dict(sqo=st(1024, 128)), dict(sqo=st(128, 512)), dict(sqo=st(2048, 256)), dict(sqo=st(128, 128), Hq=1),
    dict(sqo=st(128, 128), total=1), dict(sqo=st(2048, 128), q_out=P0), dict(sqo=st(1024, 128), total=1, q_out=P0),
    dict(sqo=st(2048, 256), Hq=1, q_out=P0)])
def test_outputs_that_do_not(L, kw):
    assert rope(L, **kw) not in (0, INVALID)             # (no B200 here)
