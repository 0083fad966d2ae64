"""The C ABI of the attention with first tokens or a shared beginning, of the
cache's way back and of the residual norm without a GPU: sizes and flags are refused first, then alignment, then null pointers, before
anything could launch (every pointer that is not the subject of a case is
null)."""
import ctypes
import math

import pytest

from test_decode_ops_abi import A16, struct

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def fp4():
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


@pytest.mark.parametrize("kw,status", [
    (dict(pdl=3), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(T=-1), 1), (dict(B=0), 1), (dict(max_blocks=0), 1),
    (dict(ldk=248), 1), (dict(ldv=248), 1), (dict(T=3, B=2), 1), (dict(B=1025, T=1025), 2), (dict(T=(1 << 30) + 1), 2),
    (dict(max_blocks=(1 << 26) + 1), 2), (dict(k=A16 + 8), 3), (dict(ldk=260), 3), (dict(ldk=258, dtype=2), 3),
    (dict(ldk=260, dtype=2), 1), (dict(), 1)])
def test_read_host_validation(fp4, kw, status):
    a = dict(k=0, ldk=256, ldv=256, dtype=0, T=1, max_blocks=4, B=1, pdl=1)
    a.update(kw)
    c = struct()
    assert fp4.lib().fp4gemv_kv_read(ctypes.addressof(c), vp(a["k"]), a["ldk"], None, a["ldv"], a["dtype"], a["T"],
                                     None, None, a["max_blocks"], None, a["B"], a["pdl"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_blocks=0), 1), (dict(fmt=2), 1), (dict(block=8), 2), (dict(dim=80), 2), (dict(codes=A16 + 8), 3)])
def test_read_cache_validation(fp4, kw, status):
    c = struct(**kw)
    assert fp4.lib().fp4gemv_kv_read(ctypes.addressof(c), None, 1 << 40, None, 1 << 40, 0, 1, None, None, 4, None, 1, 1,
                                     None) == status
    assert fp4.lib().fp4gemv_kv_read(None, None, 1 << 40, None, 1 << 40, 0, 1, None, None, 4, None, 1, 1, None) == 1


def attend(fp4, which, cache=None, q=0, ldq=512, dtype=0, heads=4, q_len=1, max_blocks=4, B=1, sm=0.1, window=0, sinks=4,
           ldo=512, out=0, pdl=1, ws=0, ws_bytes=1 << 30, prefix=0, scratch=0, always=0):
    c = ctypes.addressof(cache if cache is not None else struct())
    if which == "sinks":
        return fp4.lib().fp4gemv_kv_attention_sinks(c, vp(q), ldq, dtype, heads, q_len, None, max_blocks, None, B, sm, window,
                                                    sinks, vp(out), ldo, None, vp(ws), ws_bytes, pdl, None)
    return fp4.lib().fp4gemv_kv_attention_shared(c, vp(q), ldq, dtype, heads, q_len, None, max_blocks, None, B, vp(prefix),
                                                 sm, vp(out), ldo, None, vp(ws), ws_bytes, vp(scratch), 1 << 40, always, pdl,
                                                 None)


@pytest.mark.parametrize("which", ["sinks", "shared"])
@pytest.mark.parametrize("kw,status", [
    (dict(pdl=2), 1), (dict(dtype=2), 1), (dict(heads=0), 1), (dict(q_len=0), 1), (dict(B=0), 1), (dict(max_blocks=0), 1),
    (dict(sm=math.nan), 1), (dict(ldq=504), 1), (dict(ldo=504), 1), (dict(heads=3), 2), (dict(q_len=17), 2),
    (dict(heads=130, ldq=1 << 20, ldo=1 << 20), 2), (dict(B=1025), 2), (dict(max_blocks=(1 << 26) + 1), 2),
    (dict(q=A16 + 8), 3), (dict(ldq=516), 3), (dict(out=A16 + 2), 3), (dict(ws=A16 + 8), 3), (dict(), 1)])
def test_attention_host_validation(fp4, which, kw, status):
    assert attend(fp4, which, **kw) == status


@pytest.mark.parametrize("which,kw,status", [
    ("sinks", dict(window=-1), 1), ("sinks", dict(sinks=-1), 1), ("sinks", dict(sinks=(1 << 30) + 1), 2),
    ("shared", dict(always=2), 1), ("shared", dict(prefix=A16 + 2), 3), ("shared", dict(scratch=A16 + 8), 3),
    ("shared", dict(B=1024, q_len=16, heads=128, ldq=1 << 20, ldo=1 << 20, max_blocks=1 << 16), 2)])
def test_attention_own_arguments(fp4, which, kw, status):
    assert attend(fp4, which, **kw) == status


@pytest.mark.parametrize("args", [(0, 64, 4, 1, 1), (2, 80, 4, 1, 1), (2, 64, 3, 1, 1), (2, 64, 0, 1, 1), (2, 64, 4, 0, 1),
                                  (2, 64, 4, 17, 1), (2, 64, 4, 1, 0), (2, 64, 4, 1, 1025), (1, 64, 65, 1, 1)])
def test_shared_scratch_of_refused_sizes(fp4, args):
    assert fp4.lib().fp4gemv_kv_attention_shared_scratch_bytes(*args) == 0


def add_norm(fp4, x=0, ldx=64, x_dtype=0, y=A16, ldy=64, dtype=0, weight=0, post=0, w_dtype=0, gate=0, ldg=0, g_dtype=0,
             kind=0, sigmoid=0, scale=1.0, eps=1e-6, offset=0.0, residual=0, ldr=64, out=0, ldo=64, M=2, H=64, pdl=1):
    return fp4.lib().fp4gemv_add_norm(vp(x), ldx, x_dtype, vp(y), ldy, dtype, vp(weight), vp(post), w_dtype, vp(gate), ldg,
                                      g_dtype, kind, sigmoid, scale, eps, offset, vp(residual), ldr, vp(out), ldo, M, H,
                                      pdl, None)


@pytest.mark.parametrize("kw,status", [
    (dict(pdl=2), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(x_dtype=1), 1), (dict(x_dtype=3), 1),
    (dict(w_dtype=1), 1), (dict(gate=A16, g_dtype=1), 1), (dict(gate=A16, kind=2), 1), (dict(sigmoid=2), 1),
    (dict(M=0), 1), (dict(H=0), 1), (dict(ldx=63), 1), (dict(ldy=63), 1), (dict(ldr=63), 1), (dict(ldo=63), 1),
    (dict(gate=A16, ldg=63), 1), (dict(gate=A16, kind=1, ldg=-1), 1), (dict(scale=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(eps=-1.0), 1), (dict(offset=math.inf), 1), (dict(y=0, post=A16), 1), (dict(y=0, gate=A16), 1),
    (dict(H=32769, ldx=1 << 20, ldy=1 << 20, ldr=1 << 20, ldo=1 << 20), 2),
    (dict(x=A16 + 1), 3), (dict(x=A16 + 2, x_dtype=2), 3), (dict(weight=A16 + 2, w_dtype=2), 3), (dict(out=A16 + 1), 3),
    (dict(gate=A16 + 2, g_dtype=2), 3), (dict(), 1), (dict(y=0), 1), (dict(x=A16, weight=A16, out=A16), 1)])
def test_add_norm_host_validation(fp4, kw, status):
    assert add_norm(fp4, **kw) == status


def test_marshal_counts_arguments(fp4):
    from moe_nvfp4_gemv_gb300 import _marshal
    for fn, count in ((_marshal.kv_read, 10), (_marshal.add_norm, 12), (_marshal.kv_attention_sinks, 13),
                      (_marshal.kv_attention_shared, 15), (_marshal.bind_more, 4)):
        for n in (0, count - 1, count + 1):
            with pytest.raises(TypeError):
                fn(*([None] * n))
        with pytest.raises(TypeError):
            fn(*([None] * count))
