"""The decode operators' C ABI without a GPU: sizes and flags are refused first,
then alignment, then null pointers, before anything could launch (every pointer
that is not the subject of a case is null)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import decode_ref as ref

A16 = 1 << 20  # a fabricated, 16-byte aligned "device address"
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def fp4():
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


def struct(codes=0, scale=0, num_blocks=4, kv_heads=2, block=16, dim=128, fmt=0):
    from moe_nvfp4_gemv_gb300 import kvcache
    return kvcache._CacheStruct(codes, codes, scale, scale, num_blocks, kv_heads, block, dim, fmt)


def attend(fp4, cache=None, q=0, ldq=512, dtype=0, heads=4, q_len=1, max_blocks=4, B=1, sm=0.1, window=0, ldo=512,
           out=0, pdl=1, ws=0, ws_bytes=1 << 30, null_cache=False):
    c = cache if cache is not None else struct()
    return fp4.lib().fp4gemv_kv_attention(None if null_cache else ctypes.addressof(c), vp(q), ldq, dtype, heads, q_len,
                                          None, max_blocks, None, B, sm, window, vp(out), ldo, None, vp(ws), ws_bytes,
                                          pdl, None)


@pytest.mark.parametrize("kw,status", [
    (dict(null_cache=True), 1), (dict(pdl=2), 1), (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(heads=0), 1),
    (dict(q_len=0), 1), (dict(B=0), 1), (dict(max_blocks=0), 1), (dict(window=-1), 1), (dict(sm=math.nan), 1),
    (dict(sm=math.inf), 1), (dict(ldq=504), 1), (dict(ldo=504), 1),
    (dict(heads=3), 2), (dict(heads=130, ldq=1 << 20, ldo=1 << 20), 2), (dict(q_len=17), 2), (dict(B=1025), 2),
    (dict(max_blocks=(1 << 26) + 1), 2), (dict(B=1024, max_blocks=1 << 21), 2),
    (dict(q=A16 + 8), 3), (dict(ldq=516), 3), (dict(ldo=516), 3), (dict(out=A16 + 2), 3), (dict(ws=A16 + 8), 3),
    (dict(), 1)])
def test_attention_host_validation(fp4, kw, status):
    assert attend(fp4, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_blocks=0), 1), (dict(kv_heads=0), 1), (dict(block=0), 1), (dict(dim=0), 1), (dict(fmt=2), 1),
    (dict(block=8), 2), (dict(block=48), 2), (dict(dim=80), 2), (dict(dim=512), 2), (dict(kv_heads=65536), 2),
    (dict(codes=A16 + 8), 3), (dict(scale=A16 + 2), 3)])
def test_cache_validation(fp4, kw, status):
    c = struct(**kw)
    assert attend(fp4, cache=c, heads=c.kv_heads * 2, ldq=1 << 40, ldo=1 << 40) == status
    assert fp4.lib().fp4gemv_kv_append(ctypes.addressof(c), None, 1 << 40, None, 1 << 40, 0, 1, None, None, 4, None, 1, 1,
                                       None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(pdl=3), 1), (dict(dtype=2), 1), (dict(T=-1), 1), (dict(B=0), 1), (dict(max_blocks=0), 1), (dict(ldk=248), 1),
    (dict(ldv=248), 1), (dict(T=3, B=2), 1), (dict(B=1025, T=1025), 2), (dict(k=A16 + 8), 3), (dict(ldk=260), 3),
    (dict(), 1)])
def test_append_host_validation(fp4, kw, status):
    a = dict(k=0, ldk=256, ldv=256, dtype=0, T=1, max_blocks=4, B=1, pdl=1)
    a.update(kw)
    c = struct()
    assert fp4.lib().fp4gemv_kv_append(ctypes.addressof(c), vp(a["k"]), a["ldk"], None, a["ldv"], a["dtype"], a["T"],
                                       None, None, a["max_blocks"], None, a["B"], a["pdl"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(pdl=2), 1), (dict(dtype=3), 1), (dict(M=0), 1), (dict(E=0), 1), (dict(topk=0), 1), (dict(scores=2), 1),
    (dict(n_group=0), 1), (dict(topk_group=2), 1), (dict(group_top=3), 1), (dict(group_top=0), 1), (dict(ldl=127), 1),
    (dict(renorm=2), 1), (dict(scale=math.nan), 1),
    (dict(E=513, ldl=513), 2), (dict(topk=33), 2), (dict(E=4, topk=5), 2), (dict(n_group=3), 2),
    (dict(n_group=64), 2), (dict(n_group=16, topk_group=1, topk=9), 2), (dict(E=8, n_group=8, group_top=2, topk=1), 2),
    (dict(logits=A16 + 1), 3), (dict(logits=A16 + 2, dtype=2), 3), (dict(), 1)])
def test_route_host_validation(fp4, kw, status):
    a = dict(logits=0, ldl=128, dtype=0, M=1, E=128, topk=8, scores=0, n_group=1, topk_group=1, group_top=1, renorm=1,
             scale=1.0, pdl=1)
    a.update(kw)
    assert fp4.lib().fp4gemv_moe_route(vp(a["logits"]), a["ldl"], a["dtype"], a["M"], a["E"], a["topk"], a["scores"],
                                       None, a["n_group"], a["topk_group"], a["group_top"], a["renorm"], a["scale"],
                                       None, None, a["pdl"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(pdl=2), 1), (dict(dtype=3), 1), (dict(T=0), 1), (dict(V=0), 1), (dict(top_n=-1), 1), (dict(V=5, top_n=6), 1),
    (dict(ldl=99), 1), (dict(inv_t=0.0), 1), (dict(inv_t=math.nan), 1), (dict(inv_t=2e6), 1), (dict(top_n=33), 2),
    (dict(logits=A16 + 1), 3), (dict(logits=A16 + 2, dtype=2), 3), (dict(), 1)])
def test_logprobs_host_validation(fp4, kw, status):
    a = dict(logits=0, ldl=100, dtype=0, T=1, V=100, inv_t=1.0, top_n=4, pdl=1)
    a.update(kw)
    assert fp4.lib().fp4gemv_token_logprobs(vp(a["logits"]), a["ldl"], a["dtype"], a["T"], a["V"], None, a["inv_t"],
                                            a["top_n"], None, None, None, None, None, a["pdl"], None) == status


# ---- the tests' own restatements, worked by hand ----
def test_reference_scales():
    x = np.array([0, 448, 449, 3.5, 1e-38, 448 * 2.0 ** 100, 224.0, 225.0], np.float32)
    assert ref.page_scale(x, "e4m3").tolist() == [2.0 ** -100, 1, 2, 2.0 ** -7, 2.0 ** -100, 2.0 ** 100, 0.5, 1.0]
    assert ref.page_scale(np.array([127, 0], np.float32), "int8").tolist() == [1, 2.0 ** -100]


def test_reference_codes():
    x = torch.tensor([1.0, -448.0, 460.0, 0.0, 17.0, 2.0 ** -10])  # 17 lies between 16 and 18: to even; 2^-10 is half the least
    assert ref.decode(ref.encode(x, "e4m3"), "e4m3").tolist() == [1, -448, 448, 0, 16, 0]
    assert ref.decode(ref.encode(torch.tensor([0.5, 1.5, -127.4, 200.0, math.nan]), "int8"), "int8").tolist() == \
        [0, 2, -127, 127, 0]


def test_reference_append_grows_a_page():
    c = {p + "_codes": torch.zeros(1, 1, 16, 64, dtype=torch.uint8) for p in "kv"}
    c.update({p + "_scale": torch.zeros(1, 1) for p in "kv"})
    k = torch.full((2, 1, 64), 7.0)
    ref.append(c, k[:1], k[:1], [[0]], [1], [1], 16, "e4m3")
    assert float(c["k_scale"]) == 2.0 ** -6  # 7 = 448 / 64
    ref.append(c, 3 * k[:1], k[:1], [[0]], [2], [1], 16, "e4m3")
    assert float(c["k_scale"]) == 2.0 ** -4 and float(c["v_scale"]) == 2.0 ** -6
    assert ref.decode(c["k_codes"], "e4m3")[0, 0, :3, 0].tolist() == [112.0, 320.0, 0.0]  # 336 is halfway from 320 (even) to 352


def test_reference_route_groups():
    x = np.array([[1.0, 5.0, 4.0, 4.5, 6.0, 0.0]])  # groups (1, 5), (4, 4.5), (6, 0)
    assert ref.route(x, 2, "softmax", n_group=3, topk_group=1)[0].tolist() == [[4, 5]]
    ids, w, _ = ref.route(np.zeros((1, 4)), 2, "sigmoid")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]


# ---- the Python calls' own checks (no GPU is touched) ----
def test_python_calls_refuse_what_is_no_cuda_tensor():
    torch = pytest.importorskip("torch")
    from moe_nvfp4_gemv_gb300 import fp4gemv, kvcache
    logits = torch.zeros(2, 8)
    ids, weights = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="logits"):
        fp4gemv.moe_route(logits, 2, ids=ids, weights=weights)
    with pytest.raises(ValueError, match="logits"):
        fp4gemv.token_logprobs(logits, torch.zeros(2, dtype=torch.int32))
    for bad in (None, 3, [1.0], "x"):
        with pytest.raises(TypeError, match="logits must be a tensor"):
            fp4gemv.moe_route(bad, 2, ids=ids, weights=weights)
    cache = kvcache.KvCache8.allocate(2, 1, 64, 16, device="cpu")
    k, table, lens = torch.zeros(1, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32), \
        torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        cache.append(k, k, table, lens)
    with pytest.raises(TypeError, match="k must be a tensor"):
        cache.append(None, k, table, lens)
    with pytest.raises(ValueError, match="block_table"):
        cache.attend(k[None], table, lens, out=k[None], workspace=torch.zeros(4))


def test_marshalling_refuses_a_wrong_number_or_kind_of_arguments():
    from moe_nvfp4_gemv_gb300.fp4gemv import _marshal
    for fn, count in ((_marshal.kv_append, 10), (_marshal.kv_attention, 12), (_marshal.moe_route, 12),
                      (_marshal.token_logprobs, 10), (_marshal.bind, 4)):
        with pytest.raises(TypeError):
            fn()
        with pytest.raises(TypeError):
            fn(*[None] * (count + 1))
        with pytest.raises(TypeError):
            fn(*["x"] * count)


def test_lengths_past_thirty_bits_are_refused(fp4):
    """Places in a sequence, and new tokens, are 32-bit numbers on the device."""
    assert attend(fp4, max_blocks=(1 << 26) + 1) == 2  # 16-token pages: past 2^30 tokens
    assert attend(fp4, max_blocks=1 << 24, B=100) == 2  # too many strips in all
    many = struct(kv_heads=1 << 20)
    assert attend(fp4, cache=many, heads=1 << 20, ldq=1 << 30, ldo=1 << 30) == 2
    c = struct()
    for T, max_blocks, B in ((1, (1 << 26) + 1, 1), ((1 << 30) + 1, 4, 1)):
        assert fp4.lib().fp4gemv_kv_append(ctypes.addressof(c), None, 256, None, 256, 0, T, None, None, max_blocks, None,
                                           B, 1, None) == 2
