"""CPU-only: what the prompt, chunk, plan and packed-append calls refuse before anything is
launched, and the plan's plain statement on a case worked by hand."""
import ctypes

import pytest
import torch

from token_refs import plan_reference


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_split_gb300 import build
    build.build()
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _prompt(kvc, **kw):
    a = kvc.PromptArgs()
    a.B, a.Hq, a.Hkv, a.D, a.L = 2, 8, 2, 128, 16
    a.q = a.k = a.v = a.o = 16
    for s in (a.q_stride, a.k_stride, a.v_stride, a.o_stride):
        s[0], s[1], s[2] = 4096, 2048, 128
    for key, val in kw.items():
        if key.endswith("_stride"):
            getattr(a, key)[val[0]] = val[1]
        else:
            setattr(a, key, val)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), "INVALID_ARG"), (dict(Hq=7), "INVALID_ARG"), (dict(L=-1), "INVALID_ARG"),
    (dict(D=96), "UNSUPPORTED"), (dict(Hq=18), "UNSUPPORTED"),
    (dict(q=None), "INVALID_ARG"), (dict(v=24), "INVALID_ARG"), (dict(o=8), "INVALID_ARG"),
    (dict(q_stride=(2, 0)), "INVALID_ARG"), (dict(k_stride=(1, 12)), "INVALID_ARG"),
    (dict(v_stride=(0, -8)), "INVALID_ARG"), (dict(cu_seqlens=16, lens=16), "INVALID_ARG"),
    (dict(L=1 << 28), "UNSUPPORTED"),
])
def test_prompt_refusals(kvc, kw, code):
    a = _prompt(kvc, **kw)
    assert kvc.lib().kvc_prompt_attend(ctypes.byref(a), None) == getattr(kvc, "KVC_ERR_" + code)


def test_nothing_to_do_is_accepted(kvc):
    lib = kvc.lib()
    assert lib.kvc_prompt_attend(None, None) == kvc.KVC_ERR_INVALID_ARG
    a = _prompt(kvc, L=0, q=None, k=None, v=None, o=None)
    assert lib.kvc_prompt_attend(ctypes.byref(a), None) == kvc.KVC_OK
    c = kvc.SlotCacheDesc(1, 2, 128, 64, 16, 16, 16, 16, 16)
    s = (ctypes.c_int64 * 2)(128, 128)
    assert lib.kvc_append_packed(ctypes.byref(c), None, s, None, s, 0, None, None) == kvc.KVC_OK
    k = kvc.ChunkArgs()
    k.Hq, k.T, k.cache = 8, 0, ctypes.pointer(c)
    assert lib.kvc_chunk_attend(ctypes.byref(k), None) == kvc.KVC_OK


def _chunk(kvc, cache, **kw):
    a = kvc.ChunkArgs()
    a.Hq, a.T, a.cache = 8, 4, ctypes.pointer(cache)
    a.q = a.o = a.cu_new = 16
    for s in (a.q_stride, a.o_stride):
        s[0], s[1] = 128, 1024
    for key, val in kw.items():
        if key.endswith("_stride"):
            getattr(a, key)[val[0]] = val[1]
        else:
            setattr(a, key, val)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(Hq=3), "INVALID_ARG"), (dict(Hq=18), "UNSUPPORTED"), (dict(T=-1), "INVALID_ARG"),
    (dict(num_splits=-1), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"),
    (dict(o=24), "INVALID_ARG"), (dict(cu_new=None), "INVALID_ARG"),
    (dict(q_stride=(0, 4)), "INVALID_ARG"), (dict(o_stride=(1, 0)), "INVALID_ARG"),
])
def test_chunk_refusals(kvc, kw, code):
    cache = kvc.SlotCacheDesc(1, 2, 128, 64, 16, 16, 16, 16, 16)
    a = _chunk(kvc, cache, **kw)
    assert kvc.lib().kvc_chunk_attend(ctypes.byref(a), None) == getattr(kvc, "KVC_ERR_" + code)
    assert kvc.lib().kvc_chunk_attend(None, None) == kvc.KVC_ERR_INVALID_ARG
    assert kvc.lib().kvc_chunk_workspace_size(None) == 0


def test_plan_and_packed_refusals(kvc):
    lib, bad, uns = kvc.lib(), kvc.KVC_ERR_INVALID_ARG, kvc.KVC_ERR_UNSUPPORTED
    ref = ctypes.byref
    paged = kvc.SlotCacheDesc(1, 2, 128, 128, 16, 16, 16, 16, 16, 16, 4)
    dense = kvc.SlotCacheDesc(1, 2, 128, 128, 16, 16, 16, 16, 16)
    pool = kvc.PagePoolDesc(16, 16, 16)
    plan = lib.kvc_append_plan
    assert plan(None, None, 16, 1, 0, ref(dense), None, 16, None) == bad
    assert plan(ref(dense), None, 16, 1, 0, None, None, 16, None) == bad
    assert plan(ref(dense), None, None, 1, 0, ref(dense), None, 16, None) == bad
    assert plan(ref(dense), None, 16, 1, 0, ref(dense), None, None, None) == bad
    assert plan(ref(dense), None, 16, -1, 0, ref(dense), None, 16, None) == bad
    assert plan(ref(paged), None, 16, 1, 0, ref(paged), None, 16, None) == bad      # no pool
    assert plan(ref(paged), ref(pool), 16, 1, 0, ref(dense), ref(pool), 16, None) == bad
    hollow = kvc.PagePoolDesc(16, None, 16)
    assert plan(ref(paged), ref(pool), 16, 1, 0, ref(paged), ref(hollow), 16, None) == bad
    other = kvc.SlotCacheDesc(1, 2, 128, 192, 16, 16, 16, 16, 16, 16, 4)
    assert plan(ref(paged), ref(pool), 16, 1, 0, ref(other), ref(pool), 16, None) == bad
    many = kvc.SlotCacheDesc(kvc.PLAN_MAX_UNITS, 2, 128, 64, 16, 16, 16, 16, 16)
    assert plan(ref(many), None, 16, 1, 0, ref(many), None, 16, None) == uns
    s, odd = (ctypes.c_int64 * 2)(1024, 128), (ctypes.c_int64 * 2)(1024, 130)
    pk = lib.kvc_append_packed
    assert pk(None, 16, s, 16, s, 1, 16, None) == bad
    assert pk(ref(dense), None, s, 16, s, 1, 16, None) == bad
    assert pk(ref(dense), 16, s, 24, s, 1, 16, None) == bad
    assert pk(ref(dense), 16, odd, 16, s, 1, 16, None) == bad
    assert pk(ref(dense), 16, s, 16, s, -1, 16, None) == bad
    assert pk(ref(dense), 16, s, 16, s, 1, None, None) == bad


def test_binding_refuses_wrong_types_and_shapes(kvc):
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    with pytest.raises(ValueError, match="belong together"):
        kvc.kvc_prompt_attend(h(4, 2, 64), h(4, 1, 64), h(5, 1, 64), h(4, 2, 64),
                              cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="cu_seqlens"):
        kvc.kvc_prompt_attend(h(4, 2, 64), h(4, 1, 64), h(4, 1, 64), h(4, 2, 64),
                              cu_seqlens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="packed"):
        kvc.kvc_prompt_attend(h(4, 2, 64), h(4, 1, 64), h(4, 1, 64), h(4, 2, 64),
                              cu_seqlens=torch.zeros(2, dtype=torch.int32),
                              lens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="float16"):
        kvc.kvc_prompt_attend(h(1, 2, 4, 64).float(), h(1, 1, 4, 64), h(1, 1, 4, 64),
                              h(1, 2, 4, 64))
    with pytest.raises(ValueError, match="CUDA tensors"):
        kvc.kvc_prompt_attend(h(1, 2, 4, 64), h(1, 1, 4, 64), h(1, 1, 4, 64), h(1, 2, 4, 64))


def test_plan_reference_worked_by_hand():
    """Two sequences of one head, C = 256, stack [7, 8, 9].  Sequence 0: 60 slots in page 0 and
    six new tokens, so page 9 is taken.  Sequence 1: 10 slots left of three pages [1, 2, 3], so
    2 and 3 go back behind what is left of the stack."""
    r = plan_reference([[60], [10]], [100, 40], [6, 1], 256, 7, [[[0, -1, -1, -1]], [[1, 2, 3, -1]]],
                       [[1], [3]], [7, 8, 9], 3, True)
    assert r["table"] == [[[0, 9, -1, -1]], [[1, -1, -1, -1]]]
    assert r["pages"] == [[2], [1]] and r["stack"] == [7, 8, 2, 3]
    assert r["slots"] == [[60], [61], [62], [63], [9 * 64], [9 * 64 + 1], [64 + 10]]
    assert r["n"] == [[66], [11]] and r["seqlen"] == [106, 41] and not r["refused"]
    assert r["pos"][0, 0, 65] == 105 and r["pos"][1, 0, 10] == 40
