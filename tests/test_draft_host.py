"""CPU-only: what the calls for trees of drafted tokens refuse before anything is launched, and
their references on cases worked by hand."""
import ctypes

import numpy as np
import pytest
import torch

from draft_refs import lineage, mask_words, seen_slots, verify_sequence


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_split_gb300 import build
    build.build()
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def test_plan_refusals(kvc):
    plan, bad = kvc.lib().kvc_tree_plan, kvc.KVC_ERR_INVALID_ARG
    assert plan(16, 0, 16, 4, None, 1, 16, None, None) == bad
    assert plan(16, 1, 16, -1, None, 1, 16, None, None) == bad
    assert plan(16, 1, 16, 4, None, 0, 16, None, None) == bad
    assert plan(16, 1, 16, 4, None, kvc.TREE_MAX_NODES // 64 + 1, 16, None, None) == bad
    assert plan(None, 1, 16, 4, None, 1, 16, None, None) == bad
    assert plan(16, 1, None, 4, None, 1, 16, None, None) == bad
    assert plan(16, 1, 16, 4, None, 1, None, None, None) == bad
    assert plan(16, 1, 16, 4, None, 1, 20, None, None) == bad
    assert plan(None, 1, None, 0, None, 1, None, None, None) == kvc.KVC_OK


def _tree(kvc, cache, words=1, mask=16, **kw):
    a = kvc.TreeArgs()
    c = a.chunk
    c.Hq, c.T, c.cache = 8, 4, ctypes.pointer(cache)
    c.q = c.o = c.cu_new = 16
    for s in (c.q_stride, c.o_stride):
        s[0], s[1] = 128, 1024
    a.mask, a.words = mask, words
    for key, val in kw.items():
        if key.endswith("_stride"):
            getattr(c, key)[val[0]] = val[1]
        else:
            setattr(c, key, val)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(words=0), "INVALID_ARG"), (dict(words=5), "INVALID_ARG"), (dict(mask=None), "INVALID_ARG"),
    (dict(mask=20), "INVALID_ARG"), (dict(Hq=3), "INVALID_ARG"), (dict(Hq=18), "UNSUPPORTED"),
    (dict(T=-1), "INVALID_ARG"), (dict(num_splits=-1), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"),
    (dict(o=24), "INVALID_ARG"), (dict(cu_new=None), "INVALID_ARG"),
    (dict(q_stride=(0, 4)), "INVALID_ARG"), (dict(num_splits=2), "WORKSPACE"),
    (dict(num_splits=2, workspace=16, workspace_bytes=8), "WORKSPACE"),
])
def test_tree_refusals(kvc, kw, code):
    cache = kvc.SlotCacheDesc(1, 2, 128, 640, 16, 16, 16, 16, 16)
    a = _tree(kvc, cache, **kw)
    assert kvc.lib().kvc_tree_attend(ctypes.byref(a), None) == getattr(kvc, "KVC_ERR_" + code)
    assert kvc.lib().kvc_tree_attend(None, None) == kvc.KVC_ERR_INVALID_ARG
    assert kvc.lib().kvc_tree_workspace_size(None) == 0


def test_tree_workspace_is_a_chunk_s(kvc):
    cache = kvc.SlotCacheDesc(1, 2, 128, 4096, 16, 16, 16, 16, 16)
    a = _tree(kvc, cache, num_splits=5)
    size = kvc.lib().kvc_tree_workspace_size(ctypes.byref(a))
    assert size == kvc.lib().kvc_chunk_workspace_size(ctypes.byref(a.chunk)) > 0
    a = _tree(kvc, cache, T=0, q=None, o=None, mask=None)
    assert kvc.lib().kvc_tree_attend(ctypes.byref(a), None) == kvc.KVC_OK


def _draft(kvc, **kw):
    a = kvc.DraftArgs()
    a.B, a.T, a.V, a.max_path = 2, 6, 100, 4
    for f in ("cu_new", "tokens", "p", "u", "u_next", "path", "count", "next_token"):
        setattr(a, f, 16)
    a.p_stride = a.q_stride = 100
    for key, val in kw.items():
        setattr(a, key, val)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(V=0), "INVALID_ARG"),
    (dict(max_path=0), "INVALID_ARG"), (dict(cu_new=None), "INVALID_ARG"),
    (dict(tokens=None), "INVALID_ARG"), (dict(p=None), "INVALID_ARG"), (dict(p=18), "INVALID_ARG"),
    (dict(q=18), "INVALID_ARG"), (dict(u=None), "INVALID_ARG"),
    (dict(u_next=None), "INVALID_ARG"), (dict(path=None), "INVALID_ARG"),
    (dict(count=None), "INVALID_ARG"), (dict(next_token=None), "INVALID_ARG"),
    (dict(p_stride=99), "INVALID_ARG"), (dict(q=16, q_stride=99), "INVALID_ARG"),
    (dict(V=(1 << 24) + 1, p_stride=1 << 25), "UNSUPPORTED"),
])
def test_verify_refusals(kvc, kw, code):
    a = _draft(kvc, **kw)
    assert kvc.lib().kvc_draft_verify(ctypes.byref(a), None) == getattr(kvc, "KVC_ERR_" + code)
    assert kvc.lib().kvc_draft_verify(None, None) == kvc.KVC_ERR_INVALID_ARG


def test_commit_refusals(kvc):
    commit, bad, ref = kvc.lib().kvc_draft_commit, kvc.KVC_ERR_INVALID_ARG, ctypes.byref
    c = kvc.SlotCacheDesc(1, 2, 128, 128, 16, 16, 16, 16, 16)
    assert commit(None, 16, 4, 16, 16, 4, None, ref(c), None) == bad
    assert commit(ref(c), None, 4, 16, 16, 4, None, ref(c), None) == bad
    assert commit(ref(c), 16, -1, 16, 16, 4, None, ref(c), None) == bad
    assert commit(ref(c), 16, 4, None, 16, 4, None, ref(c), None) == bad
    assert commit(ref(c), 16, 4, 16, None, 4, None, ref(c), None) == bad
    assert commit(ref(c), 16, 4, 16, 16, 0, None, ref(c), None) == bad
    assert commit(ref(c), 16, 4, 16, 16, 4, None, None, None) == bad
    other = kvc.SlotCacheDesc(2, 2, 128, 128, 16, 16, 16, 16, 16)
    assert commit(ref(c), 16, 4, 16, 16, 4, None, ref(other), None) == bad
    hollow = kvc.SlotCacheDesc(1, 2, 128, 128, 16, 16, 16, None, 16)
    assert commit(ref(c), 16, 4, 16, 16, 4, None, ref(hollow), None) == bad


def test_packed_structs_are_the_declared_ones(kvc):
    assert len(kvc._pack_tree(*[0] * 12, 0, 0, 0.0, 0, 0)) == ctypes.sizeof(kvc.TreeArgs)
    assert len(kvc._pack_draft(*[0] * 16)) == ctypes.sizeof(kvc.DraftArgs)
    a = kvc.DraftArgs.from_buffer_copy(kvc._pack_draft(*range(1, 17)))
    names = [f for f, _ in kvc.DraftArgs._fields_]
    assert [getattr(a, f) for f in names] == list(range(1, 17))
    t = kvc.TreeArgs.from_buffer_copy(kvc._pack_tree(*range(1, 15), 0.5, 16, 17))
    assert (t.chunk.num_splits, t.chunk.softmax_scale, t.mask, t.words) == (14, 0.5, 16, 17)


def test_binding_refuses_wrong_types_and_shapes(kvc):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f32 = lambda *s: torch.zeros(*s)  # noqa: E731
    with pytest.raises(ValueError, match="parent"):
        kvc.kvc_tree_plan(i32(2), i32(5), torch.zeros(4, 1, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensors"):
        kvc.kvc_tree_plan(i32(2), i32(4), torch.zeros(4, 1, dtype=torch.int64))
    args = dict(cu_new=i32(3), tokens=i32(4), p=f32(4, 9), u=f32(4), u_next=f32(2), path=i32(2, 3),
                count=i32(2), next_token=i32(2))
    for name, wrong in (("p", f32(4, 9).double()), ("tokens", i32(5)), ("u", f32(5)),
                        ("next_token", i32(3))):
        with pytest.raises(ValueError):
            kvc.kvc_draft_verify(**{**args, name: wrong})
    with pytest.raises(ValueError, match="q must be"):
        kvc.kvc_draft_verify(**{**args, "q": f32(4, 8)})
    with pytest.raises(ValueError):
        kvc.kvc_draft_verify(**args)                   # host tensors


class DeviceTensor:
    """What the binding asks of a CUDA tensor, without a GPU."""

    def __init__(self, dtype, shape, device, address=4096):
        self.dtype, self.shape, self.index, self.address = dtype, torch.Size(shape), device, address
        self.is_cuda, self.device, self.nbytes = True, torch.device("cuda", device), 1 << 20

    def data_ptr(self): return self.address
    def get_device(self): return self.index
    def is_contiguous(self): return True
    def numel(self): return self.shape.numel()
    def stride(self, i=None):
        st = torch.empty(self.shape, device="meta").stride()
        return st if i is None else st[i]


@pytest.mark.parametrize("wrong", ["cu", "path", "mask", "p", "cache"])
def test_the_calls_refuse_tensors_of_another_device(kvc, monkeypatch, wrong):
    """With cuda:1 current, one argument of each call on cuda:0 is refused by name of the device."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(kvc, "_raw_stream", lambda dev: 0)
    on = lambda name: 0 if name == wrong else 1  # noqa: E731
    i32 = lambda name, *s: DeviceTensor(torch.int32, s, on(name))  # noqa: E731
    f32 = lambda name, *s: DeviceTensor(torch.float32, s, on(name))  # noqa: E731
    f16 = lambda name, *s: DeviceTensor(torch.float16, s, on(name))  # noqa: E731
    cache = kvc.SlotCache(K=f16("cache", 2, 2, 64, 64), V=f16("cache", 2, 2, 64, 64),
                          pos=i32("cache", 2, 2, 64), n=i32("cache", 2, 2), seqlen=i32("cache", 2))
    mask = DeviceTensor(torch.int64, (4, 1), on("mask"))
    q = f16("q", 4, 4, 64)
    calls = {
        "cu": [lambda: kvc.kvc_tree_plan(i32("cu", 3), i32("x", 4), mask),
               lambda: kvc.kvc_draft_commit(cache, i32("cu", 3), i32("path", 2, 4), i32("x", 2))],
        "path": [lambda: kvc.kvc_draft_commit(cache, i32("cu", 3), i32("path", 2, 4), i32("x", 2))],
        "mask": [lambda: kvc.kvc_tree_plan(i32("cu", 3), i32("x", 4), mask),
                 lambda: kvc.kvc_tree_attend(cache, q, i32("cu", 3), mask, q)],
        "p": [lambda: kvc.kvc_draft_verify(i32("cu", 3), i32("x", 4), f32("p", 4, 9), f32("x", 4),
                                           f32("x", 2), i32("path", 2, 4), i32("x", 2), i32("x", 2))],
        "cache": [lambda: kvc.kvc_tree_attend(cache, q, i32("cu", 3), mask, q),
                  lambda: kvc.kvc_draft_commit(cache, i32("cu", 3), i32("path", 2, 4), i32("x", 2))],
    }[wrong]
    for call in calls:
        with pytest.raises(ValueError, match="expected the current device cuda:1"):
            call()


def test_masks_worked_by_hand():
    tree = [-1, 0, 0, 1, 3, 2]
    assert lineage(tree) == [1, 0b11, 0b101, 0b1011, 0b11011, 0b100101]
    assert mask_words([tree], 1)[:, 0].tolist() == lineage(tree)
    long = mask_words([list(range(-1, 64))], 2)
    assert long[63].tolist() == [-1, 0] and long[64].tolist() == [-1, 1]
    seen = seen_slots(lineage(tree), 8, 6)
    assert seen[5].tolist() == [True, True, True, False, True, False, False, True]


def test_verification_worked_by_hand():
    """Node 0 with the children 1 (token 0) and 2 (token 1); node 2 with the child 3 (token 2)."""
    parents, tokens = [-1, 0, 0, 2], [9, 0, 1, 2]
    p = np.array([[0.2, 0.5, 0.3], [1, 0, 0], [0.0, 0.25, 0.75], [0.5, 0.0, 0.5]])
    run = lambda u, nxt, q=None, most=4: verify_sequence(parents, tokens, p, q, u, nxt, most)  # noqa: E731
    # given tokens: 0 is refused (0.3 >= 0.2), 1 then has the weight 0.5 / 0.8 = 0.625
    assert run([0, 0.3, 0.62, 0.7], 0.4) == ([0, 2, 3], 0)
    assert run([0, 0.3, 0.62, 0.7], 0.5) == ([0, 2, 3], 2)
    assert run([0, 0.3, 0.63, 0.7], 0.99) == ([0], 2)       # only token 2 is left
    assert run([0, 0.1, 0.62, 0.7], 0.9) == ([0, 1], 0)
    assert run([0, 0.3, 0.62, 0.7], 0.4, most=2) == ([0, 2], 2)
    # drawn tokens: 0 is refused when u 0.5 >= 0.2; the residual is (0, 0.25, 0.05) / 0.3
    q = np.array([[0.5, 0.25, 0.25]] * 4)
    assert run([0, 0.39, 0.1, 0.1], 0.0, q) == ([0, 1], 0)
    assert run([0, 0.41, 0.99, 0.1], 0.6, q) == ([0, 2, 3], 2)
    # the second draw may be refused only where 0.25 u >= 0.25 / 0.3: never; with less it may
    q2 = np.array([[0.1, 0.8, 0.1]] * 4)
    # 0 (accepted below 1), else the residual (0.1, 0, 0.2) / 0.3, in which token 1 has nothing
    assert run([0, 0.999, 0.5, 0.1], 0.1, q2) == ([0, 1], 0)
    p[0] = [0.05, 0.65, 0.3]
    assert run([0, 0.51, 0.0, 0.1], 0.1, q2) == ([0], 2)
