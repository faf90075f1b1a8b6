"""The append plan where its two forms meet: batches whose slot map one cluster writes and those
for which a second kernel follows give the same answers; what that kernel does with dense caches,
bad ranges and thousands of sequences; what is refused and what a chunk sees then."""
import numpy as np
import pytest
import torch

from helpers import device_status_clean
from test_gpu_append_plan import _check, _cu, _expect, _gather, _state
from token_refs import attend_rows, check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _old_positions(cache):
    """Positions of the slots that are there, all before the sequence's next one."""
    cache.seqlen.copy_(cache.n.max(1).values + 5)
    cache.pos.copy_(torch.arange(cache.C, dtype=torch.int32, device="cuda").expand_as(cache.pos))


def _without_bad_pages(want, n, m, pages):
    """The slot map's entries on table entries that are no page are -1."""
    t = 0
    for b, mb in enumerate(m):
        for i in range(int(mb)):
            for h in range(len(n[b])):
                if want["slots"][t][h] != -1:
                    e = want["table"][b][h][(n[b][h] + i) // 64]
                    if not 0 <= e < pages:
                        want["slots"][t][h] = -1
            t += 1


@pytest.mark.parametrize("Hkv", [3, 8])
@pytest.mark.parametrize("scale", [1, 9])          # 63 and 567 tokens: one kernel and two
@pytest.mark.parametrize("entry", [-1, "behind"])
def test_plan_table_entries_that_are_no_page(kvc, Hkv, scale, entry):
    """A unit whose table holds no page for its first new slot, or for a later one, takes the
    tokens that lie on its other pages; units beside it that are refused take none."""
    rng = np.random.default_rng(Hkv + scale)
    B, C = 5, 1024
    m = np.array([7, 20, 13, 15, 8]) * scale
    n = rng.integers(130, 700, (B, Hkv))
    n[1, 0], n[2, 1] = 70, 100
    n[3, 2], n[4, 0] = C - 5, C - m[4] + 1         # refused: no room
    cache, pool = _state(kvc, rng, B, Hkv, C, n, np.zeros((B, Hkv), int), 400)
    _old_positions(cache)
    num = cache.num_pages
    wrong = num if entry == "behind" else entry
    cache.block_table[1, 0, 1] = wrong              # the page of the first new slot
    cache.block_table[2, 1, 1] = wrong              # the same, and its tokens go on behind it
    T = int(m.sum())
    want = _expect(cache, pool, m, T, False)
    assert want["refused"]
    _without_bad_pages(want, n.tolist(), m, num)
    assert sum(r[0] == -1 for r in want["slots"][int(m[0]):int(m[:2].sum())]) == min(m[1], 58)
    pos0 = cache.pos.cpu().clone()
    slots = torch.full((T, Hkv), 12345, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, _cu(m), slots, pool=pool)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    _check(want, cache, pool, slots, pos0)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("T", [None, 600])         # one kernel and two
def test_plan_behind_a_unit_that_the_stack_cannot_serve(kvc, T):
    """Three pages on the stack.  The first unit takes one, the second needs five and is refused,
    the third needs two and is refused too although two are left, the fourth needs none and takes
    its token, the fifth gives a page back."""
    B, C = 5, 512
    cache = kvc.SlotCache.empty_paged(B, 1, C, 64, B * C // 64)
    pool = kvc.PagePool.empty(cache)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.n.copy_(i32([[64], [10], [60], [3], [20]]))
    cache.seqlen.copy_(i32([64, 10, 60, 3, 20]))
    cache.block_table[:, 0, :2] = i32([[0, -1], [1, -1], [2, -1], [3, -1], [4, 5]])
    pool.pages.copy_(i32([[1], [1], [1], [1], [2]]))
    pool.free[:3] = i32([6, 7, 8])
    pool.count.fill_(3)
    m = [1, 300, 100, 1, 1]
    T = T or sum(m)
    slots = torch.full((T, 1), 12345, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, _cu(m), slots, pool=pool, release=True)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert cache.n.flatten().tolist() == [65, 10, 60, 4, 21]
    assert cache.seqlen.tolist() == [65, 310, 160, 4, 21]
    assert pool.pages.flatten().tolist() == [2, 1, 1, 1, 1]
    assert pool.free[:int(pool.count)].tolist() == [6, 7, 5]
    want = [8 * 64] + [-1] * 400 + [3 * 64 + 3, 4 * 64 + 20] + [-1] * (T - 403)
    assert slots.flatten().tolist() == want
    assert device_status_clean(kvc)


def test_chunk_over_a_refused_unit(kvc):
    """One head of a sequence has no room and is refused: the status word says so, the other
    heads' rows are right, and that head's see the slots before n - m + i + 1 of what it holds."""
    g = torch.Generator(device="cuda").manual_seed(3)
    Hq, Hkv, D, C, m = 4, 2, 64, 128, [5, 30]
    cache = kvc.SlotCache.empty_paged(2, Hkv, C, D, 8)
    pool = kvc.PagePool.empty(cache)
    x = torch.randn(250, Hq + 2 * Hkv, D, generator=g, device="cuda").half()

    def enter(cu, t0, T):
        slots = torch.empty(T, Hkv, dtype=torch.int32, device="cuda")
        kvc.kvc_append_plan(cache, cu, slots, pool=pool)
        w = x[t0:t0 + T]
        kvc.kvc_append_packed(cache, w[:, Hq:Hq + Hkv], w[:, Hq + Hkv:], slots)
        return slots

    enter(_cu([100, 110]), 0, 210)
    cache.n[1, 0] = 60                       # evicted: this head has room, the other has not
    assert device_status_clean(kvc)
    slots = enter(_cu(m), 210, 35)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert cache.n.tolist() == [[105, 105], [90, 110]]
    assert (slots[5:, 1] == -1).all() and (slots[5:, 0] >= 0).all()
    q = x[210:245, :Hq]
    o, lse = torch.empty(35, Hq, D, dtype=torch.float16, device="cuda"), torch.empty(Hq, 35, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws)
    assert device_status_clean(kvc)
    for b, w in ((0, slice(0, 5)), (1, slice(5, 35))):
        for h in range(Hq):
            K, V = _gather(cache, b, h // 2)
            last = K.shape[0] - m[b] + torch.arange(m[b])
            check_rows(o[w, h], lse[h, w], attend_rows(q[w, h], K, V, last), f"b={b} h={h}")
            if (b, h // 2) != (1, 1):        # these hold the chunk
                assert torch.equal(K[-m[b]:], x[210:245, Hq + h // 2][w])


def test_plan_dense_of_many_tokens(kvc):
    """A dense cache in a batch large enough for the second kernel, some units refused."""
    rng = np.random.default_rng(11)
    B, Hkv, C = 6, 9, 500
    cache = kvc.SlotCache.empty(B, Hkv, C, 64)
    cache.n.copy_(torch.from_numpy(rng.integers(0, C + 1, (B, Hkv)).astype(np.int32)))
    _old_positions(cache)
    m = np.array([150, 0, 200, 1, 130, 64])
    T = int(m.sum()) + 7
    want = _expect(cache, None, m, T, False)
    pos0 = cache.pos.cpu().clone()
    slots = torch.full((T, Hkv), 12345, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, _cu(m), slots)
    torch.cuda.synchronize()
    assert T > 512 and want["refused"] and kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    _check(want, cache, None, slots, pos0)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("cu,m,order", [
    ([400, 700, 0, 400], [300, 0, 400], [(0, 400), (2, 0)]),    # backwards, then over again
    ([0, 300, 700, 2000], [300, 400, 0], [(0, 0), (1, 300)]),   # the last one leaves the batch
    ([-5, 300, 700, 720], [0, 400, 20], [(1, 300), (2, 700)]),  # the first one starts outside
])
@pytest.mark.parametrize("paged", [True, False])
def test_plan_of_many_tokens_with_bad_ranges(kvc, cu, m, order, paged):
    """A sequence whose range leaves the batch brings nothing; the others' tokens are where
    their ranges lie, in any order, and those of no sequence have no row."""
    rng = np.random.default_rng(sum(m))
    B, Hkv, C, T = 3, 8, 1024, 720
    n = rng.integers(0, 400, (B, Hkv))
    if paged:
        cache, pool = _state(kvc, rng, B, Hkv, C, n, np.zeros((B, Hkv), int), 300)
    else:
        cache, pool = kvc.SlotCache.empty(B, Hkv, C, 64), None
        cache.n.copy_(torch.from_numpy(n.astype(np.int32)))
    _old_positions(cache)
    want = _expect(cache, pool, m, sum(m), False)
    assert not want["refused"]
    rows, t = [[-1] * Hkv for _ in range(T)], 0
    for b, start in sorted(order):
        rows[start:start + m[b]] = want["slots"][t:t + m[b]]
        t += m[b]
    want["slots"] = rows
    pos0 = cache.pos.cpu().clone()
    slots = torch.full((T, Hkv), 12345, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, torch.tensor(cu, dtype=torch.int32, device="cuda"), slots, pool=pool)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    _check(want, cache, pool, slots, pos0)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("backwards", [False, True])
def test_plan_of_thousands_of_sequences_and_many_tokens(kvc, backwards):
    """More sequences than the second kernel keeps the starts of."""
    rng = np.random.default_rng(13)
    B, Hkv, C = 2500, 2, 128
    n = rng.integers(0, C - 3, (B, Hkv))
    cache, pool = _state(kvc, rng, B, Hkv, C, n, np.zeros((B, Hkv), int), B * Hkv)
    _old_positions(cache)
    m = rng.integers(0, 4, B)
    cu = np.concatenate([[0], np.cumsum(m)])
    T = int(cu[-1]) + 2
    if backwards:                # the last sequence brings nothing: its end lies before its start
        cu[-1] = cu[-2] - 3
        m[-1] = 0
    want = _expect(cache, pool, m, T, False)
    assert not want["refused"]
    pos0 = cache.pos.cpu().clone()
    slots = torch.full((T, Hkv), 12345, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, torch.from_numpy(cu.astype(np.int32)).cuda(), slots, pool=pool)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == (kvc.KVC_DEV_CAPACITY if backwards else 0)
    _check(want, cache, pool, slots, pos0)
    assert device_status_clean(kvc)
