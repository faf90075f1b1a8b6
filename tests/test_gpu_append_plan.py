"""The append plan and the packed append: exact against a plain statement with Python integers,
in place and into other arrays, through exhaustion of the pool, release after evictions, and
the whole path plan -> append -> attention -> eviction -> plan."""
import numpy as np
import pytest
import torch

from helpers import device_status_clean
from token_refs import attend_rows, check_rows, plan_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _state(kvc, rng, B, Hkv, C, n, extra, spare, D=64):
    """A paged cache with counts n, `extra` pages beyond them per unit, and its pool."""
    per = C // 64
    pages = np.minimum(-(-n // 64) + extra, per).astype(np.int32)
    num = int(pages.sum()) + spare
    order = rng.permutation(num).astype(np.int32)
    table = np.full((B, Hkv, per), -1, np.int32)
    i = 0
    for b in range(B):
        for h in range(Hkv):
            table[b, h, :pages[b, h]] = order[i:i + pages[b, h]]
            i += pages[b, h]
    cache = kvc.SlotCache.empty_paged(B, Hkv, C, D, num, block_table=torch.from_numpy(table))
    cache.n.copy_(torch.from_numpy(n.astype(np.int32)))
    cache.seqlen.copy_(torch.from_numpy(rng.integers(0, 9000, B).astype(np.int32)))
    free = np.full(num, -1, np.int32)
    free[:spare] = order[i:]
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    pool = kvc.PagePool(pages=dev(pages), free=dev(free), count=dev(np.array([spare])))
    return cache, pool


def _expect(cache, pool, m, T, release):
    paged = cache.block_table is not None
    return plan_reference(cache.n.tolist(), cache.seqlen.tolist(), list(m), cache.C, T,
                          cache.block_table.tolist() if paged else None,
                          pool.pages.tolist() if paged else None,
                          pool.free.tolist() if paged else None,
                          int(pool.count) if paged else 0, release)


def _check(want, cache, pool, slots, pos_before):
    assert cache.n.tolist() == want["n"] and cache.seqlen.tolist() == want["seqlen"]
    assert slots.tolist() == want["slots"]
    if want["table"] is not None:
        assert cache.block_table.tolist() == want["table"]
        assert pool.pages.tolist() == want["pages"]
        assert int(pool.count) == len(want["stack"])
        assert pool.free[:len(want["stack"])].tolist() == want["stack"]
    pos = pos_before.clone()
    for (b, h, s), p in want["pos"].items():
        pos[b, h, s] = p
    assert torch.equal(cache.pos.cpu(), pos)


CASES = [
    # B, Hkv, C, most new tokens, extra pages, spare pages, release
    (1, 1, 64, 1, 0, 1, False),
    (1, 2, 128, 64, 0, 8, False),
    (7, 3, 512, 100, 2, 200, True),
    (33, 8, 640, 130, 1, 700, True),
    (5, 8, 2048, 700, 0, 600, False),
    (16, 4, 256, 256, 1, 20, True),       # the stack runs out: later growing units are refused
    (4, 2, 256, 200, 0, 0, False),        # nothing to give
    (300, 32, 192, 2, 1, 5000, True),     # thousands of units
    (700, 30, 128, 4, 1, 9000, True),     # 21000 units: more than one per thread
    (40, 9, 640, 500, 1, 900, True),      # thousands of tokens, nine heads, the stack runs out
    (3, 2, 8192, 4000, 2, 400, False),    # a few long prompts
]


@pytest.mark.parametrize("B,Hkv,C,most,extra,spare,release", CASES)
@pytest.mark.parametrize("in_place", [True, False])
def test_plan_paged(kvc, B, Hkv, C, most, extra, spare, release, in_place):
    rng = np.random.default_rng(B * 1000 + C)
    n = rng.integers(0, C + 1, (B, Hkv))
    n[0, 0], n[-1, -1] = 0, max(0, C - most)
    ex = rng.integers(0, extra + 1, (B, Hkv))
    m = rng.integers(0, most + 1, B)
    m[rng.integers(B)] = most
    cache, pool = _state(kvc, rng, B, Hkv, C, n, ex, spare)
    T = int(m.sum()) + 3                   # three tokens behind the last sequence
    want = _expect(cache, pool, m, T, release)
    pos0 = cache.pos.cpu().clone()
    slots = torch.full((T, Hkv), 12345, dtype=torch.int32, device="cuda")
    out, pool_out = cache, pool
    if not in_place:
        before = [x.clone() for x in (cache.n, cache.seqlen, cache.block_table, pool.pages,
                                      pool.free, pool.count)]
        out = kvc.SlotCache(K=cache.K, V=cache.V, pos=cache.pos, n=torch.full_like(cache.n, -9),
                            seqlen=torch.full_like(cache.seqlen, -9),
                            block_table=torch.full_like(cache.block_table, -9))
        pool_out = kvc.PagePool(pages=torch.full_like(pool.pages, -9),
                                free=torch.full_like(pool.free, -9),
                                count=torch.full_like(pool.count, -9))
        kvc.kvc_append_plan(cache, _cu(m), slots, pool=pool, out=out, pool_out=pool_out,
                            release=release)
    else:
        kvc.kvc_append_plan(cache, _cu(m), slots, pool=pool, release=release)
    torch.cuda.synchronize()
    assert (kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY) == want["refused"]
    _check(want, out, pool_out, slots, pos0)
    if not in_place:
        for a, b in zip(before, (cache.n, cache.seqlen, cache.block_table, pool.pages, pool.free,
                                 pool.count)):
            assert torch.equal(a, b)


def test_plan_dense(kvc):
    rng = np.random.default_rng(1)
    B, Hkv, C = 6, 3, 100
    cache = kvc.SlotCache.empty(B, Hkv, C, 64)
    cache.n.copy_(torch.from_numpy(rng.integers(0, C + 1, (B, Hkv)).astype(np.int32)))
    cache.seqlen.copy_(torch.arange(B, dtype=torch.int32))
    m = rng.integers(0, 40, B)
    T = int(m.sum())
    want = _expect(cache, None, m, T, False)
    pos0 = cache.pos.cpu().clone()
    slots = torch.empty(T, Hkv, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, _cu(m), slots)
    torch.cuda.synchronize()
    assert want["refused"] and kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    _check(want, cache, None, slots, pos0)


def test_plan_range_outside_the_batch_brings_nothing(kvc):
    rng = np.random.default_rng(2)
    cache, pool = _state(kvc, rng, 3, 2, 128, np.full((3, 2), 60), np.zeros((3, 2), int), 9)
    want = _expect(cache, pool, [5, 0, 0], 9, False)
    cu = torch.tensor([0, 5, 3, 50], dtype=torch.int32, device="cuda")   # backwards, then too far
    slots = torch.empty(9, 2, dtype=torch.int32, device="cuda")
    pos0 = cache.pos.cpu().clone()
    kvc.kvc_append_plan(cache, cu, slots, pool=pool)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    want["slots"] = want["slots"][:5] + [[-1, -1]] * 4
    _check(want, cache, pool, slots, pos0)


@pytest.mark.parametrize("T,Hkv,D", [(1, 1, 64), (3, 8, 128), (257, 3, 64), (1000, 8, 128)])
def test_append_packed(kvc, T, Hkv, D):
    """Strided rows land where the map says; -1 entries and every other row stay."""
    g = torch.Generator(device="cuda").manual_seed(T)
    num = -(-T * Hkv // 64) + 2
    cache = kvc.SlotCache.empty_paged(1, Hkv, 64, D, num,
                                      block_table=torch.zeros(1, Hkv, 1, dtype=torch.int32))
    cache.K.fill_(3.0)
    cache.V.fill_(4.0)
    qkv = torch.randn(T, 3 * Hkv, D, generator=g, device="cuda").half()
    k, v = qkv[:, Hkv:2 * Hkv], qkv[:, 2 * Hkv:]
    slots = torch.randperm(num * 64, generator=g, device="cuda")[:T * Hkv].int().reshape(T, Hkv)
    slots[torch.rand(T, Hkv, generator=g, device="cuda") < 0.2] = -1
    kvc.kvc_append_packed(cache, k, v, slots.contiguous())
    assert device_status_clean(kvc)
    K, V = torch.full((num * 64, D), 3.0).half(), torch.full((num * 64, D), 4.0).half()
    sel = (slots >= 0).cpu()
    K[slots.cpu()[sel].long()] = k.cpu()[sel]
    V[slots.cpu()[sel].long()] = v.cpu()[sel]
    assert torch.equal(cache.K.cpu().view(-1, D), K) and torch.equal(cache.V.cpu().view(-1, D), V)
    bad = torch.full((T, Hkv), -1, dtype=torch.int32, device="cuda")
    bad[0, 0] = num * 64
    kvc.kvc_append_packed(cache, k, v, bad)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert torch.equal(cache.K.cpu().view(-1, D), K)


def _gather(cache, b, h):
    n = int(cache.n[b, h])
    if cache.block_table is None:
        return cache.K[b, h, :n], cache.V[b, h, :n]
    pg = cache.block_table[b, h, :-(-n // 64)].long()
    return (cache.K[pg].reshape(-1, cache.D)[:n], cache.V[pg].reshape(-1, cache.D)[:n])


def test_serving_path(kvc):
    """Prompts of different lengths enter an empty paged cache, are attended, evicted to a
    quarter per head, then three rounds of drafted tokens follow (plan with release, packed
    append, chunk attention), the last one beside a new prompt in an emptied place.  Pages are
    conserved throughout."""
    Hq, Hkv, D, C, num = 16, 4, 128, 1024, 200
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [300, 65, 513]
    B, T = len(lens), sum(lens)
    cache = kvc.SlotCache.empty_paged(B, Hkv, C, D, num)
    pool = kvc.PagePool.empty(cache)
    rand = lambda t: torch.randn(t, Hq + 2 * Hkv, D, generator=g, device="cuda").half()  # noqa: E731

    def conserved():
        held = [cache.block_table[b, h, :int(pool.pages[b, h])].tolist()
                for b in range(B) for h in range(Hkv)]
        every = sum(held, []) + pool.free[:int(pool.count)].tolist()
        assert sorted(every) == list(range(num))

    def enter(m, release=True):
        t = sum(m)
        x = rand(t)
        slots = torch.empty(t, Hkv, dtype=torch.int32, device="cuda")
        cu = _cu(m)
        kvc.kvc_append_plan(cache, cu, slots, pool=pool, release=release)
        kvc.kvc_append_packed(cache, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots)
        return x, cu

    def attend_chunk(x, cu, m):
        q = x[:, :Hq]
        o, lse = torch.empty(q.shape, dtype=torch.float16, device="cuda"), torch.empty(
            Hq, q.shape[0], device="cuda")
        ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")
        kvc.kvc_chunk_attend(cache, q, cu, o, lse=lse, workspace=ws)
        for b, mb in enumerate(m):
            w = slice(int(cu[b]), int(cu[b]) + mb)
            for h in range(Hq):
                K, V = _gather(cache, b, h // (Hq // Hkv))
                last = K.shape[0] - mb + torch.arange(mb)
                check_rows(o[w, h], lse[h, w], attend_rows(q[w, h], K, V, last), f"b={b} h={h}")
        return o

    x, cu = enter(lens)
    o = torch.empty(T, Hq, D, dtype=torch.float16, device="cuda")
    kvc.kvc_prompt_attend(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], o, cu_seqlens=cu)
    o2 = attend_chunk(x, cu, lens)         # the prompt as one chunk over the cache
    assert (o.float() - o2.float()).abs().max() < 4e-3
    conserved()
    assert cache.seqlen.tolist() == lens
    kvc.kvc_random_evict(cache, 16, 0.25, 7, 0)
    for r, m in enumerate(([4, 1, 7], [0, 3, 64], [2, 130, 1])):
        if r == 2:                          # sequence 1 ends; a new prompt takes its place
            cache.n[1] = 0
            cache.seqlen[1] = 0
        x, cu = enter(m)
        attend_chunk(x, cu, m)
        conserved()
    assert cache.seqlen[1] == 130 and cache.n[1].tolist() == [130] * Hkv
    assert device_status_clean(kvc)


def test_prompt_lse_feeds_the_heavy_hitter_scores(kvc):
    """The padded prompt attention's lse is the row normaliser of the prefill score pass: the
    scores are those of the pass that computes the normalisers itself."""
    B, Hq, Hkv, L, D = 2, 8, 2, 300, 128
    g = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn(B, Hq, L, D, generator=g, device="cuda").half()
    k = torch.randn(B, Hkv, L, D, generator=g, device="cuda").half()
    v = torch.randn(B, Hkv, L, D, generator=g, device="cuda").half()
    o, lse = torch.empty_like(q), torch.empty(B, Hq, L, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, lse=lse)
    ws = torch.empty(kvc.kvc_h2o_workspace_size(B, Hq, L) // 4, device="cuda")
    s1, s2 = torch.zeros(B, Hkv, L, device="cuda"), torch.zeros(B, Hkv, L, device="cuda")
    kvc.kvc_h2o_accumulate_prefill(q, k, s1, ws, L, lse=lse)
    kvc.kvc_h2o_accumulate_prefill(q, k, s2, ws, L)
    assert torch.allclose(s1, s2, rtol=1e-4, atol=0)
    assert abs(s1.double().sum().item() - B * Hq * L) < 1e-4 * B * Hq * L
    assert device_status_clean(kvc)


def test_captured_step_with_a_padded_batch(kvc):
    """Plan, packed append and chunk attention captured once for a fixed number of token places
    and replayed: the lengths are on the device, places behind the last sequence stay idle, and
    pages are taken and given back in place, step after step."""
    Hq, Hkv, D, C, B, T = 8, 2, 64, 512, 4, 40
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = kvc.SlotCache.empty_paged(B, Hkv, C, D, 70)
    pool = kvc.PagePool.empty(cache)
    x = torch.zeros(T, Hq + 2 * Hkv, D, dtype=torch.float16, device="cuda")
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(T, Hkv, dtype=torch.int32, device="cuda")
    o = torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")

    def step():
        kvc.kvc_append_plan(cache, cu, slots, pool=pool, release=True)
        kvc.kvc_append_packed(cache, k, v, slots)
        kvc.kvc_chunk_attend(cache, q, cu, o, workspace=ws)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()                      # nothing yet: every sequence brings no token
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    rng = np.random.default_rng(4)
    total = np.zeros(B, int)
    for it in range(12):
        m = rng.integers(0, 11, B)
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        cu.copy_(_cu(m))
        o.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        total += m
        assert cache.seqlen.tolist() == total.tolist()
        for b in range(B):
            w = slice(int(cu[b]), int(cu[b + 1]))
            for h in range(Hq):
                K, V = _gather(cache, b, h // (Hq // Hkv))
                last = K.shape[0] - m[b] + torch.arange(int(m[b]))
                check_rows(o[w, h], None, attend_rows(q[w, h], K, V, last), f"step {it} b={b} h={h}")
        assert (o[int(cu[B]):] == 7.0).all() and (slots[int(cu[B]):] == -1).all()
        held = [cache.block_table[b, h, :int(pool.pages[b, h])].tolist()
                for b in range(B) for h in range(Hkv)]
        assert sorted(sum(held, []) + pool.free[:int(pool.count)].tolist()) == list(range(70))
        if it % 4 == 3:
            kvc.kvc_random_evict(cache, 4, 0.3, 11, it)
    assert device_status_clean(kvc)


def test_captured_calls_on_forked_streams(kvc):
    """A graph in which two streams fork from one and join again, with these calls at the fork,
    on both branches and behind the join."""
    Hq, Hkv, D, C, B = 8, 2, 128, 512, 3
    g = torch.Generator(device="cuda").manual_seed(31)
    lens = [100, 64, 300]
    T = sum(lens)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").half()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    caches = [kvc.SlotCache.empty_paged(B, Hkv, C, D, 60) for _ in range(2)]
    pools = [kvc.PagePool.empty(c) for c in caches]
    slots = [torch.empty(T, Hkv, dtype=torch.int32, device="cuda") for _ in range(2)]
    os_ = [torch.empty(T, Hq, D, dtype=torch.float16, device="cuda") for _ in range(3)]
    ws = [torch.empty(max(kvc.kvc_chunk_workspace_size(caches[0], q, 3) // 4, 4), device="cuda")
          for _ in range(2)]
    cu = _cu(lens)
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def both():
        kvc.kvc_prompt_attend(q, k, v, os_[2], cu_seqlens=cu, stream=s0)
        s1.wait_stream(s0)
        for i, s in enumerate((s0, s1)):
            kvc.kvc_append_plan(caches[i], cu, slots[i], pool=pools[i], stream=s)
            kvc.kvc_append_packed(caches[i], k, v, slots[i], stream=s)
            kvc.kvc_chunk_attend(caches[i], q, cu, os_[i], workspace=ws[i], num_splits=3, stream=s)
        s0.wait_stream(s1)
        kvc.kvc_append_packed(caches[0], k, v, slots[0], stream=s0)

    def fresh():
        for c, p in zip(caches, pools):
            c.n.zero_()
            c.seqlen.zero_()
            c.block_table.fill_(-1)
            p.pages.zero_()
            p.free.copy_(torch.arange(59, -1, -1))
            p.count.fill_(60)
        torch.cuda.synchronize()

    with torch.cuda.stream(s0):
        both()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s0):
            both()
    for _ in range(3):
        fresh()
        for o in os_:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            w = slice(int(cu[b]), int(cu[b + 1]))
            for h in range(Hq):
                ref = attend_rows(q[w, h], k[w, h // 4], v[w, h // 4], torch.arange(lens[b]))
                for o in os_:
                    check_rows(o[w, h], None, ref, f"b={b} h={h}")
    assert device_status_clean(kvc)
