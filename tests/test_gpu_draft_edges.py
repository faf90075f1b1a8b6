"""Trees of drafted tokens where they can go wrong at size: batches whose units hold very
different numbers of slots, offsets beyond 32 bits, and calls that overlap on the GPU."""
import numpy as np
import pytest
import torch

from draft_refs import attend_seen, lineage, mask_words, random_tree, seen_slots, verify_batch
from helpers import device_status_clean
from token_refs import attend_rows, check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").half()


def _dense(kvc, gen, n, C, D):
    c = kvc.SlotCache.empty(len(n), len(n[0]), C, D)
    c.K.copy_(_randn(gen, *c.K.shape))
    c.V.copy_(_randn(gen, *c.V.shape))
    c.n.copy_(_i32(n))
    return c


@pytest.mark.parametrize("B,Hkv,D", [(2, 160, 64), (20, 16, 128), (32, 32, 128), (33, 10, 128)])
@pytest.mark.parametrize("tree", [True, False])
def test_units_of_very_different_lengths(kvc, B, Hkv, D, tree):
    """More items than run at once, in batches from two sequences to more than are ordered by
    length: empty sequences, units without a slot and full ones, a count above the capacity."""
    rng, gen, C, g = np.random.default_rng(B), _gen(B), 1500, 2
    m = rng.integers(0, 12, B).tolist()
    m[B // 2] = 0
    m[-1] = 9
    n = [[int(x) for x in rng.choice([mb, mb + 1, 80, 700, 1100, C], Hkv)] for mb in m]
    cache = _dense(kvc, gen, n, C, D)
    T, Hq = sum(m), g * Hkv
    q = _randn(gen, T, Hq, D)
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q, 1) // 4, 4), device="cuda")
    trees = [random_tree(rng, x, 3) if tree else list(range(-1, x - 1)) for x in m]
    bad = (B - 1, 0)                       # the first head's count orders the sequence
    cache.n[bad] = C + 1
    if tree:
        kvc.kvc_tree_attend(cache, q, _cu(m), mask_words(trees, 1).cuda(), o, lse=lse, workspace=ws,
                            num_splits=1)
    else:
        kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws, num_splits=1)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    t = 0
    for b in range(B):
        w, bits = slice(t, t + m[b]), lineage(trees[b])
        t += m[b]
        for h in range(Hq if m[b] else 0):
            nn = 0 if (b, h // g) == bad else n[b][h // g]
            ref = attend_seen(q[w, h], cache.K[b, h // g, :nn], cache.V[b, h // g, :nn],
                              seen_slots(bits, nn, m[b]))
            check_rows(o[w, h], lse[h, w], ref, f"b={b} h={h}")
    assert device_status_clean(kvc)


def test_long_items_follow_one_another(kvc):
    """Few CTAs' worth of long units behind one another: the next item is asked for while blocks
    of the one before are still to be loaded."""
    gen, B, Hkv, C, D = _gen(5), 24, 16, 3000, 128
    rng = np.random.default_rng(5)
    n = [[int(rng.integers(200, C + 1))] * Hkv for _ in range(B)]
    cache = _dense(kvc, gen, n, C, D)
    m = [5] * B
    q = _randn(gen, 5 * B, Hkv, D)
    o = torch.empty_like(q)
    ws = torch.empty(4, device="cuda")
    for _ in range(3):
        kvc.kvc_chunk_attend(cache, q, _cu(m), o, workspace=ws, num_splits=1)
    assert device_status_clean(kvc)
    for b in range(B):
        for h in range(Hkv):
            nn = n[b][h]
            check_rows(o[5 * b:5 * b + 5, h], None,
                       attend_rows(q[5 * b:5 * b + 5, h], cache.K[b, h, :nn], cache.V[b, h, :nn],
                                   nn - 5 + torch.arange(5)))


def test_offsets_beyond_32_bits(kvc):
    """Probability rows 700 million entries apart, and accepted rows in pages at the end of pools
    of more than 2^31 elements."""
    V, step, m = 1003, 700_000_000, [5]
    gen = _gen(6)
    tree = [-1, 0, 0, 1, 1]
    p = torch.softmax(torch.randn(5, V, generator=gen, device="cuda"), 1)
    q = torch.softmax(torch.randn(5, V, generator=gen, device="cuda"), 1)
    wide = torch.empty(4 * step + V, device="cuda")
    far = wide.as_strided((5, V), (step, 1))
    far.copy_(p)
    u, u_next = torch.rand(5, generator=gen, device="cuda") * 0.3, torch.rand(1, generator=gen, device="cuda")
    tokens = q.argmax(1).int()[[0, 0, 0, 1, 1]].contiguous()
    for first, second in ((far, q), (p, None), (far, None)):
        path, count, nxt = (torch.empty(*s, dtype=torch.int32, device="cuda") for s in ((1, 5), (1,), (1,)))
        kvc.kvc_draft_verify(_cu(m), tokens, first, u, u_next, path, count, nxt, parent=_i32(tree), q=second)
        n = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
        want = verify_batch([tree], n(tokens), n(p), n(second), n(u), n(u_next), 5)
        assert (path.cpu().numpy() == want[0]).all() and count.item() == want[1] and nxt.item() == want[2]
    far.copy_(q)
    kvc.kvc_draft_verify(_cu(m), tokens, p, u, u_next, path, count, nxt, parent=_i32(tree), q=far)
    want = verify_batch([tree], n(tokens), n(p), n(q), n(u), n(u_next), 5)
    assert (path.cpu().numpy() == want[0]).all() and count.item() == want[1] and nxt.item() == want[2]
    del wide, far
    num, D = 280_000, 128
    big = kvc.SlotCache(K=torch.empty(num, 64, D, dtype=torch.float16, device="cuda"),
                        V=torch.empty(num, 64, D, dtype=torch.float16, device="cuda"),
                        pos=torch.zeros(1, 1, 128, dtype=torch.int32, device="cuda"),
                        n=_i32([[70]]), seqlen=_i32([70]), block_table=_i32([[[num - 2, num - 1]]]))
    rows = _randn(gen, 128, D)
    big.K[-2:], big.V[-2:] = rows.view(2, 64, D), -rows.view(2, 64, D)
    kvc.kvc_draft_commit(big, _cu([10]), _i32([[0, 4, 9]]), _i32([3]))
    assert device_status_clean(kvc)
    assert big.n.item() == 63 and big.seqlen.item() == 63
    want = torch.cat([rows[:60], rows[[60, 64, 69]]])
    assert torch.equal(big.K[-2:].view(-1, D)[:63], want)
    assert torch.equal(big.V[-2:].view(-1, D)[:63], -want)


def test_a_captured_call_and_a_direct_one_do_not_share_state(kvc):
    """A replayed graph and direct calls of another size on another stream at the same time."""
    gen, rng = _gen(7), np.random.default_rng(7)

    def make(B, V, nodes):
        trees = [random_tree(rng, nodes, 4) for _ in range(B)]
        x = 2 * torch.randn(B * nodes, V, generator=gen, device="cuda")
        p, q = torch.softmax(x, 1), torch.softmax(x + 0.6 * torch.randn(x.shape, generator=gen, device="cuda"), 1)
        above = torch.tensor([b * nodes + max(y, 0) for b, t in enumerate(trees) for y in t], device="cuda")
        race = torch.rand(x.shape, generator=gen, device="cuda").clamp(min=1e-30)
        tokens = (-torch.log(race) / q[above].clamp(min=1e-30)).argmin(1).int()
        out = tuple(torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((B, nodes), (B,), (B,)))
        return dict(trees=trees, cu=_cu([nodes] * B), parent=_i32(sum(trees, [])), p=p, q=q, tokens=tokens,
                    u=torch.rand(B * nodes, generator=gen, device="cuda"),
                    u_next=torch.rand(B, generator=gen, device="cuda"), out=out)

    def call(a):
        kvc.kvc_draft_verify(a["cu"], a["tokens"], a["p"], a["u"], a["u_next"], *a["out"],
                             parent=a["parent"], q=a["q"])

    a, b = make(3, 50_000, 12), make(200, 3000, 6)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call(a)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(10):
                call(a)
    for x in a["out"] + b["out"]:
        x.zero_()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for _ in range(10):
            call(b)
    graph.replay()
    torch.cuda.synchronize()
    n = lambda x: x.cpu().numpy()  # noqa: E731
    for x in (a, b):
        want = verify_batch(x["trees"], *(n(x[k]) for k in ("tokens", "p", "q", "u", "u_next")),
                            x["out"][0].shape[1])
        for got, w in zip(x["out"], want):
            assert (n(got) == w).all()
    assert device_status_clean(kvc)


@pytest.mark.parametrize("policy", ["h2o", "stream"])
def test_steps_over_caches_that_are_evicted(kvc, policy):
    """Speculative steps over a budget of 48 slots: append, attention, commit, eviction.  Each unit
    holds what the policy keeps of the certain tokens, with their rows and positions; the nodes'
    attention was over that and their ancestors; slots behind a unit's have the score 0."""
    rng, gen = np.random.default_rng(3), _gen(3)
    B, Hkv, g, D, C, n_first, n_recent = 3, 2, 4, 128, 128, 16, 32
    cache = kvc.SlotCache.empty(B, Hkv, C, D)
    scores = torch.zeros(B, Hkv, C, device="cuda")
    rows_k = [[{} for _ in range(Hkv)] for _ in range(B)]      # of each unit: position -> row
    rows_v = [[{} for _ in range(Hkv)] for _ in range(B)]
    k, v = _randn(gen, B, Hkv, 70, D), _randn(gen, B, Hkv, 70, D)
    kvc.kvc_append(cache, k, v)
    scores[:, :, :70] = torch.rand(B, Hkv, 70, generator=gen, device="cuda")
    for b in range(B):
        for h in range(Hkv):
            rows_k[b][h] = {i: k[b, h, i] for i in range(70)}
            rows_v[b][h] = {i: v[b, h, i] for i in range(70)}
    length = [70] * B

    def evict():
        table = scores.clone()
        pos, n = cache.pos.tolist(), cache.n.tolist()
        if policy == "h2o":
            kvc.kvc_h2o_evict(cache, scores, n_first, n_recent)
        else:
            kvc.kvc_stream_evict(cache, n_first, n_recent)
        for b in range(B):
            for h in range(Hkv):
                held = sorted(rows_k[b][h])
                recent = [p for p in held if p >= length[b] - n_recent]
                older = [p for p in held if p < length[b] - n_recent]
                if policy == "stream":
                    keep = [p for p in older if p < n_first] + recent
                else:
                    s = {pos[b][h][j]: table[b, h, j].item() for j in range(n[b][h])}
                    keep = sorted(older, key=lambda p: (-s[p], p))[:n_first] + recent
                for rows in (rows_k, rows_v):
                    rows[b][h] = {p: rows[b][h][p] for p in keep}

    def check():
        for b in range(B):
            assert cache.seqlen[b] == length[b]
            for h in range(Hkv):
                n = int(cache.n[b, h])
                pos = cache.pos[b, h, :n].tolist()
                assert sorted(pos) == sorted(rows_k[b][h])
                assert torch.equal(cache.K[b, h, :n], torch.stack([rows_k[b][h][p] for p in pos]))
                assert torch.equal(cache.V[b, h, :n], torch.stack([rows_v[b][h][p] for p in pos]))
                if policy == "h2o":
                    assert (scores[b, h, n:] == 0).all()

    evict()
    check()
    for _ in range(5):
        m = rng.integers(1, 20, B).tolist()
        trees = [random_tree(rng, x, 4) for x in m]
        T, cu = sum(m), _cu(m)
        k, v, q = _randn(gen, T, Hkv, D), _randn(gen, T, Hkv, D), _randn(gen, T, g * Hkv, D)
        slots = torch.empty(T, Hkv, dtype=torch.int32, device="cuda")
        mask = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
        kvc.kvc_tree_plan(cu, _i32(sum(trees, [])), mask)
        kvc.kvc_append_plan(cache, cu, slots)
        kvc.kvc_append_packed(cache, k, v, slots)
        o = torch.empty_like(q)
        ws = torch.empty(max(kvc.kvc_tree_workspace_size(cache, q) // 4, 4), device="cuda")
        kvc.kvc_tree_attend(cache, q, cu, mask, o, workspace=ws)
        paths, t = [], 0
        for b, tree in enumerate(trees):
            w, bits = slice(t, t + m[b]), lineage(tree)
            t += m[b]
            for h in range(g * Hkv):
                kk = torch.cat([torch.stack(list(rows_k[b][h // g].values())), k[w, h // g]])
                vv = torch.cat([torch.stack(list(rows_v[b][h // g].values())), v[w, h // g]])
                check_rows(o[w, h], None, attend_seen(q[w, h], kk, vv, seen_slots(bits, len(kk), m[b])))
            path, i = [], int(rng.integers(0, m[b]))
            while i >= 0:
                path.append(i)
                i = tree[i]
            paths.append(path[::-1])
            for h in range(Hkv):
                for d, i in enumerate(paths[b]):
                    rows_k[b][h][length[b] + d] = k[w][i, h]
                    rows_v[b][h][length[b] + d] = v[w][i, h]
            length[b] += len(paths[b])
        most = max(map(len, paths))
        kvc.kvc_draft_commit(cache, cu, _i32([p + [-1] * (most - len(p)) for p in paths]),
                             _i32([len(p) for p in paths]), slot_map=slots)
        check()
        scores[:, :, :C] = torch.where(torch.arange(C, device="cuda") < cache.n[..., None],
                                       scores + torch.rand(scores.shape, generator=gen, device="cuda"), scores)
        evict()
        check()
    assert device_status_clean(kvc)


def test_more_sequences_than_a_grid_row_holds(kvc):
    """70 000 chains of two nodes, a few tokens each."""
    gen, B, V = _gen(9), 70_000, 5
    p = torch.softmax(torch.randn(2 * B, V, generator=gen, device="cuda"), 1)
    tokens = torch.randint(0, V, (2 * B,), generator=gen, device="cuda").int()
    u, u_next = torch.rand(2 * B, generator=gen, device="cuda"), torch.rand(B, generator=gen, device="cuda")
    path, count, nxt = (torch.empty(*s, dtype=torch.int32, device="cuda") for s in ((B, 2), (B,), (B,)))
    cu = torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda")
    mask = torch.zeros(2 * B, 1, dtype=torch.int64, device="cuda")
    kvc.kvc_tree_plan(cu, _i32([-1, 0] * B), mask)
    assert (mask[0::2] == 1).all() and (mask[1::2] == 3).all()
    kvc.kvc_draft_verify(cu, tokens, p, u, u_next, path, count, nxt)
    px = p.double()[0::2].gather(1, tokens[1::2].long()[:, None])[:, 0]
    take = u[1::2].double() < px
    assert torch.equal(count == 2, take) and torch.equal(path[:, 1] == 1, take) and (path[:, 0] == 0).all()
    w = torch.where(take[:, None], p.double()[1::2], p.double()[0::2])
    w = torch.where(take[:, None] | (torch.arange(V, device="cuda") != tokens[1::2, None]), w, 0.0)
    below = w.cumsum(1)
    want = (below <= u_next.double()[:, None] * below[:, -1:]).sum(1)
    assert torch.equal(nxt.long(), want)
    assert device_status_clean(kvc)
