"""The commit of accepted nodes behind an append that could not place all of them: units that
were refused stay as they are, units that took their nodes give the others back, whatever
the table holds for their first new slot."""
import numpy as np
import pytest
import torch

from helpers import device_status_clean
from test_gpu_append_plan import _cu, _state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _rows(cache, table, b, h, slots):
    """Row of the page array of each slot, -1 where the table entry is no page."""
    per = [int(table[b, h, s // 64]) for s in slots]
    return [x * 64 + s % 64 if 0 <= x < cache.num_pages else -1 for x, s in zip(per, slots)]


@pytest.mark.parametrize("entry", [-1, "behind"])
@pytest.mark.parametrize("scale", [1, 9])       # nodes on one bad page, and behind it
@pytest.mark.parametrize("own_counts", [False, True])
def test_commit_of_units_whose_first_slot_has_no_page(kvc, entry, scale, own_counts):
    """The slot map has -1 for node 0 of a refused unit, and of one whose first new slot lies on a
    table entry that is no page.  The first keeps its n; the second holds its other nodes, and
    only the accepted ones stay."""
    rng, gen = np.random.default_rng(scale), torch.Generator(device="cuda").manual_seed(scale)
    B, Hkv, C, D = 5, 3, 512, 64
    m = np.array([7, 20, 13, 15, 8]) * scale
    n = rng.integers(130, 300, (B, Hkv))
    n[1, 0], n[2, 1], n[3, 0] = 70, 100, 64         # no page for the first new slot
    n[3, 2], n[4, 0] = C - 5, C - m[4] + 1          # refused: no room
    cache, pool = _state(kvc, rng, B, Hkv, C, n, np.zeros((B, Hkv), int), 200, D)
    cache.seqlen.copy_(cache.n.max(1).values + 5)
    cache.pos.copy_(torch.arange(C, dtype=torch.int32, device="cuda").expand_as(cache.pos))
    wrong = cache.num_pages if entry == "behind" else entry
    pool.pages[3, 0] = 2                            # holds the page behind its rows, its entry is lost
    for b, h in ((1, 0), (2, 1), (3, 0)):
        cache.block_table[b, h, 1] = wrong
    seqlen = cache.seqlen.tolist()
    for x in (cache.K, cache.V):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda").half())
    T = int(m.sum())
    slots = torch.full((T, Hkv), 12345, dtype=torch.int32, device="cuda")
    kvc.kvc_append_plan(cache, _cu(m), slots, pool=pool)
    k, v = (torch.randn(T, Hkv, D, generator=gen, device="cuda").half() for _ in range(2))
    kvc.kvc_append_packed(cache, k, v, slots)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    refused = {(3, 2), (4, 0)}
    first = np.concatenate([[0], np.cumsum(m)])
    for b in range(B):
        for h in range(Hkv):
            assert cache.n[b, h] == n[b, h] + (0 if (b, h) in refused else m[b])
            lost = slots[int(first[b]), h].item() == -1
            assert lost == ((b, h) in refused or (b, h) in {(1, 0), (2, 1), (3, 0)})
    table = cache.block_table.cpu()
    paths = [[0, 2, 5], [0, 3, 4, 19], [0, 1], [0, 14], [0, 7]]
    if scale > 1:                                   # accepted nodes on the pages behind
        paths[1] += [60, 179]
        paths[2] += [40, 100, 116]
    path = torch.full((B, 8), -1, dtype=torch.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = torch.tensor(x, dtype=torch.int32)
    count = torch.tensor([len(x) for x in paths], dtype=torch.int32, device="cuda")
    want_k, want_v = cache.K.clone().view(-1, D), cache.V.clone().view(-1, D)
    want_n = n.copy()
    for b, x in enumerate(paths):
        for h in range(Hkv):
            if (b, h) in refused:
                continue
            want_n[b, h] += len(x)
            src = _rows(cache, table, b, h, [int(n[b, h]) + i for i in x])
            dst = _rows(cache, table, b, h, [int(n[b, h]) + i for i in range(len(x))])
            for s, d in zip(src, dst):
                if s >= 0 and d >= 0:
                    want_k[d], want_v[d] = want_k[s].clone(), want_v[s].clone()
    out = None
    if own_counts:
        out = kvc.SlotCache(K=cache.K, V=cache.V, pos=cache.pos, n=torch.full_like(cache.n, 77),
                            seqlen=torch.full_like(cache.seqlen, 77), block_table=cache.block_table)
    before = cache.n.clone()
    kvc.kvc_draft_commit(cache, _cu(m), path.cuda(), count, slot_map=slots, out=out)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() in (0, kvc.KVC_DEV_CAPACITY)
    got = out or cache
    assert got.n.tolist() == want_n.tolist()
    assert got.seqlen.tolist() == [s + len(x) for s, x in zip(seqlen, paths)]
    assert torch.equal(cache.K.view(-1, D), want_k) and torch.equal(cache.V.view(-1, D), want_v)
    assert not own_counts or torch.equal(cache.n, before)
    assert device_status_clean(kvc)


def test_commit_of_refused_units_that_hold_fewer_slots_than_nodes(kvc):
    """Refused units with less in them than the tree has nodes, and with nothing: left as they are,
    without a report by the commit."""
    rng = np.random.default_rng(3)
    n, m = np.array([[3, 30, 0], [0, 64, 10]]), np.array([70, 60])
    cache, pool = _state(kvc, rng, 2, 3, 64, n, np.zeros((2, 3), int), 0, 64)
    slots = torch.full((130, 3), 12345, dtype=torch.int32, device="cuda")
    seqlen = cache.seqlen.tolist()
    kvc.kvc_append_plan(cache, _cu(m), slots, pool=pool)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert (slots == -1).all() and cache.n.tolist() == n.tolist()
    path = torch.tensor([[0, 5], [0, -1]], dtype=torch.int32, device="cuda")
    count = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    kvc.kvc_draft_commit(cache, _cu(m), path, count, slot_map=slots)
    assert device_status_clean(kvc)
    assert cache.n.tolist() == n.tolist()
    assert cache.seqlen.tolist() == [seqlen[0] + 2, seqlen[1] + 1]
