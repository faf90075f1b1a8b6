"""The append plan where its two forms meet: batches whose slot map one cluster writes and those
for which a second kernel follows give the same answers."""
import numpy as np
import pytest
import torch

from helpers import device_status_clean
from test_gpu_append_plan import _check, _cu, _expect, _state

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
