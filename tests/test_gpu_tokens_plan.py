"""The plan of chunk and tree attention as the workspace sizes show it: it follows the sizes of a
call, not what divides what."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _splits(kvc, cache, Hq, T):
    """Ranges that a call of T tokens divides each unit into: a part holds D + 2 numbers per row."""
    q = torch.empty(T, Hq, cache.D, dtype=torch.float16, device="cuda")
    size = kvc.kvc_chunk_workspace_size(cache, q)
    assert size == kvc.kvc_tree_workspace_size(cache, q)
    parts, rest = divmod(max(size - 16, 0), T * Hq * (cache.D + 2) * 4)
    assert rest == 0
    return max(parts, 1)


@pytest.mark.parametrize("B,Hq,Hkv,D,C", [(8, 64, 8, 128, 16384), (3, 64, 8, 128, 3008), (12, 16, 4, 128, 4096),
                                          (24, 64, 8, 64, 8192), (5, 8, 1, 64, 2048),
                                          (40, 24, 3, 64, 8192), (16, 32, 32, 128, 1024)])
def test_a_batch_that_divides_evenly_is_planned_like_its_neighbours(kvc, B, Hq, Hkv, D, C):
    """Batches of B k tokens: between those of one token less and one more.  Equal lengths and
    lengths that happen to add up to such a number are not told apart."""
    cache = kvc.SlotCache.empty_paged(B, Hkv, C, D, 64)
    for k in list(range(1, 40)) + [64, 100, 128]:
        T = B * k
        if T == 1:
            continue
        less, here, more = (_splits(kvc, cache, Hq, T + i) for i in (-1, 0, 1))
        assert min(less, more) <= here <= max(less, more), (T, less, here, more)


@pytest.mark.parametrize("B,Hq,Hkv,D,C", [(8, 64, 8, 128, 16384), (1, 8, 1, 64, 2048), (96, 32, 32, 128, 1024)])
@pytest.mark.parametrize("splits", [0, 5])
def test_no_tokens_need_no_workspace(kvc, B, Hq, Hkv, D, C, splits):
    cache = kvc.SlotCache.empty_paged(B, Hkv, C, D, 64)
    q = torch.empty(0, Hq, D, dtype=torch.float16, device="cuda")
    assert kvc.kvc_chunk_workspace_size(cache, q, splits) == 0
    assert kvc.kvc_tree_workspace_size(cache, q, splits) == 0
