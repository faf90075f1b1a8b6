"""Prompt attention and chunk attention over the slot cache against a plain 64-bit reference:
group sizes that do and do not divide a tile, lengths from one token on, odd and ragged
batches, strided rows, padded rows and slots that hold NaN, empty sequences and units, pages
that end inside a tile, graphs and streams."""
import numpy as np
import pytest
import torch

from helpers import device_status_clean
from token_refs import attend_rows, check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").half()


def check_prompt(q, k, v, o, lse, cu, lens, Hq, Hkv, what=""):
    """Packed tensors, sequence by sequence and head by head."""
    g = Hq // Hkv
    for b, n in enumerate(lens):
        w = slice(int(cu[b]), int(cu[b]) + n)
        for h in range(Hq):
            ref = attend_rows(q[w, h], k[w, h // g], v[w, h // g], torch.arange(n))
            check_rows(o[w, h], None if lse is None else lse[h, w], ref, f"{what} b={b} h={h}")


PACKED = [
    # Hq, Hkv, D, lengths
    (4, 4, 64, [64]),
    (8, 1, 128, [1]),
    (8, 1, 128, [1, 2, 3, 0, 5, 0]),
    (1, 1, 128, [127, 128, 129]),
    (1, 1, 64, [255, 256, 257]),
    (7, 1, 128, [18, 19, 37, 200]),
    (10, 2, 64, [25, 26, 130]),
    (6, 2, 128, [333, 42]),
    (16, 2, 128, [511, 17, 640]),
    (2, 2, 128, [1111]),
    (8, 8, 64, [700, 3]),
    # above 1024 tokens on average: two tiles per item with 128 channels
    (8, 1, 128, [1500, 5, 1800]),
    (16, 2, 128, [1061, 1120]),
    (7, 1, 128, [1111, 1040]),
    (3, 3, 128, [1025]),
    (8, 2, 64, [1500]),
]


@pytest.mark.parametrize("Hq,Hkv,D,lens", PACKED)
def test_prompt_packed(kvc, Hq, Hkv, D, lens):
    """q, k, v are column ranges of one projection; a gap of NaN tokens in front of and behind
    the sequences is neither read into a result nor written."""
    pad = 5
    T = sum(lens) + 2 * pad
    qkv = _randn(_gen(T + Hq), T, Hq + 2 * Hkv, D)
    qkv[:pad] = float("nan")
    qkv[T - pad:] = float("nan")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = _cu(lens) + pad
    o = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((Hq, T), 7.0, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=cu, lse=lse)
    assert device_status_clean(kvc)
    check_prompt(q, k, v, o, lse, cu, lens, Hq, Hkv)
    for x in (o[:pad], o[T - pad:], lse[:, :pad], lse[:, T - pad:]):
        assert (x == 7.0).all()


@pytest.mark.parametrize("Hq,Hkv,D,L,lens", [(8, 2, 128, 300, [300, 1, 0, 257]),
                                             (4, 4, 64, 129, None), (5, 1, 128, 77, [77, 76])])
def test_prompt_padded(kvc, Hq, Hkv, D, L, lens):
    """Padded batch with a wider key capacity; rows past a sequence's length hold NaN."""
    B = 4 if lens is None else len(lens)
    gen = _gen(L)
    q = _randn(gen, B, Hq, L, D)
    k, v = _randn(gen, B, Hkv, L + 9, D), _randn(gen, B, Hkv, L + 9, D)
    real = [L] * B if lens is None else lens
    for b, n in enumerate(real):
        q[b, :, n:] = k[b, :, n:] = v[b, :, n:] = float("nan")
    o = torch.full_like(q, 7.0)
    lse = torch.full((B, Hq, L), 7.0, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, lens=dl, lse=lse)
    assert device_status_clean(kvc)
    g = Hq // Hkv
    for b, n in enumerate(real):
        for h in range(Hq):
            ref = attend_rows(q[b, h, :n], k[b, h // g, :n], v[b, h // g, :n], torch.arange(n))
            check_rows(o[b, h, :n], lse[b, h, :n], ref, f"b={b} h={h}")
        assert (o[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()


def test_prompt_large_scores_and_given_scale(kvc):
    """Scores that spread over hundreds, a growing maximum along the keys, and a scale."""
    gen = _gen(3)
    L, D = 600, 128
    q, k, v = _randn(gen, L, 2, D) * 3, _randn(gen, L, 1, D) * 3, _randn(gen, L, 1, D)
    k *= torch.linspace(0.1, 3.0, L, device="cuda")[:, None, None].half()
    o = torch.empty_like(q)
    lse = torch.empty(2, L, device="cuda")
    cu = _cu([L])
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=cu, lse=lse, softmax_scale=0.2)
    for h in range(2):
        check_rows(o[:, h], lse[h], attend_rows(q[:, h], k[:, 0], v[:, 0], torch.arange(L), 0.2))
    assert device_status_clean(kvc)


def test_prompt_range_outside_the_batch_is_an_empty_sequence(kvc):
    gen = _gen(4)
    q, k, v = _randn(gen, 50, 2, 64), _randn(gen, 50, 1, 64), _randn(gen, 50, 1, 64)
    o = torch.full_like(q, 7.0)
    cu = torch.tensor([0, 20, 90], dtype=torch.int32, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert (o[20:] == 7.0).all()
    check_prompt(q, k, v, o, None, cu, [20], 2, 1)
    assert device_status_clean(kvc)


def test_prompt_ranges_that_run_backwards(kvc):
    """A range of negative length is an empty sequence; rows that one other range alone holds
    are right."""
    gen = _gen(31)
    q, k, v = _randn(gen, 50, 4, 64), _randn(gen, 50, 2, 64), _randn(gen, 50, 2, 64)
    o = torch.full_like(q, 7.0)
    cu = torch.tensor([0, 40, 10, 50], dtype=torch.int32, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    for h in range(4):
        check_rows(o[:10, h], None, attend_rows(q[:10, h], k[:10, h // 2], v[:10, h // 2],
                                                torch.arange(10)))
        check_rows(o[40:, h], None, attend_rows(q[40:, h], k[10:, h // 2], v[10:, h // 2],
                                                torch.arange(30, 40)))
    assert device_status_clean(kvc)


# ---------------------------------------------------------------- chunks

def _cache(kvc, gen, n, C, D, paged, spare=3):
    """A slot cache with counts n [B, Hkv]; rows behind n, and pages nobody holds, are NaN."""
    B, Hkv = len(n), len(n[0])
    K, V = _randn(gen, B, Hkv, C, D), _randn(gen, B, Hkv, C, D)
    for b in range(B):
        for h in range(Hkv):
            K[b, h, n[b][h]:] = V[b, h, n[b][h]:] = float("nan")
    nt = torch.tensor(n, dtype=torch.int32, device="cuda")
    if not paged:
        c = kvc.SlotCache.empty(B, Hkv, C, D)
        c.K.copy_(K)
        c.V.copy_(V)
    else:
        need = [[-(-x // 64) for x in row] for row in n]
        num = sum(map(sum, need)) + spare
        order = np.random.default_rng(num).permutation(num)
        table = np.full((B, Hkv, C // 64), -1, np.int32)
        i = 0
        for b in range(B):
            for h in range(Hkv):
                table[b, h, :need[b][h]] = order[i:i + need[b][h]]
                i += need[b][h]
        c = kvc.SlotCache.empty_paged(B, Hkv, C, D, num, block_table=torch.from_numpy(table))
        c.K.fill_(float("nan"))
        c.V.fill_(float("nan"))
        for b in range(B):
            for h in range(Hkv):
                for j in range(need[b][h]):
                    c.K[table[b, h, j]] = K[b, h, 64 * j:64 * j + 64]
                    c.V[table[b, h, j]] = V[b, h, 64 * j:64 * j + 64]
    c.n.copy_(nt)
    c.seqlen.copy_(nt.max(1).values)
    return c, K, V


def check_chunk(q, K, V, n, m, o, lse, Hq, what=""):
    Hkv = len(n[0])
    g = Hq // Hkv
    t = 0
    for b, mb in enumerate(m):
        w = slice(t, t + mb)
        for h in range(Hq):
            nn = n[b][h // g]
            last = nn - mb + torch.arange(mb)
            ref = attend_rows(q[w, h], K[b, h // g, :nn], V[b, h // g, :nn], last)
            check_rows(o[w, h], None if lse is None else lse[h, w], ref, f"{what} b={b} h={h}")
        t += mb


CHUNKS = [
    # Hq, Hkv, D, C, paged, n, m
    (8, 1, 128, 64, True, [[1]], [1]),
    (8, 1, 128, 128, True, [[64]], [64]),
    (8, 2, 128, 320, True, [[65, 300], [64, 128], [1, 320]], [5, 0, 1]),
    (4, 4, 64, 200, False, [[200, 199, 130, 17], [63, 64, 65, 16]], [17, 16]),
    (7, 1, 128, 500, False, [[500], [333], [40]], [3, 40, 40]),
    (16, 2, 64, 1024, True, [[1000, 513], [700, 1024]], [300, 2]),
    (6, 2, 128, 2048, True, [[2048, 1500]], [129]),
    (8, 8, 128, 700, False, [[600, 700, 512, 384, 129, 128, 127, 640]], [127]),
    (2, 1, 128, 4096, True, [[4000], [10], [0], [3333]], [1, 10, 0, 4]),
    # batches that two tiles per item suit: long chunks, and many sequences over long caches
    (32, 4, 128, 1536, True, [[1500, 1499, 1408, 1345], [777, 900, 1024, 600]], [600, 555]),
    (6, 2, 128, 1400, False, [[1399, 1300], [1400, 400]], [400, 333]),
    (64, 8, 128, 4096, True, [[4096 - 3 * i] * 8 for i in range(16)],
     [16, 17, 1, 0, 15, 16, 33, 16, 16, 9, 16, 16, 16, 20, 16, 16]),
]


@pytest.mark.parametrize("Hq,Hkv,D,C,paged,n,m", CHUNKS)
@pytest.mark.parametrize("splits", [0, 1, 3, 7])
def test_chunk(kvc, Hq, Hkv, D, C, paged, n, m, splits):
    gen = _gen(C + Hq)
    cache, K, V = _cache(kvc, gen, n, C, D, paged)
    T, pad = sum(m), 2
    q = _randn(gen, T + pad, Hq, D)
    o = torch.full_like(q, 7.0)
    lse = torch.full((Hq, T + pad), 7.0, device="cuda")
    ws = torch.full((max(kvc.kvc_chunk_workspace_size(cache, q, splits) // 4, 4),), float("nan"),
                    device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws, num_splits=splits)
    assert device_status_clean(kvc)
    check_chunk(q, K, V, n, m, o, lse, Hq)
    assert (o[T:] == 7.0).all() and (lse[:, T:] == 7.0).all()


@pytest.mark.parametrize("splits", [2, 4, 5, 16, 17, 33, 64])
def test_chunk_merge_of_few_rows(kvc, splits):
    """Every number of parts per warp of the merge, its rows ending inside a group of eight;
    parts without a key of some row, and tokens of no sequence before and between."""
    gen = _gen(40 + splits)
    n, m = [[2500, 1700], [64, 4096]], [3, 2]
    cache, K, V = _cache(kvc, gen, n, 4096, 128, True)
    q = _randn(gen, 9, 10, 128)
    o, lse = torch.full_like(q, 7.0), torch.full((10, 9), 7.0, device="cuda")
    cu = torch.tensor([2, 5, 7], dtype=torch.int32, device="cuda")
    ws = torch.full((kvc.kvc_chunk_workspace_size(cache, q, splits) // 4,), float("nan"),
                    device="cuda")
    kvc.kvc_chunk_attend(cache, q, cu, o, lse=lse, workspace=ws, num_splits=splits)
    assert device_status_clean(kvc)
    check_chunk(q[2:7], K, V, n, m, o[2:7], lse[:, 2:7], 10)
    for x in (o[:2], o[7:], lse[:, :2], lse[:, 7:]):
        assert (x == 7.0).all()


@pytest.mark.parametrize("D,splits", [(128, 2), (128, 5), (128, 9), (64, 6)])
def test_chunk_merge_of_many_rows(kvc, D, splits):
    """More rows than the merge shares out among a block's warps."""
    gen = _gen(50 + splits)
    n, m = [[900, 640], [1000, 333]], [400 if D == 128 else 700, 33]
    cache, K, V = _cache(kvc, gen, n, 1024, D, False)
    q = _randn(gen, sum(m), 14, D)
    o, lse = torch.full_like(q, 7.0), torch.full((14, sum(m)), 7.0, device="cuda")
    ws = torch.full((kvc.kvc_chunk_workspace_size(cache, q, splits) // 4,), float("nan"),
                    device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws, num_splits=splits)
    assert device_status_clean(kvc)
    check_chunk(q, K, V, n, m, o, lse, 14)


@pytest.mark.parametrize("splits", [1, 3, 20])
def test_chunk_ranges_that_run_backwards(kvc, splits):
    """A range of negative length is an empty sequence; the others', in any order, are right."""
    gen = _gen(33)
    n = [[150, 640], [700, 3], [64, 1500]]
    cache, K, V = _cache(kvc, gen, n, 1536, 128, True)
    q = _randn(gen, 30, 4, 128)
    o, lse = torch.full_like(q, 7.0), torch.full((4, 30), 7.0, device="cuda")
    cu = torch.tensor([20, 30, 0, 10], dtype=torch.int32, device="cuda")
    ws = torch.full((max(kvc.kvc_chunk_workspace_size(cache, q, splits) // 4, 4),), float("nan"),
                    device="cuda")
    kvc.kvc_chunk_attend(cache, q, cu, o, lse=lse, workspace=ws, num_splits=splits)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    for b, w in ((0, slice(20, 30)), (2, slice(0, 10))):
        check_chunk(q[w], K[b:b + 1], V[b:b + 1], n[b:b + 1], [10], o[w], lse[:, w], 4, f"{b}")
    assert (o[10:20] == 7.0).all() and (lse[:, 10:20] == 7.0).all()
    assert device_status_clean(kvc)


def test_chunk_of_more_tokens_than_slots_has_empty_rows(kvc):
    """A unit that holds fewer slots than the chunk has tokens: the first rows see nothing."""
    gen = _gen(9)
    cache, K, V = _cache(kvc, gen, [[3, 0]], 64, 64, True)
    q = _randn(gen, 5, 4, 64)
    o, lse = torch.full_like(q, 7.0), torch.full((4, 5), 7.0, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu([5]), o, lse=lse, workspace=ws)
    check_chunk(q, K, V, [[3, 0]], [5], o, lse, 4)
    assert (o[:2] == 0).all() and torch.isneginf(lse[:, :2]).all()
    assert (o[:, 2:] == 0).all() and torch.isneginf(lse[2:]).all()
    assert device_status_clean(kvc)


def test_chunk_bad_counts_and_pages_are_reported(kvc):
    """A count above C is an empty unit; a table entry outside the pool yields no data."""
    gen = _gen(10)
    cache, K, V = _cache(kvc, gen, [[100, 128]], 128, 128, True)
    q = _randn(gen, 2, 2, 128)
    o = torch.empty_like(q)
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")
    cache.n[0, 0] = 129
    kvc.kvc_chunk_attend(cache, q, _cu([2]), o, workspace=ws)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert (o[:, 0] == 0).all()
    check_rows(o[:, 1], None, attend_rows(q[:, 1], K[0, 1], V[0, 1], torch.tensor([126, 127])))
    cache.n[0, 0] = 100
    cache.block_table[0, 0, 1] = cache.num_pages
    kvc.kvc_chunk_attend(cache, q, _cu([2]), o, workspace=ws)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() & kvc.KVC_DEV_CAPACITY
    assert torch.isfinite(o).all()
    check_rows(o[:, 1], None, attend_rows(q[:, 1], K[0, 1], V[0, 1], torch.tensor([126, 127])))


def test_chunk_of_one_token_is_a_decode_step(kvc):
    gen = _gen(11)
    n = [[300, 64], [65, 511], [1, 448]]
    cache, K, V = _cache(kvc, gen, n, 512, 128, True)
    q = _randn(gen, 3, 8, 128)
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4,
                         kvc.kvc_workspace_size(cache, q) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu([1, 1, 1]), o, workspace=ws)
    for x in (cache.K, cache.V):            # the decode call takes finite rows only
        x.nan_to_num_(0.0)
    kvc.kvc_decode_attend(cache, q, o2, workspace=ws)
    assert (o.float() - o2.float()).abs().max() < 4e-3
    check_chunk(q, K, V, n, [1, 1, 1], o, None, 8)
    assert device_status_clean(kvc)


def test_graph_replay_follows_device_lengths(kvc):
    """One captured graph of both calls, replayed after the lengths on the device changed, on a
    stream of its own."""
    gen = _gen(12)
    Hq, Hkv, D, T = 8, 2, 128, 400
    qkv = _randn(gen, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    o, lse = torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda"), torch.zeros(Hq, T, device="cuda")
    n = [[400, 380], [200, 390]]
    cache, K, V = _cache(kvc, gen, n, 448, D, True)
    o2 = torch.zeros_like(o)
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")
    cu = _cu([150, 250])
    cu2 = _cu([100, 50])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        for _ in range(2):
            kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=cu, lse=lse)
            kvc.kvc_chunk_attend(cache, q, cu2, o2, workspace=ws)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=cu, lse=lse)
            kvc.kvc_chunk_attend(cache, q, cu2, o2, workspace=ws)
    for lens, m in (([150, 250], [100, 50]), ([400, 0], [1, 199]), ([3, 333], [0, 60])):
        cu.copy_(_cu(lens))
        cu2.copy_(_cu(m))
        o.zero_()
        o2.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_prompt(q, k, v, o, lse, cu, lens, Hq, Hkv, what=str(lens))
        check_chunk(q, K, V, n, m, o2, None, Hq, what=str(m))
    assert device_status_clean(kvc)


@pytest.mark.parametrize("Hq,Hkv,D,L", [(8, 1, 128, 300), (4, 4, 64, 200), (6, 2, 128, 90),
                                        (8, 1, 128, 1300), (3, 3, 128, 1200)])
def test_prompt_non_finite_rows_stay_with_the_rows_that_attend_them(kvc, Hq, Hkv, D, L):
    """Infinities and NaN in single key and value rows: rows before them, which do not attend
    them, are what they are without them; rows from them on are what the formula gives: NaN
    where a key is NaN, and in a channel whose attended values hold an infinity or NaN, that."""
    gen = _gen(D + L)
    q, k, v = _randn(gen, L, Hq, D), _randn(gen, L, Hkv, D), _randn(gen, L, Hkv, D)
    clean_k, clean_v = k.clone(), v.clone()
    inf_at, nan_at, key_at = L // 3, L // 2, 3 * L // 4
    v[inf_at, 0, 5] = float("inf")
    v[nan_at, 0, 9] = float("nan")
    k[key_at, 0] = float("nan")
    o, lse = torch.empty_like(q), torch.empty(Hq, L, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=_cu([L]), lse=lse)
    g = Hq // Hkv
    for h in range(Hq):
        ref = attend_rows(q[:, h], clean_k[:, h // g], clean_v[:, h // g], torch.arange(L))
        if h // g > 0:
            check_rows(o[:, h], lse[h], ref, f"h={h}")
            continue
        assert torch.isnan(o[key_at:, h]).all() and torch.isnan(lse[h, key_at:]).all()
        keep = torch.ones(D, dtype=torch.bool, device="cuda")
        keep[5] = keep[9] = False
        part = [x[:key_at] for x in ref]
        check_rows(o[:key_at, h][:, keep], lse[h, :key_at],
                   (part[0][:, keep], part[1], part[2][:, keep], part[3]), f"h={h}")
        assert torch.isposinf(o[inf_at:key_at, h, 5]).all()
        assert torch.isnan(o[nan_at:key_at, h, 9]).all()
        for c, first in ((5, inf_at), (9, nan_at)):
            err = (o[:first, h, c].double() - ref[0][:first, c]).abs()
            assert (err <= ref[2][:first, c]).all()
    assert device_status_clean(kvc)


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("m", [[3, 1], [60, 1], [150, 2], [400, 390]])
def test_chunk_non_finite_values_behind_a_row(kvc, m, splits):
    """The chunk's later value rows are infinite or NaN: the earlier rows do not attend them."""
    gen = _gen(sum(m))
    n = [[500, 700], [650, 513]]
    cache, K, V = _cache(kvc, gen, n, 704, 128, False)
    clean = V.clone()
    for h in range(2):
        last = n[0][h] - 1
        V[0, h, last, 3] = cache.V[0, h, last, 3] = float("inf")
        V[0, h, last, 77] = cache.V[0, h, last, 77] = float("nan")
    q = _randn(gen, sum(m), 8, 128)
    o, lse = torch.empty_like(q), torch.empty(8, sum(m), device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q, splits) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws, num_splits=splits)
    assert torch.isposinf(o[m[0] - 1, :, 3]).all() and torch.isnan(o[m[0] - 1, :, 77]).all()
    o[m[0] - 1, :, 3] = o[m[0] - 1, :, 77] = 0
    for b, w in ((0, slice(0, m[0])), (1, slice(m[0], sum(m)))):
        for h in range(8):
            nn = n[b][h // 4]
            ref = attend_rows(q[w, h], K[b, h // 4, :nn], clean[b, h // 4, :nn],
                              nn - m[b] + torch.arange(m[b]))
            if b == 0:
                ref[0][-1, 3] = ref[0][-1, 77] = 0
            check_rows(o[w, h], lse[h, w], ref, f"b={b} h={h}")
    assert device_status_clean(kvc)


@pytest.mark.parametrize("D,most", [(128, 8), (64, 3), (128, 40)])
def test_chunk_many_items_per_cta(kvc, D, most):
    """More (sequence, head) items than run at once, with odd and even block counts and heads
    evicted apart: what one item leaves in a CTA's pipeline must not reach the next."""
    B, Hkv, g, C = 72, 8, 2, 640
    rng = np.random.default_rng(D + most)
    m = rng.integers(0, most + 1, B).tolist()
    n = [[int(x) for x in rng.integers(mb, C + 1, Hkv)] for mb in m]
    gen = _gen(D)
    cache, K, V = _cache(kvc, gen, n, C, D, True)
    T, Hq = sum(m), g * Hkv
    q = _randn(gen, T, Hq, D)
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q) // 4, 4), device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda")
    for _ in range(3):
        kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws)
    assert device_status_clean(kvc)
    check_chunk(q, K, V, n, m, o, lse, Hq)
    first = o.clone()
    for _ in range(5):
        kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws)
        assert torch.equal(o, first)          # the same inputs give the same bits
    assert device_status_clean(kvc)


def test_prompt_lens_outside_the_padding_are_empty(kvc):
    gen = _gen(21)
    q, k, v = _randn(gen, 3, 2, 40, 64), _randn(gen, 3, 1, 40, 64), _randn(gen, 3, 1, 40, 64)
    o = torch.full_like(q, 7.0)
    lens = torch.tensor([41, -1, 40], dtype=torch.int32, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, lens=lens)
    torch.cuda.synchronize()
    assert kvc.kvc_read_device_status() == kvc.KVC_DEV_CAPACITY
    assert (o[:2] == 7.0).all()
    for h in range(2):
        check_rows(o[2, h], None, attend_rows(q[2, h], k[2, 0], v[2, 0], torch.arange(40)))


def test_element_offsets_beyond_32_bits(kvc):
    """Rows 8 million elements apart in a prompt, and pages at the end of pools of more than
    2^31 elements in a chunk."""
    gen = _gen(22)
    T, D, step = 300, 128, 8_000_000
    wide = torch.zeros(T * step, dtype=torch.float16, device="cuda")
    view = wide.as_strided((T, 4, D), (step, D, 1))
    x = _randn(gen, T, 4, D)
    view.copy_(x)
    o = torch.empty(T, 2, D, dtype=torch.float16, device="cuda")
    kvc.kvc_prompt_attend(view[:, :2], view[:, 2:3], view[:, 3:], o, cu_seqlens=_cu([T]))
    check_prompt(x[:, :2], x[:, 2:3], x[:, 3:], o, None, _cu([T]), [T], 2, 1)
    del wide, view
    num = 280_000
    n = [[500, 77]]
    small, K, V = _cache(kvc, gen, n, 512, D, True)
    big = kvc.SlotCache(K=torch.empty(num, 64, D, dtype=torch.float16, device="cuda"),
                        V=torch.empty(num, 64, D, dtype=torch.float16, device="cuda"),
                        pos=small.pos, n=small.n, seqlen=small.seqlen,
                        block_table=torch.where(small.block_table >= 0,
                                                num - 1 - small.block_table, -1).int())
    for j in range(small.num_pages):
        big.K[num - 1 - j], big.V[num - 1 - j] = small.K[j], small.V[j]
    assert big.K.numel() > 2 ** 31
    q = _randn(gen, 3, 8, D)
    o = torch.empty_like(q)
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(big, q) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(big, q, _cu([3]), o, workspace=ws)
    check_chunk(q, K, V, n, [3], o, None, 8)
    # the packed append at the same end
    new = _randn(gen, 5, 2, D)
    slots = torch.arange(num * 64 - 10, num * 64, dtype=torch.int32, device="cuda").reshape(5, 2)
    kvc.kvc_append_packed(big, new, new, slots)
    assert torch.equal(big.K.view(-1, D)[-10:], new.reshape(-1, D))
    assert torch.equal(big.V.view(-1, D)[-10:], new.reshape(-1, D))
    assert device_status_clean(kvc)


def test_two_streams_at_once(kvc):
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    gen = _gen(23)
    n = [[900, 1000], [700, 1024], [513, 64]]
    cache, K, V = _cache(kvc, gen, n, 1024, 128, True)
    m = [3, 1, 5]
    qs = [_randn(gen, 9, 8, 128) for _ in range(2)]
    os_ = [torch.empty_like(q) for q in qs]
    wss = [torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q, 4) // 4, 4), device="cuda") for q in qs]
    L = 700
    x = _randn(gen, L, 10, 128)
    po, cu, cum = torch.empty(L, 8, 128, dtype=torch.float16, device="cuda"), _cu([L]), _cu(m)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            kvc.kvc_chunk_attend(cache, qs[i], cum, os_[i], workspace=wss[i], num_splits=4,
                                 stream=streams[i])
        kvc.kvc_prompt_attend(x[:, :8], x[:, 8:9], x[:, 9:], po, cu_seqlens=cu, stream=streams[0])
    torch.cuda.synchronize()
    for i in range(2):
        check_chunk(qs[i], K, V, n, m, os_[i], None, 8)
    check_prompt(x[:, :8], x[:, 8:9], x[:, 9:], po, None, cu, [L], 8, 1)
    assert device_status_clean(kvc)
