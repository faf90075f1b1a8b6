"""Prompt and chunk attention where they can go wrong at length: value rows that are not finite
far from the rows that are computed again, and many keys of little weight beside a strong one; layouts: padded batches in the two-tile form,
projections whose tokens lie further apart than their heads, results that are a column range."""
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


@pytest.mark.parametrize("Hq,D,at", [(8, 128, 200_003 - 10), (8, 128, 5), (8, 64, 200_003 - 30),
                                     (1, 128, 200_003 - 100)])
def test_long_prompt_with_a_value_row_that_is_not_finite(kvc, Hq, D, at):
    """An infinity and a NaN in one value row of 200 003, in the last tile or the first one: the
    rows before it are what they are without it, the rows from it on have them in those two
    channels, and no wait inside the kernel runs out meanwhile."""
    L = 200_003
    gen = _gen(at + D)
    q, k, v = _randn(gen, L, Hq, D), _randn(gen, L, 1, D), _randn(gen, L, 1, D)
    clean = v.clone()
    v[at, 0, 5], v[at, 0, 41] = float("-inf"), float("nan")
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, L), 7.0, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=_cu([L]), lse=lse)
    assert device_status_clean(kvc)
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[5] = keep[41] = False
    before = torch.arange(max(0, at - 130), at)
    behind = torch.unique(torch.cat([torch.arange(at, min(L, at + 40)), torch.arange(at, L, 19_001)]))
    for h in {0, Hq - 1}:
        check_rows(o[before, h], lse[h, before],
                   attend_rows(q[before, h], k[:at, 0], clean[:at, 0], before), f"before, h={h}")
        ro, rl, to, tl = attend_rows(q[behind, h], k[:, 0], clean[:, 0], behind)
        check_rows(o[behind, h][:, keep], lse[h, behind], (ro[:, keep], rl, to[:, keep], tl),
                   f"behind, h={h}")
    assert torch.isneginf(o[at:, :, 5]).all() and torch.isnan(o[at:, :, 41]).all()
    assert torch.isfinite(o[:at]).all() and torch.isfinite(o[at:][:, :, keep]).all()


@pytest.mark.parametrize("D,splits", [(128, 0), (128, 1), (64, 3)])
def test_long_chunk_with_values_that_are_not_finite(kvc, D, splits):
    """A chunk over 100 000 slots whose newest value row is NaN throughout: the chunk's other
    tokens do not attend it."""
    C, n, m, Hq = 100_032, 100_001, 9, 8
    gen = _gen(D + splits)
    cache = kvc.SlotCache.empty(1, 2, C, D)
    cache.K.copy_(_randn(gen, 1, 2, C, D))
    cache.V.copy_(_randn(gen, 1, 2, C, D))
    cache.n.fill_(n)
    clean = cache.V.clone()
    cache.V[0, 0, n - 1] = float("nan")
    cache.V[0, 1, n - 1, 7] = float("inf")
    q = _randn(gen, m, Hq, D)
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, m), 7.0, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q, splits) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu([m]), o, lse=lse, workspace=ws, num_splits=splits)
    assert device_status_clean(kvc)
    assert torch.isnan(o[-1, :4]).all() and torch.isposinf(o[-1, 4:, 7]).all()
    last = n - m + torch.arange(m)
    for h in range(Hq):
        ref = attend_rows(q[:, h], cache.K[0, h // 4, :n], clean[0, h // 4, :n], last)
        check_rows(o[:-1, h], lse[h, :-1], tuple(x[:-1] for x in ref), f"h={h}")


def _weak(D, n, dev="cuda"):
    """n keys of which the first has the score 17.5 (25.2 in powers of two) and the others 0, so
    that their weights are below 2^-25 of the first one's, each; together they are 0.3% of the
    131 072 keys' weight, with values a hundred times the first one's."""
    k = torch.zeros(n, D, dtype=torch.float16, device=dev)
    k[0, 0] = 3.5
    v = torch.full((n, D), 100.0, dtype=torch.float16, device=dev)
    v[:, 1::2] = -50.0
    v[0] = 1.0
    return k, v


def _check_weak(o, lse, q, k, v, last):
    """As check_rows, with weights rounded by 2^-32 of the row's largest at most where they are
    not held to 2^-11 (the references in token_refs allow 2^-25)."""
    ro, rl, to, tl = attend_rows(q, k, v, last, 1.0)
    count = (last + 1).clamp(0, k.shape[0]).double().to(to.device)[:, None]
    to = to - count * (2.0 ** -25 - 2.0 ** -32) * v.double().abs().max()
    check_rows(o, lse, (ro, rl, to, tl))


@pytest.mark.parametrize("Hq,D,L", [(1, 128, 131_072), (8, 128, 131_072), (2, 64, 131_072),
                                    (8, 128, 1000)])
def test_prompt_many_keys_of_little_weight(kvc, Hq, D, L):
    k, v = _weak(D, L)
    q = torch.zeros(L, Hq, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 5.0
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, L), 7.0, device="cuda")
    kvc.kvc_prompt_attend(q, k[:, None], v[:, None], o, cu_seqlens=_cu([L]), lse=lse,
                          softmax_scale=1.0)
    assert device_status_clean(kvc)
    rows = torch.unique(torch.cat([torch.arange(0, L, max(1, L // 20)), torch.arange(L - 5, L)]))
    for h in range(Hq):
        _check_weak(o[rows, h], lse[h, rows], q[rows, h], k, v, rows)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_chunk_many_keys_of_little_weight(kvc, D, splits):
    C, m = 131_072, 3
    k, v = _weak(D, C)
    cache = kvc.SlotCache.empty(1, 1, C, D)
    cache.K[0, 0], cache.V[0, 0] = k, v
    cache.n.fill_(C)
    q = torch.zeros(m, 8, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 5.0
    o, lse = torch.full_like(q, 7.0), torch.full((8, m), 7.0, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q, splits) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu([m]), o, lse=lse, workspace=ws, num_splits=splits,
                         softmax_scale=1.0)
    assert device_status_clean(kvc)
    for h in range(8):
        _check_weak(o[:, h], lse[h], q[:, h], k, v, C - m + torch.arange(m))


def test_chunk_workspace_of_several_sizes(kvc):
    """A small batch is split and needs a workspace where a large one needs none: the size of
    the largest T does not do for the others (refused before anything is launched), the largest
    of the sizes does for all."""
    B, C, Hq, Hkv, D = 4, 4096, 32, 4, 128
    gen = _gen(2)
    cache = kvc.SlotCache.empty(B, Hkv, C, D)
    cache.K.copy_(_randn(gen, B, Hkv, C, D))
    cache.V.copy_(_randn(gen, B, Hkv, C, D))
    n = [[1000, 3000, 4096, 70], [4000, 129, 2048, 800], [3333] * 4, [64, 4000, 500, 1]]
    cache.n.copy_(torch.tensor(n, dtype=torch.int32))
    q = _randn(gen, 2048, Hq, D)
    sizes = {T: kvc.kvc_chunk_workspace_size(cache, q[:T]) for T in (4, 8, 64, 256, 2048)}
    assert sizes[2048] < sizes[8] and sizes[2048] < max(sizes.values())
    o = torch.full_like(q, 7.0)
    small = torch.empty(sizes[2048] // 4 + 4, device="cuda")
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_chunk_attend(cache, q[:8], _cu([2] * 4), o[:8], workspace=small)
    assert e.value.status == kvc.KVC_ERR_WORKSPACE and (o == 7.0).all()
    ws = torch.full((max(sizes.values()) // 4,), float("nan"), device="cuda")
    for T in sizes:
        m = T // B
        kvc.kvc_chunk_attend(cache, q[:T], _cu([m] * B), o[:T], workspace=ws)
        for b in range(B):
            w = slice(b * m, b * m + m)
            for h in range(0, Hq, 5):
                nn = n[b][h // 8]
                ref = attend_rows(q[w, h], cache.K[b, h // 8, :nn], cache.V[b, h // 8, :nn],
                                  nn - m + torch.arange(m))
                check_rows(o[w, h], None, ref, f"T={T} b={b} h={h}")
    assert device_status_clean(kvc)


@pytest.mark.parametrize("Hq,Hkv,D,L,lens", [(8, 1, 128, 1500, [1500, 3, 700, 1499]),
                                             (3, 3, 128, 1100, [1025, 0, 1100]),
                                             (14, 2, 128, 1300, None),
                                             (4, 2, 64, 1200, [1200, 1001])])
@pytest.mark.parametrize("token_major", [False, True])
def test_padded_prompts_of_more_than_a_thousand_tokens(kvc, Hq, Hkv, D, L, lens, token_major):
    """Two tiles per item over a padded batch.  token_major: q, k, v are [B, L, H, D] column ranges
    of one projection, transposed, and o is a column range of a wider result, so that a token's
    stride is larger than a head's; what lies beside them stays as it was."""
    B = 3 if lens is None else len(lens)
    real = [L] * B if lens is None else lens
    gen = _gen(L + Hq)
    if token_major:
        wide = _randn(gen, B, L, Hq + 2 * Hkv + 1, D)
        q, k, v = (wide[:, :, a:b].transpose(1, 2) for a, b in
                   ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        room = torch.full((B, L, Hq + 3, D), 7.0, dtype=torch.float16, device="cuda")
        o = room[:, :, 1:1 + Hq].transpose(1, 2)
    else:
        q = _randn(gen, B, Hq, L, D)
        k, v = _randn(gen, B, Hkv, L + 30, D), _randn(gen, B, Hkv, L + 30, D)
        o = torch.full_like(q, 7.0)
    for b, n in enumerate(real):
        q[b, :, n:] = k[b, :, n:] = v[b, :, n:] = float("nan")
    lse = torch.full((B, Hq, L), 7.0, device="cuda")
    dl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    kvc.kvc_prompt_attend(q, k, v, o, lens=dl, lse=lse)
    assert device_status_clean(kvc)
    for b, n in enumerate(real):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            ref = attend_rows(q[b, h, :n], k[b, g, :n], v[b, g, :n], torch.arange(n))
            check_rows(o[b, h, :n], lse[b, h, :n], ref, f"b={b} h={h}")
        assert (o[b, :, n:] == 7.0).all() and (lse[b, :, n:] == 7.0).all()
    if token_major:
        assert (room[:, :, 0] == 7.0).all() and (room[:, :, 1 + Hq:] == 7.0).all()


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(8, 2, 128, [200, 17, 1, 63]), (5, 1, 64, [90, 333]),
                                           (8, 1, 128, [1400, 1100])])
def test_packed_result_in_a_column_range(kvc, Hq, Hkv, D, lens):
    """o is a column range of a wider buffer, with the heads' stride larger than D."""
    T = sum(lens)
    gen = _gen(T)
    qkv = _randn(gen, T, Hq + 2 * Hkv, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    room = torch.full((T + 2, Hq + 1, D + 8), 7.0, dtype=torch.float16, device="cuda")
    o = room[1:T + 1, 1:, :D]
    kvc.kvc_prompt_attend(q, k, v, o, cu_seqlens=_cu(lens))
    assert device_status_clean(kvc)
    t = 0
    for n in lens:
        for h in range(Hq):
            g = h // (Hq // Hkv)
            ref = attend_rows(q[t:t + n, h], k[t:t + n, g], v[t:t + n, g], torch.arange(n))
            check_rows(o[t:t + n, h], None, ref, f"t={t} h={h}")
        t += n
    room[1:T + 1, 1:, :D] = 7.0
    assert (room == 7.0).all()


@pytest.mark.parametrize("D,splits", [(128, 1), (128, 4), (64, 1), (64, 5)])
@pytest.mark.parametrize("m", [[3, 40], [300, 450]])
def test_chunk_with_a_given_scale_and_strided_rows(kvc, D, splits, m):
    """softmax_scale, q a column range and o one of a wider buffer."""
    Hq, Hkv, C, n = 8, 2, 1024, [[900, 1024], [450, 777]]
    gen = _gen(D + splits + m[0])
    cache = kvc.SlotCache.empty(2, Hkv, C, D)
    cache.K.copy_(_randn(gen, 2, Hkv, C, D) * 2)
    cache.V.copy_(_randn(gen, 2, Hkv, C, D))
    cache.n.copy_(torch.tensor(n, dtype=torch.int32))
    T = sum(m)
    q = _randn(gen, T, Hq + 3, D)[:, 2:2 + Hq]
    room = torch.full((T, Hq + 2, D + 16), 7.0, dtype=torch.float16, device="cuda")
    o, lse = room[:, 1:1 + Hq, 8:8 + D], torch.full((Hq, T), 7.0, device="cuda")
    ws = torch.empty(max(kvc.kvc_chunk_workspace_size(cache, q, splits) // 4, 4), device="cuda")
    kvc.kvc_chunk_attend(cache, q, _cu(m), o, lse=lse, workspace=ws, num_splits=splits,
                         softmax_scale=0.21)
    assert device_status_clean(kvc)
    for b, w in ((0, slice(0, m[0])), (1, slice(m[0], T))):
        for h in range(Hq):
            nn = n[b][h // 4]
            ref = attend_rows(q[w, h], cache.K[b, h // 4, :nn], cache.V[b, h // 4, :nn],
                              nn - m[b] + torch.arange(m[b]), 0.21)
            check_rows(o[w, h], lse[h, w], ref, f"b={b} h={h}")
    room[:, 1:1 + Hq, 8:8 + D] = 7.0
    assert (room == 7.0).all()
