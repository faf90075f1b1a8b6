"""Trees of drafted tokens: masks and positions, attention, verification and commit against
plain 64-bit references; odd sizes, strides, empty rows and sequences, values that are not
finite, refused units, graphs and streams, and a whole step."""
import numpy as np
import pytest
import torch

from draft_refs import (attend_seen, lineage, mask_words, random_tree, seen_slots, verify_batch)
from helpers import device_status_clean
from token_refs import check_rows

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


def _status(kvc):
    torch.cuda.synchronize()
    return kvc.kvc_read_device_status()


# ---------------------------------------------------------------- masks and positions

@pytest.mark.parametrize("sizes,fan,words", [([1], 0, 1), ([64, 1, 0, 63], 3, 1), ([65, 128, 7], 9, 2),
                                             ([0, 0, 2], 0, 3), ([256, 255, 193, 1], 40, 4),
                                             ([256], 0, 4), ([17] * 300, 5, 1)])
def test_tree_plan(kvc, sizes, fan, words):
    rng = np.random.default_rng(sum(sizes) + fan)
    trees = [random_tree(rng, m, fan) for m in sizes]
    T, pad = sum(sizes), 3
    parent = _i32(sum(trees, []) + [7] * pad)
    mask = torch.full((T + pad, words), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((T + pad,), 77, dtype=torch.int32, device="cuda")
    seqlen = _i32(rng.integers(0, 9000, len(sizes)))
    kvc.kvc_tree_plan(_cu(sizes), parent, mask, pos=pos, seqlen=seqlen)
    assert device_status_clean(kvc)
    assert torch.equal(mask[:T].cpu(), mask_words(trees, words))
    depth = [bin(x).count("1") - 1 for tree in trees for x in lineage(tree)]
    want = np.array(depth, dtype=np.int64) + np.repeat(seqlen.cpu().numpy(), sizes)
    assert (pos[:T].cpu().numpy() == want).all()
    assert (mask[T:] == 77).all() and (pos[T:] == 77).all()
    # without positions, and positions without lengths
    mask.fill_(77)
    kvc.kvc_tree_plan(_cu(sizes), parent, mask)
    assert torch.equal(mask[:T].cpu(), mask_words(trees, words))
    kvc.kvc_tree_plan(_cu(sizes), parent, mask, pos=pos)
    assert (pos[:T].cpu().numpy() == depth).all()
    assert device_status_clean(kvc)


def test_tree_plan_bad_parents_sizes_and_ranges(kvc):
    """Parents that are no earlier node count as none; a tree of more nodes than the mask has bits
    and ranges outside the batch are left alone.  Each is reported."""
    parent = _i32([-1, 0, 2, -5, 3, 900])
    mask = torch.full((6, 1), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((6,), 77, dtype=torch.int32, device="cuda")
    kvc.kvc_tree_plan(_cu([6]), parent, mask, pos=pos)
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert mask[:, 0].tolist() == [1, 3, 4, 8, 24, 32]
    assert pos.tolist() == [0, 1, 0, 0, 1, 0]
    chain = _i32([i - 1 for i in range(65)] + [-1])
    mask = torch.full((66, 1), 77, dtype=torch.int64, device="cuda")
    kvc.kvc_tree_plan(_cu([65, 1]), chain, mask)
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert (mask[:65] == 77).all() and mask[65, 0] == 1
    for cu in ([-1, 1], [0, 67], [5, 3]):
        mask.fill_(77)
        kvc.kvc_tree_plan(_i32(cu), chain, mask)
        assert _status(kvc) == kvc.KVC_DEV_CAPACITY
        assert (mask == 77).all()
    assert device_status_clean(kvc)


# ---------------------------------------------------------------- attention

def _cache(kvc, gen, n, C, D, paged, spare=3):
    """A slot cache with counts n [B, Hkv]; rows behind n, and pages nobody holds, are NaN."""
    B, Hkv = len(n), len(n[0])
    K, V = _randn(gen, B, Hkv, C, D), _randn(gen, B, Hkv, C, D)
    for b in range(B):
        for h in range(Hkv):
            K[b, h, n[b][h]:] = V[b, h, n[b][h]:] = float("nan")
    nt = _i32(n)
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


def check_tree(q, K, V, n, bits, o, lse, Hq, what=""):
    """bits: per sequence the nodes' masks as Python integers."""
    g, t = Hq // len(n[0]), 0
    for b, rows in enumerate(bits):
        m = len(rows)
        w = slice(t, t + m)
        for h in range(Hq):
            nn = n[b][h // g]
            ref = attend_seen(q[w, h], K[b, h // g, :nn], V[b, h // g, :nn],
                              seen_slots(rows, nn, m))
            check_rows(o[w, h], None if lse is None else lse[h, w], ref, f"{what} b={b} h={h}")
        t += m


def _ws(kvc, cache, q, splits=0):
    return torch.full((max(kvc.kvc_tree_workspace_size(cache, q, splits) // 4, 4),), float("nan"),
                      device="cuda")


TREES = [
    # Hq, Hkv, D, C, paged, n, nodes, fan, words
    (8, 1, 128, 64, True, [[1]], [1], 0, 1),
    (8, 1, 128, 128, True, [[64]], [64], 5, 1),
    (8, 1, 128, 128, True, [[65]], [64], 63, 1),
    (8, 2, 128, 320, True, [[65, 300], [64, 128], [1, 320]], [5, 0, 1], 2, 1),
    (4, 4, 64, 200, False, [[200, 199, 130, 17], [63, 64, 65, 16]], [17, 16], 4, 2),
    (7, 1, 128, 500, False, [[500], [333], [40]], [3, 40, 40], 12, 1),
    (16, 2, 64, 1024, True, [[1000, 513], [700, 1024]], [200, 2], 30, 4),
    (6, 2, 128, 2048, True, [[2048, 1500]], [129], 1, 3),
    (8, 8, 128, 700, False, [[600, 700, 512, 384, 256, 255, 257, 640]], [255], 200, 4),
    (2, 1, 128, 4096, True, [[4000], [10], [0], [3333]], [1, 10, 0, 4], 3, 1),
    # batches that two tiles per item suit: big trees, and many sequences over long caches
    (32, 4, 128, 1536, True, [[1500, 1499, 1408, 1345], [777, 900, 1024, 600]], [256, 190], 50, 4),
    (6, 2, 128, 1400, False, [[1399, 1300], [1400, 400]], [250, 233], 8, 4),
    (64, 8, 128, 4096, True, [[4096 - 3 * i] * 8 for i in range(16)],
     [16, 17, 1, 0, 15, 16, 33, 16, 16, 9, 16, 16, 16, 20, 16, 16], 6, 1),
]


@pytest.mark.parametrize("Hq,Hkv,D,C,paged,n,m,fan,words", TREES)
@pytest.mark.parametrize("splits", [0, 1, 3, 7])
def test_tree_attend(kvc, Hq, Hkv, D, C, paged, n, m, fan, words, splits):
    gen, rng = _gen(C + Hq), np.random.default_rng(C + fan)
    cache, K, V = _cache(kvc, gen, n, C, D, paged)
    trees = [random_tree(rng, x, fan) for x in m]
    T, pad = sum(m), 2
    q = _randn(gen, T + pad, Hq, D)
    o = torch.full_like(q, 7.0)
    lse = torch.full((Hq, T + pad), 7.0, device="cuda")
    mask = torch.cat([mask_words(trees, words), torch.full((pad, words), -1)]).cuda()
    kvc.kvc_tree_attend(cache, q, _cu(m), mask, o, lse=lse, workspace=_ws(kvc, cache, q, splits),
                        num_splits=splits)
    assert device_status_clean(kvc)
    check_tree(q, K, V, n, [lineage(t) for t in trees], o, lse, Hq)
    assert (o[T:] == 7.0).all() and (lse[:, T:] == 7.0).all()


@pytest.mark.parametrize("D,splits", [(128, 1), (128, 5), (64, 1), (64, 4)])
def test_any_mask(kvc, D, splits):
    """Masks that are no trees: bits above the node are not looked at, nodes that do not see
    themselves, and rows that see no slot at all where the unit holds nothing older."""
    gen, rng = _gen(D), np.random.default_rng(D + splits)
    m, words = [100, 70, 130], 3
    n = [[100, 600], [69, 70], [577, 130]]
    bits = [[int.from_bytes(rng.bytes(24), "little") for _ in range(x)] for x in m]
    bits[0][3] = bits[0][99] = bits[2][0] = bits[2][129] = bits[1][69] = 0
    bits[1][1] = 1 << 1          # sees itself alone, whose slot is 0 in a unit of 69
    bits[1][0] = 1               # a slot before the unit's first
    flat = np.array([[(x >> 64 * w) & (2 ** 64 - 1) for w in range(words)] for r in bits for x in r],
                    dtype=np.uint64)
    cache, K, V = _cache(kvc, gen, n, 640, D, True)
    q = _randn(gen, sum(m), 6, D)
    o, lse = torch.full_like(q, 7.0), torch.full((6, sum(m)), 7.0, device="cuda")
    mask = torch.from_numpy(flat.view(np.int64)).cuda()
    kvc.kvc_tree_attend(cache, q, _cu(m), mask, o, lse=lse, workspace=_ws(kvc, cache, q, splits),
                        num_splits=splits)
    assert device_status_clean(kvc)
    check_tree(q, K, V, n, bits, o, lse, 6)
    assert (o[3, :3] == 0).all() and torch.isneginf(lse[:3, 3]).all()
    assert (o[100, :3] == 0).all() and torch.isneginf(lse[:3, 100]).all()


@pytest.mark.parametrize("Hq,Hkv,D,C,n,m,splits", [
    (64, 8, 128, 576, [[576 - 7 * i] * 8 for i in range(9)], [8, 1, 7, 3, 8, 0, 8, 5, 6], 0),
    (4, 1, 128, 8192, [[8000]], [5], 0), (8, 2, 64, 300, [[300, 299]], [130], 2)])
def test_a_chain_is_a_chunk(kvc, Hq, Hkv, D, C, n, m, splits):
    gen = _gen(Hq + D)
    cache, K, V = _cache(kvc, gen, n, C, D, False)
    q = _randn(gen, sum(m), Hq, D)
    words = -(-max(m) // 64)
    mask = mask_words([list(range(-1, x - 1)) for x in m], words).cuda()
    o, o2, lse, lse2 = torch.empty_like(q), torch.empty_like(q), *(
        torch.empty(Hq, sum(m), device="cuda") for _ in range(2))
    ws = _ws(kvc, cache, q, splits)
    kvc.kvc_tree_attend(cache, q, _cu(m), mask, o, lse=lse, workspace=ws, num_splits=splits)
    kvc.kvc_chunk_attend(cache, q, _cu(m), o2, lse=lse2, workspace=ws, num_splits=splits)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("splits", [1, 4])
def test_tree_of_more_nodes_than_bits(kvc, splits):
    """Such a sequence counts as empty and is reported; the others are right."""
    gen, rng = _gen(7), np.random.default_rng(7)
    m, n = [10, 65, 3], [[200], [300], [250]]
    cache, K, V = _cache(kvc, gen, n, 320, 128, True)
    trees = [random_tree(rng, x, 3) for x in m]
    q = _randn(gen, sum(m), 4, 128)
    o, lse = torch.full_like(q, 7.0), torch.full((4, sum(m)), 7.0, device="cuda")
    mask = mask_words(trees, 1).cuda()
    kvc.kvc_tree_attend(cache, q, _cu(m), mask, o, lse=lse, workspace=_ws(kvc, cache, q, splits),
                        num_splits=splits)
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert (o[10:75] == 7.0).all() and (lse[:, 10:75] == 7.0).all()
    for b, w in ((0, slice(0, 10)), (2, slice(75, 78))):
        check_tree(q[w], K[b:b + 1], V[b:b + 1], n[b:b + 1], [lineage(trees[b])], o[w], lse[:, w], 4)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("Hq,D,m,splits", [(8, 128, 9, 1), (8, 128, 60, 1), (4, 64, 33, 1),
                                           (2, 128, 200, 1), (8, 128, 40, 3)])
def test_non_finite_values_of_nodes(kvc, Hq, D, m, splits):
    """An infinity and a NaN in value rows of nodes, one in an older slot, and a NaN key: rows that
    attend them have them in those channels, the others are what they are without."""
    gen, rng = _gen(D + m), np.random.default_rng(m)
    n = [[300 + m]]
    cache, K, V = _cache(kvc, gen, n, 640, D, False)
    tree = random_tree(rng, m, 6)
    bits = lineage(tree)
    base = n[0][0] - m
    # nodes that some later node does not continue
    hidden = [j for j in range(1, m) if any(not bits[i] >> j & 1 for i in range(j + 1, m))]
    inf_at, nan_at, key_at = hidden[0], hidden[len(hidden) // 2], hidden[-1]
    clean_k, clean_v = K.clone(), V.clone()
    for X, at, c, x in ((cache.V, base + inf_at, 5, float("-inf")), (cache.V, base + nan_at, 9, float("nan")),
                        (cache.V, base - 200, 11, float("inf")), (cache.K, base + key_at, None, float("nan"))):
        X[0, 0, at] = x if c is None else X[0, 0, at]
        if c is not None:
            X[0, 0, at, c] = x
    q = _randn(gen, m, Hq, D)
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, m), 7.0, device="cuda")
    kvc.kvc_tree_attend(cache, q, _cu([m]), mask_words([tree], -(-m // 64)).cuda(), o, lse=lse,
                        workspace=_ws(kvc, cache, q, splits), num_splits=splits)
    assert device_status_clean(kvc)
    has = lambda j: torch.tensor([bool(x >> j & 1) for x in bits], device="cuda")  # noqa: E731
    lost = has(key_at)
    for h in range(Hq):
        assert torch.isnan(o[lost, h]).all() and torch.isnan(lse[h, lost]).all()
        ro, rl, to, tl = attend_seen(q[:, h], clean_k[0, 0, :n[0][0]], clean_v[0, 0, :n[0][0]],
                                     seen_slots(bits, n[0][0], m))
        row = ~lost
        assert torch.isposinf(o[row, h, 11]).all()
        assert torch.isneginf(o[row & has(inf_at), h, 5]).all()
        assert torch.isnan(o[row & has(nan_at), h, 9]).all()
        good = torch.ones(m, D, dtype=torch.bool, device="cuda")
        good[lost] = False
        good[:, 11] = False
        good[has(inf_at), 5] = False
        good[has(nan_at), 9] = False
        err = (o[:, h].double() - ro).abs()
        assert torch.isfinite(o[:, h][good]).all()
        assert (err[good] <= to[good]).all(), (err / to)[good].max()
        assert ((lse[h].double() - rl).abs()[row] <= tl[row]).all()
    assert device_status_clean(kvc)


def test_tree_rows_of_a_projection_and_results_in_a_column_range(kvc):
    gen, rng = _gen(19), np.random.default_rng(19)
    n, m = [[400, 350], [90, 333]], [20, 13]
    cache, K, V = _cache(kvc, gen, n, 448, 128, True)
    trees = [random_tree(rng, x, 4) for x in m]
    wide = _randn(gen, sum(m), 14, 128)
    out = torch.full((sum(m), 12, 128), 7.0, dtype=torch.float16, device="cuda")
    q, o = wide[:, 2:10], out[:, 1:9]
    kvc.kvc_tree_attend(cache, q, _cu(m), mask_words(trees, 1).cuda(), o,
                        workspace=_ws(kvc, cache, q), softmax_scale=0.07)
    g = 4
    t = 0
    for b, tree in enumerate(trees):
        w = slice(t, t + m[b])
        for h in range(8):
            nn = n[b][h // g]
            check_rows(o[w, h], None, attend_seen(q[w, h], K[b, h // g, :nn], V[b, h // g, :nn],
                                                  seen_slots(lineage(tree), nn, m[b]), 0.07))
        t += m[b]
    assert (out[:, 0] == 7.0).all() and (out[:, 9:] == 7.0).all()
    assert device_status_clean(kvc)


@pytest.mark.parametrize("D,most", [(128, 8), (64, 3), (128, 40)])
def test_tree_many_items_per_cta(kvc, D, most):
    """More (sequence, head) items than run at once, and the same bits from the same inputs."""
    B, Hkv, g, C = 72, 8, 2, 640
    rng = np.random.default_rng(D + most)
    m = rng.integers(0, most + 1, B).tolist()
    n = [[int(x) for x in rng.integers(mb, C + 1, Hkv)] for mb in m]
    trees = [random_tree(rng, x, 3) for x in m]
    gen = _gen(D)
    cache, K, V = _cache(kvc, gen, n, C, D, True)
    T, Hq = sum(m), g * Hkv
    q = _randn(gen, T, Hq, D)
    mask, ws = mask_words(trees, 1).cuda(), _ws(kvc, cache, q)
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda")
    for _ in range(3):
        kvc.kvc_tree_attend(cache, q, _cu(m), mask, o, lse=lse, workspace=ws)
    assert device_status_clean(kvc)
    check_tree(q, K, V, n, [lineage(t) for t in trees], o, lse, Hq)
    first = o.clone()
    for _ in range(5):
        kvc.kvc_tree_attend(cache, q, _cu(m), mask, o, lse=lse, workspace=ws)
        assert torch.equal(o, first)


# ---------------------------------------------------------------- verification

def _probs(gen, T, V, spread=2.0, near=0.6):
    x = spread * torch.randn(T, V, generator=gen, device="cuda")
    p = torch.softmax(x, 1)
    return p, torch.softmax(x + near * torch.randn(T, V, generator=gen, device="cuda"), 1)


def _drafts(gen, trees, q, V):
    """Tokens drawn from the parents' rows of q."""
    above, t = [], 0
    for tree in trees:
        above += [t + max(x, 0) for x in tree]
        t += len(tree)
    if t == 0:
        return torch.zeros(0, dtype=torch.int32, device="cuda")
    race = torch.rand(t, V, generator=gen, device="cuda").clamp(min=1e-30)
    return (-torch.log(race) / q[above].clamp(min=1e-30)).argmin(1).int()


def _verify(kvc, m, tokens, p, u, u_next, max_path, parent=None, q=None, **kw):
    B = len(m)
    path = torch.full((B, max_path), 77, dtype=torch.int32, device="cuda")
    count, nxt = (torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    kvc.kvc_draft_verify(_cu(m), tokens, p, u, u_next, path, count, nxt, parent=parent, q=q, **kw)
    return path, count, nxt


def check_verify(got, trees, tokens, p, q, u, u_next, max_path):
    n = lambda x: None if x is None else x.cpu().numpy()  # noqa: E731
    path, count, nxt = verify_batch(trees, n(tokens), n(p), n(q), n(u), n(u_next), max_path)
    assert (got[1].cpu().numpy() == count).all()
    assert (got[0].cpu().numpy() == path).all()
    assert (got[2].cpu().numpy() == nxt).all()
    return count


VERIFY = [
    # vocabulary, nodes, fan
    (1, [1, 2, 3], 1), (5, [4, 0, 9, 1], 3), (31, [33, 64, 65], 20), (1000, [7] * 40, 2),
    (4099, [12, 3, 1, 30, 0, 2], 6), (32000, [5, 60, 1], 10), (32000, [3] * 70, 0),
    (50001, [256, 100], 120), (128000, [4], 1),
]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V,m,fan", VERIFY)
def test_verify(kvc, V, m, fan, drawn):
    gen, rng = _gen(V + len(m)), np.random.default_rng(V + fan)
    trees = [random_tree(rng, x, fan) for x in m]
    T, B = sum(m), len(m)
    p, q = _probs(gen, T, V)
    tokens = _drafts(gen, trees, q, V)
    u = torch.rand(T, generator=gen, device="cuda")
    u_next = torch.rand(B, generator=gen, device="cuda")
    q = q if drawn else None
    most = max(m)
    for max_path in {most, 2, 1}:
        got = _verify(kvc, m, tokens, p, u, u_next, max_path, parent=_i32(sum(trees, [])), q=q)
        assert device_status_clean(kvc)
        check_verify(got, trees, tokens, p, q, u, u_next, max_path)
    # chains need no parents
    got = _verify(kvc, m, tokens, p, u, u_next, most, q=q)
    check_verify(got, m, tokens, p, q, u, u_next, most)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("V,po,qo", [(1001, 0, 0), (1001, 1, 1), (999, 2, 3), (4000, 3, 0), (3, 1, 2),
                                     (128, 1, 0)])
def test_verify_rows_of_any_alignment(kvc, V, po, qo):
    """Rows that begin anywhere, p's and q's apart, in wider arrays whose other entries are NaN."""
    gen, rng = _gen(V + po), np.random.default_rng(V)
    m = [6, 1, 9, 20]
    trees = [random_tree(rng, x, 5) for x in m]
    T = sum(m)
    p, q = _probs(gen, T, V)
    tokens = _drafts(gen, trees, q, V)
    wp = torch.full((T, V + 7), float("nan"), device="cuda")
    wq = torch.full((T, V + 5), float("nan"), device="cuda")
    wp[:, po:po + V], wq[:, qo:qo + V] = p, q
    u, u_next = torch.rand(T, generator=gen, device="cuda"), torch.rand(4, generator=gen, device="cuda")
    for vq in (wq[:, qo:qo + V], None):
        got = _verify(kvc, m, tokens, wp[:, po:po + V], u, u_next, 20, parent=_i32(sum(trees, [])), q=vq)
        check_verify(got, trees, tokens, p, None if vq is None else q, u, u_next, 20)
    assert device_status_clean(kvc)


def test_verify_numbers_at_their_ends(kvc):
    """u of 0 accepts every token of positive probability and no other one; u_next of 0 draws the
    first token with a weight, the largest number below 1 the last one."""
    V, m = 300, [2, 2, 1, 1]
    p = torch.zeros(6, V, device="cuda")
    p[:, 40:60] = 1 / 20
    tokens = _i32([0, 45, 0, 39, 0, 0])
    u = torch.zeros(6, device="cuda")
    u_next = torch.tensor([0.0, 1 - 2.0 ** -24, 0.0, 1 - 2.0 ** -24], device="cuda")
    for q in (None, torch.full((6, V), 1 / V, device="cuda")):
        path, count, nxt = _verify(kvc, m, tokens, p, u, u_next, 2, q=q)
        assert count.tolist() == [2, 1, 1, 1]
        assert nxt.tolist() == [40, 59, 40, 59]
    # numbers outside [0, 1) count as its ends, NaN as 0
    _, _, nxt = _verify(kvc, m, tokens, p, u, torch.tensor([-1.0, 1.0, float("nan"), 5.0],
                                                           device="cuda"), 2)
    assert nxt.tolist() == [40, 59, 40, 59]
    assert device_status_clean(kvc)


def test_verify_rows_without_mass(kvc):
    """A row of zeros accepts nothing and draws -1; a draft that covers the target wholly leaves
    the target itself; refused tokens that were all of p, too; a sure token is drawn."""
    V = 64
    p = torch.zeros(8, V, device="cuda")
    p[2:4, 7] = 1.0                      # one sure token, whose draft is a bit larger or another
    p[4:6] = 1 / 64
    p[6:8, 9] = 1.0
    q = torch.zeros(8, V, device="cuda")
    q[0:2] = 1 / 64
    q[2:4, 3] = 1.0
    q[4:6] = 1 / 64 + 2.0 ** -20
    q[6:8, 9] = 1.0
    m, tokens = [2, 2, 2, 2], _i32([0, 5, 0, 3, 0, 30, 0, 9])
    u = torch.full((8,), 1 - 2.0 ** -24, device="cuda")
    u_next = torch.tensor([0.5, 0.5, 0.51, 0.5], device="cuda")
    path, count, nxt = _verify(kvc, m, tokens, p, u, u_next, 4, q=q)
    assert count.tolist() == [1, 1, 1, 2]
    assert nxt.tolist() == [-1, 7, 32, 9]
    path, count, nxt = _verify(kvc, m, tokens, p, u, u_next, 4)
    assert count.tolist() == [1, 1, 1, 2] and nxt.tolist()[:2] == [-1, 7]
    assert path.tolist() == [[0, -1, -1, -1]] * 3 + [[0, 1, -1, -1]]
    check_verify((path, count, nxt), m, tokens, p, None, u, u_next, 4)
    # the only token there is, refused: u of 1 is outside its range
    _, count, nxt = _verify(kvc, [2], _i32([0, 7]), p[2:4], torch.ones(2, device="cuda"), u_next[:1], 4)
    assert count.tolist() == [1] and nxt.tolist() == [7]
    assert device_status_clean(kvc)


def test_verify_siblings_of_the_same_token_and_tokens_outside(kvc):
    gen = _gen(3)
    V, m = 50, [9] * 30
    tree = [-1, 0, 0, 0, 0, 1, 1, 2, 0]
    T = 270
    p, q = _probs(gen, T, V, 1.0, 1.0)
    tokens = torch.randint(0, 3, (T,), generator=gen, device="cuda").int()
    tokens[4::9] = V
    tokens[2::18] = -1
    u, u_next = torch.rand(T, generator=gen, device="cuda"), torch.rand(30, generator=gen, device="cuda")
    for vq in (None, q):
        got = _verify(kvc, m, tokens, p, u, u_next, 9, parent=_i32(tree * 30), q=vq)
        check_verify(got, [tree] * 30, tokens, p, vq, u, u_next, 9)
    assert device_status_clean(kvc)


def test_verify_entries_that_are_no_probabilities(kvc):
    """NaN and negative entries count as 0, such above 1 as 1, in p and in q."""
    gen = _gen(5)
    V, m = 777, [5, 5, 5]
    p, q = _probs(gen, 15, V)
    tokens = _drafts(gen, [[-1, 0, 0, 1, 1]] * 3, q, V)
    for x, k in ((p, 3), (q, 5)):
        x[:, ::k] = float("nan")
        x[:, 1::7 * k] = -0.25
        x[:, 2::11 * k] = float("-inf")
    q[:, 500] = float("inf")
    u, u_next = torch.rand(15, generator=gen, device="cuda"), torch.rand(3, generator=gen, device="cuda")
    for vq in (None, q):
        got = _verify(kvc, m, tokens, p, u, u_next, 5, parent=_i32([-1, 0, 0, 1, 1] * 3), q=vq)
        check_verify(got, [[-1, 0, 0, 1, 1]] * 3, tokens, p, vq, u, u_next, 5)
    # a row far from a distribution: some token of positive weight
    big = torch.zeros(1, 100000, device="cuda")
    big[:, 1::2] = 1e30
    for x in (0.0, 0.3, 1 - 2.0 ** -24):
        _, count, nxt = _verify(kvc, [1], _i32([0]), big, torch.zeros(1, device="cuda"),
                                torch.full((1,), x, device="cuda"), 1)
        assert count.item() == 1 and nxt.item() % 2 == 1 and nxt.item() < 100000
    assert device_status_clean(kvc)


def test_verify_bad_parents_sizes_and_ranges(kvc):
    gen = _gen(6)
    V, T = 100, 300
    p, q = _probs(gen, T, V)
    u, u_next = torch.rand(T, generator=gen, device="cuda"), torch.rand(2, generator=gen, device="cuda")
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda").int()
    # a parent that is not before its node: the node is nobody's child
    tree = [-1, 0, 2, 9, -7, 1]
    got = _verify(kvc, [6], tokens, p, u * 0, u_next[:1], 6, parent=_i32(tree + [0] * 294))
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert got[0].tolist() == [[0, 1, 5, -1, -1, -1]] and got[1].item() == 3
    for cu, good in (([0, 257, 300], 1), ([-1, 5, 10], 1), ([0, 5, 301], 0), ([9, 5, 10], 1)):
        path = torch.full((2, 4), 77, dtype=torch.int32, device="cuda")
        count, nxt = (torch.full((2,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        kvc.kvc_draft_verify(_i32(cu), tokens, p, u, u_next, path, count, nxt)
        assert _status(kvc) == kvc.KVC_DEV_CAPACITY
        bad = 1 - good
        assert count[bad] == 0 and nxt[bad] == -1 and (path[bad] == -1).all()
        w = slice(cu[good], cu[good + 1])
        check_verify((path[good:good + 1], count[good:good + 1], nxt[good:good + 1]),
                     [cu[good + 1] - cu[good]], tokens[w], p[w], None, u[w], u_next[good:], 4)
    assert device_status_clean(kvc)


@pytest.mark.parametrize("drawn", [True, False])
def test_tokens_are_distributed_as_the_target_s(kvc, drawn):
    """The first new token (accepted or drawn) of many sequences over the same rows has the
    target's distribution, whatever the draft."""
    gen = _gen(8)
    V, B, tree = 12, 40000, [-1, 0, 0, 0, 1]
    p1, q1 = _probs(gen, 1, V, 1.0, 1.5)
    p, q = p1.expand(5 * B, V).contiguous(), q1.expand(5 * B, V).contiguous()
    tokens = _drafts(gen, [tree] * B, q, V) if drawn else _i32([0, 3, 1, 7, 3] * B)
    u = torch.rand(5 * B, generator=gen, device="cuda")
    u_next = torch.rand(B, generator=gen, device="cuda")
    path, count, nxt = _verify(kvc, [5] * B, tokens, p, u, u_next, 5, parent=_i32(tree * B),
                               q=q if drawn else None)
    second = path[:, 1].clamp(min=0) + 5 * torch.arange(B, device="cuda")
    first = torch.where(count > 1, tokens[second], nxt)
    # Bernstein: a frequency of n trials is off by 5 sigma + 25 / (3 n) or more with a probability
    # of at most 2 exp(-12.5)
    def close(sample):
        n, want = sample.numel(), p1[0].double()
        got = torch.bincount(sample.long(), minlength=V).double() / n
        assert ((got - want).abs() <= 5 * (want * (1 - want) / n).sqrt() + 25 / (3 * n)).all()

    assert (count > 1).any() and (count == 1).any()
    close(first)
    # the token behind an accepted second node is the target's too
    deep = count == 3
    assert deep.any()
    close(nxt[deep])
    assert device_status_clean(kvc)


def test_verify_is_the_same_whatever_the_batch(kvc):
    """A sequence's path and token do not depend on how many others are in the call."""
    gen, rng = _gen(9), np.random.default_rng(9)
    V, B = 9001, 400
    trees = [random_tree(rng, int(x), 4) for x in rng.integers(1, 7, B)]
    m = [len(t) for t in trees]
    p, q = _probs(gen, sum(m), V)
    tokens, u = _drafts(gen, trees, q, V), torch.rand(sum(m), generator=gen, device="cuda")
    u_next = torch.rand(B, generator=gen, device="cuda")
    path, count, nxt = _verify(kvc, m, tokens, p, u, u_next, 6, parent=_i32(sum(trees, [])), q=q)
    first = np.concatenate([[0], np.cumsum(m)])
    for b in list(range(0, B, 37)) + [B - 1]:
        w = slice(int(first[b]), int(first[b + 1]))
        one = _verify(kvc, m[b:b + 1], tokens[w], p[w], u[w], u_next[b:b + 1], 6,
                      parent=_i32(trees[b]), q=q[w])
        assert torch.equal(one[0][0], path[b]) and one[1][0] == count[b] and one[2][0] == nxt[b]
    assert device_status_clean(kvc)


# ---------------------------------------------------------------- commit

def _random_path(rng, tree):
    path, i = [], int(rng.integers(0, len(tree))) if tree else -1
    while i >= 0:
        path.append(i)
        i = tree[i]
    return path[::-1]


def _unit_rows(cache, X, b, h, n):
    if cache.block_table is None:
        return X[b, h, :n]
    return X[cache.block_table[b, h, :-(-n // 64)].long()].reshape(-1, cache.D)[:n]


@pytest.mark.parametrize("D,Hkv,C,paged,n,m,fan", [
    (128, 1, 64, False, [[1]], [1], 0), (128, 2, 320, True, [[65, 300], [64, 128], [1, 320]], [5, 0, 1], 2),
    (64, 3, 200, False, [[200, 199, 130], [63, 64, 65], [16, 17, 18]], [17, 63, 16], 4),
    (128, 1, 512, True, [[500], [333], [256]], [256, 200, 256], 1),
    (64, 1, 512, True, [[500], [333], [256]], [100, 200, 256], 0),
    (128, 8, 192, True, [[70 + 7 * h for h in range(8)]] * 40, [33] * 40, 8)])
@pytest.mark.parametrize("own_counts", [False, True])
def test_commit(kvc, D, Hkv, C, paged, n, m, fan, own_counts):
    gen, rng = _gen(C + D), np.random.default_rng(C + fan)
    cache, K, V = _cache(kvc, gen, n, C, D, paged)
    paths = [_random_path(rng, random_tree(rng, x, fan)) for x in m]
    most = max(max(map(len, paths)), 2)
    path = _i32([x + [-1] * (most - len(x)) for x in paths])
    count = _i32([len(x) for x in paths])
    seqlen = cache.seqlen.clone()
    out = None
    if own_counts:
        out = kvc.SlotCache(K=cache.K, V=cache.V, pos=cache.pos, n=torch.full_like(cache.n, 77),
                            seqlen=torch.full_like(seqlen, 77), block_table=cache.block_table)
    before_k, before_v = cache.K.clone(), cache.V.clone()
    kvc.kvc_draft_commit(cache, _cu(m), path, count, out=out)
    assert device_status_clean(kvc)
    got = out or cache
    if own_counts:
        assert cache.n.tolist() == n and torch.equal(cache.seqlen, seqlen)
    touched = torch.zeros(before_k.shape[:-1], dtype=torch.bool, device="cuda")
    for b, x in enumerate(paths):
        assert got.seqlen[b] == seqlen[b] - m[b] + len(x)
        for h in range(Hkv):
            base = n[b][h] - m[b]
            assert got.n[b, h] == base + len(x)
            rows = list(range(base)) + [base + i for i in x]
            assert torch.equal(_unit_rows(cache, cache.K, b, h, len(rows)), K[b, h][rows])
            assert torch.equal(_unit_rows(cache, cache.V, b, h, len(rows)), V[b, h][rows])
            for s in range(base, base + len(x)):
                if paged:
                    touched[cache.block_table[b, h, s // 64].long(), s % 64] = True
                else:
                    touched[b, h, s] = True
    same = torch.equal
    assert same(cache.K[~touched].view(torch.int16), before_k[~touched].view(torch.int16))
    assert same(cache.V[~touched].view(torch.int16), before_v[~touched].view(torch.int16))


def test_commit_refused_units_bad_paths_and_pages(kvc):
    gen = _gen(4)
    n = [[100, 90], [80, 70], [60, 50], [128, 3], [64, 65]]
    cache, K, V = _cache(kvc, gen, n, 128, 64, True)
    m = [6, 6, 6, 6, 6]
    seqlen = cache.seqlen.tolist()
    path = _i32([[0, 2, 5], [0, 3, 3], [0, 2, 6], [0, 2, 5], [0, 1, 4]])
    count = _i32([3, 3, 3, 3, 3])
    slot_map = torch.zeros(30, 2, dtype=torch.int32, device="cuda")
    slot_map[0, 1] = -1                       # refused: left as it is
    kvc.kvc_draft_commit(cache, _cu(m), path, count, slot_map=slot_map)
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert cache.n.tolist() == [[97, 90], [80, 70], [60, 50], [125, 3], [61, 62]]
    assert cache.seqlen.tolist() == [seqlen[0] - 3, *seqlen[1:3], seqlen[3] - 3, seqlen[4] - 3]
    for b, h in ((0, 1), (1, 0), (1, 1), (2, 0), (2, 1), (3, 1)):
        assert torch.equal(_unit_rows(cache, cache.K, b, h, n[b][h]), K[b, h, :n[b][h]])
    for b, h, p in ((0, 0, [0, 2, 5]), (3, 0, [0, 2, 5]), (4, 0, [0, 1, 4]), (4, 1, [0, 1, 4])):
        rows = list(range(n[b][h] - 6)) + [n[b][h] - 6 + i for i in p]
        assert torch.equal(_unit_rows(cache, cache.V, b, h, len(rows)), V[b, h][rows])
    # counts and ranges outside; a table entry that is no page
    cache, K, V = _cache(kvc, gen, [[100], [90], [80], [100]], 128, 64, True)
    cu = _i32([0, 6, 12, 11, 17])             # sequence 2 runs backwards
    cache.block_table[3, 0, 1] = -3
    kvc.kvc_draft_commit(cache, cu, _i32([[0, 2], [0, 2], [0, 2], [0, 2]]), _i32([3, -1, 1, 2]))
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert cache.n.view(-1).tolist() == [100, 90, 80, 96]
    for b in range(3):
        assert torch.equal(_unit_rows(cache, cache.K, b, 0, cache.n[b, 0]), K[b, 0, :cache.n[b, 0]])
    kvc.kvc_draft_commit(cache, _i32([0, 6, 12, 13, 18]), _i32([[0]] * 4), _i32([1] * 4),
                         slot_map=torch.zeros(17, 1, dtype=torch.int32, device="cuda"))
    assert _status(kvc) == kvc.KVC_DEV_CAPACITY
    assert cache.n.view(-1).tolist() == [95, 85, 80, 96]       # the last range leaves [0, 17]
    # nothing accepted: all nodes leave
    kvc.kvc_draft_commit(cache, _cu([5, 5, 5, 5]), _i32([[7, 7]] * 4), _i32([0] * 4))
    assert cache.n.view(-1).tolist() == [90, 80, 75, 91]
    assert device_status_clean(kvc)


# ---------------------------------------------------------------- a step of all of them

@pytest.mark.parametrize("Hq,Hkv,D,V", [(8, 2, 128, 500), (6, 6, 64, 33)])
def test_steps_of_speculative_decoding(kvc, Hq, Hkv, D, V):
    """Several steps over a paged cache: plan, append, attention, verification, commit.  After
    every step each unit holds the certain tokens' rows, in order, at their positions, and the
    nodes' attention was over them and their ancestors."""
    gen, rng = _gen(V), np.random.default_rng(V)
    B, C = 5, 192
    cache = kvc.SlotCache.empty_paged(B, Hkv, C, D, B * Hkv * 3)
    pool = kvc.PagePool.empty(cache)
    keys = [torch.zeros(0, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(B)]
    values = [x.clone() for x in keys]

    def append(m):
        cu, T = _cu(m), sum(m)
        k, v = _randn(gen, T, Hkv, D), _randn(gen, T, Hkv, D)
        slots = torch.empty(T, Hkv, dtype=torch.int32, device="cuda")
        kvc.kvc_append_plan(cache, cu, slots, pool, release=True)
        kvc.kvc_append_packed(cache, k, v, slots)
        return cu, k, v, slots

    m = [40, 0, 63, 1, 64]                     # prompts
    cu, k, v, _ = append(m)
    for b in range(B):
        keys[b], values[b] = k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]
    for step in range(6):
        m = rng.integers(0, 14, B).tolist()
        m[step % B] = 14
        trees = [random_tree(rng, x, 4) for x in m]
        T = sum(m)
        parent = _i32(sum(trees, []))
        mask = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
        pos = torch.zeros(T, dtype=torch.int32, device="cuda")
        kvc.kvc_tree_plan(_cu(m), parent, mask, pos=pos, seqlen=cache.seqlen)
        cu, k, v, slots = append(m)
        q = _randn(gen, T, Hq, D)
        o, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device="cuda")
        kvc.kvc_tree_attend(cache, q, cu, mask, o, lse=lse, workspace=_ws(kvc, cache, q))
        p, qd = _probs(gen, T, V)
        tokens = _drafts(gen, trees, qd, V)
        u, u_next = torch.rand(T, generator=gen, device="cuda"), torch.rand(B, generator=gen, device="cuda")
        path, count, nxt = (torch.empty(*s, dtype=torch.int32, device="cuda") for s in ((B, 14), (B,), (B,)))
        kvc.kvc_draft_verify(cu, tokens, p, u, u_next, path, count, nxt, parent=parent, q=qd)
        kvc.kvc_draft_commit(cache, cu, path, count, slot_map=slots)
        assert device_status_clean(kvc)
        check_verify((path, count, nxt), trees, tokens, p, qd, u, u_next, 14)
        g = Hq // Hkv
        for b in range(B):
            w, bits, held = slice(int(cu[b]), int(cu[b + 1])), lineage(trees[b]), keys[b].shape[0]
            assert pos[w].tolist() == [held + bin(x).count("1") - 1 for x in bits]
            kk, vv = torch.cat([keys[b], k[w]]), torch.cat([values[b], v[w]])
            for h in range(Hq if m[b] else 0):
                ref = attend_seen(q[w, h], kk[:, h // g], vv[:, h // g], seen_slots(bits, held + m[b], m[b]))
                check_rows(o[w, h], lse[h, w], ref, f"step {step} b={b} h={h}")
            kept = path[b, :count[b]].long()
            keys[b], values[b] = torch.cat([keys[b], k[w][kept]]), torch.cat([values[b], v[w][kept]])
            n = keys[b].shape[0]
            assert cache.seqlen[b] == n and cache.n[b].tolist() == [n] * Hkv
            for h in range(Hkv):
                assert torch.equal(_unit_rows(cache, cache.K, b, h, n), keys[b][:, h])
                assert torch.equal(_unit_rows(cache, cache.V, b, h, n), values[b][:, h])
                assert cache.pos[b, h, :n].tolist() == list(range(n))


def test_captured_step_follows_the_device(kvc):
    """All four calls in one captured graph, on a stream of its own, replayed after lengths, trees,
    tokens and numbers on the device changed."""
    gen = _gen(12)
    Hq, Hkv, D, V, T, B = 8, 2, 128, 3000, 40, 3
    n0 = [[300, 280], [150, 290], [64, 65]]
    cache, K, V_ = _cache(kvc, gen, n0, 320, D, True)
    n1, s1 = cache.n.clone(), cache.seqlen.clone()
    after = kvc.SlotCache(K=cache.K, V=cache.V, pos=cache.pos, n=torch.zeros_like(n1),
                          seqlen=torch.zeros_like(s1), block_table=cache.block_table)
    cu = _cu([20, 10, 10])
    parent, tokens = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    mask = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    q, o = _randn(gen, T, Hq, D), torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda")
    p, qd = torch.zeros(T, V, device="cuda"), torch.zeros(T, V, device="cuda")
    u, u_next = torch.zeros(T, device="cuda"), torch.zeros(B, device="cuda")
    path, count, nxt = (torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((B, 20), (B,), (B,)))
    ws = _ws(kvc, cache, q)

    def step():
        kvc.kvc_tree_plan(cu, parent, mask)
        kvc.kvc_tree_attend(cache, q, cu, mask, o, workspace=ws)
        kvc.kvc_draft_verify(cu, tokens, p, u, u_next, path, count, nxt, parent=parent, q=qd)
        kvc.kvc_draft_commit(cache, cu, path, count, out=after)

    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    parent.fill_(-1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    kvc.kvc_read_device_status()
    for seed, m in ((1, [20, 10, 10]), (2, [0, 39, 1]), (3, [13, 0, 7])):
        rng = np.random.default_rng(seed)
        trees = [random_tree(rng, x, 3) for x in m]
        cu.copy_(_cu(m))
        parent.copy_(_i32((sum(trees, []) + [-1] * T)[:T]))
        pp, qq = _probs(gen, T, V)
        p.copy_(pp)
        qd.copy_(qq)
        tokens[:sum(m)] = _drafts(gen, trees, qd, V)
        u.copy_(torch.rand(T, generator=gen, device="cuda"))
        u_next.copy_(torch.rand(B, generator=gen, device="cuda"))
        K0, V0 = cache.K.clone(), cache.V.clone()
        units = [[(_unit_rows(cache, K0, b, h, n0[b][h]), _unit_rows(cache, V0, b, h, n0[b][h]))
                  for h in range(Hkv)] for b in range(B)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        t = 0
        for b, tree in enumerate(trees):
            w = slice(t, t + m[b])
            t += m[b]
            for h in range(Hq if m[b] else 0):
                kk, vv = units[b][h // 4]
                check_rows(o[w, h], None, attend_seen(q[w, h], kk, vv, seen_slots(lineage(tree), n0[b][h // 4], m[b])))
        check_verify((path, count, nxt), trees, tokens[:sum(m)], p[:sum(m)], qd[:sum(m)], u, u_next, 20)
        kept = count - _i32(m)
        assert torch.equal(after.n, n1 + kept[:, None]) and torch.equal(after.seqlen, s1 + kept)
        assert torch.equal(cache.n, n1)
    assert device_status_clean(kvc)


def test_two_streams_at_once(kvc):
    gen, rng = _gen(23), np.random.default_rng(23)
    V, B = 20000, 9
    trees = [[random_tree(rng, 12, 5) for _ in range(B)] for _ in range(2)]
    T = 12 * B
    rows = [_probs(gen, T, V) for _ in range(2)]
    tokens = [_drafts(gen, trees[i], rows[i][1], V) for i in range(2)]
    us = [(torch.rand(T, generator=gen, device="cuda"), torch.rand(B, generator=gen, device="cuda"))
          for _ in range(2)]
    parents, cu = [_i32(sum(t, [])) for t in trees], _cu([12] * B)
    outs = [tuple(torch.zeros(*s, dtype=torch.int32, device="cuda") for s in ((B, 12), (B,), (B,)))
            for _ in range(2)]
    masks = [torch.zeros(T, 1, dtype=torch.int64, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            kvc.kvc_tree_plan(cu, parents[i], masks[i], stream=streams[i])
            kvc.kvc_draft_verify(cu, tokens[i], rows[i][0], *us[i], *outs[i], parent=parents[i],
                                 q=rows[i][1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        check_verify(outs[i], trees[i], tokens[i], *rows[i], *us[i], 12)
        assert torch.equal(masks[i].cpu(), mask_words(trees[i], 1))
    assert device_status_clean(kvc)
