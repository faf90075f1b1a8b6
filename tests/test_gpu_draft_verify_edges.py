"""Verification of drafted tokens where several CTAs share a sequence's row: rows of p and q that
begin at different places of a 16-byte vector, residuals of which nothing is left, refused tokens
that were all of p, and draws at the border between two tokens, in batches of 1 to 200."""
import numpy as np
import pytest
import torch

from draft_refs import random_tree
from helpers import device_status_clean
from test_gpu_draft import _cu, _drafts, _gen, _i32, _probs, _verify, check_verify

pytestmark = pytest.mark.gpu

BELOW_ONE = 1 - 2.0 ** -24


@pytest.fixture(scope="module")
def kvc():
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


@pytest.mark.parametrize("V", [32000, 50001, 128000])
@pytest.mark.parametrize("B,nodes", [(1, 14), (16, 7), (130, 4)])
def test_rows_of_different_alignment_in_long_vocabularies(kvc, V, B, nodes):
    """Rows begin anywhere, p's and q's apart, in wider arrays whose other entries are NaN; numbers
    near 1 refuse many siblings, so that walks end at residuals and take several passes."""
    gen, rng = _gen(V + B), np.random.default_rng(V + B)
    trees = [random_tree(rng, int(rng.integers(2, nodes + 1)), 4) for _ in range(B)]
    m = [len(t) for t in trees]
    T, parent = sum(m), _i32(sum(trees, []))
    p, q = _probs(gen, T, V)
    tokens = _drafts(gen, trees, q, V)
    u = torch.rand(T, generator=gen, device="cuda") ** 0.25
    u = torch.where(u < 1, u, BELOW_ONE)
    u_next = torch.rand(B, generator=gen, device="cuda")
    for po, qo, width in ((0, 1, 0), (3, 1, 0), (2, 0, 1), (1, 1, 0)):
        wp = torch.full((T, V + 8 - V % 4 + width), float("nan"), device="cuda")
        wq = torch.full((T, V + 8 - V % 4), float("nan"), device="cuda")
        wp[:, po:po + V], wq[:, qo:qo + V] = p, q
        got = _verify(kvc, m, tokens, wp[:, po:po + V], u, u_next, nodes, parent=parent,
                      q=wq[:, qo:qo + V])
        assert device_status_clean(kvc)
        check_verify(got, trees, tokens, p, q, u, u_next, nodes)
    best = p[[t + max(x, 0) for t, tree in zip(np.cumsum([0] + m), trees) for x in tree]].argmax(1).int()
    given = torch.where(torch.arange(T, device="cuda") % 2 == 0, best, tokens)
    got = _verify(kvc, m, given, wp[:, 1:1 + V], u, u_next, nodes, parent=parent)
    assert device_status_clean(kvc)
    check_verify(got, trees, given, p, None, u, u_next, nodes)


@pytest.mark.parametrize("V", [32000, 50001, 128000])
@pytest.mark.parametrize("B", [1, 16, 130])
def test_nothing_left_of_a_row_in_long_vocabularies(kvc, V, B):
    """A draft that lies above the target within rounding everywhere, and refused tokens that were
    all of p: the next token is drawn from p itself, by a pass over the row of its own."""
    gen = _gen(V + B)
    T = 3 * B
    tree = [-1, 0, 0]
    p, _ = _probs(gen, T, V)
    q = p * (1 + 2.0 ** -18)
    tokens = _drafts(gen, [tree] * B, p, V)
    u = torch.full((T,), BELOW_ONE, device="cuda")
    u_next = torch.rand(B, generator=gen, device="cuda")
    got = _verify(kvc, [3] * B, tokens, p, u, u_next, 3, parent=_i32(tree * B), q=q)
    assert device_status_clean(kvc)
    assert got[1].eq(1).all()
    check_verify(got, [tree] * B, tokens, p, q, u, u_next, 3)
    # the row's only tokens, each refused by a number of 1
    at = torch.randint(0, V // 3, (T, 3), generator=gen, device="cuda") + \
        torch.arange(3, device="cuda") * (V // 3)
    p = torch.zeros(T, V, device="cuda").scatter_(1, at, torch.tensor(
        [[0.5, 0.25, 0.25]], device="cuda").expand(T, 3))
    four = [-1, 0, 0, 0]
    tokens = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    tokens[:, 1:] = at[0::3].int()
    tokens = tokens.view(-1)
    p4 = p.view(B, 3, V)[:, [0, 1, 2, 2]].reshape(4 * B, V)
    u = torch.ones(4 * B, device="cuda")
    got = _verify(kvc, [4] * B, tokens, p4, u, u_next, 4, parent=_i32(four * B))
    assert device_status_clean(kvc)
    assert got[1].eq(1).all()
    check_verify(got, [four] * B, tokens, p4, None, u, u_next, 4)


def _draw(kvc, p, u_next):
    """Tokens drawn from the rows of p by sequences of one node."""
    B = p.shape[0]
    zero = torch.zeros(B, device="cuda")
    _, count, nxt = _verify(kvc, [1] * B, _i32([0] * B), p, zero, u_next, 1)
    assert count.eq(1).all() and device_status_clean(kvc)
    return nxt.tolist()


@pytest.mark.parametrize("V", [1000, 32000, 128000])
@pytest.mark.parametrize("B", [1, 16, 200])
def test_draws_at_borders_that_sums_hold_exactly(kvc, V, B):
    """Entries are multiples of 2^-24 and sum to 1, so every running sum is exact: a number that is
    one draws the token behind it, 2^-24 less the token that ends there."""
    rng = np.random.default_rng(V)
    rows, us, want = [], [], []
    for i in range(8):
        c = rng.multinomial(2 ** 24, rng.dirichlet(np.full(V, 0.2)))
        cum = np.cumsum(c)
        k = int(rng.choice(np.flatnonzero((c > 0) & (cum < 2 ** 24))))
        for line in (int(cum[k]), int(cum[k]) - 1):
            rows.append(c)
            us.append(line)
            want.append(int(np.searchsorted(cum, line, side="right")))
    assert want[0] > want[1]
    p = torch.from_numpy(np.stack(rows)).cuda().double().mul(2.0 ** -24).float()
    u = torch.tensor(us, dtype=torch.float64, device="cuda").mul(2.0 ** -24).float()
    if B == 1:
        assert [_draw(kvc, p[i:i + 1], u[i:i + 1])[0] for i in range(16)] == want
    else:
        which = torch.arange(B, device="cuda") % 16
        assert _draw(kvc, p[which].contiguous(), u[which]) == [want[i % 16] for i in range(B)]


def _row_with_border(rng, V, off):
    """A row of fp32 probabilities and an fp32 number u such that the sum up to some token k is off
    (in units of 2^-80) above u times the row's sum, in exact arithmetic.  Returns the row, u and
    the token that is drawn."""
    x = rng.standard_normal(V) * 2.5
    e = np.exp(x - x.max())
    e[:2] = 0
    row = (e / e.sum()).astype(np.float32)
    row[row < 2.0 ** -50] = 0
    exact = lambda r: np.array([int(v) for v in np.ldexp(r.astype(np.float64), 80)], dtype=object)  # noqa: E731
    cum0 = np.cumsum(exact(row))
    total0 = int(cum0[-1])
    while True:                                              # a number just above a token's sum
        k = int(rng.integers(V // 20, V - V // 20))
        u = np.nextafter(np.float32(int(cum0[k]) / total0), np.float32(1))
        num = int(np.ldexp(np.float64(u), 40))               # u = num / 2^40
        assert num / 2 ** 40 == float(u)
        gap = (num * total0 >> 40) - int(cum0[k]) + off
        if gap > 0 and min(row[k], row[k + 1]) > 1e-6 and float(u) < 0.95:
            break
    # two entries in front, the second the rounding of the first: their sum moves the border
    delta = (gap << 40) // (2 ** 40 - num)
    row[0] = np.float32(delta / 2 ** 80)
    rest = delta - int(np.ldexp(np.float64(row[0]), 80))
    if rest < 0:
        row[0] = np.nextafter(row[0], np.float32(0))
        rest = delta - int(np.ldexp(np.float64(row[0]), 80))
    row[1] = np.float32(rest / 2 ** 80)
    cum = np.cumsum(exact(row))
    line = num * int(cum[-1])                                # of 2^-120
    assert abs(int(cum[-1]) - 2 ** 80) < 2 ** 61             # still a distribution within rounding
    margin = (int(cum[k]) << 40) - line
    assert abs(margin - (off << 40)) < abs(off << 40) // 8
    want = next(i for i in range(k - 1, k + 2) if (int(cum[i]) << 40) > line)
    return row, u, want


@pytest.mark.parametrize("V", [9001, 32000, 128000])
def test_draws_near_a_border_do_not_depend_on_the_batch(kvc, V):
    """Numbers V 2^-50 beside a border, the distance from which on the token is the one of exact
    arithmetic: each batch, whose CTAs divide a row in their own way, draws that token."""
    rng = np.random.default_rng(V)
    off = V << 30                                            # V 2^-50, of 2^-80
    made = [_row_with_border(rng, V, off * s) for s in (1, -1) * 8]
    p = torch.from_numpy(np.stack([r for r, _, _ in made])).cuda()
    u = torch.from_numpy(np.array([x for _, x, _ in made], dtype=np.float32)).cuda()
    want = [w for _, _, w in made]
    assert [_draw(kvc, p[i:i + 1], u[i:i + 1])[0] for i in range(16)] == want
    for B in (16, 64, 200, 520):
        which = torch.arange(B, device="cuda") % 16
        assert _draw(kvc, p[which].contiguous(), u[which]) == [want[i % 16] for i in range(B)]


def test_the_largest_vocabulary(kvc):
    """2^24 tokens: trees with siblings, drawn and given, and the first and last tokens of a row."""
    gen, V, tree = _gen(24), 1 << 24, [-1, 0, 0]
    assert V == kvc.DRAFT_MAX_VOCAB
    p, q = _probs(gen, 3, V)
    tokens = _drafts(gen, [tree], q, V)
    for seed in range(4):
        u = torch.rand(3, generator=gen, device="cuda") ** 0.25
        u_next = torch.rand(1, generator=gen, device="cuda")
        for vq in (q, None):
            got = _verify(kvc, [3], tokens, p, u, u_next, 3, parent=_i32(tree), q=vq)
            assert device_status_clean(kvc)
            check_verify(got, [tree], tokens, p, vq, u, u_next, 3)
    p = torch.zeros(2, V, device="cuda")
    p[:, 0] = p[:, -1] = 0.5
    tokens = _i32([0, V - 1])
    for x, u_next, want in ((0.9, 0.25, [1, 0]), (0.9, 0.75, [1, V - 1]), (0.1, 0.75, [2, V - 1])):
        _, count, nxt = _verify(kvc, [2], tokens, p, torch.full((2,), x, device="cuda"),
                                torch.full((1,), u_next, device="cuda"), 2)
        # a refused last token leaves the first one alone
        assert count.item() == want[0] and nxt.item() == (0 if x == 0.9 else want[1])
    assert device_status_clean(kvc)
