"""Plain 64-bit references for trees of drafted tokens (test infrastructure)."""
import math

import numpy as np
import torch

from token_refs import F, H


def random_tree(rng, m, fan):
    """Parents of m nodes, each one of the fan + 1 nodes before."""
    return [int(rng.integers(max(0, i - 1 - fan), i)) if i else -1 for i in range(m)]


def lineage(parents):
    """Ancestors of each node, itself included, as bits of a Python integer."""
    bits = []
    for i, x in enumerate(parents):
        bits.append((bits[x] if x >= 0 else 0) | 1 << i)
    return bits


def mask_words(trees, words):
    """[T, words] int64 masks of all sequences' nodes."""
    rows = [[(x >> 64 * w) & (2 ** 64 - 1) for w in range(words)]
            for tree in trees for x in lineage(tree)]
    a = np.array(rows, dtype=np.uint64).reshape(-1, words)
    return torch.from_numpy(a.view(np.int64))


def seen_slots(bits, n, m):
    """[m, n] truth values: node i sees the slots before n - m, and slot n - m + j when bit j <= i
    of bits[i] is set."""
    seen = torch.zeros(m, n, dtype=torch.bool)
    seen[:, :max(0, n - m)] = True
    for i in range(m):
        for j in range(i + 1):
            if bits[i] >> j & 1 and n - m + j >= 0:
                seen[i, n - m + j] = True
    return seen


def attend_seen(q, k, v, seen, scale=None):
    """float64 attention of rows q [R, D] over the keys with seen[r], and each output's bound, as
    token_refs.attend_rows derives it: the probabilities and the result are rounded to binary16
    once each (probabilities under 2^-14 to a multiple of 2^-24), scores and sums are held in 32
    bits."""
    R, D = q.shape
    n = k.shape[0]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    hide = ~seen.to(q.device)
    if n == 0:
        zero = torch.zeros(R, dtype=torch.float64, device=q.device)
        return zero[:, None].expand(R, D), zero - math.inf, zero[:, None].expand(R, D), zero
    some = (~hide).any(0)
    k, v = (torch.where(some[:, None], x, 0.0) for x in (k, v))   # nobody attends: may be anything
    s = (q @ k.t()) * scale
    size = torch.where(hide, 0.0, (q.abs() @ k.abs().t()) * scale)
    s = s.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(s, 1)
    w = torch.where(torch.isfinite(lse)[:, None], torch.exp(s - lse[:, None]), 0.0)
    w = torch.where(hide, 0.0, w)
    o, heavy = w @ v, w @ v.abs()
    count = (~hide).sum(1).double()
    s_off = (D + 4) * F * size.max(1).values + 2 * F * s.masked_fill(hide, 0.0).abs().max(1).values
    p_off = 2 * (s_off + 2.0 ** -21) + count * F
    tol_o = heavy * (H + p_off[:, None]) + o.abs() * H + \
        count[:, None] * 2.0 ** -25 * v.abs().max().clamp(min=1.0) + 1e-7
    tol_lse = s_off + 2.0 ** -20 + count * F + 4 * F * torch.where(torch.isfinite(lse), lse, 0.0).abs()
    return o, lse, tol_o, tol_lse


def _clean(x):
    x = np.asarray(x, dtype=np.float64)
    return np.minimum(np.where(x > 0, x, 0.0), 1.0)


def verify_sequence(parents, tokens, p, q, u, u_next, max_path):
    """kvc_draft_verify of one sequence in Python: the residual is kept as a distribution.
    parents None: a chain.  Returns path and next token."""
    m, V = len(tokens), p.shape[1]
    if m == 0:
        return [], -1
    parents = list(range(-1, m - 1)) if parents is None else parents
    path, cur, going = [0], 0, True
    rest = _clean(p[0])
    while going and len(path) < max_path:
        going = False
        rest, mass = _clean(p[cur]), 1.0      # the residual is rest / mass
        for j in range(cur + 1, m):
            if parents[j] != cur:
                continue
            x = int(tokens[j])
            r = rest[x] / mass if 0 <= x < V and mass > 0 else 0.0
            if q is None:
                going = r > 0 and u[j] < r
                if not going and 0 <= x < V:
                    mass -= rest[x]
                    rest[x] = 0.0
            else:
                draft = _clean(q[cur])
                going = r > 0 and u[j] * draft[x] < r
                if not going:
                    rest = np.maximum((rest / mass if mass > 0 else rest) - draft, 0.0)
                    mass = math.fsum(rest)
            if going:
                cur = j
                path.append(j)
                rest = _clean(p[cur])
                break
    if not rest.sum() > 0:
        rest = _clean(p[cur])
    below = np.cumsum(rest)
    return path, int((below <= u_next * below[-1]).sum()) if below[-1] > 0 else -1


def verify_batch(trees, tokens, p, q, u, u_next, max_path):
    """All sequences; trees: a list of parents per sequence (or of node counts for chains)."""
    paths, counts, nexts, t = [], [], [], 0
    for b, tree in enumerate(trees):
        m = tree if isinstance(tree, int) else len(tree)
        w = slice(t, t + m)
        path, nxt = verify_sequence(None if isinstance(tree, int) else tree, tokens[w], p[w],
                                    None if q is None else q[w], u[w], u_next[b], max_path)
        paths.append(path + [-1] * (max_path - len(path)))
        counts.append(len(path))
        nexts.append(nxt)
        t += m
    return np.array(paths).reshape(len(trees), max_path), np.array(counts), np.array(nexts)
