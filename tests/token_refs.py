"""Plain 64-bit references and derived tolerances of the prompt and chunk attention, and a
plain statement of the append plan (test infrastructure)."""
import math

import torch

H = 2.0 ** -11          # half a step of binary16, relative
F = 2.0 ** -24          # half a step of binary32, relative


def attend_rows(q, k, v, last, scale=None):
    """float64 attention of rows q [R, D] over keys 0 .. last[r] (none when last < 0).
    Returns o, lse, and each output's bound: the probabilities and the result are rounded to
    binary16 once each (probabilities under 2^-14 to a multiple of 2^-24, off by 2^-25 at
    most), the scores and sums are held in 32 bits."""
    R, D = q.shape
    n = k.shape[0]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    last = last.to(q.device)
    hide = torch.arange(n, device=q.device)[None, :] > last[:, None]
    s = (q @ k.t()) * scale
    size = torch.where(hide, 0.0, (q.abs() @ k.abs().t()) * scale)
    s = s.masked_fill(hide, -math.inf)
    if n == 0:
        o = torch.zeros(R, D, dtype=torch.float64, device=q.device)
        lse = torch.full((R,), -math.inf, dtype=torch.float64, device=q.device)
        return o, lse, torch.zeros_like(o), torch.zeros(R, dtype=torch.float64, device=q.device)
    lse = torch.logsumexp(s, 1)
    w = torch.where(torch.isfinite(lse)[:, None], torch.exp(s - lse[:, None]), 0.0)
    w = torch.where(hide, 0.0, w)
    seen = (~hide).any(0)
    v = torch.where(seen[:, None], v, 0.0)      # rows that nobody attends may hold anything
    o = w @ v
    heavy = w @ v.abs()
    count = (last + 1).clamp(0, n).double()
    # scores: D products summed in 32 bits, the scale folded in; exp2's argument and result
    s_off = (D + 4) * F * size.max(1).values + 2 * F * s.masked_fill(hide, 0.0).abs().max(1).values
    p_off = 2 * (s_off + 2.0 ** -21) + count * F
    tol_o = heavy * (H + p_off[:, None]) + o.abs() * H + \
        count[:, None] * 2.0 ** -25 * v.abs().max().clamp(min=1.0) + 1e-7
    tol_lse = s_off + 2.0 ** -20 + count * F + 4 * F * torch.where(torch.isfinite(lse), lse, 0.0).abs()
    return o, lse, tol_o, tol_lse


def check_rows(o, lse, ref, what=""):
    ro, rl, to, tl = ref
    err = (o.double() - ro).abs()
    assert torch.isfinite(o).all(), f"{what}: not finite"
    assert (err <= to).all(), f"{what}: o off by {(err / to).max():.2f} of its bound"
    if lse is not None:
        empty = torch.isinf(rl)
        assert torch.equal(torch.isneginf(lse), empty), f"{what}: lse of empty rows"
        off = torch.where(empty, 0.0, (lse.double() - rl).abs())
        assert (off <= tl).all(), f"{what}: lse off by {(off / tl.clamp(min=1e-30)).max():.2f}"


def plan_reference(n, seqlen, m, C, T, table, pages, free, count, release):
    """kvc_append_plan stated with Python integers.  table is None for a dense cache."""
    B, Hkv = len(n), len(n[0])
    n2 = [row[:] for row in n]
    seq2 = [s + x for s, x in zip(seqlen, m)]
    table2 = None if table is None else [[r[:] for r in row] for row in table]
    pages2 = None if pages is None else [row[:] for row in pages]
    stack = None if free is None else free[:count]
    back, given, ask = [], {}, 0
    for b in range(B):
        for h in range(Hkv):
            ok = n[b][h] + m[b] <= C
            if ok and table is not None:
                need = -(-(n[b][h] + m[b]) // 64)
                held = pages[b][h]
                grow = max(0, need - held)
                if grow and ask + grow > count:
                    ok = False
                elif grow:
                    for j in range(grow):
                        table2[b][h][held + j] = stack.pop()
                    pages2[b][h] = need
                elif release and held > need:
                    back += table[b][h][need:held]
                    for j in range(need, held):
                        table2[b][h][j] = -1
                    pages2[b][h] = need
                ask += grow
            given[b, h] = ok
            if ok:
                n2[b][h] = n[b][h] + m[b]
    if stack is not None:
        stack += back
    slots = [[-1] * Hkv for _ in range(T)]
    pos = {}
    t = 0
    for b in range(B):
        for i in range(m[b]):
            for h in range(Hkv):
                if given[b, h]:
                    slot = n[b][h] + i
                    pos[b, h, slot] = seqlen[b] + i
                    slots[t][h] = (b * Hkv + h) * C + slot if table is None else \
                        table2[b][h][slot // 64] * 64 + slot % 64
            t += 1
    return dict(n=n2, seqlen=seq2, table=table2, pages=pages2, stack=stack, slots=slots, pos=pos,
                refused=not all(given.values()))
