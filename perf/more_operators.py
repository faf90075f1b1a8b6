"""Cases of the operators that check trees of drafted tokens over the slot caches.

Four operators, in the order a step of speculative decoding uses them:

  plan    ancestor masks and positions of the drafted nodes, from their parents
  tree    attention of the nodes over the slot cache, each over its own ancestors
  verify  which nodes are accepted, and the token behind them, from the target's
          probabilities and given random numbers
  commit  the slots of the accepted path stay, those of the other nodes are given back

A sequence's nodes are packed like new tokens; node 0 is the last token that is certain, and
a node comes behind its parent.  run() computes the operators in plain torch operations, or,
where `own` is true, makes the library's calls.  exact() states them again in 64 bits.  Heads,
slots and batches are those of the library's workloads (64 query heads over 8 KV heads of 128
channels, 32 heads of 128, 4 heads of 64; caches of 512 to 32768 slots; up to 512 sequences);
trees have up to 128 nodes and vocabularies 1000 to 128000 tokens.
"""
import math
import random

import torch

own = False

PAGE = 64           # slots per page of the paged layout
WORD = 64           # nodes per word of a mask


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a small tree over the shortest cache of the library's workloads: latency
        dict(name="tree tiny", op="tree", batch=1, new_lo=7, new_hi=7, fan=3, kv_lo=96, kv_hi=96,
             cap=96, per_head=False, mix=1, hq=4, hkv=4, d=64, paged=False),
        # trees of a decode batch over 512-slot budgets whose heads were evicted apart
        dict(name="tree evicted", op="tree", batch=64, new_lo=8, new_hi=24, fan=6, kv_lo=300,
             kv_hi=576, cap=576, per_head=True, mix=2, hq=64, hkv=8, d=128, paged=True),
        # one sequence's tree over a long cache: few units, the long axis is split
        dict(name="tree long", op="tree", batch=1, new_lo=60, new_hi=60, fan=12, kv_lo=32000,
             kv_hi=32000, cap=32768, per_head=False, mix=3, hq=64, hkv=8, d=128, paged=True),
        # wide trees, more than one word of nodes, over mixed caches: the largest case
        dict(name="tree wide", op="tree", batch=16, new_lo=33, new_hi=100, fan=20, kv_lo=1000,
             kv_hi=8192, cap=8192, per_head=False, mix=4, hq=32, hkv=32, d=128, paged=True),
        # masks of a few trees: latency
        dict(name="plan few", op="plan", batch=4, new_lo=1, new_hi=9, fan=3, mix=5),
        # masks of a large batch's trees
        dict(name="plan batch", op="plan", batch=512, new_lo=30, new_hi=64, fan=8, mix=6),
        # one sequence's chain of drawn tokens: latency
        dict(name="verify chain", op="verify", batch=1, new_lo=5, new_hi=5, fan=0, vocab=32000,
             drawn=True, mix=7),
        # trees of a draft's most likely tokens
        dict(name="verify likely", op="verify", batch=64, new_lo=8, new_hi=24, fan=6, vocab=32000,
             drawn=False, mix=8),
        # trees whose siblings were drawn: a pass over a row for every sibling but one
        dict(name="verify drawn", op="verify", batch=16, new_lo=20, new_hi=33, fan=10,
             vocab=127999, drawn=True, mix=9),
        # chains of a large batch and a large vocabulary: bandwidth
        dict(name="verify batch", op="verify", batch=512, new_lo=2, new_hi=4, fan=0, vocab=128000,
             drawn=True, mix=10),
        # one sequence's accepted path: latency
        dict(name="commit one", op="commit", batch=1, new_lo=16, new_hi=16, fan=4, kv_lo=500,
             kv_hi=500, cap=576, per_head=False, mix=11, hkv=8, d=128, paged=False),
        # a large batch of trees over evicted caches
        dict(name="commit batch", op="commit", batch=256, new_lo=16, new_hi=64, fan=8, kv_lo=300,
             kv_hi=576, cap=640, per_head=True, mix=12, hkv=8, d=128, paged=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "verify", "verify", "verify", "plan", "commit"])
    mix = rng.randrange(1 << 20)
    new_hi = _log_int(rng, 1, 128)
    case = dict(op=op, mix=mix, new_hi=new_hi, new_lo=rng.randint(0, new_hi),
                fan=_log_int(rng, 1, 1 + new_hi) - 1)
    if op == "plan":
        case["batch"] = _log_int(rng, 1, 512)
        return case
    if op == "verify":
        vocab = _log_int(rng, 1000, 128000)
        most = max(1, min(512, (1 << 27) // (new_hi * vocab)))
        return dict(case, vocab=vocab, batch=_log_int(rng, 1, most), drawn=rng.random() < 0.6)
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    case.update(hkv=hkv, d=rng.choice([64, 128, 128]), paged=rng.random() < 0.6,
                per_head=rng.random() < 0.4)
    cap = _log_int(rng, new_hi + 64, 16384 if op == "tree" else 2048)
    if case["paged"]:
        cap = -(-cap // PAGE) * PAGE
    case.update(cap=cap, kv_lo=rng.randint(0, cap), kv_hi=cap)
    if op == "commit":
        return dict(case, batch=_log_int(rng, 1, max(1, min(256, (1 << 20) // (cap * hkv)))))
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 8])
    most = max(1, min(64, (1 << 28) // (hq * new_hi * cap), (1 << 18) // cap))
    return dict(case, hq=hq, batch=_log_int(rng, 1, most))


# ------------------------------------------------------------------ lengths and trees of a case

def _new(case):
    """Nodes of each sequence; at least one sequence has the most."""
    r = random.Random(case["mix"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    new[r.randrange(len(new))] = case["new_hi"]
    return new


def _held(case, at_least):
    """Slots each unit holds: one count per sequence, or one per head where evictions differ."""
    r = random.Random(case["mix"] + 1)
    out = []
    for need in at_least:
        row = [r.randint(min(max(case["kv_lo"], need), case["kv_hi"]), case["kv_hi"])
               for _ in range(case["hkv"])]
        out.append(row if case["per_head"] else [row[0]] * case["hkv"])
    return out


def _trees(case):
    """Parents of each sequence's nodes: one of the fan + 1 nodes before (a chain for fan 0)."""
    r = random.Random(case["mix"] + 2)
    return [[r.randint(max(0, i - 1 - case["fan"]), i - 1) if i else -1 for i in range(m)]
            for m in _new(case)]


def _paths(case):
    """An accepted path of each sequence: from the root to one of its nodes."""
    r = random.Random(case["mix"] + 3)
    out = []
    for tree in _trees(case):
        path, i = [], r.randrange(len(tree)) if tree else -1
        while i >= 0:
            path.append(i)
            i = tree[i]
        out.append(path[::-1])
    return out


def _lineage(tree):
    """Ancestors of each node, itself included, as bits."""
    bits = []
    for i, parent in enumerate(tree):
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << i)
    return bits


def _words(case):
    return max(1, -(-case["new_hi"] // WORD))


def work(case):
    new, op = _new(case), case["op"]
    t = sum(new)
    if op == "plan":
        return {"bytes": 4 * t + 8 * t * _words(case) + 4 * t, "flops": t}
    if op == "verify":
        # each node's token, parent, number and probabilities; of each sequence the last node's
        # row, and the draft's row where the walk ended at a refusal: two of three, about
        rows = case["batch"] * (5 / 3 if case["drawn"] else 1)
        return {"bytes": 20 * t + 4 * rows * case["vocab"], "flops": 2 * rows * case["vocab"]}
    hkv, d = case["hkv"], case["d"]
    if op == "commit":
        moved = sum(sum(1 for i, x in enumerate(path) if i != x) for path in _paths(case))
        # K and V rows of 2 d bytes: appended (read and written), then moved
        return {"bytes": 8 * d * hkv * (t + moved), "flops": 0}
    held, hq = _held(case, new), case["hq"]
    slots = sum(n for m, row in zip(new, held) for n in row if m)
    seen = 0
    for tree, row in zip(_trees(case), held):
        inside = sum(bin(x).count("1") for x in _lineage(tree))
        seen += sum(len(tree) * (n - len(tree)) + inside for n in row)
    return {"bytes": 4 * t * hq * d + 4 * t * hq + 4 * slots * d + 8 * t * _words(case),
            "flops": 4 * d * (hq // hkv) * seen}


# ------------------------------------------------------------------ inputs

def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return _int(c)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).half()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"plan": _prepare_plan, "tree": _prepare_tree, "verify": _prepare_verify,
            "commit": _prepare_commit}[case["op"]](case, g)


def _parents(case):
    return _int([x for tree in _trees(case) for x in tree])


def _prepare_plan(case, g):
    # the case has the trees' sizes; which of the nodes before is a node's parent is an input
    new = _new(case)
    cu, t = _cu(new), sum(new)
    tok = torch.arange(t, device="cuda")
    i = tok - cu[torch.searchsorted(cu[1:], tok, right=True)]
    back = torch.randint(0, case["fan"] + 1, (t,), generator=g, device="cuda")
    parent = torch.where(i > 0, (i - 1 - back).clamp(min=0), -1).int()
    return dict(op="plan", cu=cu, most=max(new), parent=parent,
                seqlen=torch.randint(0, 9000, (len(new),), generator=g, device="cuda",
                                     dtype=torch.int32),
                mask=torch.zeros(t, _words(case), dtype=torch.int64, device="cuda"),
                pos=torch.zeros(t, dtype=torch.int32, device="cuda"))


def _signed(x):
    return x - (1 << 64) if x >> 63 else x


def _cache_arrays(case, held, g):
    """K and V of a dense or paged cache; the pages of a unit come from a shuffled pool."""
    b, hkv, cap, d = len(held), case["hkv"], case["cap"], case["d"]
    n = _int(held)
    if not case["paged"]:
        return n, None, _normal((b, hkv, cap, d), g), _normal((b, hkv, cap, d), g)
    flat = ((n + PAGE - 1) // PAGE).reshape(-1)
    pool = sum(-(-x // PAGE) for row in held for x in row) + 5
    order = torch.randperm(pool, generator=g, device="cuda").int()
    j = torch.arange(cap // PAGE, device="cuda")
    at = (torch.cumsum(flat, 0) - flat)[:, None] + j
    table = torch.where(j < flat[:, None], order[at.clamp(max=pool - 1)], -1).int()
    return (n, table.reshape(b, hkv, -1).contiguous(), _normal((pool, PAGE, d), g),
            _normal((pool, PAGE, d), g))


def _prepare_tree(case, g):
    new, hq, d, cap = _new(case), case["hq"], case["d"], case["cap"]
    held = _held(case, new)
    t, words = sum(new), _words(case)
    mask = [[_signed(x >> WORD * w & (1 << WORD) - 1) for w in range(words)]
            for tree in _trees(case) for x in _lineage(tree)]
    s = dict(op="tree", hq=hq, hkv=case["hkv"], d=d, cap=cap, most=max(new), cu=_cu(new),
             q=_normal((t, hq, d), g), o=torch.zeros(t, hq, d, dtype=torch.float16, device="cuda"),
             lse=torch.zeros(hq, t, device="cuda"),
             mask=torch.tensor(mask, dtype=torch.int64, device="cuda").reshape(t, words))
    s["n"], s["table"], s["k"], s["v"] = _cache_arrays(case, held, g)
    if own:   # the cache handle and the scratch that a serving loop keeps
        import kv_cache_compression_split_gb300 as kvc
        s["cache"] = kvc.SlotCache(
            K=s["k"], V=s["v"], n=s["n"], seqlen=s["n"].max(1).values.int(), block_table=s["table"],
            pos=torch.zeros(len(new), case["hkv"], cap, dtype=torch.int32, device="cuda"))
        need = kvc.kvc_tree_workspace_size(s["cache"], s["q"])
        s["ws"] = torch.empty(max(need // 4, 4), device="cuda")
    return s


def _prepare_verify(case, g):
    new, vocab, trees = _new(case), case["vocab"], _trees(case)
    t, b = sum(new), len(new)
    rank, above, first = [], [], 0      # a node's place among its siblings, its parent's row
    for tree in trees:
        born = [0] * len(tree)
        for x in tree:
            rank.append(born[x] if x >= 0 else 0)
            above.append(first + max(x, 0))
            if x >= 0:
                born[x] += 1
        first += len(tree)
    rank = torch.tensor(rank, device="cuda")
    above = torch.tensor(above, device="cuda")
    p = torch.empty(t, vocab, device="cuda")
    q = torch.empty(t, vocab, device="cuda") if case["drawn"] else None
    tokens = torch.empty(t, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // vocab)
    likely = []
    for r in range(0, t, step):         # the draft's distribution is near the target's
        x = 2.5 * torch.randn(min(step, t - r), vocab, generator=g, device="cuda")
        p[r:r + step] = torch.softmax(x, 1)
        x += 0.6 * torch.randn(x.shape, generator=g, device="cuda")
        if case["drawn"]:
            q[r:r + step] = torch.softmax(x, 1)
        else:
            likely.append(torch.topk(x, min(vocab, case["new_hi"]), dim=1).indices)
    if case["drawn"]:                   # siblings are drawn from the parent's row
        for r in range(0, t, step):
            race = torch.rand(min(step, t - r), vocab, generator=g, device="cuda")
            race = -torch.log(race.clamp(min=1e-30)) / q[above[r:r + step]].clamp(min=1e-30)
            tokens[r:r + step] = race.argmin(1).int()
    elif t:
        tokens.copy_(torch.cat(likely)[above, rank])
    return dict(op="verify", cu=_cu(new), most=max(new), vocab=vocab, tokens=tokens,
                parent=_parents(case), p=p, q=q,
                u=torch.rand(t, generator=g, device="cuda"),
                u_next=torch.rand(b, generator=g, device="cuda"),
                path=torch.zeros(b, max(new), dtype=torch.int32, device="cuda"),
                count=torch.zeros(b, dtype=torch.int32, device="cuda"),
                next=torch.zeros(b, dtype=torch.int32, device="cuda"))


def _prepare_commit(case, g):
    new, hkv, d, cap = _new(case), case["hkv"], case["d"], case["cap"]
    held, paths = _held(case, new), _paths(case)
    b, t, most = len(new), sum(new), max(new)
    s = dict(op="commit", hkv=hkv, d=d, cap=cap, cu=_cu(new),
             path=_int([x + [-1] * (most - len(x)) for x in paths]),
             count=_int([len(x) for x in paths]),
             n_out=torch.zeros(b, hkv, dtype=torch.int32, device="cuda"),
             seqlen=torch.randint(4000, 9000, (b,), generator=g, device="cuda", dtype=torch.int32),
             seqlen_out=torch.zeros(b, dtype=torch.int32, device="cuda"))
    s["n"], s["table"], s["k"], s["v"] = _cache_arrays(case, held, g)
    # the nodes' rows and where they go: the step writes them, then keeps the accepted ones
    s["k_new"], s["v_new"] = _normal((t, hkv, d), g), _normal((t, hkv, d), g)
    seq, node = _nodes(s["cu"], t)
    s["slots"] = _rows(s, seq[:, None], node[:, None] + s["n"][seq] - _new_of(s)[seq]).int()
    if own:   # the cache handles that a serving loop keeps
        import kv_cache_compression_split_gb300 as kvc
        pos = torch.zeros(b, hkv, cap, dtype=torch.int32, device="cuda")
        s["cache"] = kvc.SlotCache(K=s["k"], V=s["v"], pos=pos, n=s["n"], seqlen=s["seqlen"],
                                   block_table=s["table"])
        s["after"] = kvc.SlotCache(K=s["k"], V=s["v"], pos=pos, n=s["n_out"],
                                   seqlen=s["seqlen_out"], block_table=s["table"])
    return s


def _nodes(cu, t):
    """Sequence and node of each packed token."""
    tok = torch.arange(t, device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return seq, tok - cu[seq]


def _new_of(s):
    return (s["cu"][1:] - s["cu"][:-1])[:, None]


def _rows(s, seq, slot):
    """Rows of the K / V arrays that slots [.., Hkv] of sequences [.., 1] occupy."""
    head = torch.arange(s["hkv"], device="cuda")
    if s["table"] is None:
        return (seq * s["hkv"] + head) * s["cap"] + slot
    return s["table"].long()[seq, head, slot // PAGE] * PAGE + slot % PAGE


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"plan": _own_plan, "tree": _own_tree, "verify": _own_verify,
                "commit": _own_commit}[s["op"]](s)
    return {"plan": _plain_plan, "tree": _plain_tree, "verify": _plain_verify,
            "commit": _plain_commit}[s["op"]](s)


def _own_plan(s):
    import kv_cache_compression_split_gb300 as kvc
    kvc.kvc_tree_plan(s["cu"], s["parent"], s["mask"], pos=s["pos"], seqlen=s["seqlen"])
    return {"mask": s["mask"], "pos": s["pos"]}


def _own_tree(s):
    import kv_cache_compression_split_gb300 as kvc
    kvc.kvc_tree_attend(s["cache"], s["q"], s["cu"], s["mask"], s["o"], lse=s["lse"],
                        workspace=s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_verify(s):
    import kv_cache_compression_split_gb300 as kvc
    kvc.kvc_draft_verify(s["cu"], s["tokens"], s["p"], s["u"], s["u_next"], s["path"], s["count"],
                         s["next"], parent=s["parent"], q=s["q"])
    return {"path": s["path"], "count": s["count"], "next": s["next"]}


def _own_commit(s):
    import kv_cache_compression_split_gb300 as kvc
    kvc.kvc_append_packed(s["cache"], s["k_new"], s["v_new"], s["slots"])
    kvc.kvc_draft_commit(s["cache"], s["cu"], s["path"], s["count"], slot_map=s["slots"],
                         out=s["after"])
    return {"k": s["k"], "v": s["v"], "n": s["n_out"], "seqlen": s["seqlen_out"]}


def _plain_plan(s):
    most, t, words = s["most"], s["mask"].shape[0], s["mask"].shape[1]
    first, m = s["cu"][:-1].long(), _new_of(s)[:, 0]
    b = torch.arange(m.shape[0], device="cuda")
    kin = torch.zeros(m.shape[0], most, WORD * words, dtype=torch.bool, device="cuda")
    depth = torch.zeros(m.shape[0], most, dtype=torch.int64, device="cuda")
    for j in range(most):
        parent = s["parent"].long()[(first + j).clamp(max=t - 1)]
        under = parent >= 0
        up = parent.clamp(min=0, max=most - 1)
        kin[:, j] = kin[b, up] & under[:, None]
        kin[:, j, j] = True
        depth[:, j] = torch.where(under, depth[b, up] + 1, 0)
    seq, node = _nodes(s["cu"], t)
    bit = torch.ones(WORD, dtype=torch.int64, device="cuda") << torch.arange(WORD, device="cuda")
    s["mask"].copy_((kin[seq, node].reshape(t, words, WORD) * bit).sum(2))
    s["pos"].copy_(s["seqlen"][seq] + depth[seq, node])
    return {"mask": s["mask"], "pos": s["pos"]}


def _plain_tree(s):
    hq, hkv, d, cap, most = s["hq"], s["hkv"], s["d"], s["cap"], s["most"]
    t, b, g = s["q"].shape[0], s["n"].shape[0], s["hq"] // s["hkv"]
    slot, i = torch.arange(cap, device="cuda"), torch.arange(most, device="cuda")
    if s["table"] is None:
        k, v = s["k"].float(), s["v"].float()
    else:
        row = s["table"].long().clamp(min=0)[..., slot // PAGE] * PAGE + slot % PAGE
        k, v = (s[x].reshape(-1, d)[row].float() for x in "kv")
    tok = (s["cu"][:-1, None] + i).clamp(max=t - 1)
    q = s["q"].float()[tok].transpose(1, 2).reshape(b, hkv, g * most, d)
    scores = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    # a node sees the slots before the tree, and of the tree those of its mask
    m, n = _new_of(s), s["n"]
    kin = (s["mask"][:, i // WORD] >> i % WORD & 1).bool()[tok]              # [B, node, node]
    kin &= (i <= i[:, None]) & (i < m)[:, None]
    node = slot - (n - m)[..., None]                                         # [B, Hkv, slot]
    inside = kin[:, None].expand(b, hkv, most, most).gather(
        3, node.clamp(0, most - 1)[:, :, None].expand(b, hkv, most, cap))
    seen = (node[:, :, None] < 0) | (inside & (node < m[..., None])[:, :, None])
    seen = seen[:, :, None].expand(b, hkv, g, most, cap).reshape(b, hkv, g * most, cap)
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    w = scores.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).reshape(b, hq, most, d)
    lse = (top + torch.log(total)).reshape(b, hq, most)
    seq, at = _nodes(s["cu"], t)
    s["o"].copy_(o[seq, :, at].half())
    s["lse"].copy_(lse[seq, :, at].t())
    return {"o": s["o"], "lse": s["lse"]}


def _plain_verify(s):
    # 64 bits: a border of the running sum is decided between neighbours of 2^-24
    p, q, tokens, most, vocab = s["p"], s["q"], s["tokens"].long(), s["most"], s["vocab"]
    first, m = s["cu"][:-1].long(), _new_of(s)[:, 0]
    b, t = m.shape[0], tokens.shape[0]
    if t == 0:
        s["path"].fill_(-1)
        s["count"].zero_()
        s["next"].fill_(-1)
        return {"path": s["path"], "count": s["count"], "next": s["next"]}
    each = torch.arange(b, device="cuda")
    first = first.clamp(max=t - 1)
    cur = torch.zeros(b, dtype=torch.int64, device="cuda")
    a = torch.zeros(b, dtype=torch.float64, device="cuda")      # the residual is p - a q
    left = torch.ones_like(a)                                   # its mass
    gone = torch.full((b, most), -1, dtype=torch.int64, device="cuda")   # refused here
    path = torch.full((b, most + 1), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = torch.where(m > 0, 0, -1)
    count = (m > 0).long()
    for j in range(1, most):
        tok, row = (first + j).clamp(max=t - 1), first + cur
        child = (j < m) & (s["parent"][tok] == cur)
        x, u = tokens[tok], s["u"][tok].double()
        w = p[row, x].double()
        if q is not None:
            qx = q[row, x].double()
            rest = (p[row].double() - a[:, None] * q[row].double()).clamp_(min=0).sum(1)
            left = torch.where(a > 0, rest, 1.0)
            w = w - a * qx
            take = child & (w > 0) & (u * qx * left < w)
            a = torch.where(take, 0.0, torch.where(child, a + left, a))
        else:
            w = torch.where((gone == x[:, None]).any(1), 0.0, w)
            take = child & (w > 0) & (u * left < w)
            left = torch.where(take, 1.0, torch.where(child, left - w, left))
            gone[:, j] = torch.where(child, x, -1)
            gone = torch.where(take[:, None], -1, gone)
        cur = torch.where(take, j, cur)
        path.scatter_(1, torch.where(take, count, most)[:, None], torch.full_like(cur, j)[:, None])
        count = count + take
    row = first + cur
    weight = p[row].double()
    if q is not None:
        weight.sub_(a[:, None] * q[row].double()).clamp_(min=0)
    else:
        weight = torch.cat([weight, weight[:, :1]], 1)
        weight[each[:, None], torch.where(gone < 0, vocab, gone)] = 0.0
        weight = weight[:, :vocab]
    weight = torch.where(weight.sum(1, keepdim=True) > 0, weight, p[row].double())
    total = torch.cumsum(weight, 1)
    line = s["u_next"].double() * total[:, -1]
    pick = (total <= line[:, None]).sum(1)
    s["path"].copy_(path[:, :most])
    s["count"].copy_(count)
    s["next"].copy_(torch.where((m > 0) & (total[:, -1] > 0), pick, -1))
    return {"path": s["path"], "count": s["count"], "next": s["next"]}


def _plain_commit(s):
    d, t = s["d"], s["slots"].shape[0]
    k, v = s["k"].view(-1, d), s["v"].view(-1, d)
    rows = s["slots"].long()
    k[rows], v[rows] = s["k_new"], s["v_new"]
    most = s["path"].shape[1]
    i = torch.arange(most, device="cuda")
    kept = i < s["count"][:, None]
    tok = s["cu"][:-1, None].long()
    to = rows[(tok + i).clamp(max=t - 1)]                       # [B, path, Hkv]
    source = rows[(tok + s["path"].clamp(min=0)).clamp(max=t - 1)]
    new_k, new_v = k[source], v[source]
    k[to[kept]], v[to[kept]] = new_k[kept], new_v[kept]
    m = _new_of(s)[:, 0]
    s["n_out"].copy_(s["n"] - (m - s["count"])[:, None])
    s["seqlen_out"].copy_(s["seqlen"] - m + s["count"])
    return {"k": s["k"], "v": s["v"], "n": s["n_out"], "seqlen": s["seqlen_out"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "tree": _exact_tree, "verify": _exact_verify,
            "commit": _exact_commit}[case["op"]](case, s)


def _exact_plan(case, s):
    parent, seqlen = s["parent"].tolist(), s["seqlen"].tolist()
    mask, pos, first = [], [], 0
    for b, m in enumerate(_new(case)):
        bits = _lineage(parent[first:first + m])
        mask += [[_signed(x >> WORD * w & (1 << WORD) - 1) for w in range(_words(case))]
                 for x in bits]
        pos += [seqlen[b] + bin(x).count("1") - 1 for x in bits]
        first += m
    return {"mask": torch.tensor(mask, dtype=torch.int64).reshape(-1, _words(case)),
            "pos": torch.tensor(pos, dtype=torch.int64)}


def _exact_tree(case, s):
    g, d, new, start = case["hq"] // case["hkv"], case["d"], _new(case), 0
    held, trees = _held(case, new), _trees(case)
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, m in enumerate(new):
        w = slice(start, start + m)
        start += m
        kin = torch.tensor([[bits >> j & 1 for j in range(m)] for bits in _lineage(trees[b])],
                           dtype=torch.bool, device="cuda").reshape(m, m)
        for hk in range(case["hkv"] if m else 0):
            n = held[b][hk]
            if s["table"] is None:
                k, v = s["k"][b, hk, :n].double(), s["v"][b, hk, :n].double()
            else:
                pg = s["table"][b, hk, :-(-n // PAGE)].long()
                k, v = (s[x][pg].reshape(-1, d)[:n].double() for x in "kv")
            x = s["q"][w, hk * g:(hk + 1) * g].double() @ k.t() / math.sqrt(d)   # [m, g, n]
            x[:, :, n - m:] = x[:, :, n - m:].masked_fill(~kin[:, None], -math.inf)
            total = torch.logsumexp(x, 2)
            o[w, hk * g:(hk + 1) * g] = torch.exp(x - total[..., None]) @ v
            lse[hk * g:(hk + 1) * g, w] = total.t()
    return {"o": o, "lse": lse}


def _exact_verify(case, s):
    tokens, u, u_next = s["tokens"].tolist(), s["u"].tolist(), s["u_next"].tolist()
    paths, counts, nexts, first = [], [], [], 0
    for b, tree in enumerate(_trees(case)):
        path, token = [], -1
        if tree:
            path, cur, stay = [0], 0, True
            while stay:
                stay = False
                rest = s["p"][first + cur].double()       # the residual, a distribution
                for j in (j for j in range(len(tree)) if tree[j] == cur):
                    x = tokens[first + j]
                    r = float(rest[x])
                    if s["q"] is None:
                        stay = r > 0 and u[first + j] < r
                        if not stay:
                            rest = rest.clone()
                            scale = 1.0 - r
                            rest[x] = 0.0
                            rest = rest / scale if scale > 0 else rest
                    else:
                        draft = s["q"][first + cur].double()
                        stay = r > 0 and u[first + j] * float(draft[x]) < r
                        if not stay:
                            rest = (rest - draft).clamp(min=0)
                            total = float(rest.sum())
                            rest = rest / total if total > 0 else rest
                    if stay:
                        cur = j
                        path.append(j)
                        break
            if float(rest.sum()) <= 0:
                rest = s["p"][first + cur].double()
            below = torch.cumsum(rest, 0)
            if float(below[-1]) > 0:
                token = int((below <= u_next[b] * below[-1]).sum())
        paths.append(path + [-1] * (s["path"].shape[1] - len(path)))
        counts.append(len(path))
        nexts.append(token)
        first += len(tree)
    return {"path": torch.tensor(paths), "count": torch.tensor(counts),
            "next": torch.tensor(nexts)}


def _exact_commit(case, s):
    d = case["d"]
    k, v = s["k"].double().view(-1, d), s["v"].double().view(-1, d)
    slots = s["slots"].long()
    k[slots.reshape(-1)] = s["k_new"].double().reshape(-1, d)
    v[slots.reshape(-1)] = s["v_new"].double().reshape(-1, d)
    n, seqlen, first = s["n"].long().clone(), s["seqlen"].long().clone(), 0
    for b, (m, path) in enumerate(zip(_new(case), _paths(case))):
        if path:
            source = slots[[first + i for i in path]]
            kept = k[source], v[source]
            k[slots[first:first + len(path)]], v[slots[first:first + len(path)]] = kept
        n[b] += len(path) - m
        seqlen[b] += len(path) - m
        first += m
    return {"k": k.reshape(s["k"].shape), "v": v.reshape(s["v"].shape), "n": n, "seqlen": seqlen}
