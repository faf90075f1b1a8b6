"""Cases of the operators that bring tokens into the slot caches and attend them.

Four operators, in the order a serving step uses them:

  plan    block tables, slot map, positions and lengths of a ragged batch of new tokens
  append  the new tokens' K/V rows written to the slots of the slot map
  chunk   attention of a chunk of new tokens per sequence over the slot cache
  prompt  causal attention over whole prompts, packed or padded

run() computes them in plain torch operations, or, where `own` is true, makes the library's
calls.  exact() states them again in 64 bits.  Sizes are those of the library's workloads
(64 query heads over 8 KV heads of 128 channels, 32 heads of 128, 4 heads of 64; caches of
512 to 32768 slots; prompts of 2048) and ragged ones around them.
"""
import math
import random

import torch

own = False

PAGE = 64           # slots per page of the paged layout


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest prompt of the library's workloads: one short sequence, latency
        dict(name="prompt tiny", op="prompt", batch=1, lo=64, hi=64, mix=1, hq=4, hkv=4, d=64,
             padded=False),
        # packed prompts of mixed odd lengths, as continuous batching meets them
        dict(name="prompt packed gqa", op="prompt", batch=8, lo=37, hi=2047, mix=2, hq=64, hkv=8,
             d=128, padded=False),
        # a padded batch of full 2048-token prompts, 32 heads; its lse feeds the score pass
        dict(name="prompt padded mha", op="prompt", batch=4, lo=2048, hi=2048, mix=3, hq=32,
             hkv=32, d=128, padded=True),
        # one long prompt: the largest case
        dict(name="prompt long", op="prompt", batch=1, lo=8192, hi=8192, mix=4, hq=64, hkv=8,
             d=128, padded=False),
        # a few drafted tokens per sequence over 512-slot budgets whose heads were evicted apart
        dict(name="chunk draft evicted", op="chunk", batch=64, new_lo=1, new_hi=8, kv_lo=300,
             kv_hi=576, cap=576, per_head=True, mix=5, hq=64, hkv=8, d=128, paged=True),
        # one sequence's drafted tokens over a long cache: few units, the long axis is split
        dict(name="chunk draft long", op="chunk", batch=1, new_lo=5, new_hi=5, kv_lo=32000,
             kv_hi=32000, cap=32768, per_head=False, mix=6, hq=64, hkv=8, d=128, paged=True),
        # chunks of prompts that are taken in pieces, over what the cache already holds
        dict(name="chunk prefill", op="chunk", batch=4, new_lo=257, new_hi=512, kv_lo=2000,
             kv_hi=8192, cap=8192, per_head=False, mix=7, hq=64, hkv=8, d=128, paged=True),
        # a dense cache of 64-channel heads, odd lengths
        dict(name="chunk dense d64", op="chunk", batch=3, new_lo=1, new_hi=130, kv_lo=131,
             kv_hi=1000, cap=1000, per_head=False, mix=8, hq=12, hkv=4, d=64, paged=False),
        # one token for each sequence of a large decode batch
        dict(name="plan decode", op="plan", batch=512, new_lo=1, new_hi=1, kv_lo=100, kv_hi=2047,
             cap=2112, per_head=False, mix=9, hkv=8, release=False),
        # ragged prompts enter a batch whose other units gave slots back by eviction
        dict(name="plan mixed", op="plan", batch=96, new_lo=0, new_hi=700, kv_lo=0, kv_hi=1300,
             cap=2048, per_head=True, mix=10, hkv=8, release=True),
        # one token per sequence: latency
        dict(name="append decode", op="append", batch=64, new_lo=1, new_hi=1, hkv=8, d=128,
             mix=11),
        # the packed prompts' rows: bandwidth
        dict(name="append prompts", op="append", batch=32, new_lo=200, new_hi=2047, hkv=8, d=128,
             mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "chunk", "chunk", "plan", "append"])
    mix = rng.randrange(1 << 20)
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 8])
    if op == "prompt":
        hi = _log_int(rng, 1, 4096)
        most = max(1, min(32, (64 * 4096 * 4096) // (hq * hi * hi), 16384 // hi))
        return dict(op=op, batch=_log_int(rng, 1, most), lo=max(1, int(hi * rng.uniform(0, 1))),
                    hi=hi, mix=mix, hq=hq, hkv=hkv, d=d, padded=rng.random() < 0.4)
    if op == "chunk":
        new_hi = _log_int(rng, 1, 600)
        cap = _log_int(rng, new_hi + 64, 16384)
        paged = rng.random() < 0.6
        if paged:
            cap = -(-cap // PAGE) * PAGE
        most = max(1, min(64, (1 << 29) // (hq * new_hi * cap), (1 << 18) // cap))
        return dict(op=op, batch=_log_int(rng, 1, most), new_lo=rng.randint(0, new_hi),
                    new_hi=new_hi, kv_lo=rng.randint(0, cap), kv_hi=cap, cap=cap,
                    per_head=rng.random() < 0.4, mix=mix, hq=hq, hkv=hkv, d=d, paged=paged)
    if op == "plan":
        cap = PAGE * _log_int(rng, 2, 64)
        new_hi = _log_int(rng, 1, cap // 2)
        return dict(op=op, batch=_log_int(rng, 1, 512), new_lo=rng.randint(0, new_hi),
                    new_hi=new_hi, kv_lo=0, kv_hi=cap - new_hi, cap=cap,
                    per_head=rng.random() < 0.5, mix=mix, hkv=hkv, release=rng.random() < 0.5)
    new_hi = _log_int(rng, 1, 2047)
    most = max(1, min(256, 40000 // new_hi))
    return dict(op=op, batch=_log_int(rng, 1, most), new_lo=rng.randint(0, new_hi),
                new_hi=new_hi, hkv=hkv, d=d, mix=mix)


# ------------------------------------------------------------------ lengths of a case

def _lens(case):
    """Prompt lengths; one of them is the longest of the range."""
    r = random.Random(case["mix"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    lens[r.randrange(len(lens))] = case["hi"]
    return lens


def _new(case):
    """New tokens of each sequence; at least one sequence has some."""
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


def work(case):
    if case["op"] == "prompt":
        lens = _lens(case)
        t, hq, hkv, d = sum(lens), case["hq"], case["hkv"], case["d"]
        return {"bytes": 2 * t * d * (2 * hq + 2 * hkv) + 4 * t * hq,
                "flops": 4 * d * hq * sum(n * (n + 1) // 2 for n in lens)}
    if case["op"] == "chunk":
        new = _new(case)
        held = _held(case, new)
        t, hq, hkv, d = sum(new), case["hq"], case["hkv"], case["d"]
        seen = sum(m * (n - m) + m * (m + 1) // 2 for m, row in zip(new, held) for n in row)
        slots = sum(n for m, row in zip(new, held) for n in row if m)
        return {"bytes": 4 * t * hq * d + 4 * t * hq + 4 * slots * d,
                "flops": 4 * d * (hq // hkv) * seen}
    if case["op"] == "plan":
        t, units = sum(_new(case)), case["batch"] * case["hkv"]
        grow = sum(-(-(n + m) // PAGE) for m, row in zip(_new(case), _held(case, [0] * case["batch"]))
                   for n in row)
        # tables in and out, counts in and out, slot map and positions out, free pages
        return {"bytes": 4 * (2 * units * (case["cap"] // PAGE) + 4 * units + 2 * t * case["hkv"]
                              + grow), "flops": units}
    t = sum(_new(case))
    return {"bytes": 8 * t * case["hkv"] * case["d"] + 4 * t * case["hkv"], "flops": 0}


# ------------------------------------------------------------------ inputs

def _cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).half()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"prompt": _prepare_prompt, "chunk": _prepare_chunk, "plan": _prepare_plan,
            "append": _prepare_append}[case["op"]](case, g)


def _prepare_prompt(case, g):
    lens, hq, hkv, d = _lens(case), case["hq"], case["hkv"], case["d"]
    b, longest, t = len(lens), max(lens), sum(lens)
    s = dict(op="prompt", longest=longest, hq=hq, hkv=hkv, d=d, padded=case["padded"],
             cu=_cu(lens), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["padded"]:
        s["q"] = _normal((b, hq, longest, d), g)
        s["k"] = _normal((b, hkv, longest, d), g)
        s["v"] = _normal((b, hkv, longest, d), g)
        s["lse"] = torch.zeros(b, hq, longest, device="cuda")
    else:
        # one fused projection's output: q, k and v are its column ranges
        qkv = _normal((t, hq + 2 * hkv, d), g)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["lse"] = torch.zeros(hq, t, device="cuda")
    s["o"] = torch.zeros(s["q"].shape, dtype=torch.float16, device="cuda")
    return s


def _tables(held, pages_per_unit, pool, g):
    """Pages of each unit, taken in order from a shuffled pool; -1 beyond.  Also the shuffle."""
    pages = (held + PAGE - 1) // PAGE
    order = torch.randperm(pool, generator=g, device="cuda").int()
    flat = pages.reshape(-1)
    first = torch.cumsum(flat, 0) - flat
    j = torch.arange(pages_per_unit, device="cuda")
    at = (first[:, None] + j).clamp(max=pool - 1)
    table = torch.where(j < flat[:, None], order[at], -1).int()
    return table.reshape(*held.shape, pages_per_unit), pages.int(), order


def _prepare_chunk(case, g):
    new, hq, hkv, d, cap = _new(case), case["hq"], case["hkv"], case["d"], case["cap"]
    held = torch.tensor(_held(case, new), dtype=torch.int32, device="cuda")
    b, t = len(new), sum(new)
    s = dict(op="chunk", hq=hq, hkv=hkv, d=d, cap=cap, most=max(new), cu=_cu(new), n=held,
             q=_normal((t, hq, d), g), o=torch.zeros(t, hq, d, dtype=torch.float16, device="cuda"),
             lse=torch.zeros(hq, t, device="cuda"),
             seqlen=held.max(1).values.int(),
             pos=torch.arange(cap, dtype=torch.int32, device="cuda").expand(b, hkv, cap).contiguous())
    if case["paged"]:
        pool = int(sum(-(-n // PAGE) for row in _held(case, new) for n in row)) + 5
        s["table"], _, _ = _tables(held, cap // PAGE, pool, g)
        s["k"], s["v"] = _normal((pool, PAGE, d), g), _normal((pool, PAGE, d), g)
    else:
        s["table"] = None
        s["k"], s["v"] = _normal((b, hkv, cap, d), g), _normal((b, hkv, cap, d), g)
    if own:   # the cache handle and the scratch that a serving loop keeps
        import kv_cache_compression_split_gb300 as kvc
        s["cache"] = kvc.SlotCache(K=s["k"], V=s["v"], pos=s["pos"], n=s["n"],
                                   seqlen=s["seqlen"], block_table=s["table"])
        need = kvc.kvc_chunk_workspace_size(s["cache"], s["q"])
        s["ws"] = torch.empty(max(need // 4, 4), device="cuda")
    return s


def _prepare_plan(case, g):
    new, hkv, cap = _new(case), case["hkv"], case["cap"]
    b, t = len(new), sum(new)
    rows = _held(case, [0] * b)
    n = torch.tensor(rows, dtype=torch.int32, device="cuda")
    # with release, some units hold pages beyond their slots, as after an eviction
    spare = torch.randint(0, 9, n.shape, generator=g, device="cuda") if case["release"] else 0
    kept = torch.clamp(n + PAGE * spare, max=cap)
    per = cap // PAGE
    pool = b * hkv * per + 3
    table, pages, order = _tables(kept, per, pool, g)
    used = pages.sum()
    free = torch.where(torch.arange(pool, device="cuda") < pool - used,
                       order[(used + torch.arange(pool, device="cuda")).clamp(max=pool - 1)], -1)
    seqlen = torch.randint(4000, 9000, (b,), generator=g, device="cuda", dtype=torch.int32)
    s = dict(op="plan", hkv=hkv, cap=cap, release=case["release"], pool=pool, cu=_cu(new), tokens=t,
             n=n, seqlen=seqlen, table=table.contiguous(), pages=pages, free=free.int(),
             count=(pool - used).reshape(1).int())
    # the step's own state: written here while attention still reads the last step's
    s["out"] = dict(n=torch.empty_like(n), seqlen=torch.empty_like(seqlen),
                    table=torch.empty_like(table), pages=torch.empty_like(pages),
                    free=torch.full_like(s["free"], -1), count=torch.empty_like(s["count"]),
                    slots=torch.empty(t, hkv, dtype=torch.int32, device="cuda"),
                    pos=torch.full((b, hkv, cap), -1, dtype=torch.int32, device="cuda"))
    if own:   # the handles that a serving loop keeps
        import kv_cache_compression_split_gb300 as kvc
        kv = torch.empty(pool, PAGE, 64, dtype=torch.float16, device="cuda")
        o = s["out"]
        s["cache"] = kvc.SlotCache(K=kv, V=kv, pos=o["pos"], n=n, seqlen=seqlen,
                                   block_table=s["table"])
        s["next"] = kvc.SlotCache(K=kv, V=kv, pos=o["pos"], n=o["n"], seqlen=o["seqlen"],
                                  block_table=o["table"])
        s["pool_in"] = kvc.PagePool(pages=pages, free=s["free"], count=s["count"])
        s["pool_out"] = kvc.PagePool(pages=o["pages"], free=o["free"], count=o["count"])
    return s


def _prepare_append(case, g):
    new, hkv, d = _new(case), case["hkv"], case["d"]
    t = sum(new)
    pool = -(-t * hkv // PAGE) + 9 * hkv
    # the rows of each (sequence, head) follow one another inside a page, pages are shuffled
    seq = torch.searchsorted(_cu(new)[1:], torch.arange(t, device="cuda"), right=True)
    line = torch.argsort((seq[:, None] * hkv + torch.arange(hkv, device="cuda")).reshape(-1),
                         stable=True)
    rank = torch.empty_like(line)
    rank[line] = torch.arange(t * hkv, device="cuda")
    order = torch.randperm(pool, generator=g, device="cuda")
    slots = (order[rank // PAGE] * PAGE + rank % PAGE).reshape(t, hkv).int()
    qkv = _normal((t, 3 * hkv, d), g)
    s = dict(op="append", k_new=qkv[:, hkv:2 * hkv], v_new=qkv[:, 2 * hkv:], slots=slots,
             k=torch.zeros(pool, PAGE, d, dtype=torch.float16, device="cuda"),
             v=torch.zeros(pool, PAGE, d, dtype=torch.float16, device="cuda"))
    if own:   # the cache handle that a serving loop keeps
        import kv_cache_compression_split_gb300 as kvc
        i32 = dict(dtype=torch.int32, device="cuda")
        s["cache"] = kvc.SlotCache(K=s["k"], V=s["v"], pos=torch.zeros(1, hkv, PAGE, **i32),
                                   n=torch.zeros(1, hkv, **i32), seqlen=torch.zeros(1, **i32),
                                   block_table=torch.zeros(1, hkv, 1, **i32))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return {"prompt": _own_prompt, "chunk": _own_chunk, "plan": _own_plan,
                "append": _own_append}[s["op"]](s)
    return {"prompt": _plain_prompt, "chunk": _plain_chunk, "plan": _plain_plan,
            "append": _plain_append}[s["op"]](s)


def _own_prompt(s):
    import kv_cache_compression_split_gb300 as kvc
    if s["padded"]:
        kvc.kvc_prompt_attend(s["q"], s["k"], s["v"], s["o"], lens=s["lens"], lse=s["lse"])
    else:
        kvc.kvc_prompt_attend(s["q"], s["k"], s["v"], s["o"], cu_seqlens=s["cu"], lse=s["lse"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_chunk(s):
    import kv_cache_compression_split_gb300 as kvc
    kvc.kvc_chunk_attend(s["cache"], s["q"], s["cu"], s["o"], lse=s["lse"], workspace=s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _own_plan(s):
    import kv_cache_compression_split_gb300 as kvc
    o = s["out"]
    kvc.kvc_append_plan(s["cache"], s["cu"], o["slots"], pool=s["pool_in"], out=s["next"],
                        pool_out=s["pool_out"], release=s["release"])
    return o


def _own_append(s):
    import kv_cache_compression_split_gb300 as kvc
    kvc.kvc_append_packed(s["cache"], s["k_new"], s["v_new"], s["slots"])
    return {"k": s["k"], "v": s["v"]}


def _softmax_rows(scores, seen, v):
    """Rows of masked scores -> weighted values and log-sum-exp (0 and -inf for an empty row)."""
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o, (top + torch.log(total)).squeeze(-1)


def _grouped(q, hkv):
    """[B, Hq, L, D] -> [B, Hkv, g * L, D]: the query heads of one KV head side by side."""
    b, hq, n, d = q.shape
    return q.reshape(b, hkv, hq // hkv * n, d)


def _plain_prompt(s):
    hq, hkv, d, longest = s["hq"], s["hkv"], s["d"], s["longest"]
    at = torch.arange(longest, device="cuda")
    if s["padded"]:
        q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    else:
        t = s["q"].shape[0]
        rows = (s["cu"][:-1, None] + at).clamp(max=t - 1)
        q, k, v = (s[x].float()[rows].transpose(1, 2) for x in "qkv")
    b = q.shape[0]
    scores = torch.matmul(_grouped(q, hkv), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    seen = (at[:, None] >= at).repeat(hq // hkv, 1)
    o, lse = _softmax_rows(scores, seen, v)
    o, lse = o.reshape(b, hq, longest, d), lse.reshape(b, hq, longest)
    if s["padded"]:
        real = at < s["lens"][:, None]
        s["o"].copy_(torch.where(real[:, None, :, None], o.half(), s["o"]))
        s["lse"].copy_(torch.where(real[:, None, :], lse, s["lse"]))
    else:
        tok = torch.arange(t, device="cuda")
        seq = torch.searchsorted(s["cu"][1:], tok, right=True)
        i = tok - s["cu"][seq]
        s["o"].copy_(o[seq, :, i].half())
        s["lse"].copy_(lse[seq, :, i].t())
    return {"o": s["o"], "lse": s["lse"]}


def _plain_chunk(s):
    hq, hkv, d, cap, most = s["hq"], s["hkv"], s["d"], s["cap"], s["most"]
    t, b = s["q"].shape[0], s["n"].shape[0]
    g = hq // hkv
    slot = torch.arange(cap, device="cuda")
    if s["table"] is None:
        k, v = s["k"].float(), s["v"].float()
    else:
        row = s["table"].long().clamp(min=0)[..., slot // PAGE] * PAGE + slot % PAGE
        k, v = (s[x].reshape(-1, d)[row].float() for x in "kv")
    i = torch.arange(most, device="cuda")
    m = s["cu"][1:] - s["cu"][:-1]
    q = s["q"].float()[(s["cu"][:-1, None] + i).clamp(max=t - 1)].transpose(1, 2)
    scores = torch.matmul(_grouped(q, hkv), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    last = (s["n"] - m[:, None])[..., None] + i          # the last slot each query sees
    seen = (slot <= last[..., None]) & (slot < s["n"][..., None, None])
    seen = seen[:, :, None].expand(b, hkv, g, most, cap).reshape(b, hkv, g * most, cap)
    o, lse = _softmax_rows(scores, seen, v)
    o, lse = o.reshape(b, hq, most, d), lse.reshape(b, hq, most)
    tok = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["cu"][1:], tok, right=True)
    i = tok - s["cu"][seq]
    s["o"].copy_(o[seq, :, i].half())
    s["lse"].copy_(lse[seq, :, i].t())
    return {"o": s["o"], "lse": s["lse"]}


def _plain_plan(s):
    hkv, cap, pool, o = s["hkv"], s["cap"], s["pool"], s["out"]
    b, per = s["n"].shape[0], cap // PAGE
    n, pages, count = s["n"].long(), s["pages"].long(), s["count"].long()
    m = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    fits = n + m <= cap
    need = (n + m + PAGE - 1) // PAGE
    grow = torch.where(fits, (need - pages).clamp(min=0), 0).reshape(-1)
    before = torch.cumsum(grow, 0) - grow
    given = ((grow == 0) | (before + grow <= count)).reshape(b, hkv) & fits
    grow = torch.where(given.reshape(-1), grow, 0)
    back = torch.where(given, (pages - need).clamp(min=0), 0).reshape(-1) if s["release"] \
        else torch.zeros_like(grow)
    left = count - grow.sum()
    # tables: kept, newly given from the top of the stack, given back
    j = torch.arange(per, device="cuda")
    old = s["table"].reshape(-1, per)
    held, want = pages.reshape(-1, 1), need.reshape(-1, 1)
    fresh = (j >= held) & (j < held + grow[:, None])
    gone = (j >= want) & (j < held) & (back[:, None] > 0)
    at = (count - 1 - before[:, None] - (j - held)).clamp(0, pool - 1)
    o["table"].copy_(torch.where(fresh, s["free"][at], torch.where(gone, -1, old))
                     .reshape(b, hkv, per))
    o["pages"].copy_((held[:, 0] + grow - back).reshape(b, hkv))
    # the stack: what is left, then the returned pages in unit order
    i = torch.arange(pool, device="cuda")
    stack = torch.cat([torch.where(i < left, s["free"], o["free"]), s["free"][:1]])
    first = left + torch.cumsum(back, 0) - back
    to = torch.where(gone, first[:, None] + j - want, pool).clamp(max=pool)
    stack[to.reshape(-1)] = old.reshape(-1)
    o["free"].copy_(stack[:pool])
    o["count"].copy_(left + back.sum())
    # slot map, positions and lengths
    tok = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:], tok, right=True)
    step = tok - s["cu"][seq]
    slot = n[seq] + step[:, None]
    ok = given[seq]
    inside = torch.where(ok, slot, 0)
    head = torch.arange(hkv, device="cuda")
    page = o["table"].long()[seq[:, None], head, inside // PAGE]
    o["slots"].copy_(torch.where(ok, page * PAGE + inside % PAGE, -1))
    old_pos = o["pos"][seq[:, None], head, inside]
    o["pos"][seq[:, None], head, inside] = torch.where(
        ok, (s["seqlen"][seq] + step)[:, None].expand(-1, hkv).int(), old_pos)
    o["n"].copy_(torch.where(given, n + m, n))
    o["seqlen"].copy_(s["seqlen"] + m[:, 0])
    return o


def _plain_append(s):
    d = s["k"].shape[-1]
    rows = s["slots"].long()
    s["k"].reshape(-1, d)[rows] = s["k_new"]
    s["v"].reshape(-1, d)[rows] = s["v_new"]
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(case, s)
    if case["op"] == "chunk":
        return _exact_chunk(case, s)
    if case["op"] == "append":
        return _exact_append(s)
    return None      # whole numbers: the plain form is the definition


def _exact_rows(q, k, v, last):
    """Row r of q [R, D] attends keys 0 .. last[r]: float64 outputs and log-sum-exp."""
    x = (q.double() @ k.double().t()) / math.sqrt(q.shape[-1])
    hide = torch.arange(k.shape[0], device=q.device)[None, :] > last[:, None]
    x = x.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - lse[:, None])
    w = torch.where(torch.isfinite(lse)[:, None], w, torch.zeros_like(w))
    return w @ v.double(), lse


def _exact_prompt(case, s):
    g = case["hq"] // case["hkv"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for b, n in enumerate(_lens(case)):
        last = torch.arange(n, device="cuda")
        for h in range(case["hq"]):
            if case["padded"]:
                o[b, h, :n], lse[b, h, :n] = _exact_rows(s["q"][b, h, :n], s["k"][b, h // g, :n],
                                                         s["v"][b, h // g, :n], last)
            else:
                w = slice(start, start + n)
                o[w, h], lse[h, w] = _exact_rows(s["q"][w, h], s["k"][w, h // g],
                                                 s["v"][w, h // g], last)
        start += n
    return {"o": o, "lse": lse}


def _exact_chunk(case, s):
    g, d = case["hq"] // case["hkv"], case["d"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    new, start = _new(case), 0
    held = _held(case, new)
    for b, m in enumerate(new):
        w = slice(start, start + m)
        for hk in range(case["hkv"] if m else 0):
            n = held[b][hk]
            if s["table"] is None:
                k, v = s["k"][b, hk, :n], s["v"][b, hk, :n]
            else:
                pg = s["table"][b, hk, :-(-n // PAGE)].long()
                k, v = (s[x][pg].reshape(-1, d)[:n] for x in "kv")
            q = s["q"][w, hk * g:(hk + 1) * g].transpose(0, 1).reshape(g * m, d)
            last = (n - m + torch.arange(m, device="cuda")).repeat(g)
            ow, lw = _exact_rows(q, k, v, last)
            o[w, hk * g:(hk + 1) * g] = ow.reshape(g, m, d).transpose(0, 1)
            lse[hk * g:(hk + 1) * g, w] = lw.reshape(g, m)
        start += m
    return {"o": o, "lse": lse}


def _exact_append(s):
    out = {}
    for x in "kv":
        flat = s[x].double().reshape(-1, s[x].shape[-1])
        flat[s["slots"].reshape(-1).long()] = s[x + "_new"].double().reshape(-1, flat.shape[-1])
        out[x] = flat.reshape(s[x].shape)
    return out
