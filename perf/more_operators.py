"""What a speculative serving step costs over the paged cache: attention of a chunk of new tokens of every cursor (a prompt's
next part, or drafted tokens to be checked), the same with a sliding window and first tokens that stay visible, and the
verification of drafted tokens against the target's logits.  Each in a plain form of elementary torch operations and as the
calls that a user of the framework makes."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ----
# Attention: `roots` prompts of `prefix` tokens, each forked into `branches` of `length` tokens; with `mount`, a branch then
# reads that many of its next sibling's tokens; `new` tokens follow in every branch, and they are the rows.  ragged: lengths
# and new tokens differ from branch to branch, some branches have no row.  window 0: the whole context.
# Verification: `cursors` sequences of `new` rows, the token agreed on last and new - 1 drafted ones behind it.

def _attn(name, roots, branches, prefix, length, new, **more):
    case = {"name": name, "op": "attn", "roots": roots, "branches": branches, "prefix": prefix, "length": length, "new": new, "mount": 0,
            "ragged": 0, "page": 64, "kv_heads": 4, "group": 4, "head_dim": 128, "dtype": "bf16", "window": 0, "sink": 0}
    return {**case, **more}


def _verify(name, cursors, new, vocab, **more):
    case = {"name": name, "op": "verify", "cursors": cursors, "new": new, "ragged": 0, "vocab": vocab, "dtype": "bf16", "draft": 1, "greedy": 0,
            "inv_temp": 1.0, "masked": 0}
    return {**case, **more}


def listed():
    return [
        # one request's four drafted tokens over a short context: latency alone
        _attn("chunk_1_cursor", 1, 1, 1200, 300, 5),
        # the check of four drafted tokens for 64 agents of eight episodes, siblings' spans mounted, lengths differ
        _attn("chunk_drafts_64_cursors", 8, 8, 8192, 6000, 5, mount=512, ragged=1),
        # one agent with a very long context, eight tokens
        _attn("chunk_long_context", 1, 1, 120000, 11000, 8),
        # prompts' next parts behind a shared prefix of 16,384 tokens: arithmetic alone
        _attn("chunk_prefill", 1, 4, 16384, 64, 2048),
        # fp32 pool, small pages and heads, three query heads a kv head, odd and empty chunks, mounts
        _attn("chunk_odd_f32", 2, 3, 777, 451, 37, mount=129, ragged=1, page=16, kv_heads=2, group=3, head_dim=64, dtype="f32"),
        # a step of single tokens that see their last 1,024 positions and four sinks
        _attn("window_single_96_cursors", 8, 12, 4096, 4096, 1, window=1024, sink=4),
        # two prompts' parts of 4,096 tokens under a window of 2,048
        _attn("window_prefill", 1, 2, 4096, 100, 4096, window=2048, sink=16),
        # small heads and pages, eight query heads a kv head, a window that ends inside pages, mounts, odd and empty chunks
        _attn("window_odd_d64", 2, 4, 1000, 333, 70, mount=150, ragged=1, page=32, kv_heads=2, group=8, head_dim=64, window=301, sink=5),
        # one request's four drafted tokens: latency alone
        _verify("verify_1_cursor", 1, 5, 151936),
        # a serving step of 256 cursors with four drafted tokens each
        _verify("verify_256_cursors", 256, 5, 151936),
        # greedy decoding, drafts of a look-up (no draft logits), lengths differ
        _verify("verify_greedy_ragged", 61, 9, 151936, ragged=1, draft=0, greedy=1),
        # fp32 logits with most tokens masked, odd sizes, a temperature
        _verify("verify_odd_f32", 37, 4, 50001, ragged=1, dtype="f32", inv_temp=1.25, masked=1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.35:
        vocab = _log(rng, 256, 160000)
        new = _log(rng, 1, 16)
        greedy = rng.choice([0, 0, 1])
        case = {"cursors": _log(rng, 1, max(2, min(400, 190000000 // (vocab * new)))), "new": new, "ragged": rng.choice([0, 1]), "vocab": vocab,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "greedy": greedy, "draft": 0 if greedy else rng.choice([0, 1, 1]),
                "inv_temp": rng.choice([1.0, round(rng.uniform(0.4, 2.0), 3)]), "masked": rng.choice([0, 0, 1])}
        case = _verify(None, **case)
        del case["name"]
        return case
    f32 = rng.random() < 0.2
    group, kv, d = rng.choice([1, 2, 3, 4, 4, 4, 5, 8]), rng.choice([1, 2, 4, 4, 8]), rng.choice([64, 128, 128])
    single = rng.random() < 0.25
    new = 1 if single else _log(rng, 2, 300 if f32 else 2500)
    roots, branches = rng.randint(1, 6), rng.randint(1, 8)
    # pairs of a row and a key that a query head may cost, and tokens that the pool may hold
    pairs = (1 << 27 if f32 else 1 << 30) // (group * kv)
    tokens = 1 << 19
    ctx = max(8, min(pairs // (roots * branches * new), tokens // (roots * branches), 16000 if f32 else 100000))
    ctx = _log(rng, min(ctx, 64), ctx)
    prefix = max(1, int(ctx * rng.uniform(0.1, 0.9)))
    length = max(1, ctx - prefix)
    window = _log(rng, 1, 6000) if rng.random() < 0.45 else 0
    case = _attn(None, roots, branches, prefix, length, new, mount=rng.choice([0, 0, rng.randint(1, length)]), ragged=rng.choice([0, 1]),
                 page=rng.choice([64, 64, 64, 16, 32, 128]), kv_heads=kv, group=group, head_dim=d, dtype="f32" if f32 else "bf16", window=window,
                 sink=rng.choice([0, rng.randint(1, 80)]) if window else 0)
    del case["name"]
    return case


# ---- the episodes of the attention cases ----

def _lengths(case):
    """(tokens before the rows, rows) of every branch, in cursor order."""
    out = []
    for c in range(case["roots"] * case["branches"]):
        n, new = case["length"], case["new"]
        if case["ragged"]:
            n -= (c * 37) % (n // 2 + 1)
            new = 0 if c % 5 == 4 else 1 + (c * 7 + new - 1) % new
        out.append((n, new))
    return out


def _appends(case):
    """The tokens appended to each segment, in order: (segment, tokens), segment 0 .. roots - 1 the prompts."""
    R, B = case["roots"], case["branches"]
    lens = _lengths(case)
    ops = [(r, case["prefix"]) for r in range(R)]
    part = 16 * case["page"]                       # branches grow side by side: their pages alternate in the pool
    for at in range(0, case["length"], part):
        ops += [(R + c, min(part, n - at)) for c, (n, _) in enumerate(lens) if n > at]
    return ops, [(R + c, new) for c, (_, new) in enumerate(lens) if new]


def _mounted(case, c):
    """The span of the next sibling that cursor c reads: (cursor, first token, end), or None."""
    B = case["branches"]
    if not case["mount"] or B < 2:
        return None
    sib = c - c % B + (c % B + 1) % B
    n = _lengths(case)[sib][0]
    b = min(n, case["mount"] + 11)
    return sib, max(0, b - case["mount"]), b


def _pages(case):
    """The pool's pages of each segment, taken in the order of the appends, and how many there are."""
    P = case["page"]
    pages, lens, used = {}, {}, 0
    first, then = _appends(case)
    for s, n in first + then:
        lens[s] = lens.get(s, 0) + n
        own_pages = pages.setdefault(s, [])
        need = -(-lens[s] // P) - len(own_pages)
        own_pages += range(used, used + need)
        used += need
    return pages, used


def _context(case):
    """Every cursor's context, as arrays [cursors][most tokens]: slot in the pool (page * page_size + slot, 0 behind the end), position,
    and the row from which on it is seen (behind the end: never); then each cursor's rows [cursors][most rows] (-1: none) and their
    positions."""
    R, B, P, f = case["roots"], case["branches"], case["page"], case["prefix"]
    pages, _ = _pages(case)
    slots = {s: (np.repeat(np.array(p, dtype=np.int64), P) * P + np.tile(np.arange(P), len(p))) if p else np.zeros(0, np.int64) for s, p in pages.items()}
    lens = _lengths(case)
    ctx, rows, at = [], [], 0
    for c, (n, new) in enumerate(lens):
        root = c // B
        slot, pos, seen = [slots[root][:f]], [np.arange(f)], [np.full(f, -1)]
        jump, m = 0, _mounted(case, c)
        if m:
            sib, a, b = m
            slot.append(slots[R + sib][a:b])
            pos.append(f + np.arange(a, b))
            seen.append(np.full(b - a, -1))
            jump = max(0, f + b + 1 - (f + n))         # positions go on after the mounted span's last
        mine = np.arange(n + new)
        slot.append(slots[R + c][:n + new])
        pos.append(f + mine + np.where(mine >= n, jump, 0))
        seen.append(mine - n)
        ctx.append([np.concatenate(x) for x in (slot, pos, seen)])
        rows.append((at, new, f + n + jump))
        at += new
    L, T = max(len(x[0]) for x in ctx), max(1, max(n for _, n, _ in rows))
    out = [np.full((len(ctx), L), v, dtype=np.int64) for v in (0, 0, 1 << 40)]
    for c, x in enumerate(ctx):
        for o, v in zip(out, x):
            o[c, :len(v)] = v
    t = np.arange(T)[None, :]
    first, count, p0 = (np.array(x)[:, None] for x in zip(*rows))
    return out + [np.where(t < count, first + t, -1), p0 + t]


def _pairs(case):
    """(rows, visible pairs of a row and a key, tokens that some row sees, counted once)."""
    f, W, S = case["prefix"], case["window"], case["sink"]
    rows = pairs = 0
    slots, spos, seen, row, rpos = _context(case)
    used = np.zeros(_pages(case)[1] * case["page"], dtype=bool)
    for c in range(len(slots)):
        new = int((row[c] >= 0).sum())
        rows += new
        if not new:
            continue
        live = seen[c] < (1 << 40)
        far = seen[c] < 0
        if W:
            keep = live & ((spos[c] > rpos[c, 0] - W) | (spos[c] < S))
            used[slots[c][keep]] = True
            p = np.sort(spos[c][far])
            inside = len(p) - np.searchsorted(p, rpos[c, :new] - W, side="right")
            sinks = np.searchsorted(p, np.minimum(S, rpos[c, :new] - W + 1), side="left")
            pairs += int(inside.sum() + np.maximum(sinks, 0).sum()) + sum(min(t + 1, W) for t in range(new))
        else:
            used[slots[c][live]] = True
            pairs += int(far.sum()) * new + new * (new + 1) // 2
    return rows, pairs, int(used.sum())


def _rows_of(case):
    """Rows of each cursor of a verification."""
    n = case["new"]
    return [0 if c % 7 == 5 else 1 + (c * 5 + n - 1) % n for c in range(case["cursors"])] if case["ragged"] else [n] * case["cursors"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "verify":
        rows = _rows_of(case)
        n, V = sum(rows), case["vocab"]
        drafts, live = sum(max(0, r - 1) for r in rows), sum(r > 0 for r in rows)
        read = n * V * es + (drafts * V * es if case["draft"] else 0) + (0 if case["greedy"] else live * V * 4)
        return {"bytes": read + 4 * n * (2 if case["greedy"] else 3) + 12 * case["cursors"], "flops": 4 * (n + drafts * case["draft"]) * V}
    rows, pairs, tokens = _pairs(case)
    heads, d = case["kv_heads"] * case["group"], case["head_dim"]
    return {"bytes": tokens * case["kv_heads"] * d * 2 * es + rows * heads * (2 * d * es + 4), "flops": 4 * d * heads * pairs}


# ---- inputs ----

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _prepare_verify(case, g) if case["op"] == "verify" else _prepare_attn(case, g)


def _prepare_attn(case, g):
    dt = DTYPES[case["dtype"]]
    kv, d, P = case["kv_heads"], case["head_dim"], case["page"]
    heads = kv * case["group"]
    pages = _pages(case)[1]
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(dt)
    index = _context(case)
    n = int((index[3] >= 0).sum())
    s = {"case": case, "k": randn(pages, kv, P, d), "v": randn(pages, kv, P, d), "q": randn(n, heads, d) * 2, "scale": 1 / math.sqrt(d), "n": n}
    s["o"] = torch.zeros((n, heads, d), dtype=dt, device="cuda")
    s["lse"] = torch.zeros((n, heads), dtype=torch.float32, device="cuda")
    if own:
        s["plan"], s["ws"] = _chunk_plan(case)
    else:
        s["index"] = [torch.from_numpy(x).cuda() for x in index]
    return s


def _chunk_plan(case):
    import packed_tree_attention_gb300 as pta
    R, B, P = case["roots"], case["branches"], case["page"]
    pool = pta.Pool(_pages(case)[1], P, case["kv_heads"], case["head_dim"], pta.DTYPE_BF16 if case["dtype"] == "bf16" else pta.DTYPE_F32)
    first, then = _appends(case)
    cur = [pool.root() for _ in range(R)]
    for s, n in first:
        if s == R and len(cur) == R:
            for r in range(R):
                cur += pool.fork(cur[r], B)
        pool.append(cur[s], n)
    mounts = [(c, _mounted(case, c)) for c in range(R * B)]
    for c, m in mounts:
        if m:
            pool.mount(cur[R + c], cur[R + m[0]], m[1], m[2])
    for s, n in then:
        pool.append(cur[s], n)
    plan = pool.chunk_plan(cur[R:], [n for _, n in _lengths(case)], case["kv_heads"] * case["group"], window=case["window"], n_sink=case["sink"])
    return plan, torch.empty(max(256, plan.chunk_attn_workspace_size()), dtype=torch.uint8, device="cuda")


def _prepare_verify(case, g):
    dt = DTYPES[case["dtype"]]
    V, c = case["vocab"], case["inv_temp"]
    rows = _rows_of(case)
    n, cursors = sum(rows), case["cursors"]
    ld = -(-V // 8) * 8                                # rows on 16-byte boundaries
    f32 = {"dtype": torch.float32, "device": "cuda"}
    i32 = {"dtype": torch.int32, "device": "cuda"}
    logits = torch.full((n, ld), float("nan"), dtype=dt, device="cuda")
    x = torch.randn((n, V), generator=g, device="cuda").mul_(3)
    if case["masked"]:
        x.masked_fill_(torch.rand((n, V), generator=g, device="cuda") < 0.95, float("-inf"))
    logits[:, :V] = x
    start = np.concatenate([[0], np.cumsum(rows)])
    T = max(1, max(rows))
    table = np.arange(T)[None, :] + start[:-1, None]
    table = np.where(np.arange(T)[None, :] < np.array(rows)[:, None], table, -1)
    s = {"case": case, "logits": logits, "rows": torch.from_numpy(table).cuda()}
    # drafted by a model near the target, or looked up: the target's favourite three times in four
    near = x.add_(torch.randn((n, V), generator=g, device="cuda")) if case["draft"] else x
    if case["draft"]:
        s["draft_logits"] = torch.full((n, ld), float("nan"), dtype=dt, device="cuda")
        s["draft_logits"][:, :V] = near
        near = s["draft_logits"][:, :V].float()
        race = torch.empty((n, V), device="cuda").exponential_(generator=g)
        guess = (near.mul_(c).nan_to_num_(neginf=-1e30) - race.log_()).argmax(1)
    else:
        guess = torch.where(torch.rand(n, generator=g, device="cuda") < 0.75, logits[:, :V].float().argmax(1),
                            torch.randint(0, V, (n,), generator=g, device="cuda"))
    s["ids"] = torch.zeros(n, **i32)
    s["ids"][1:] = guess[:-1].to(torch.int32)          # row r + 1 holds what row r led to
    if not case["greedy"]:
        s["u"] = torch.rand(n, generator=g, device="cuda")
        s["noise"] = torch.empty((cursors, ld), device="cuda").exponential_(generator=g).clamp_min_(1e-30)
    s.update(n_accept=torch.zeros(cursors, **i32), next_id=torch.zeros(cursors, **i32), next_logp=torch.zeros(cursors, **f32), accept_p=torch.zeros(n, **f32))
    if own:
        import packed_tree_attention_gb300 as pta
        pool = pta.Pool(sum(-(-max(r, 1) // 64) for r in rows), 64, 1, 64, pta.DTYPE_BF16)
        cur = [pool.root() for _ in rows]
        for a, r in zip(cur, rows):
            pool.append(a, max(r, 1))
        s["plan"] = pool.chunk_plan(cur, rows, 1)
        s["ws"] = torch.empty(max(256, s["plan"].verify_drafts_workspace_size(0, cursors)), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ----

def run(s):
    if s["case"]["op"] == "verify":
        return _run_verify(s)
    if own:
        s["plan"].chunk_attn(s["q"], s["o"], s["lse"], s["scale"], s["ws"], k_pool=s["k"], v_pool=s["v"])
        return {"o": s["o"], "lse": s["lse"]}
    return _attend(s)


def _run_verify(s):
    case = s["case"]
    if own:
        s["plan"].verify_drafts(0, case["cursors"], s["logits"], case["vocab"], s["ids"], s["n_accept"], s["next_id"], s["ws"], u=s.get("u"),
                                noise=s.get("noise"), draft_logits=s.get("draft_logits"), accept_p=s["accept_p"], next_logp=s["next_logp"],
                                inv_temp=case["inv_temp"], draft_inv_temp=case["inv_temp"])
        return {k: s[k] for k in ("n_accept", "next_id", "next_logp", "accept_p")}
    return _greedy(s, case) if case["greedy"] else _sampled(s, case)


# ---- the plain forms ----

def _attend(s):
    case = s["case"]
    slot, kpos, seen, row, rpos = s["index"]
    P, G, W = case["page"], case["group"], case["window"]
    c, T = row.shape
    k = s["k"][slot // P, :, slot % P].float()                               # [cursors][tokens][kv heads][d]
    v = s["v"][slot // P, :, slot % P].float()
    q = s["q"][row.clamp_min(0)].float().reshape(c, T, case["kv_heads"], G, -1)
    # [cursors][kv heads][G T][tokens]
    q = q.permute(0, 2, 3, 1, 4).reshape(c, case["kv_heads"], G * T, -1)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).reshape(c, case["kv_heads"], G, T, -1)
    t = torch.arange(T, device=row.device)[:, None]
    keep = seen[:, None, :] <= t
    if W:
        keep &= (kpos[:, None, :] > rpos[:, :, None] - W) | (kpos[:, None, :] < case["sink"])
    x.masked_fill_(~keep[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    S = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(c, case["kv_heads"], G * T, -1), v.permute(0, 2, 1, 3)).reshape(c, case["kv_heads"], G, T, -1) / S
    lse = m + torch.log(S)
    live = row >= 0
    o = o.permute(0, 3, 1, 2, 4)[live].reshape(s["n"], case["kv_heads"] * G, -1)
    lse = lse.permute(0, 3, 1, 2, 4)[live].reshape(s["n"], -1)
    return {"o": o.to(DTYPES[case["dtype"]]), "lse": lse}


def _log_sums(x, c):
    """Largest entry and the log of the sum of exponentials relative to it, the sum in 64 bits: both lie next to borders."""
    m = x.amax(1, keepdim=True)
    e = torch.exp((x - m.masked_fill(m == float("-inf"), 0)) * c)
    return m, torch.log(e.sum(1, keepdim=True, dtype=torch.float64))


def _log_p(x, m, ls, c):
    return torch.where(m == float("-inf"), float("-inf"), (x.double() - m) * c - ls)


def _first(score, floor):
    """The lowest index of each row's largest score; -1 where none is above `floor`."""
    best = score.amax(1, keepdim=True)
    at = torch.arange(score.shape[1], device=score.device)
    i = torch.where(score == best, at, score.shape[1]).amin(1)
    return torch.where(best[:, 0] > floor, i, -1)


def _drafted(s):
    """Which rows hold a drafted token, and its id (row - 1 has its distribution)."""
    rows = s["rows"]
    n = s["ids"].shape[0]
    held = torch.zeros(n + 1, dtype=torch.bool, device=rows.device)
    held[torch.where(rows[:, 1:] >= 0, rows[:, 1:], n)] = True
    return held[:n]


def _accepted(s, ok):
    """Accepted drafts of each cursor, the row of the distribution that its next token is from (-1: no rows), and whether a draft was
    rejected there."""
    rows = s["rows"]
    count = (rows >= 0).sum(1)
    held = rows[:, 1:] >= 0
    run = (ok[rows[:, 1:].clamp_min(0)] & held).to(torch.int32).cumprod(1)
    acc = run.sum(1)
    return acc, torch.where(count > 0, rows[:, 0] + acc, -1), acc < count - 1


def _finish(s, acc, at, out, m, ls, x, accept_p):
    """next_logp, and acceptance probabilities up to the first rejected draft."""
    c = s["case"]["inv_temp"]
    r, i = at.clamp_min(0), out.clamp_min(0)
    lp = _log_p(x[r, i].float(), m[r, 0], ls[r, 0], c)
    rows = s["rows"][:, 1:]
    t = torch.arange(rows.shape[1], device=rows.device)
    shown = (rows >= 0) & (t <= acc[:, None])
    n = accept_p.shape[0]
    p = torch.zeros(n + 1, device=rows.device)
    p[torch.where(shown, rows, n)] = accept_p[rows.clamp_min(0)].float()
    return {"n_accept": acc.to(torch.int32), "next_id": out.to(torch.int32), "next_logp": torch.where(out < 0, float("-inf"), lp).float(), "accept_p": p[:n]}


def _greedy(s, case):
    x = s["logits"][:, :case["vocab"]]
    m, ls = _log_sums(x.float(), case["inv_temp"])
    best = _first(x, float("-inf"))
    held = _drafted(s)
    ok = torch.zeros_like(held)
    ok[1:] = (s["ids"][1:] == best[:-1]) & held[1:]
    acc, at, _ = _accepted(s, ok)
    out = torch.where(at < 0, -1, best[at.clamp_min(0)])
    return _finish(s, acc, at, out, m, ls, x, ok.float())


def _sampled(s, case):
    V, c = case["vocab"], case["inv_temp"]
    x = s["logits"][:, :V]
    m, ls = _log_sums(x.float(), c)
    held = _drafted(s)
    r = held.nonzero()[:, 0]
    tok = s["ids"][r].long()
    lp = _log_p(x[r - 1, tok].float(), m[r - 1, 0], ls[r - 1, 0], c)
    lq = torch.zeros_like(lp)
    if case["draft"]:
        y = s["draft_logits"][:, :V]
        mq, lsq = _log_sums(y.float(), c)
        lq = _log_p(y[r - 1, tok].float(), mq[r - 1, 0], lsq[r - 1, 0], c)
    a = torch.zeros(held.shape[0], dtype=torch.float64, device=x.device)
    a[r] = torch.where(lp == float("-inf"), 0.0, torch.exp(lp - lq).clamp_max(1.0))
    ok = held & (s["u"] < a)
    acc, at, rejected = _accepted(s, ok)
    j = at.clamp_min(0)
    p = torch.exp(_log_p(x[j].float(), m[j], ls[j], c)).float()
    w = p
    if case["draft"]:
        q = torch.exp(_log_p(y[j].float(), mq[j], lsq[j], c)).float()
        w = torch.where(rejected[:, None], p - q, p)
    elif held.shape[0]:
        last = s["ids"][(j + 1).clamp_max(held.shape[0] - 1)].long()
        w = torch.where(rejected[:, None] & (torch.arange(V, device=x.device) == last[:, None]), 0.0, p)
    noise = s["noise"][:, :V]
    out = _first(w / noise, 0.0)
    out = torch.where(out < 0, _first(p / noise, 0.0), out)                  # nothing left: the target's own
    return _finish(s, acc, at, torch.where(at < 0, -1, out), m, ls, x, a)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s, case)
    rows, pairs, _ = _pairs(case)
    if 4 * case["head_dim"] * case["kv_heads"] * case["group"] * pairs > 4e12:
        return None
    return _exact_attn(s, case)


def _exact_attn(s, case):
    """Cursor by cursor and head by head, from the episode's description: token t of a segment is in slot t % page of its page t // page."""
    R, B, P, G, f = case["roots"], case["branches"], case["page"], case["group"], case["prefix"]
    pages, _ = _pages(case)
    lens = _lengths(case)
    o, lse = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    row = 0

    def tokens(pool, seg, a, b, h):
        p = torch.tensor(pages[seg][a // P:-(-b // P)], device="cuda", dtype=torch.long)
        return pool[p, h].reshape(len(p) * P, -1)[a % P:a % P + b - a].double()

    for c, (n, new) in enumerate(lens):
        if not new:
            continue
        m = _mounted(case, c)
        spans = [(c // B, 0, f, 0)] + ([(R + m[0], m[1], m[2], f + m[1])] if m else []) + [(R + c, 0, n, f)]
        p0 = max(f + n, f + m[2] + 1) if m else f + n
        spans.append((R + c, n, n + new, p0))
        kpos = torch.cat([torch.arange(p, p + b - a, device="cuda") for _, a, b, p in spans])
        before = sum(b - a for _, a, b, _ in spans[:-1])
        t = torch.arange(new, device="cuda")[:, None]
        gone = torch.arange(len(kpos), device="cuda")[None, :] > before + t
        if case["window"]:
            gone |= (kpos <= p0 + t - case["window"]) & (kpos >= case["sink"])
        for h in range(case["kv_heads"]):
            k, v = (torch.cat([tokens(s[x], seg, a, b, h) for seg, a, b, _ in spans]) for x in "kv")
            for i in range(h * G, h * G + G):
                x = (s["q"][row:row + new, i].double() @ k.T * s["scale"]).masked_fill_(gone, float("-inf"))
                lse[row:row + new, i] = torch.logsumexp(x, 1)
                o[row:row + new, i] = torch.exp(x - lse[row:row + new, i, None]) @ v
        row += new
    return {"o": o, "lse": lse}


def _exact_verify(s, case):
    V, c, none = case["vocab"], case["inv_temp"], float("-inf")
    out = {"n_accept": [], "next_id": [], "next_logp": []}
    accept = torch.zeros(s["ids"].shape[0], dtype=torch.float64)
    ids = s["ids"].cpu()
    u = s["u"].cpu().double() if not case["greedy"] else None

    def probabilities(x, r):
        x = x[r, :V].double() * c
        top = x.max()
        e = torch.exp(x - top) if top > none else torch.zeros_like(x)
        return e / e.sum() if top > none else e

    row = 0
    for i, n in enumerate(_rows_of(case)):
        end, r, w = row + n, row, None
        while r + 1 < end:
            p, tok = probabilities(s["logits"], r), int(ids[r + 1])
            if case["greedy"]:
                top = p.max()
                a = float(top > 0 and int((p == top).nonzero()[0]) == tok)
                taken = a > 0
            else:
                q = probabilities(s["draft_logits"], r) if case["draft"] else None
                px, qx = float(p[tok]), float(q[tok]) if case["draft"] else 1.0
                a = 0.0 if px == 0 else 1.0 if px >= qx else px / qx
                taken = bool(u[r + 1] < a)
            accept[r + 1] = a
            if not taken:
                if not case["greedy"]:
                    w = (p - q).clamp_min(0) if case["draft"] else p.clone().index_fill_(0, torch.tensor([tok], device="cuda"), 0)
                break
            r += 1
        if n:
            p = probabilities(s["logits"], r)
            if case["greedy"]:
                score = p
            else:
                w = p if w is None or not bool((w > 0).any()) else w
                score = w / s["noise"][i, :V].double()
            best = int(score.argmax()) if float(score.max()) > 0 else -1
        else:
            best = -1
        out["n_accept"].append(r - row if n else 0)
        out["next_id"].append(best)
        out["next_logp"].append(float(torch.log(p[best])) if best >= 0 else none)
        row = end
    return {"n_accept": torch.tensor(out["n_accept"], dtype=torch.int32), "next_id": torch.tensor(out["next_id"], dtype=torch.int32),
            "next_logp": torch.tensor(out["next_logp"], dtype=torch.float64), "accept_p": accept}
