"""What the row-wise loss operators cost: token scoring (log-probabilities of given tokens, entropy, top
alternatives), its gradient, and distillation from a teacher's top logits, each in a plain form of elementary
torch operations and as the calls that a user of the framework makes."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ----
# A packed plan is a shared prefix of `prefix` tokens forked into `branches` of `length` tokens each (rows =
# prefix + branches * length); a decode plan has one row for each of `cursors`.

def listed():
    return [
        # one request that asks for the log-probabilities of its sampled token: latency alone
        {"name": "score_1_cursor", "op": "score", "plan": "decode", "cursors": 1, "vocab": 151936, "dtype": "bf16", "k": 20,
         "inv_temp": 1.0, "masked": 0},
        # a serving step of the paged decode's 256 cursors
        {"name": "score_256_cursors", "op": "score", "plan": "decode", "cursors": 256, "vocab": 151936, "dtype": "bf16", "k": 20,
         "inv_temp": 1.0, "masked": 0},
        # constrained decoding: all but a few tokens at -inf, rows with nothing left among them; odd sizes, a temperature
        {"name": "score_masked_odd_f32", "op": "score", "plan": "decode", "cursors": 37, "vocab": 50001, "dtype": "f32", "k": 5,
         "inv_temp": 1.25, "masked": 1},
        # the policy's log-probabilities and entropies over packed rows (no alternatives)
        {"name": "score_packed", "op": "score", "plan": "pack", "prefix": 1024, "branches": 6, "length": 1536, "vocab": 151936,
         "dtype": "bf16", "k": 0, "inv_temp": 1.0, "masked": 0},
        # the teacher's pass of a distillation: its top 64 of every packed row
        {"name": "score_packed_top64", "op": "score", "plan": "pack", "prefix": 512, "branches": 4, "length": 384, "vocab": 151936,
         "dtype": "bf16", "k": 64, "inv_temp": 0.5, "masked": 0},
        # gradient of a policy loss with an entropy bonus over packed rows
        {"name": "score_bwd_packed", "op": "score_bwd", "plan": "pack", "prefix": 1024, "branches": 5, "length": 1024, "vocab": 151936,
         "dtype": "bf16", "k": 0, "inv_temp": 1.0, "masked": 0},
        # the same of a short ragged episode in fp32
        {"name": "score_bwd_odd_f32", "op": "score_bwd", "plan": "pack", "prefix": 61, "branches": 3, "length": 77, "vocab": 32003,
         "dtype": "f32", "k": 0, "inv_temp": 0.8, "masked": 1},
        # the student's step against a teacher's renormalised top 64
        {"name": "distill_packed", "op": "distill", "plan": "pack", "prefix": 2048, "branches": 4, "length": 1536, "vocab": 151936,
         "dtype": "bf16", "k": 64, "inv_temp": 0.5, "masked": 0, "tail": 0, "grad": 1},
        # a small batch of a small vocabulary, the teacher's remaining mass as one more class
        {"name": "distill_small_tail", "op": "distill", "plan": "pack", "prefix": 24, "branches": 2, "length": 20, "vocab": 32000,
         "dtype": "bf16", "k": 8, "inv_temp": 1.0, "masked": 0, "tail": 1, "grad": 1},
        # fp32 logits with masked entries, odd sizes, remaining mass
        {"name": "distill_odd_f32", "op": "distill", "plan": "pack", "prefix": 101, "branches": 3, "length": 133, "vocab": 50001,
         "dtype": "f32", "k": 17, "inv_temp": 0.7, "masked": 1, "tail": 1, "grad": 1},
        # an evaluation pass: the divergence alone
        {"name": "distill_eval", "op": "distill", "plan": "pack", "prefix": 256, "branches": 3, "length": 256, "vocab": 151936,
         "dtype": "bf16", "k": 32, "inv_temp": 1.0, "masked": 0, "tail": 1, "grad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "score", "score_bwd", "distill", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    vocab = _log(rng, 256, 160000)
    case = {"op": op, "vocab": vocab, "dtype": dtype, "inv_temp": rng.choice([1.0, round(rng.uniform(0.4, 2.0), 3)]),
            "masked": rng.choice([0, 0, 1]), "k": 0}
    most = max(1, min(6000, 400000000 // vocab))
    if op == "score":
        case["k"] = rng.choice([0, min(vocab, _log(rng, 1, 128))])
    if op == "score" and rng.random() < 0.5:
        return {**case, "plan": "decode", "cursors": _log(rng, 1, min(most, 600))}
    branches = rng.randint(1, 6)
    rows = max(2 + branches, _log(rng, 4, max(5, most)))
    length = max(1, rows // (branches + 1))
    case.update(plan="pack", prefix=max(1, rows - branches * length), branches=branches, length=length)
    if op == "distill":
        case.update(k=min(vocab, _log(rng, 1, 128)), tail=rng.choice([0, 1]), grad=rng.choice([1, 1, 0]))
    return case


def _rows(case):
    return case["cursors"] if case["plan"] == "decode" else case["prefix"] + case["branches"] * case["length"]


def work(case):
    n, V, k = _rows(case), case["vocab"], case["k"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "score":
        return {"bytes": n * V * es + n * (4 + 4 + 8 + 4 + 8 * k), "flops": 6 * n * V}
    if case["op"] == "score_bwd":
        return {"bytes": 2 * n * V * es + n * (8 + 4 + 4 + 4 + 4), "flops": 7 * n * V}
    return {"bytes": (2 if case["grad"] else 1) * n * V * es + n * (8 * k + 4 + 4) + 4, "flops": (8 if case["grad"] else 4) * n * V}


# ---- inputs ----

def _tree(case, device):
    """Row of the token before each packed token on its path (-1: none)."""
    P, B, L = case["prefix"], case["branches"], case["length"]
    pred = torch.arange(-1, P + B * L - 1, device=device)
    pred[P::L] = P - 1
    return pred


def _plan(case):
    import packed_tree_attention_gb300 as pta
    page = 64
    if case["plan"] == "decode":
        pool = pta.Pool(case["cursors"], page, 1, 64, pta.DTYPE_BF16)
        cursors = [pool.root() for _ in range(case["cursors"])]
        for c in cursors:
            pool.append(c, 1)
        return pool.decode_plan(cursors)
    pages = lambda n: -(-n // page)
    pool = pta.Pool(pages(case["prefix"]) + case["branches"] * pages(case["length"]), page, 1, 64, pta.DTYPE_BF16)
    root = pool.root()
    pool.append(root, case["prefix"])
    for c in pool.fork(root, case["branches"]):
        pool.append(c, case["length"])
    return pool.pack_tree([root], 128)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, V, k, c = _rows(case), case["vocab"], case["k"], case["inv_temp"]
    dt = DTYPES[case["dtype"]]
    ld = -(-V // 8) * 8                                     # rows on 16-byte boundaries
    logits = torch.full((n, ld), float("nan"), dtype=dt, device="cuda")
    logits[:, :V] = torch.randn((n, V), generator=g, device="cuda").mul_(3)
    if case["masked"]:
        keep = torch.rand((n, V), generator=g, device="cuda") < 4.0 / V + 0.3 * (torch.arange(n, device="cuda")[:, None] % 2)
        keep[n // 3] = False
        logits[:, :V].masked_fill_(~keep, float("-inf"))
    s = {"case": case, "logits": logits, "n": n}
    f32 = {"dtype": torch.float32, "device": "cuda"}
    s["ids"] = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    s["pred"] = torch.arange(n, device="cuda") if case["plan"] == "decode" else _tree(case, "cuda")
    if case["op"] == "score":
        s.update(logp=torch.zeros(n, **f32), row_stat=torch.zeros((n, 2), **f32), entropy=torch.zeros(n, **f32))
        s.update(top_ids=torch.zeros((n, k), dtype=torch.int32, device="cuda") if k else None, top_logp=torch.zeros((n, k), **f32) if k else None)
    elif case["op"] == "score_bwd":
        s["row_stat"], s["entropy"] = _stats(logits[:, :V], c)
        s["g_logp"] = torch.randn(n, generator=g, device="cuda")
        s["g_entropy"] = torch.randn(n, generator=g, device="cuda").mul_(0.1)
        s["dlogits"] = torch.zeros((n, ld), dtype=dt, device="cuda")
    else:
        teacher = logits[:, :V].float().add_(torch.randn((n, V), generator=g, device="cuda"))
        val, ids = torch.topk(teacher, k, dim=1)
        s["teach_ids"] = torch.where(val == float("-inf"), -1, ids).to(torch.int32)
        if case["tail"]:
            val = val * c - torch.logsumexp(teacher.mul_(c), dim=1, keepdim=True).clamp_min(-1e30)
        s["teach_val"] = val.contiguous()
        s["weight"] = torch.rand(n, generator=g, device="cuda") * (torch.rand(n, generator=g, device="cuda") < 0.9)
        s.update(row_kl=torch.zeros(n, **f32), loss=torch.zeros(1, **f32))
        s["dlogits"] = torch.zeros((n, ld), dtype=dt, device="cuda") if case["grad"] else None
        s["ws"] = torch.empty(max(256, 8 * n), dtype=torch.uint8, device="cuda")
    if own:
        s["plan"] = _plan(case)
    return s


# ---- one pass ----

def run(s):
    case = s["case"]
    V = case["vocab"]
    if own:
        return _run_own(s, case, V)
    x = s["logits"][:, :V]
    if case["op"] == "score":
        return _score(x, s["ids"], s["pred"], case["inv_temp"], case["k"])
    if case["op"] == "score_bwd":
        return {"dlogits": _score_bwd(x, s["row_stat"], s["entropy"], s["ids"], s["pred"], s["g_logp"], s["g_entropy"], case["inv_temp"])}
    return _distill(x, s["teach_ids"], s["teach_val"], s["weight"], case["inv_temp"], case["tail"], case["grad"])


def _run_own(s, case, V):
    plan, n, c = s["plan"], s["n"], case["inv_temp"]
    if case["op"] == "score":
        plan.token_score(0, n, s["logits"], V, s["row_stat"], entropy=s["entropy"], ids=s["ids"], logp=s["logp"], top_ids=s["top_ids"],
                         top_logp=s["top_logp"], inv_temp=c)
        out = {"logp": s["logp"], "entropy": s["entropy"], "row_stat": s["row_stat"]}
        return {**out, "top_ids": s["top_ids"], "top_logp": s["top_logp"]} if case["k"] else out
    if case["op"] == "score_bwd":
        plan.token_score_bwd(0, n, s["logits"], V, s["row_stat"], s["entropy"], s["ids"], s["g_logp"], s["g_entropy"], s["dlogits"], inv_temp=c)
        return {"dlogits": s["dlogits"][:, :V]}
    plan.distill_topk(0, n, s["logits"], V, s["teach_ids"], s["teach_val"], s["row_kl"], s["ws"], weight=s["weight"], tail=bool(case["tail"]),
                      inv_temp=c, dlogits=s["dlogits"], loss=s["loss"])
    out = {"row_kl": s["row_kl"], "loss": s["loss"]}
    return {**out, "dlogits": s["dlogits"][:, :V]} if case["grad"] else out


# ---- the plain forms ----

def _stats(x, c):
    """(max, log of the sum of exponentials relative to it) and the entropy of each row."""
    x = x.float()
    m = x.amax(1, keepdim=True)
    empty = m == float("-inf")
    t = (x - m.masked_fill(empty, 0)) * c
    e = torch.exp(t)
    S = e.sum(1, keepdim=True)
    ent = torch.log(S) - (e * t.clamp_min(-1e30)).sum(1, keepdim=True) / S
    return torch.cat([m, torch.log(S)], 1), ent.masked_fill(empty, 0)[:, 0]


def _score(x, ids, pred, c, k):
    stat, entropy = _stats(x, c)
    m, ls = stat[:, 0], stat[:, 1]
    r = pred.clamp_min(0)
    xi = x[r, ids.long()].float()
    logp = torch.where(m[r] == float("-inf"), m[r], (xi - m[r]) * c - ls[r])
    out = {"logp": torch.where(pred < 0, 0.0, logp), "entropy": entropy, "row_stat": stat}
    if k:
        # a stable descending sort keeps the lowest id first among equal values
        v, i = torch.sort(x, dim=1, descending=True, stable=True)
        v = v[:, :k].float()
        out["top_ids"] = i[:, :k].to(torch.int32)
        out["top_logp"] = torch.where(v == float("-inf"), v, (v - m[:, None]) * c - ls[:, None])
    return out


def _score_bwd(x, stat, entropy, ids, pred, g_logp, g_entropy, c):
    n, V = x.shape
    dt = x.dtype
    m, ls = stat[:, :1], stat[:, 1:]
    empty = m == float("-inf")
    lp = torch.where(empty, m, (x.float() - m.masked_fill(empty, 0)) * c - ls.masked_fill(empty, 0))
    p = torch.exp(lp)
    has = pred >= 0
    G = torch.zeros(n, device=x.device).index_add_(0, pred[has], g_logp[has])
    d = -p * (G[:, None] + g_entropy[:, None] * (lp.clamp_min(-1e30) + entropy[:, None]))
    d = d.index_put_((pred[has], ids.long()[has]), g_logp[has], accumulate=True) * c
    return d.masked_fill_(empty, 0).to(dt)


def _distill(x, ids, val, weight, c, tail, grad):
    dt = x.dtype
    stat, _ = _stats(x, c)
    m, ls = stat[:, :1], stat[:, 1:]
    live = ids >= 0
    idx = ids.clamp_min(0).long()
    z = (val if tail else val * c).masked_fill(~live, float("-inf"))
    none = (z == float("-inf")).all(1, keepdim=True)
    if tail:
        lnP = z
    else:
        z = z - z.amax(1, keepdim=True).masked_fill(none, 0)
        lnP = z - torch.log(torch.exp(z).sum(1, keepdim=True)).masked_fill(none, 0)
    P = torch.exp(lnP)
    x = x.float()
    t = (x - m.masked_fill(m == float("-inf"), 0)) * c
    lnq = t.gather(1, idx) - ls
    kl = torch.where(P > 0, P * (lnP - lnq), 0.0).sum(1)
    q = torch.exp(t - ls)
    d = q * P.sum(1, keepdim=True)
    if tail:
        rest = (1 - P.sum(1, keepdim=True)).clamp_min(0)
        inside = torch.zeros_like(x, dtype=torch.bool).scatter_(1, torch.where(live, idx, idx[:, :1].clamp_min(0)), live.any(1, keepdim=True).expand_as(live))
        qR = q.masked_fill(inside, 0).sum(1, keepdim=True)
        rest = rest.masked_fill(qR == 0, 0)
        kl = kl + torch.where(rest > 0, rest * (torch.log(rest) - torch.log(qR)), 0.0)[:, 0]
        d = d + rest * q * (1 - (~inside).float() / qR.masked_fill(qR == 0, 1))
    skip = (m[:, 0] == float("-inf")) | (weight == 0) | (none[:, 0] & (not tail))
    kl = kl.masked_fill(skip, 0)
    out = {"row_kl": kl, "loss": (weight * kl).sum().reshape(1)}
    if grad:
        d = d.scatter_add_(1, idx, -P) * (weight * c)[:, None]
        out["dlogits"] = d.masked_fill_(skip[:, None], 0).to(dt)
    return out


# ---- the definitions in 64 bits, row by row ----

def _row(x, c):
    """Log-probabilities of a row, or None where every logit is -inf."""
    m = x.max()
    if m == float("-inf"):
        return None
    return (x - m) * c - torch.log(torch.exp((x - m) * c).sum())


def exact(case, seed):
    n, V, c = _rows(case), case["vocab"], case["inv_temp"]
    if n * V > 2000000000:
        return None
    s = prepare(case, seed)
    x = s["logits"][:, :V]
    inf = float("inf")
    if case["op"] == "score":
        lps, H, stat = [], [], []
        logp = torch.zeros(n, dtype=torch.float64, device="cuda")
        tops = []
        for r in range(n):
            row = x[r].double()
            lp = _row(row, c)
            if lp is None:
                lp = torch.full_like(row, -inf)
                H.append(torch.zeros((), dtype=torch.float64, device="cuda"))
                stat.append(torch.full((2,), -inf, dtype=torch.float64, device="cuda"))
            else:
                p = torch.exp(lp)
                H.append(-torch.where(p > 0, p * lp, 0.0).sum())
                stat.append(torch.stack([row.max(), -lp.max()]))
            if case["k"]:
                tops.append(torch.topk(lp, case["k"]).values)
            at = (s["pred"] == r).nonzero()[:, 0] if case["plan"] == "decode" or r == case["prefix"] - 1 else (r + 1) if _follows(case, r) else None
            if at is not None:
                logp[at] = lp[s["ids"][at].long()]
        out = {"logp": logp, "entropy": torch.stack(H), "row_stat": torch.stack(stat)}
        return {**out, "top_ids": None, "top_logp": torch.stack(tops)} if case["k"] else out
    if case["op"] == "score_bwd":
        d = torch.zeros((n, V), dtype=torch.float64, device="cuda")
        for r in range(n):
            lp = _row(x[r].double(), c)
            if lp is None:
                continue
            p = torch.exp(lp)
            plp = torch.where(p > 0, p * lp, 0.0)
            kids = _kids(case, r)
            d[r] = -s["g_entropy"][r].double() * (plp - p * plp.sum())
            for t in kids:
                d[r] -= s["g_logp"][t].double() * p
                d[r, s["ids"][t].long()] += s["g_logp"][t].double()
            d[r] *= c
        return {"dlogits": d}
    kl = torch.zeros(n, dtype=torch.float64, device="cuda")
    d = torch.zeros((n, V), dtype=torch.float64, device="cuda") if case["grad"] else None
    ids, val, w = s["teach_ids"].cpu(), s["teach_val"].double(), s["weight"].double()
    for r in range(n):
        live = (ids[r] >= 0).cuda()
        lp = _row(x[r].double(), c)
        if lp is None or w[r] == 0 or (not case["tail"] and not bool(live.any())):
            continue
        at = s["teach_ids"][r].long()[live]
        lnP = val[r][live] if case["tail"] else _row(val[r][live], c)
        P, q = torch.exp(lnP), torch.exp(lp)
        kl[r] = torch.where(P > 0, P * (lnP - lp[at]), 0.0).sum()
        g = q * P.sum()
        if case["tail"]:
            R = (1 - P.sum()).clamp_min(0)
            out = q.clone()
            out[at] = 0
            qR = out.sum()
            if qR > 0 and R > 0:
                kl[r] += R * (torch.log(R) - torch.log(qR))
                g += R * (q - out / qR)
        if d is not None:
            g.index_add_(0, at, -P)
            d[r] = g * (w[r] * c)
    out = {"row_kl": kl, "loss": (w * kl).sum().reshape(1)}
    return {**out, "dlogits": d} if case["grad"] else out


def _follows(case, r):
    """Whether row r + 1 is the next token of row r's own segment."""
    P, L = case["prefix"], case["length"]
    return r + 1 < _rows(case) and (r < P - 1 or (r >= P and (r - P) % L < L - 1))


def _kids(case, r):
    """Tokens that row r predicts."""
    P, B, L = case["prefix"], case["branches"], case["length"]
    return [P + b * L for b in range(B)] if r == P - 1 else [r + 1] if _follows(case, r) else []
