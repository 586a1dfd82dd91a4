"""GPU parity of octo_verify_drafts against the fp64 reference in oracle/verify.py.

Ids and counts are equal: the inputs' draws and thresholds are random reals, a decision that 1e-5 of a
probability's relative error could turn is told apart beforehand and not compared.  accept_p and
next_logp: exponents of at most ~60 with two fp32 roundings, 1e-5 (1 + |ref|)."""
import numpy as np
import pytest

from oracle import verify as ov
from oracle.token_score import log_softmax

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import packed_tree_attention_gb300 as pta
    pta.load()
    return pta


def chunk_plan(lib, rows, before=0):
    pool = lib.Pool(sum(-(-max(r, 1) // 16) for r in rows) + 1, 16, 1, 64, lib.DTYPE_BF16)
    cur = [pool.root() for _ in rows]
    for c, r in zip(cur, rows):
        pool.append(c, max(r, 1))
    return pool.chunk_plan(cur, rows, 1)


def on_gpu(x, dtype, pad=8):
    ld = -(-x.shape[1] // 8) * 8 + pad
    full = np.full((x.shape[0], ld), np.nan, dtype=np.float32)
    full[:, :x.shape[1]] = x
    t = torch.from_numpy(full).to(DT[dtype]).cuda()
    return t, t[:, :x.shape[1]].float().cpu().numpy().astype(np.float64)


def run(plan, rows, V, x, ids, y=None, u=None, noise=None, c=1.0, cq=1.0, cur0=0, n_cur=None):
    n_cur = len(rows) if n_cur is None else n_cur
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    N = plan.info["n_rows"]
    acc, nxt = (torch.full((n_cur,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    logp, ap = torch.full((n_cur,), -7.0, device="cuda"), torch.full((N,), -7.0, device="cuda")
    ws = torch.full((max(1, plan.verify_drafts_workspace_size(cur0, n_cur)),), 255, dtype=torch.uint8, device="cuda")
    plan.verify_drafts(cur0, n_cur, x, V, i32(ids), acc, nxt, ws, u=None if u is None else torch.tensor(u, dtype=torch.float32, device="cuda"),
                       noise=noise, draft_logits=y, accept_p=ap, next_logp=logp, inv_temp=c, draft_inv_temp=cq)
    return [a.cpu().numpy() for a in (acc, nxt, logp, ap)]


def close(got, ref, what):
    ref, got = np.asarray(ref, dtype=np.float64), np.asarray(got, dtype=np.float64)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), what
    assert np.all(np.abs(got[fin] - ref[fin]) <= 1e-5 * (1 + np.abs(ref[fin]))), "%s: %g" % (what, np.abs(got[fin] - ref[fin]).max())


def inputs(rng, rows, V, masked, draft, near=1.0):
    n = sum(rows)
    x = rng.standard_normal((n, V)) * 3
    if masked:
        x[rng.random((n, V)) < masked] = -np.inf
    y = x + near * rng.standard_normal((n, V)) if draft else None
    ids = np.zeros(n, dtype=np.int32)
    for r in range(n - 1):
        row = np.where(np.isfinite(y[r] if draft else x[r]), y[r] if draft else x[r], -1e9)
        ids[r + 1] = np.argmax(row - np.log(rng.exponential(size=V))) if draft or rng.random() < 0.3 else np.argmax(row)
    return x, y, ids, rng.random(n).astype(np.float32), rng.exponential(size=(len(rows), V)).astype(np.float32)


def clear(x, rows, ids, y, u, noise, c, cq):
    """Cursors whose decisions 1e-5 of relative error does not turn: no u within that of a_r, and the same winner when each weight's
    share of p and q moves by as much."""
    acc, nxt, _, ap = ov.verify(x, rows, ids, y, u, noise, c, cq)
    keep, r0 = [], 0
    lp = log_softmax(x, c)[0]
    lq = None if y is None else log_softmax(y, cq)[0]
    for i, n in enumerate(rows):
        ok = all(ap[r] == 0 or abs(u[r] - ap[r]) > 1e-5 * ap[r] for r in range(r0 + 1, min(r0 + n, r0 + 2 + acc[i])))
        if n and nxt[i] >= 0:
            r = r0 + acc[i]
            p = np.exp(lp[r])
            w = p.copy()
            if acc[i] + 1 < n:
                if lq is not None:
                    w = np.maximum(p - np.exp(lq[r]), 0)
                elif 0 <= ids[r + 1] < len(w):
                    w[ids[r + 1]] = 0
                if not w.max() > 0:
                    w = p
            err = 1e-5 * (p + (np.exp(lq[r]) if lq is not None else 0))
            hi = (w + err) / noise[i]
            hi[nxt[i]] = 0
            ok &= bool(hi.max() < (w[nxt[i]] - err[nxt[i]]) / noise[i, nxt[i]])
        keep.append(ok)
        r0 += n
    return np.array(keep)


def check(lib, rows, V, dtype, masked=0.0, draft=True, c=1.0, cq=1.0, seed=0, near=1.0):
    rng = np.random.default_rng(seed)
    x, y, ids, u, noise = inputs(rng, rows, V, masked, draft, near)
    xt, xr = on_gpu(x, dtype)
    yt, yr = (None, None) if y is None else on_gpu(y, dtype, 16)
    nt, nr = on_gpu(noise, "f32", 4 if V % 8 else 8)
    plan = chunk_plan(lib, rows)
    got = run(plan, rows, V, xt, ids, yt, u, nt, c, cq)
    plan.sync()
    ref = ov.verify(xr, rows, ids, yr, u, nr, c, cq)
    keep = clear(xr, rows, ids, yr, u, nr, c, cq)
    assert keep.mean() > 0.9
    assert np.array_equal(got[0][keep], ref[0][keep]) and np.array_equal(got[1][keep], ref[1][keep])
    close(got[2][keep], ref[2][keep], "next_logp")
    rk = np.repeat(keep, rows)
    close(got[3][rk], ref[3][rk], "accept_p")
    again = run(plan, rows, V, xt, ids, yt, u, nt, c, cq)
    assert all(np.array_equal(a, b) for a, b in zip(got, again))
    return ref


ROWS = [1, 5, 0, 2, 9, 1, 17, 3, 0, 4]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 257, 1000, 4099, 50001])
@pytest.mark.parametrize("draft", [True, False])
def test_sampled(lib, dtype, V, draft):
    check(lib, ROWS, V, dtype, draft=draft, c=1.25, cq=0.8, seed=V)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_vocabulary_of_the_benchmarks(lib, dtype):
    ref = check(lib, [5, 3, 1, 4], 151936, dtype, seed=3)
    assert ref[0].max() > 0


@pytest.mark.parametrize("draft", [True, False])
def test_masked(lib, draft):
    check(lib, ROWS, 999, "bf16", masked=0.95, draft=draft, seed=4)


def test_many_cursors(lib):
    check(lib, [4] * 400, 300, "bf16", seed=5)
    check(lib, [1] * 700, 64, "f32", seed=6)


@pytest.mark.parametrize("dtype,V", [("f32", 31003), ("bf16", 62003)])
@pytest.mark.parametrize("draft,near", [(True, 1.0), (True, 0.0), (True, 3.0), (False, 1.0)])
def test_many_cursors_of_a_large_vocabulary(lib, dtype, V, draft, near):
    """Enough of both that rows behind a rejected draft are passed over; all drafts accepted (near 0), few, ragged cursors."""
    n = 230 if draft else 460
    check(lib, [(1, 4, 3, 0, 4, 4, 3)[i % 7] for i in range(n)], V, dtype, masked=0.2 if near == 1 else 0, draft=draft, seed=15, near=near)


def test_many_cursors_greedily(lib):
    rng = np.random.default_rng(16)
    V, rows = 31003, [(3, 4, 1, 4)[i % 4] for i in range(470)]
    x = np.round(rng.standard_normal((sum(rows), V)) * 3)    # ties: the lowest id
    xt, xr = on_gpu(x, "f32")
    ids = np.where(rng.random(len(x)) < 0.7, np.roll(np.argmax(xr, axis=1), 1), 5)
    plan = chunk_plan(lib, rows)
    got = run(plan, rows, V, xt, ids, c=0.7)
    plan.sync()
    ref = ov.verify(xr, rows, ids, c=0.7)
    assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1]) and np.array_equal(got[3], ref[3])
    close(got[2], ref[2], "next_logp")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_greedy(lib, dtype):
    rng = np.random.default_rng(7)
    for V in (1, 3, 33, 5000, 151936):
        rows = ROWS if V < 10000 else [5, 2]
        x, _, ids, _, _ = inputs(rng, rows, V, 0.3 if V > 3 else 0, False)
        x = np.round(x)                                  # ties: the lowest id
        x[min(3, len(x) - 1)] = -np.inf
        xt, xr = on_gpu(x, dtype)
        for r in range(1, len(ids)):
            if rng.random() < 0.8:
                ids[r] = np.argmax(xr[r - 1])
        plan = chunk_plan(lib, rows)
        got = run(plan, rows, V, xt, ids, c=0.7)
        plan.sync()
        ref = ov.verify(xr, rows, ids, c=0.7)
        assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1]) and np.array_equal(got[3], ref[3])
        close(got[2], ref[2], "next_logp")


def test_certain_and_impossible_drafts(lib):
    """Equal distributions are always accepted; a draft that the target cannot say never is; one that the draft could not say is
    taken where the target can; certain targets leave nothing but themselves; a target without tokens draws none."""
    V, inf = 40, float("inf")
    rng = np.random.default_rng(8)
    x = rng.standard_normal((12, V))
    y = x.copy()
    x[3, 5] = -inf                     # impossible for the target
    y[5, 6] = -inf                     # impossible for the draft, not for the target
    x[7], y[7] = -inf, -inf
    x[7, 9] = y[7, 9] = 0.0            # certain
    x[9] = -inf                        # no token left
    rows = [3, 2, 2, 2, 3]
    ids = np.array([0, 1, 2, 0, 5, 0, 6, 0, 9, 0, 4, 4])
    u = np.full(12, 0.999999, dtype=np.float32)
    noise = rng.exponential(size=(5, V)).astype(np.float32)
    xt, xr = on_gpu(x, "f32")
    yt, yr = on_gpu(y, "f32")
    nt, nr = on_gpu(noise, "f32")
    plan = chunk_plan(lib, rows)
    acc, nxt, logp, ap = run(plan, rows, V, xt, ids, yt, u, nt)
    plan.sync()
    ref = ov.verify(xr, rows, ids, yr, u, nr)
    assert acc.tolist() == [2, 0, 1, 1, 0] == ref[0].tolist()
    assert nxt.tolist() == ref[1].tolist() and nxt[4] == -1 and nxt[1] != 5
    close(logp, ref[2], "next_logp")
    close(ap, ref[3], "accept_p")
    # drafts of certain distributions, the target certain of another token and of the same one
    acc, nxt, logp, ap = run(chunk_plan(lib, [2, 2]), [2, 2], V, xt[[7, 0, 7, 0]], [0, 3, 0, 9], None, u[:4], nt[:2].contiguous())
    assert acc.tolist() == [0, 1] and nxt[0] == 9 and ap.tolist() == [0, 0, 0, 1]


def test_nan_and_ids_out_of_range(lib):
    V, rows = 64, [3, 3, 2]
    rng = np.random.default_rng(9)
    x, y, ids, u, noise = inputs(rng, rows, V, 0, True)
    u[:] = 0
    ids[1], ids[4] = V, -3
    x[6, 3] = np.nan
    xt, xr = on_gpu(x, "f32")
    yt, yr = on_gpu(y, "f32")
    nt, nr = on_gpu(noise, "f32")
    plan = chunk_plan(lib, rows)
    acc, nxt, logp, ap = run(plan, rows, V, xt, ids, yt, u, nt)
    with pytest.raises(lib.OctoError):
        plan.sync()
    assert acc.tolist() == [0, 0, 0] and nxt[2] == -1 and logp[2] == -np.inf
    ref = ov.verify(xr[:6], rows[:2], ids, yr[:6], u, nr[:2])
    assert nxt[:2].tolist() == ref[1].tolist() and ap[:6].tolist() == ref[3].tolist()


def test_some_of_the_cursors(lib):
    """A range of the plan's cursors: their logits, the plan's ids and u; other rows of accept_p stay."""
    rng = np.random.default_rng(10)
    rows, V = [4, 3, 5, 2], 500
    x, y, ids, u, noise = inputs(rng, rows, V, 0, True)
    xt, xr = on_gpu(x, "bf16")
    yt, yr = on_gpu(y, "bf16")
    nt, nr = on_gpu(noise, "f32")
    plan = chunk_plan(lib, rows)
    whole = run(plan, rows, V, xt, ids, yt, u, nt)
    part = run(plan, rows, V, xt[4:12], ids, yt[4:12], u, nt[1:3], cur0=1, n_cur=2)
    plan.sync()
    assert all(np.array_equal(a[1:3], b) for a, b in zip(whole[:3], part[:3]))
    assert np.array_equal(whole[3][4:12], part[3][4:12]) and (part[3][:4] == -7).all() and (part[3][12:] == -7).all()


def test_capture_and_replay(lib):
    """A graph of a verification, replayed on other logits and draws with a dirty workspace; greedy and sampled."""
    rng = np.random.default_rng(13)
    rows, V = [5, 0, 3, 4], 3001
    plan = chunk_plan(lib, rows)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    for greedy in (False, True):
        sets = []
        for _ in range(2):
            x, y, ids, u, noise = inputs(rng, rows, V, 0, True)
            sets.append((on_gpu(x, "bf16")[0], on_gpu(y, "bf16")[0], torch.tensor(ids, device="cuda"), torch.tensor(u, device="cuda"), on_gpu(noise, "f32")[0]))
        xt, yt, it, ut, nt = (a.clone() for a in sets[0])
        acc, nxt, ap, lp = i32(4), i32(4), torch.zeros(12, device="cuda"), torch.zeros(4, device="cuda")
        ws = torch.full((plan.verify_drafts_workspace_size(0, 4),), 255, dtype=torch.uint8, device="cuda")
        kw = {} if greedy else dict(u=ut, noise=nt, draft_logits=yt)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.verify_drafts(0, 4, xt, V, it, acc, nxt, ws, accept_p=ap, next_logp=lp, **kw)
        for s in (sets[1], sets[0]):
            for a, b in zip((xt, yt, it, ut, nt), s):
                a.copy_(b)
            ws.fill_(77)
            g.replay()
            torch.cuda.synchronize()
            got = [a.cpu().numpy() for a in (acc, nxt, lp, ap)]
            want = run(plan, rows, V, s[0], s[2].cpu().numpy(), None if greedy else s[1], None if greedy else s[3].cpu().numpy(), None if greedy else s[4])
            assert all(np.array_equal(a, b) for a, b in zip(got, want))
    plan.sync()


def test_nothing_left_of_the_target(lib):
    """A rejected draft where the target is nowhere above the draft's distribution (equal rows, u = 1 - 2^-24 or the draft's own id masked):
    the next token is drawn from the target itself."""
    V, n = 1000, 6
    rng = np.random.default_rng(14)
    x = rng.standard_normal((2 * n, V))
    noise = rng.exponential(size=(n, V)).astype(np.float32)
    ids = np.zeros(2 * n, dtype=np.int32)
    ids[1::2] = V + 5                      # rejected whatever u is
    xt, xr = on_gpu(x, "f32")
    nt, nr = on_gpu(noise, "f32")
    plan = chunk_plan(lib, [2] * n)
    acc, nxt, lp, ap = run(plan, [2] * n, V, xt, ids, xt.clone(), np.zeros(2 * n, dtype=np.float32), nt)
    with pytest.raises(lib.OctoError):
        plan.sync()
    p = np.exp(log_softmax(xr, 1.0)[0])[::2]
    assert acc.tolist() == [0] * n and nxt.tolist() == np.argmax(p / nr, axis=1).tolist() and (ap == 0).all()


def test_distribution_of_the_emitted_token(lib):
    """Over many draws the first emitted token has the target's own distribution, whatever the draft's: frequencies of 40,000 within
    five standard deviations."""
    n, V = 40000, 8
    rng = np.random.default_rng(11)
    x0, y0 = rng.standard_normal(V), 2 * rng.standard_normal(V)
    p, q = (np.exp(z - np.logaddexp.reduce(z)) for z in (x0, y0))
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = np.zeros(2 * n, dtype=np.int32)
    ids[1::2] = rng.choice(V, size=n, p=q)
    xt = torch.tensor(x0, dtype=torch.float32, device="cuda").repeat(2 * n, 1)
    yt = torch.tensor(y0, dtype=torch.float32, device="cuda").repeat(2 * n, 1)
    noise = torch.empty((n, V), device="cuda").exponential_(generator=g)
    rows = [2] * n
    plan = chunk_plan(lib, rows)
    acc, nxt, _, _ = run(plan, rows, V, xt, ids, yt, rng.random(2 * n).astype(np.float32), noise)
    plan.sync()
    first = np.where(acc > 0, ids[1::2], nxt)
    freq = np.bincount(first, minlength=V) / n
    assert np.all(np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / n))


def test_refusals(lib):
    rows, V = [3, 2], 64
    rng = np.random.default_rng(12)
    x, y, ids, u, noise = inputs(rng, rows, V, 0, True)
    xt, yt, nt = on_gpu(x, "bf16")[0], on_gpu(y, "bf16")[0], on_gpu(noise, "f32")[0]
    plan = chunk_plan(lib, rows)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    need = plan.verify_drafts_workspace_size(0, 2)
    ut, it, ws = torch.tensor(u, device="cuda"), torch.tensor(ids, device="cuda"), torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    call = lambda cur0=0, n_cur=2, x=xt, V=V, ids=it, a=i32(2), b=i32(2), ws=ws, **kw: plan.verify_drafts(cur0, n_cur, x, V, ids, a, b, ws, **kw)
    for kw in (dict(cur0=1), dict(n_cur=3), dict(cur0=-1), dict(ws=None), dict(ws=ws[:need - 1].contiguous()), dict(ws=ws[4:]), dict(u=ut), dict(noise=nt),
               dict(draft_logits=yt), dict(inv_temp=0.0), dict(inv_temp=float("nan")), dict(u=ut, noise=nt, draft_logits=yt, draft_inv_temp=-1.0),
               dict(V=0), dict(ids=None), dict(a=None), dict(x=xt[:, 1:])):
        with pytest.raises((lib.OctoError, ValueError)):
            call(**kw)
    for kw in (dict(x=xt[:4]), dict(x=xt.half()), dict(x=xt.cpu()), dict(u=ut, noise=nt[:1]), dict(u=ut, noise=nt.bfloat16()), dict(u=ut[:4], noise=nt),
               dict(u=ut, noise=nt, draft_logits=yt.float()), dict(u=ut, noise=nt, draft_logits=yt[:4]), dict(ids=it.long()), dict(a=i32(1)),
               dict(accept_p=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    call(n_cur=0, x=xt[:0])
    call()
    plan.sync()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
def test_greedy_rows_with_a_nan(lib, dtype, many):
    """A NaN anywhere in a row that is needed, a +inf beside it or not: its draft is rejected and no token is drawn.  A +inf without one is
    the largest logit.  Few cursors, and enough of a large vocabulary that rows behind a rejected draft are passed over."""
    V = (24007 if dtype == "f32" else 48011) if many else 1003
    n_cur, n = 480 if many else 40, 4
    N = n_cur * n
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.full((N, -(-V // 8) * 8 + 8), float("nan"), dtype=DT[dtype], device="cuda")
    for r0 in range(0, N, 256):
        x[r0:r0 + 256, :V] = torch.randn((min(256, N - r0), V), generator=g, device="cuda").to(DT[dtype])
    rng = np.random.default_rng(18)
    top = rng.integers(0, V - 1, N)
    x[torch.arange(N), torch.from_numpy(top)] = 40.0
    ids = np.concatenate([[0], top[:-1]]).astype(np.int32)
    acc, nxt, ap, logp = [], [], np.zeros(N, dtype=np.float32), []
    for i in range(n_cur):
        j, kind = int(rng.integers(0, n)), i % 6
        r = i * n + j
        if kind in (3, 4):
            x[r, top[r]] = float("inf")
        if kind in (1, 2, 3, 5):
            x[r, {1: int(rng.integers(0, V)), 2: V - 1, 3: top[r] ^ 1 if top[r] ^ 1 < V else top[r] - 1, 5: top[r]}[kind]] = float("nan")
        k = j if kind in (1, 2, 3, 5) else n - 1
        acc.append(k)
        nxt.append(-1 if kind in (1, 2, 3, 5) else top[i * n + n - 1])
        ap[i * n + 1:i * n + k + 1] = 1
        logp.append(-np.inf if nxt[-1] < 0 else np.nan if kind == 4 and j == n - 1 else 0.0)
    plan = chunk_plan(lib, [n] * n_cur)
    got = run(plan, [n] * n_cur, V, x, ids)
    plan.sync()
    assert got[0].tolist() == acc and got[1].tolist() == nxt and np.array_equal(got[3], ap)
    # the other V - 1 logits take less than V e^(5.5 - 40) of the mass
    assert np.allclose(got[2], logp, rtol=0, atol=1e-6, equal_nan=True)


def test_acceptance_of_unlikely_drafts(lib):
    """Ratios of probabilities far below the types' range: what is off is the two sums and one exponential, not the exponents.

    Each sum: exponentials to 2^-22, exponents of at most 8 (those further down weigh less than 2^-24) times the rounded inverse
    temperature and rounded once, 2 * 8 * 2^-24 ln 2, 64 terms in a tree of at most 9 roundings: 1.5e-6.  Two of them, the exponential
    (2^-22), a quotient and two products: below 4e-6."""
    V, n = 64, 400
    rng = np.random.default_rng(19)
    x, y = rng.standard_normal((2 * n, V)), rng.standard_normal((2 * n, V))
    x[::2, 7] = -rng.uniform(20, 500, n)
    y[::2, 7] = x[::2, 7] + rng.uniform(-0.5, 2.5, n)
    xt, xr = on_gpu(x, "f32")
    yt, yr = on_gpu(y, "f32")
    nt, nr = on_gpu(rng.exponential(size=(n, V)).astype(np.float32), "f32")
    ids = np.full(2 * n, 7, dtype=np.int32)
    for c, cq in ((1.0, 1.0), (0.7, 0.7)):
        c32, cq32 = float(np.float32(c)), float(np.float32(cq))
        plan = chunk_plan(lib, [2] * n)
        _, _, _, ap = run(plan, [2] * n, V, xt, ids, yt, np.ones(2 * n, dtype=np.float32), nt, c, cq)
        plan.sync()
        lp, lq = log_softmax(xr, c32)[0][::2, 7], log_softmax(yr, cq32)[0][::2, 7]
        a = np.exp(np.minimum(lp - lq, 0))
        assert (a < 1).mean() > 0.5 and np.all(np.abs(ap[1::2] - a) <= 4e-6 * a), np.abs(ap[1::2] / a - 1).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_masked_by_the_lowest_value(lib, dtype):
    """A drafted token that the target masks with its type's lowest value has no probability, whatever the draft's distribution has there
    (the same value, -inf, a logit, or no distribution); one that only the draft masks so is taken."""
    V = 40
    low = float(torch.finfo(DT[dtype]).min)
    rng = np.random.default_rng(20)
    x, y = rng.standard_normal((8, V)), rng.standard_normal((8, V))
    x[[0, 2, 4], 5] = low
    y[0, 5], y[2, 5], y[6, 5] = low, -np.inf, low
    ids = np.full(8, 5, dtype=np.int32)
    xt, xr = on_gpu(x, dtype)
    yt, yr = on_gpu(y, dtype)
    nt, nr = on_gpu(rng.exponential(size=(4, V)).astype(np.float32), "f32")
    for c in (1.0, 0.25, 2.0):
        plan = chunk_plan(lib, [2] * 4)
        acc, nxt, lp, ap = run(plan, [2] * 4, V, xt, ids, yt, np.zeros(8, dtype=np.float32), nt, c, c)
        assert acc.tolist() == [0, 0, 0, 1] and ap[1::2].tolist() == [0, 0, 0, 1] and (nxt[:3] != 5).all()
        acc, nxt, lp, ap = run(plan, [2] * 4, V, xt, ids, None, np.zeros(8, dtype=np.float32), nt, c, c)
        assert acc.tolist() == [0, 0, 0, 1] and (ap[1:6] == 0).all() and ap[7] > 0 and (nxt[:3] != 5).all()
        plan.sync()


@pytest.mark.parametrize("dtype,V", [("f32", 24007), ("bf16", 48011)])
@pytest.mark.parametrize("draft", [True, False])
def test_many_cursors_with_broken_rows(lib, dtype, V, draft):
    """Enough of a large vocabulary that rows behind a rejected draft are passed over: NaN in the target's rows and in the draft's, +inf,
    rows without a token, ids out of range; a range of the plan's cursors gives what the whole gives."""
    n_cur, n = 240 if draft else 470, 4
    N = n_cur * n
    rng = np.random.default_rng(21)
    g = torch.Generator(device="cuda").manual_seed(22)

    def rand():
        t = torch.full((N, -(-V // 8) * 8), float("nan"), dtype=DT[dtype], device="cuda")
        for r0 in range(0, N, 256):
            t[r0:r0 + 256, :V] = (3 * torch.randn((min(256, N - r0), V), generator=g, device="cuda")).to(DT[dtype])
        return t
    x, y = rand(), rand() if draft else None
    ids = np.zeros(N, dtype=np.int32)
    best = x[:, :V].float().argmax(1).cpu().numpy()      # likely drafts, u = 0 below: taken
    ids[1:] = best[:-1]
    u = np.zeros(N, dtype=np.float32)
    noise = torch.empty((n_cur, -(-V // 4) * 4), device="cuda").exponential_(generator=g)
    acc, kinds = [], []
    for i in range(n_cur):
        j, kind = int(rng.integers(0, n - 1)), i % 8      # row r0 + j leads to a draft
        r = i * n + j
        if kind == 0:
            u[r + 1] = 2                                  # rejected in the usual way
        elif kind == 1:
            x[r, int(rng.integers(0, V))] = float("nan")
        elif kind == 2:
            x[r, V - 1] = float("nan")
        elif kind == 3:
            x[r, int(rng.integers(0, V))] = float("inf")
        elif kind == 4:
            x[r, :V] = -float("inf")
        elif kind == 5:
            ids[r + 1] = V + i if i % 16 < 8 else -1 - i
        elif kind == 6 and draft:
            y[r, int(rng.integers(0, V))] = float("nan")
        acc.append(j if kind < 6 or (kind == 6 and draft) else n - 1), kinds.append(kind)
    plan = chunk_plan(lib, [n] * n_cur)
    got = run(plan, [n] * n_cur, V, x, ids, y, u, noise)
    with pytest.raises(lib.OctoError):
        plan.sync()
    assert got[0].tolist() == acc
    ap = got[3].reshape(n_cur, n)
    for i, (k, kind) in enumerate(zip(acc, kinds)):
        assert (ap[i, 1:k + 1] > 0).all() and (ap[i, k + 2:] == 0).all() and (kind in (0, 7) or k == n - 1 or ap[i, k + 1] == 0)
        if 1 <= kind <= 4:
            assert got[1][i] == -1 and got[2][i] == -np.inf
            continue
        # the next token: p - q, p without the rejected draft, or p
        r = i * n + k
        lp = torch.log_softmax(x[r, :V].double(), 0)
        p = lp.exp()
        w, err = p, 1e-5 * p
        if k < n - 1 and draft and kind != 6:
            q = torch.softmax(y[r, :V].double(), 0)
            w, err = (p - q).clamp_min(0), 1e-5 * (p + q)
        elif k < n - 1 and not draft and kind != 5:
            w = p.index_fill(0, torch.tensor([int(ids[r + 1])], device="cuda"), 0)
        t = int(got[1][i])
        lo, hi = (w - err) / noise[i, :V].double(), (w + err) / noise[i, :V].double()
        assert hi[t] >= lo.max(), i
        assert abs(got[2][i] - float(lp[t])) <= 1e-5 * (1 + abs(float(lp[t])))
    part = run(plan, [n] * n_cur, V, x[3 * n:-2 * n], ids, None if y is None else y[3 * n:-2 * n], u, noise[3:-2], cur0=3, n_cur=n_cur - 5)
    with pytest.raises(lib.OctoError):
        plan.sync()
    assert all(np.array_equal(a[3:-2], b) for a, b in zip(got[:3], part[:3]))
    assert np.array_equal(got[3][3 * n:-2 * n], part[3][3 * n:-2 * n]) and (part[3][:3 * n] == -7).all() and (part[3][-2 * n:] == -7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_nothing_left_of_the_target_over_several_ctas(lib, dtype, n):
    """As above with a vocabulary that several CTAs draw from: whichever of them ends last draws from the target itself."""
    V = 151936 if n < 40 else 20003
    rng = np.random.default_rng(23)
    x = rng.standard_normal((2 * n, V))
    noise = rng.exponential(size=(n, V)).astype(np.float32)
    ids = np.zeros(2 * n, dtype=np.int32)
    ids[1::2] = V
    xt, xr = on_gpu(x, dtype)
    nt, nr = on_gpu(noise, "f32")
    plan = chunk_plan(lib, [2] * n)
    s = np.exp(log_softmax(xr, 1.0)[0])[::2] / nr
    two = np.partition(s, V - 2, axis=1)[:, -2:]
    sure = two[:, 0] < two[:, 1] * (1 - 2e-5)
    assert sure.mean() > 0.9
    want = np.argmax(s, axis=1)
    for _ in range(5):
        acc, nxt, lp, ap = run(plan, [2] * n, V, xt, ids, xt.clone(), np.zeros(2 * n, dtype=np.float32), nt)
        with pytest.raises(lib.OctoError):
            plan.sync()
        assert acc.tolist() == [0] * n and (ap == 0).all()
        same = np.abs(s[np.arange(n), nxt] - two[:, 1]) <= 2e-5 * two[:, 1]
        assert np.array_equal(nxt[sure], want[sure]) and same.all()


@pytest.mark.parametrize("n_cur,V,draft", [(3, 50001, True), (240, 24007, True), (470, 24007, None)])
def test_two_verifications_at_once(lib, n_cur, V, draft):
    """One plan, calls under way on two streams with logits, draws and workspaces of their own; greedily (draft None) too."""
    n = 4
    plan = chunk_plan(lib, [n] * n_cur)
    g = torch.Generator(device="cuda").manual_seed(24)
    ld = -(-V // 4) * 4
    rnd = lambda rows: torch.randn((rows, ld), generator=g, device="cuda")
    i32 = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")
    sets, size = [], plan.verify_drafts_workspace_size(0, n_cur)
    for _ in range(2):
        x = rnd(n * n_cur)
        kw = {}
        if draft:
            kw = dict(draft_logits=x + rnd(n * n_cur), u=torch.rand(n * n_cur, generator=g, device="cuda"),
                      noise=torch.empty((n_cur, ld), device="cuda").exponential_(generator=g))
        ids = i32(n * n_cur)
        ids[1:] = x[:-1, :V].argmax(1).int()
        ids[n // 2::n] = 1
        out = (i32(n_cur), i32(n_cur), torch.zeros(n * n_cur, device="cuda"), torch.zeros(n_cur, device="cuda"))
        sets.append((x, ids, kw, out, torch.full((size,), 255, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    call = lambda s, o, ws, st: plan.verify_drafts(0, n_cur, s[0], V, s[1], o[0], o[1], ws, accept_p=o[2], next_logp=o[3], stream=st, **s[2])
    want = []
    for s in sets:
        o = tuple(t.clone() for t in s[3])
        call(s, o, torch.empty(size, dtype=torch.uint8, device="cuda"), None)
        want.append(o)
    plan.sync()
    torch.cuda.synchronize()
    for _ in range(20):
        for s in sets:
            call(s, s[3], s[4], s[5])
    torch.cuda.synchronize()
    for s, o in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(s[3], o))
    plan.sync()
