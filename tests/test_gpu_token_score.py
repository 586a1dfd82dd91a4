"""GPU parity of octo_token_score, octo_token_score_bwd and octo_distill_topk against the
fp64 reference in oracle/token_score.py.

Tolerances.  fp32 results: an exponent c (x - m) of at most ~60 in size carries two fp32
roundings (60 * 2^-23 = 7e-6), as a log-probability directly, as a relative error of a
probability <= 1 otherwise; sums of positive terms and the exponential add less than 1e-6:
within 1e-5 + 1e-5 |ref|.  bf16 gradients add half a step, 2^-8 |ref|.  Ids are equal."""
import numpy as np
import pytest

import synth
from oracle import token_score as ts
from test_gpu_token_logprob import _plans

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


def close(got, ref, what, bf16=False, scale=1.0):
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin], equal_nan=True), what + ": non-finite values"
    err = np.abs(got[fin] - ref[fin])
    tol = 1e-5 * scale + (1e-5 + (2.0 ** -8 if bf16 else 0)) * np.abs(ref[fin])
    assert np.all(err <= tol), "%s: %g over %g" % (what, err[err > tol].max(), tol[err > tol].min())


def decode_plan(lib, n):
    pool = lib.Pool(n, 16, 1, 64, lib.DTYPE_BF16)
    cur = [pool.root() for _ in range(n)]
    for c in cur:
        pool.append(c, 1)
    return pool.decode_plan(cur)


def chain_plan(lib, n):
    pool = lib.Pool(-(-n // 16), 16, 1, 64, lib.DTYPE_BF16)
    r = pool.root()
    pool.append(r, n)
    return pool.pack_tree([r], 128)


def rows_on_gpu(x, dtype, pad=True):
    """x with a row pitch of whole 16-byte vectors, NaN in the padding; and x as stored."""
    N, V = x.shape
    ld = -(-V // 8) * 8 + (8 if pad else 0)
    full = np.full((N, ld), np.nan, dtype=np.float32)
    full[:, :V] = x
    t = torch.from_numpy(full).to(DT[dtype]).cuda()
    return t, t[:, :V].float().cpu().numpy().astype(np.float64)


def gpu(a, dt=torch.float32):
    return None if a is None else torch.as_tensor(np.ascontiguousarray(a)).to(dt).cuda()


def run_score(plan, xt, V, ids=None, k=0, c=1.0, row0=0, n=None, stream=None):
    N = plan.info["n_rows"]
    n = N - row0 if n is None else n
    logp = torch.full((N,), -7.0, device="cuda")
    stat, H = torch.full((max(n, 1), 2), -7.0, device="cuda"), torch.full((max(n, 1),), -7.0, device="cuda")
    ti = torch.full((n, k), -7, dtype=torch.int32, device="cuda") if k else None
    tl = torch.full((n, k), -7.0, device="cuda") if k else None
    plan.token_score(row0, n, xt, V, stat, entropy=H, ids=gpu(ids, torch.int32), logp=None if ids is None else logp, top_ids=ti,
                     top_logp=tl, inv_temp=c, stream=stream)
    return [None if a is None else a.cpu().numpy() for a in (logp, stat[:n], H[:n], ti, tl)]


def check_score(plan, pred, x, dtype, ids, k, c=1.0):
    V = x.shape[1]
    xt, xr = rows_on_gpu(x, dtype)
    logp, stat, H, ti, tl = run_score(plan, xt, V, ids, k, c)
    plan.sync()
    rlogp, rstat, rH, rti, rtl = ts.score(xr, ids, pred, c, k)
    close(logp, rlogp, "logp")
    close(stat, rstat, "row_stat")
    close(H, rH, "entropy")
    if k:
        assert np.array_equal(ti, rti), "top ids"
        close(tl, rtl, "top logp")
    return xt, xr, stat, H


# ---- scoring ----

@pytest.mark.parametrize("dtype,V,k,c", [("f32", 997, 7, 1.0), ("bf16", 1037, 20, 0.5), ("bf16", 4096, 128, 1.0), ("f32", 4097, 0, 1.7),
                                         ("bf16", 1200, 0, 1.0)])
@pytest.mark.parametrize("seed", [5, 19])
def test_score_random_dags(lib, dtype, V, k, c, seed):
    ep = synth.random_dag(seed, page_size=16, max_segments=16, max_len=300)
    pool, plan, pred = _plans(lib, ep)
    N = plan.info["n_rows"]
    rng = np.random.default_rng(seed)
    check_score(plan, pred, rng.normal(0, 3, (N, V)), dtype, rng.integers(0, V, N), k, c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,k", [(1, 1, 1), (1, 2, 2), (3, 7, 7), (1, 8, 3), (2, 9, 9), (5, 128, 128), (1, 151936, 20), (2, 50001, 128),
                                   (19, 32003, 5), (160, 5000, 20), (311, 2048, 64), (700, 513, 40)])
def test_score_sizes(lib, dtype, n, V, k):
    """One row to more than the GPU holds at once, one entry to a full vocabulary."""
    rng = np.random.default_rng(n * 7 + V)
    plan = decode_plan(lib, n)
    check_score(plan, np.arange(n), rng.normal(0, 3, (n, V)), dtype, rng.integers(0, V, n), k)


def awkward_rows(V, rng):
    low = {"f32": np.finfo(np.float32).min, "bf16": -3.3895313892515355e38}
    few = np.full(V, -np.inf)
    few[rng.choice(V, 3, replace=False)] = [1.0, -2.0, 1.0]
    one = np.full(V, -np.inf)
    one[V - 1] = -5.0
    zeros = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    steps = np.round(rng.normal(0, 2, V))
    last = rng.normal(0, 1, V)
    last[-20:] = 9.0
    return [few, one, np.full(V, -np.inf), np.full(V, 2.5), zeros, steps, np.arange(V) / V * 20, -np.arange(V) / V * 20, last,
            rng.normal(5000, 2, V), rng.normal(-5000, 2, V), np.where(np.arange(V) % 512 < 30, 8.0, -8.0) + rng.normal(0, .1, V),
            np.where(np.arange(V) % 4096 < 8, 10.0, 0.0), rng.normal(0, 40, V), low, rng.normal(0, 3, V),
            np.where((np.arange(V) % 4096 < 800) & (np.arange(V) < 16384), rng.normal(20, 1, V), 0.0),
            np.where((np.arange(V) % 2048 < 400) & (np.arange(V) < 16384), rng.normal(20, 1, V), -np.inf)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,k", [(700, 64), (40003, 20), (40003, 128)])
def test_score_awkward_rows(lib, dtype, V, k):
    """Masked rows (-inf, the type's lowest value), an empty row, ties everywhere, signed
    zeros, sorted and periodic rows, far offsets, flat and very peaked ones."""
    rng = np.random.default_rng(V + k)
    rows = awkward_rows(V, rng)
    low = rows[14][dtype]
    lowest = np.full(V, low)
    some = lowest.copy()
    some[[3, V - 2]] = [0.5, 0.25]
    x = np.stack([r for r in rows if not isinstance(r, dict)] + [lowest, some])
    n = len(x)
    ids = rng.integers(0, V, n)
    ids[0] = int(np.argmax(x[0]))
    plan = decode_plan(lib, n)
    xt, xr = rows_on_gpu(x, dtype)
    logp, stat, H, ti, tl = run_score(plan, xt, V, ids, k)
    plan.sync()
    rlogp, rstat, rH, rti, rtl = ts.score(xr, ids, np.arange(n), 1.0, k)
    # rows whose logits differ by more than ~60: a difference of the size d rounds by
    # 2^-23 d in its log-probability, relative to |ref| ~ d: inside 1e-5 |ref|
    close(stat, rstat, "row_stat")
    # (x - m) of the lowest fp32 value overflows to -inf, where the formula's is -3.4e38
    rlogp, rtl = np.where(rlogp < -1e38, -np.inf, rlogp), np.where(rtl < -1e38, -np.inf, rtl)
    logp, tl = np.where(logp < -1e38, -np.inf, logp), np.where(tl < -1e38, -np.inf, tl)
    close(logp, rlogp, "logp")
    close(H, rH, "entropy")
    assert np.array_equal(ti, rti)
    close(tl, rtl, "top logp")


def test_score_nan_and_inf_stay_in_their_rows(lib):
    V, k = 3001, 8
    rng = np.random.default_rng(3)
    x = rng.normal(0, 3, (5, V))
    x[1, 77] = np.nan
    x[2, 500] = np.inf
    x[3] = np.nan
    plan = decode_plan(lib, 5)
    ids = rng.integers(0, V, 5)
    for dtype in ("f32", "bf16"):
        xt, xr = rows_on_gpu(x, dtype)
        logp, stat, H, ti, tl = run_score(plan, xt, V, ids, k)
        for r in (1, 2, 3):
            assert np.isnan(stat[r, 1]) and np.isnan(H[r]) and np.isnan(tl[r]).all()
        rl, rs, rH, rti, rtl = ts.score(xr[[0, 4]], ids[[0, 4]], np.arange(2), 1.0, k)
        close(logp[[0, 4]], rl, "logp")
        close(tl[[0, 4]], rtl, "top logp")
        assert np.array_equal(ti[[0, 4]], rti) and ti[2, 0] == 500
        assert np.array_equal(ti[1], np.argsort(np.where(np.isnan(xr[1]), np.inf, -xr[1]), kind="stable")[:k])
        assert (ti[3] == -1).all()
        d = torch.zeros_like(xt)
        plan.token_score_bwd(0, 5, xt, V, gpu(stat), gpu(H), gpu(ids, torch.int32), gpu(np.ones(5)), gpu(np.ones(5)), d)
        d = d[:, :V].float().cpu().numpy()
        assert np.isfinite(d[[0, 4]]).all() and np.isnan(d[[1, 2, 3]]).any(axis=1).all()
    plan.sync()


def test_score_chunks_options_and_repeats(lib):
    """Chunks equal the whole bit for bit, an output left out changes no other, a second run
    gives the same bits, rows past the chunk and columns past the vocabulary stay as they were."""
    ep = synth.random_dag(23, page_size=16, max_segments=14, max_len=200)
    pool, plan, pred = _plans(lib, ep)
    N, V, k = plan.info["n_rows"], 5003, 20
    rng = np.random.default_rng(8)
    ids = rng.integers(0, V, N)
    xt, xr = rows_on_gpu(rng.normal(0, 3, (N, V)), "bf16")
    whole = run_score(plan, xt, V, ids, k)
    for a, b in zip(whole, run_score(plan, xt, V, ids, k)):
        assert np.array_equal(a, b)
    cuts = [0, 1, N // 3 + 1, (2 * N) // 3 + 5, N]
    for a, b in zip(cuts[:-1], cuts[1:]):
        part = run_score(plan, xt[a:b], V, ids, k, row0=a, n=b - a)
        own = ((pred >= a) & (pred < b)) | ((pred < 0) & (np.arange(N) >= a) & (np.arange(N) < b))
        close(part[0][own], whole[0][own], "chunk logp")
        assert (part[0][~own] == -7.0).all()
        assert np.array_equal(part[3], whole[3][a:b])
        for i in (1, 2, 4):
            close(part[i], whole[i][a:b], "chunk")
    bare = run_score(plan, xt, V)
    close(bare[1], whole[1], "row_stat alone")
    st = torch.full((N + 3, 2), -7.0, device="cuda")
    plan.token_score(0, N, xt, V, st)
    assert (st[N:] == -7.0).all()
    close(st[:N].cpu().numpy(), whole[1], "row_stat, no entropy")
    plan.token_score(N, 0, xt[:0], V, st)            # no rows: nothing to do
    plan.sync()


def test_score_bad_ids_and_refusals(lib):
    plan = chain_plan(lib, 40)
    N, V = 40, 300
    rng = np.random.default_rng(1)
    xt, xr = rows_on_gpu(rng.normal(0, 3, (N, V)), "f32")
    ids = rng.integers(0, V, N)
    pred = np.arange(-1, N - 1)
    bad = ids.copy()
    bad[5], bad[9] = V, -1
    logp, stat, H, _, _ = run_score(plan, xt, V, bad)
    with pytest.raises(lib.OctoError) as e:
        plan.sync()
    assert e.value.code == lib.EINVAL
    plan.sync()
    ok = np.ones(N, bool)
    ok[[5, 9]] = False
    assert np.isnan(logp[~ok]).all()
    close(logp[ok], ts.score(xr, ids, pred)[0][ok], "the other tokens")
    # a bad id adds nothing to the gradient, nor to its row's sum
    g, gb = rng.normal(size=N), None
    d = torch.zeros_like(xt)
    plan.token_score_bwd(0, N, xt, V, gpu(stat), None, gpu(bad, torch.int32), gpu(g), None, d)
    with pytest.raises(lib.OctoError):
        plan.sync()
    gb = g.astype(np.float32).astype(np.float64)
    gb[[5, 9]] = 0.0
    close(d[:, :V].cpu().numpy(), ts.score_bwd(xr, ids, pred, gb, None), "gradient")

    st, f, i = torch.zeros((N, 2), device="cuda"), torch.zeros(N, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda")
    top = torch.zeros((N, 129), dtype=torch.int32, device="cuda"), torch.zeros((N, 129), device="cuda")

    def refused(**kw):
        a = dict(row0=0, n_rows=N, logits=xt, vocab=V, row_stat=st)
        a.update(kw)
        with pytest.raises((lib.OctoError, ValueError)):
            plan.token_score(**a)

    refused(row0=1)
    refused(row0=-1)
    refused(n_rows=N + 1)
    refused(n_rows=-1)
    refused(vocab=0)
    refused(vocab=xt.shape[1] + 1)
    refused(ids=i)
    refused(logp=f)
    refused(inv_temp=0.0)
    refused(inv_temp=float("nan"))
    refused(inv_temp=float("inf"))
    refused(top_ids=top[0], top_logp=top[1])                        # k > 128
    refused(vocab=4, top_ids=top[0][:, :5].contiguous(), top_logp=top[1][:, :5].contiguous())
    refused(top_ids=top[0])
    refused(row_stat=st[:1])
    refused(logits=xt[:, 1:])                                       # rows off the 16-byte boundaries
    refused(logits=torch.zeros((N, V + 1), device="cuda"))          # pitch of no whole vectors
    refused(logits=xt.half())
    for a in (dict(entropy=None), dict(ids=None), dict(dlogits=d[:, 1:]), dict(dlogits=d.bfloat16()), dict(row_stat=None)):
        b = dict(row0=0, n_rows=N, logits=xt, vocab=V - 1, row_stat=st, entropy=f, ids=i, g_logp=f, g_entropy=f, dlogits=d)
        b.update(a)
        with pytest.raises((lib.OctoError, ValueError)):
            plan.token_score_bwd(**b)
    plan.sync()


def test_many_rows_a_cta(lib):
    """Dozens of rows for each CTA: slots, barriers and buffers go round many times."""
    n, V, k = 8000, 20011, 9
    plan = decode_plan(lib, n)
    g = torch.Generator(device="cuda").manual_seed(5)
    xt = torch.empty((n, 20016), dtype=torch.bfloat16, device="cuda").normal_(0, 3, generator=g)
    xt[:, V:] = float("nan")
    x = xt[:, :V].double()
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    lp = torch.log_softmax(x, 1)
    H = -(lp.exp() * lp).sum(1)
    for kk in (0, k):
        logp, stat, ent, ti, tl = run_score(plan, xt, V, ids.cpu().numpy(), kk)
        plan.sync()
        close(stat.sum(1), torch.logsumexp(x, 1).cpu().numpy(), "lse")
        close(ent, H.cpu().numpy(), "entropy")
        close(logp, lp.gather(1, ids[:, None])[:, 0].cpu().numpy(), "logp")
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    assert np.array_equal(ti, i[:, :k].cpu().numpy())
    w = torch.rand(n, generator=g, device="cuda") * (torch.rand(n, generator=g, device="cuda") < 0.8)
    t_lp = torch.log_softmax(x + 0.3 * torch.randn(x.shape, generator=g, device="cuda"), 1)
    val, at = torch.topk(t_lp, k, dim=1)
    P = val.exp()
    inside = torch.zeros_like(x, dtype=torch.bool).scatter_(1, at, True)
    q = lp.exp()
    for tail in (False, True):
        lnP = val if tail else val - torch.logsumexp(val, 1, keepdim=True)
        P = lnP.exp()
        R = (1 - P.sum(1)) if tail else torch.zeros(n, device="cuda", dtype=torch.float64)
        qR = q.masked_fill(inside, 0).sum(1)
        kl = (P * (lnP - lp.gather(1, at))).sum(1) + torch.where(R > 0, R * (R.log() - qR.log()), 0.0)
        d = q * (P.sum(1) + R)[:, None] - (R / qR)[:, None] * q.masked_fill(inside, 0)
        d = d.scatter_add(1, at, -P) * w[:, None].double()
        live = (w != 0).cpu().numpy()
        got_kl, _, got = run_distill(plan, xt, V, at.cpu().numpy(), val.cpu().numpy().astype(np.float32), w.cpu().numpy(), 1.0, tail, "sep")
        plan.sync()
        close(got_kl, np.where(live, kl.cpu().numpy(), 0.0), "row_kl", scale=5.0)
        close(got[:, :V], d.cpu().numpy(), "dlogits", True, scale=2.0)


@pytest.mark.parametrize("tail", [False, True])
def test_first_calls_equal_later_ones(lib, tail):
    """A kernel's start on inputs that no cache holds: slots of the ring given back before the
    loads of them were served would hold the data of a later stage here and there."""
    n, V, k = 1200, 151936, 64
    plan = decode_plan(lib, n)
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        xt = torch.empty((n, V), dtype=torch.bfloat16, device="cuda").normal_(0, 3, generator=g)
        ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(16)]).repeat(n // 16, 1).to(torch.int32)
        val = torch.randn((n, k), generator=g, device="cuda") - (6 if tail else 0)
        tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
        d = torch.empty_like(xt)
        torch.cuda.synchronize()
        got = []
        for _ in range(3):
            kl, logp, st = (torch.zeros(s, device="cuda") for s in (n, n, (n, 2)))
            ti, tl = torch.zeros((n, k), dtype=torch.int32, device="cuda"), torch.zeros((n, k), device="cuda")
            plan.distill_topk(0, n, xt, V, ids, val, kl, tail=tail, inv_temp=0.5, dlogits=d)
            plan.token_score(0, n, xt, V, st, ids=tok, logp=logp, top_ids=ti, top_logp=tl)
            got.append((kl, d.clone(), st, logp, ti, tl))
        plan.sync()
        for a in got[1:]:
            assert all(torch.equal(x, y) for x, y in zip(a, got[0]))
        del xt, d, got


# ---- gradient ----

@pytest.mark.parametrize("dtype,V,c", [("f32", 997, 1.0), ("bf16", 1037, 0.5), ("bf16", 4096, 1.0), ("f32", 4097, 1.7), ("f32", 3, 1.0)])
@pytest.mark.parametrize("seed", [5, 19])
def test_score_bwd_random_dags(lib, dtype, V, c, seed):
    ep = synth.random_dag(seed, page_size=16, max_segments=16, max_len=300)
    pool, plan, pred = _plans(lib, ep)
    N = plan.info["n_rows"]
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, V, N)
    xt, xr, stat, H = check_score(plan, pred, rng.normal(0, 3, (N, V)), dtype, ids, 0, c)
    gl = rng.uniform(-1, 1, N).astype(np.float32)
    gh = rng.uniform(-1, 1, N).astype(np.float32)
    gl[rng.random(N) < 0.2] = 0
    bf = dtype == "bf16"
    for l, h in ((gl, gh), (gl, None), (None, gh), (None, None)):
        d = torch.full_like(xt, -7.0)
        plan.token_score_bwd(0, N, xt, V, gpu(stat), gpu(H), gpu(ids, torch.int32), gpu(l), gpu(h), d, inv_temp=c)
        got = d.float().cpu().numpy()
        assert (got[:, V:] == -7.0).all()
        # a row feeds up to a few tokens and p (ln p + H) stays below ~ max(H, 1) p: scale 4
        close(got[:, :V], ts.score_bwd(xr, ids, pred, l, h, c), "dlogits", bf, scale=4.0)
    both = torch.full_like(xt, -7.0)
    plan.token_score_bwd(0, N, xt, V, gpu(stat), gpu(H), gpu(ids, torch.int32), gpu(gl), gpu(gh), both, inv_temp=c)
    cut = N // 2
    part = torch.full_like(xt, -7.0)
    for a, b in ((0, cut), (cut, N)):
        plan.token_score_bwd(a, b - a, xt[a:b], V, gpu(stat[a:b]), gpu(H[a:b]), gpu(ids, torch.int32), gpu(gl), gpu(gh[a:b]), part[a:b],
                             inv_temp=c)
    assert torch.equal(part, both)
    pads = xt[:, V:].clone()
    plan.token_score_bwd(0, N, xt, V, gpu(stat), gpu(H), gpu(ids, torch.int32), gpu(gl), gpu(gh), xt, inv_temp=c)   # in place
    assert torch.equal(xt[:, :V], both[:, :V]) and torch.equal(xt[:, V:].isnan(), pads.isnan())
    plan.sync()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(1, 1), (1, 151936), (3, 50001), (257, 9001)])
def test_score_bwd_sizes_and_masks(lib, dtype, n, V):
    rng = np.random.default_rng(V)
    x = rng.normal(0, 3, (n, V))
    if V > 1:
        x[rng.random((n, V)) < 0.5] = -np.inf
    x[n // 2, 1:] = -np.inf                           # one entry left: its gradient is zero
    if n > 2:
        x[0] = -np.inf
        x[1] = rng.normal(3000, 3, V)                 # far from zero
    plan = decode_plan(lib, n)
    ids = rng.integers(0, V, n)
    xt, xr = rows_on_gpu(x, dtype)
    _, stat, H, _, _ = run_score(plan, xt, V, ids)
    gl, gh = rng.uniform(-1, 1, n).astype(np.float32), rng.uniform(-1, 1, n).astype(np.float32)
    d = torch.full_like(xt, -7.0)
    plan.token_score_bwd(0, n, xt, V, gpu(stat), gpu(H), gpu(ids, torch.int32), gpu(gl), gpu(gh), d)
    plan.sync()
    close(d[:, :V].float().cpu().numpy(), ts.score_bwd(xr, ids, np.arange(n), gl, gh), "dlogits", dtype == "bf16", scale=4.0)


# ---- distillation ----

def teacher(rng, n, V, k, tail):
    """Entries in no order, some empty, some repeated; rows with none."""
    ids = rng.integers(0, V, (n, k))
    ids[rng.random((n, k)) < 0.15] = -1
    val = rng.normal(0, 2, (n, k))
    val[rng.random((n, k)) < 0.1] = -np.inf
    if tail:
        val = np.log(rng.dirichlet(np.ones(k + 1), n)[:, :k]) + np.where(np.isinf(val), val, 0.0)
    if n > 4:
        ids[3] = -1
        val[4] = -np.inf
    return ids.astype(np.int32), val.astype(np.float32)


def run_distill(plan, xt, V, ids, val, w, c, tail, grad, gs=1.0, row0=0, n=None):
    N = plan.info["n_rows"]
    n = N - row0 if n is None else n
    kl = torch.full((N,), -7.0, device="cuda")
    loss = torch.full((1,), -7.0, device="cuda")
    ws = torch.full((max(plan.distill_topk_workspace_size(n), 1),), 255, dtype=torch.uint8, device="cuda")
    d = None if grad is None else xt if grad == "inplace" else torch.full_like(xt, -7.0)
    plan.distill_topk(row0, n, xt, V, gpu(ids, torch.int32), gpu(val), kl, ws, weight=gpu(w), tail=tail, inv_temp=c, dlogits=d, grad_scale=gs,
                      loss=loss)
    return kl.cpu().numpy(), loss.item(), None if d is None else d.float().cpu().numpy()


def check_distill(plan, x, dtype, ids, val, w, c, tail, gs=1.0):
    N, V = x.shape
    xt, xr = rows_on_gpu(x, dtype)
    kl, loss, d = run_distill(plan, xt, V, ids, val, w, c, tail, "sep", gs)
    plan.sync()
    rkl, rloss, rd = ts.distill(xr, ids, val, w, c, tail, gs)
    # P_R = 1 - sum of up to 128 fp32 terms: off by up to 2^-24 * 10, times |ln| up to ~60
    close(kl, rkl, "row_kl", scale=5.0)
    fin = np.isfinite(rkl)
    if fin.all():
        close([loss], [rloss], "loss", scale=5.0 * N)
    close(d[:, :V], rd, "dlogits", dtype == "bf16", scale=2.0)
    assert (d[:, V:] == -7.0).all()
    kl2, loss2, _ = run_distill(plan, xt, V, ids, val, w, c, tail, None)
    close(kl2, rkl, "row_kl without a gradient", scale=5.0)
    kl3, loss3, d3 = run_distill(plan, xt, V, ids, val, w, c, tail, "inplace", gs)
    assert np.array_equal(kl3, kl, equal_nan=True) and np.array_equal(d3[:, :V], d[:, :V], equal_nan=True)
    assert np.isnan(d3[:, V:]).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V,k,c", [("f32", 997, 7, 1.0), ("bf16", 1037, 20, 0.5), ("bf16", 4096, 128, 1.0), ("f32", 4097, 1, 1.7),
                                         ("f32", 40, 128, 1.0), ("bf16", 9, 64, 1.0)])
def test_distill_random_dags(lib, dtype, V, k, c, tail):
    ep = synth.random_dag(11, page_size=16, max_segments=16, max_len=300)
    pool, plan, _ = _plans(lib, ep)
    N = plan.info["n_rows"]
    rng = np.random.default_rng(V + k)
    ids, val = teacher(rng, N, V, k, tail)
    w = rng.uniform(-1, 1, N).astype(np.float32)
    w[rng.random(N) < 0.2] = 0.0
    check_distill(plan, rng.normal(0, 3, (N, V)), dtype, ids, val, w, c, tail, 0.5)
    check_distill(plan, rng.normal(0, 3, (N, V)), dtype, ids, val, None, c, tail)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,k", [(1, 1, 1), (1, 151936, 64), (2, 50001, 128), (19, 32003, 8), (170, 5000, 20), (400, 513, 3), (3, 300007, 9)])
def test_distill_sizes(lib, dtype, n, V, k, tail):
    rng = np.random.default_rng(n + V)
    plan = decode_plan(lib, n)
    ids, val = teacher(rng, n, V, k, tail)
    check_distill(plan, rng.normal(0, 3, (n, V)), dtype, ids, val, None, 1.0, tail)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_masks(lib, dtype, tail):
    """Students masked at listed ids (an infinite divergence with a finite gradient), at all
    others (the rest drops out), everywhere; far offsets; lists of one id; teacher = student."""
    V, k = 2003, 16
    rng = np.random.default_rng(7)
    n = 9
    x = rng.normal(0, 3, (n, V))
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(n)]).astype(np.int32)
    val = (np.log(rng.dirichlet(np.ones(k + 1), n)[:, :k]) if tail else rng.normal(0, 2, (n, k))).astype(np.float32)
    x[0, ids[0, 2]] = -np.inf
    keep = np.zeros(V, bool)
    keep[ids[1]] = True
    x[1, ~keep] = -np.inf
    x[2] = -np.inf
    x[3] += 4000
    ids[4] = ids[4, 0]
    x[5, ids[5]] = -np.inf                             # no listed id has mass
    x[6, 0] = 80.0                                     # almost all of the mass on one id, outside
    ids[7] = np.argsort(-x[7], kind="stable")[:k]
    x[7, ids[7, 0]] = 80.0                             # and inside the list
    check_distill(decode_plan(lib, n), x, dtype, ids, val, None, 1.0, tail)


@pytest.mark.parametrize("noise", [0.0, 1e-5, 1e-3, 0.1, 0.7])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_distill_of_a_student_near_its_teacher(lib, dt, noise):
    """With the rest class the error of a divergence falls with the divergence: an error e of a
    class's d = ln P - ln q is felt as P |d| e + P e^2.  e: two roundings (2^-24) of ln P, of ln q and
    of the numbers up to 2 that they are made of."""
    N, V, k = 48, 3001, 20
    plan = chain_plan(lib, N)
    rng = np.random.default_rng(7)
    xt, xr = rows_on_gpu(rng.normal(0, 3, (N, V)), dt)
    z = xr + noise * rng.normal(size=(N, V))
    z = z - np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) - z.max(1, keepdims=True)
    ids = np.argsort(-z, axis=1)[:, :k].copy()
    ids[3, 1] = ids[3, 0] = -1                                      # empty entries: their mass is the rest's
    val = np.take_along_axis(z, np.maximum(ids, 0), 1).astype(np.float32)
    kl, _, _ = run_distill(plan, xt, V, ids, val, None, 1.0, True, None)
    plan.sync()
    rkl = ts.distill(xr, ids, val, tail=True)[0]
    lq = xr - xr.max(1, keepdims=True)
    lq = lq - np.log(np.exp(lq).sum(1, keepdims=True))
    lqi = np.take_along_axis(lq, np.maximum(ids, 0), 1)
    P = np.where(ids < 0, 0.0, np.exp(val.astype(np.float64)))
    q = np.where(ids < 0, 0.0, np.exp(lqi))
    pr, qr = 1 - P.sum(1), 1 - q.sum(1)
    d, dr = np.abs(val - lqi), np.abs(np.log(pr / qr))
    eps = 2.0 ** -24
    # P_R and q_R are sums of 1 and of exponentials, each good to 4 roundings
    bound = (P * d * 2 * eps * (np.abs(val) + np.abs(lqi) + 2)).sum(1) + dr * 8 * eps + pr * dr * 2 * eps * (np.abs(np.log(qr)) + 4)
    bound = bound + ((2 * eps * (np.abs(val) + np.abs(lqi) + 2)) ** 2 * P).sum(1) + (16 * eps) ** 2 / pr + 16 * eps * rkl
    assert (kl >= 0).all()
    assert (np.abs(kl - rkl) <= bound).all(), np.max(np.abs(kl - rkl) / bound)


def test_distill_refuses_unfit_workspaces(lib):
    """A workspace that its floats cannot be stored in: off a 4-byte boundary, or expanded from
    fewer bytes than it seems to have."""
    N, V, k = 30, 300, 5
    plan = chain_plan(lib, N)
    rng = np.random.default_rng(3)
    xt, _ = rows_on_gpu(rng.normal(0, 3, (N, V)), "f32")
    ids, val = teacher(rng, N, V, k, False)
    ti, tv, f, loss = gpu(ids, torch.int32), gpu(val), torch.zeros(N, device="cuda"), torch.zeros(1, device="cuda")
    need = plan.distill_topk_workspace_size(N)
    big = torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    for ws in (big[1:], big[2:], big[:1].expand(need), big.repeat(2)[::2]):
        with pytest.raises((lib.OctoError, ValueError)):
            plan.distill_topk(0, N, xt, V, ti, tv, f, ws=ws, loss=loss)
    plan.distill_topk(0, N, xt, V, ti, tv, f, ws=big[4:], loss=loss)
    plan.sync()
    torch.cuda.synchronize()
    assert abs(loss.item() - f.double().sum().item()) <= 1e-5 * (1 + abs(loss.item()))



def test_distill_bad_ids_and_refusals(lib):
    N, V, k = 30, 300, 5
    plan = chain_plan(lib, N)
    rng = np.random.default_rng(2)
    xt, xr = rows_on_gpu(rng.normal(0, 3, (N, V)), "f32")
    ids, val = teacher(rng, N, V, k, False)
    bad = ids.copy()
    bad[7, 2], bad[8, 0] = V, 2 ** 31 - 1
    kl, loss, d = run_distill(plan, xt, V, bad, val, None, 1.0, False, "sep")
    with pytest.raises(lib.OctoError) as e:
        plan.sync()
    assert e.value.code == lib.EINVAL
    plan.sync()
    rkl, rloss, rd = ts.distill(xr, bad, val)
    close(kl, rkl, "row_kl", scale=5.0)
    close(d[:, :V], rd, "dlogits", scale=2.0)
    ti, tv, f = gpu(ids, torch.int32), gpu(val), torch.zeros(N, device="cuda")
    ws = torch.zeros(plan.distill_topk_workspace_size(N), dtype=torch.uint8, device="cuda")
    g = torch.zeros_like(xt)

    def refused(**kw):
        a = dict(row0=0, n_rows=N, logits=xt, vocab=V, teach_ids=ti, teach_val=tv, row_kl=f, ws=ws, loss=f[:1].clone())
        a.update(kw)
        with pytest.raises((lib.OctoError, ValueError)):
            plan.distill_topk(**a)

    refused(ws=None)
    refused(ws=ws[:8])
    refused(row0=1)
    refused(n_rows=-1)
    refused(teach_ids=ti[:, :0], teach_val=tv[:, :0])
    refused(teach_ids=ti.long())
    refused(teach_ids=ti[:2])
    refused(teach_ids=ti.repeat(1, 30), teach_val=tv.repeat(1, 30))   # k > 128
    refused(row_kl=f[:3])
    refused(weight=f[:3])
    refused(inv_temp=-1.0)
    refused(dlogits=g[:, 1:])
    refused(dlogits=g.bfloat16())
    plan.sync()
    plan.distill_topk(0, 0, xt, V, ti, tv, f, loss=kl_loss(f), ws=ws)
    plan.sync()


def test_many_successors(lib):
    """A row that 40 branches continue, one that is rewound to again and again; more than 64
    successors are refused where tokens are asked for, and not otherwise."""
    def tree(children):
        pool = lib.Pool(256, 16, 1, 64, lib.DTYPE_BF16)
        r = pool.root()
        pool.append(r, 50)
        for c in pool.fork(r, children):
            pool.append(c, 2)
        a = r
        pool.append(a, 3)
        for _ in range(20):
            a = pool.rewind(a, 1) if pool.seg_info(a)["len"] > 1 else a
            pool.append(a, 2)
        plan = pool.pack_tree([r], 64)
        out = plan.copy_out()
        pred = np.full(plan.info["n_rows"], -1)
        base = {int(s): int(b) for s, b in zip(out["seg_order"], out["seg_row_base"])}
        for s, b in base.items():
            i = pool.seg_info(s)
            pred[b + 1:b + i["len"]] = np.arange(b, b + i["len"] - 1)
            if i["parent"] >= 0 and i["len"]:
                pred[b] = base[i["parent"]] + i["fork"] - 1
        return pool, plan, pred

    pool, plan, pred = tree(40)
    N, V = plan.info["n_rows"], 601
    assert 32 < np.bincount(pred[pred >= 0]).max() <= 64
    rng = np.random.default_rng(6)
    ids = rng.integers(0, V, N)
    bad = ids.copy()
    bad[int(np.nonzero(pred == 49)[0][35])] = V       # one of the fork's
    xt, xr, stat, H = check_score(plan, pred, rng.normal(0, 3, (N, V)), "f32", ids, 4)
    g = rng.uniform(-1, 1, N).astype(np.float32)
    d = torch.zeros_like(xt)
    plan.token_score_bwd(0, N, xt, V, gpu(stat), None, gpu(ids, torch.int32), gpu(g), None, d)
    # up to 41 terms of size 1 in a row
    close(d[:, :V].cpu().numpy(), ts.score_bwd(xr, ids, pred, g, None), "dlogits", scale=40.0)
    run_score(plan, xt, V, bad)
    with pytest.raises(lib.OctoError):
        plan.sync()
    pool, plan, pred = tree(64)
    N = plan.info["n_rows"]
    xt, xr = rows_on_gpu(rng.normal(0, 3, (N, V)), "f32")
    with pytest.raises(lib.OctoError) as e:
        run_score(plan, xt, V, rng.integers(0, V, N))
    assert e.value.code == lib.ENOTSUP
    _, stat, H, _, _ = run_score(plan, xt, V)
    close(H, ts.score(xr, np.zeros(N, int), np.full(N, -1))[2], "entropy")
    plan.sync()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_huge_vocabularies(lib, dtype):
    """A million entries, and a refusal past what the table of listed vectors holds."""
    V, k = 1000003, 20
    rng = np.random.default_rng(12)
    plan = decode_plan(lib, 2)
    x = rng.normal(0, 3, (2, V))
    check_score(plan, np.arange(2), x, dtype, rng.integers(0, V, 2), k)
    ids, val = teacher(rng, 2, V, k, True)
    check_distill(plan, x, dtype, ids, val, None, 1.0, True)
    check_distill(plan, x, dtype, ids, val, None, 1.0, False)
    big = torch.zeros((1, 40000000), dtype=DT[dtype], device="cuda")
    one = decode_plan(lib, 1)
    kl = torch.zeros(1, device="cuda")
    with pytest.raises(lib.OctoError) as e:
        one.distill_topk(0, 1, big, 40000000, gpu(ids[:1], torch.int32), gpu(val[:1]), kl, tail=True)
    assert e.value.code == lib.ENOTSUP
    one.distill_topk(0, 1, big, 40000000, gpu(ids[:1], torch.int32), gpu(val[:1]), kl)
    one.sync()
    # a flat student: ln V plus the teacher's negative entropy
    _, z = ids[0] >= 0, val[0].astype(np.float64)[(ids[0] >= 0) & np.isfinite(val[0])]
    P = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
    close(kl.cpu().numpy(), [np.log(4e7) + (P * np.log(P)).sum()], "row_kl", scale=5.0)


def kl_loss(f):
    return torch.full_like(f[:1], 3.0)


# ---- together ----

def test_teacher_to_student(lib):
    """A distillation step: the teacher's rows scored into their top alternatives, the student
    held to them; gradients against autograd in 64 bits.  Then the same calls captured into a
    graph on another stream and replayed on new logits."""
    ep = synth.random_dag(31, page_size=16, max_segments=12, max_len=120)
    pool, plan, pred = _plans(lib, ep)
    N, V, k, c = plan.info["n_rows"], 2500, 12, 0.8
    rng = np.random.default_rng(4)
    tt, tr = rows_on_gpu(rng.normal(0, 3, (N, V)), "f32")
    st, sr = rows_on_gpu(rng.normal(0, 3, (N, V)), "f32")
    ids = gpu(rng.integers(0, V, N), torch.int32)
    w = rng.uniform(0, 1, N).astype(np.float32)
    wd = gpu(w)
    f = lambda *s: torch.zeros(s, device="cuda")
    logp, stat, H, top, tlp = f(N), f(N, 2), f(N), torch.zeros((N, k), dtype=torch.int32, device="cuda"), f(N, k)
    kl, loss, d1, d2 = f(N), f(1), torch.zeros_like(st), torch.zeros_like(st)
    gl, gh = gpu(rng.normal(size=N)), gpu(rng.normal(size=N))
    ws = torch.empty(plan.distill_topk_workspace_size(N), dtype=torch.uint8, device="cuda")

    def step(stream=None):
        plan.token_score(0, N, tt, V, stat, top_ids=top, top_logp=tlp, inv_temp=c, stream=stream)
        plan.distill_topk(0, N, st, V, top, tlp, kl, ws, weight=wd, tail=True, inv_temp=c, dlogits=d1, loss=loss, stream=stream)
        plan.token_score(0, N, st, V, stat, entropy=H, ids=ids, logp=logp, inv_temp=c, stream=stream)
        plan.token_score_bwd(0, N, st, V, stat, H, ids, gl, gh, d2, inv_temp=c, stream=stream)

    def check(tr, sr):
        x = torch.from_numpy(sr).requires_grad_()
        lp = torch.log_softmax(x * c, 1)
        t = torch.log_softmax(torch.from_numpy(tr) * c, 1)
        at = torch.from_numpy(top.cpu().numpy().astype(np.int64))
        P = torch.exp(t.gather(1, at))
        inside = torch.zeros((N, V), dtype=torch.bool).scatter_(1, at, True)
        R = 1 - P.sum(1)
        qR = torch.exp(lp).masked_fill(inside, 0).sum(1)
        rk = (P * (t.gather(1, at) - lp.gather(1, at))).sum(1) + R * (R.log() - qR.log())
        total = (torch.from_numpy(w).double() * rk).sum()
        g1, = torch.autograd.grad(total, x, retain_graph=True)
        has = torch.from_numpy(pred >= 0)
        r = torch.from_numpy(np.maximum(pred, 0))
        ent = -(lp.exp() * lp).sum(1)
        obj = (gl.cpu().double() * lp[r, ids.cpu().long()])[has].sum() + (gh.cpu().double() * ent).sum()
        g2, = torch.autograd.grad(obj, x)
        close(kl.cpu().numpy(), rk.detach().numpy(), "row_kl", scale=5.0)
        close(loss.cpu().numpy(), [total.item()], "loss", scale=5.0 * N)
        close(d1[:, :V].cpu().numpy(), g1.numpy(), "distillation gradient", scale=2.0)
        close(d2[:, :V].cpu().numpy(), g2.numpy(), "score gradient", scale=8.0)

    step()
    plan.sync()
    check(tr, sr)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side)
    tn, trn = rows_on_gpu(rng.normal(0, 2, (N, V)), "f32")
    sn, srn = rows_on_gpu(rng.normal(0, 4, (N, V)), "f32")
    tt.copy_(tn)
    st.copy_(sn)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check(trn, srn)


def test_score_after_a_decode_step(lib):
    """Serving: the plan of live cursors, advanced by a token, scores the next ones."""
    P, n = 16, 6
    pool = lib.Pool(4 * n, P, 1, 64, lib.DTYPE_BF16)
    cur = [pool.root() for _ in range(n)]
    for i, c in enumerate(cur):
        pool.append(c, 1 + 5 * i)
    plan = pool.decode_plan(cur)
    rng = np.random.default_rng(9)
    for step in range(3):
        check_score(plan, np.arange(n), rng.normal(0, 3, (n, 4001)), "bf16", rng.integers(0, 4001, n), 10)
        pool.append_step(cur)
        plan.advance()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,c", [(2003, 1.0), (2003, 0.5), (50, 1.0), (70001, 1.0)])
def test_distill_rest_outside_64_bits(lib, dtype, V, c):
    """The rest class drops out where no unlisted id has a probability that 64 bits can hold:
    masked with the type's lowest value, a far one, -inf, or several of them; it stays where one
    has, however small."""
    k, n = 8, 9
    low = -3.3895313892515355e38 if dtype == "bf16" else np.finfo(np.float32).min
    rng = np.random.default_rng(V)
    x = rng.normal(0, 1, (n, V))
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(n)]).astype(np.int32)
    val = np.log(rng.dirichlet(np.ones(k + 1), n)[:, :k]).astype(np.float32)
    out = np.ones((n, V), bool)
    np.put_along_axis(out, ids, False, 1)
    for r, far in enumerate([low, -1e30, -9984.0, low, -700.0 / c, -800.0 / c, low, low]):
        x[r, out[r]] = far
    at = np.flatnonzero(out[3])[V // 3]
    x[3, at] = 0.5                                     # one of them lives
    x[6, out[6] & (np.arange(V) % 3 == 0)] = -np.inf
    x[7, ~out[7]] += 5000.0                            # far from zero
    check_distill(decode_plan(lib, n), x, dtype, ids, val, None, c, True)
    # the row masked with the lowest value is the row masked with -inf
    y = x.copy()
    y[x < -1e29] = -np.inf
    a, b = (run_distill(decode_plan(lib, n), rows_on_gpu(z, dtype)[0], V, ids, val, None, c, True, "sep") for z in (x, y))
    for r in (0, 1, 6, 7):
        close(a[0][r], b[0][r], "row_kl", scale=5.0)
        close(a[2][r, :V], b[2][r, :V], "dlogits", dtype == "bf16", scale=2.0)


@pytest.mark.parametrize("branches,goes_on,fits", [(64, False, True), (63, True, True), (65, False, False), (64, True, False)])
def test_most_successors(lib, branches, goes_on, fits):
    """64 successors are taken, whether one of them is the row's own next or all are branches."""
    pool = lib.Pool(256, 16, 1, 64, lib.DTYPE_BF16)
    r = pool.root()
    P = 20
    pool.append(r, P)
    kids = pool.fork(r, branches)
    for c in kids:
        pool.append(c, 2)
    if goes_on:
        pool.append(r, 3)
    plan = pool.pack_tree([r], 64)
    out = plan.copy_out()
    N, V = plan.info["n_rows"], 601
    pred = np.arange(-1, N - 1)
    base = {int(s): int(b) for s, b in zip(out["seg_order"], out["seg_row_base"])}
    pred[base[r]] = -1
    for c in kids:
        pred[base[c]] = base[r] + P - 1
    assert (np.bincount(pred[pred >= 0]).max() <= 64) == fits
    rng = np.random.default_rng(branches)
    ids = rng.integers(0, V, N)
    g = rng.uniform(-1, 1, N).astype(np.float32)
    x = rng.normal(0, 3, (N, V))
    if not fits:
        xt, _ = rows_on_gpu(x, "f32")
        d, st = torch.zeros_like(xt), torch.zeros((N, 2), device="cuda")
        for call in (lambda: run_score(plan, xt, V, ids),
                     lambda: plan.token_score_bwd(0, N, xt, V, st, None, gpu(ids, torch.int32), gpu(g), None, d)):
            with pytest.raises(lib.OctoError) as e:
                call()
            assert e.value.code == lib.ENOTSUP
        return
    xt, xr, stat, _ = check_score(plan, pred, x, "f32", ids, 3)
    d = torch.zeros_like(xt)
    plan.token_score_bwd(0, N, xt, V, gpu(stat), None, gpu(ids, torch.int32), gpu(g), None, d)
    plan.sync()
    # up to 64 terms of size 1 in a row
    close(d[:, :V].cpu().numpy(), ts.score_bwd(xr, ids, pred, g, None), "dlogits", scale=64.0)
    logp = torch.zeros(N, device="cuda")
    ws = torch.empty(plan.token_logprob_workspace_size(N), dtype=torch.uint8, device="cuda")
    plan.token_logprob(0, N, xt, V, gpu(ids, torch.int32), None, logp, ws)
    plan.sync()
    close(logp.cpu().numpy(), ts.score(xr, ids, pred)[0], "token_logprob's")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3001, 12])
def test_score_masked_entries_of_bad_rows(lib, dtype, V):
    """A NaN or +inf logit makes every log-probability of its row NaN, those of entries masked at
    -inf too."""
    k = 8
    rng = np.random.default_rng(V)
    x = np.where(rng.random((7, V)) < 0.6, -np.inf, rng.normal(0, 3, (7, V)))
    x[0, 2] = np.nan
    x[1, 2] = np.inf
    x[2] = -np.inf
    x[2, 5] = np.nan                                   # nothing else: the alternatives are masked ones
    x[3] = -np.inf
    x[3, 5] = np.inf
    x[4] = -np.inf                                     # an empty row is no bad one
    ids = np.zeros(7, int)
    x[:, 0] = -np.inf                                  # every row's token is masked
    plan = decode_plan(lib, 7)
    xt, xr = rows_on_gpu(x, dtype)
    logp, stat, H, ti, tl = run_score(plan, xt, V, ids, k)
    plan.sync()
    assert np.isnan(logp[:4]).all() and np.isnan(tl[:4]).all() and np.isnan(stat[:4, 1]).all() and np.isnan(H[:4]).all()
    assert ti[1, 0] == 2 and ti[3, 0] == 5
    assert np.array_equal(ti[2], [0, 1, 2, 3, 4, 6, 7, 8])
    good = slice(4, 7)
    rl, rs, rH, rti, rtl = ts.score(xr[good], ids[good], np.arange(3), 1.0, k)
    close(logp[good], rl, "logp")
    close(H[good], rH, "entropy")
    assert np.array_equal(ti[good], rti)
    close(tl[good], rtl, "top logp")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_row_against_a_buffer_of_several(lib, dtype):
    """A last chunk of one row: the pitch of a single row matters to nobody."""
    V, k, N = 1001, 6, 5
    plan = chain_plan(lib, N)
    rng = np.random.default_rng(4)
    x = np.full((N, 1104), np.nan)
    x[:, :V] = rng.normal(0, 3, (N, V))
    xt = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).cuda()
    xr = xt[:, :V].double().cpu().numpy()
    ids, val = teacher(rng, N, V, k, False)
    tok = rng.integers(0, V, N)
    g = rng.uniform(-1, 1, N).astype(np.float32)
    stat = gpu(ts.score(xr, tok, np.arange(-1, N - 1))[1])
    want = ts.score_bwd(xr, tok, np.arange(-1, N - 1), g, None)
    _, _, want_d = ts.distill(xr, ids, val)
    kl = torch.zeros(N, device="cuda")
    last = slice(N - 2, N - 1)
    for logits, grad in ((xt[N - 2:], torch.full((1, 1104), -7.0, device="cuda", dtype=DT[dtype])),
                         (xt[last], torch.full((N, 1104), -7.0, device="cuda", dtype=DT[dtype])),
                         (xt[last], torch.full((N, 1208), -7.0, device="cuda", dtype=DT[dtype])),
                         (xt[last].clone(), torch.full((3, 1008), -7.0, device="cuda", dtype=DT[dtype]))):
        plan.token_score_bwd(N - 2, 1, logits, V, stat[last], None, gpu(tok, torch.int32), gpu(g), None, grad)
        close(grad[0, :V].float().cpu().numpy(), want[N - 2], "dlogits", dtype == "bf16", scale=4.0)
        plan.distill_topk(N - 2, 1, logits, V, gpu(ids[last], torch.int32), gpu(val[last]), kl, dlogits=grad)
        close(grad[0, :V].float().cpu().numpy(), want_d[N - 2], "distillation's", dtype == "bf16", scale=2.0)
        assert (grad[0, V:] == -7.0).all() and (grad[1:] == -7.0).all()
    for n in (2, 3):
        with pytest.raises(ValueError):
            plan.token_score_bwd(0, n, xt, V, stat, None, gpu(tok, torch.int32), gpu(g), None, torch.zeros((N, 1208), device="cuda", dtype=DT[dtype]))
    plan.sync()


@pytest.mark.parametrize("n", [1, 900, 5000])
def test_losses_of_calls_in_a_row(lib, n):
    """Calls that follow one another on one workspace, each sum of row losses started while the rows
    are still in work: every loss is that of its own call's rows, launched and replayed."""
    V, k, calls = 640, 3, 24
    plan = chain_plan(lib, n)
    g = torch.Generator(device="cuda").manual_seed(n)
    xt = torch.randn((n, V), generator=g, device="cuda")
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(n)]).to(torch.int32)
    val = torch.randn((n, k), generator=g, device="cuda")
    tok = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((calls, n), generator=g, device="cuda") * torch.arange(1, calls + 1, device="cuda")[:, None]
    kl, logp = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    ws = torch.empty(plan.distill_topk_workspace_size(n), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(plan.token_logprob_workspace_size(n), dtype=torch.uint8, device="cuda")
    loss, loss2 = torch.zeros((calls, 1), device="cuda"), torch.zeros((calls, 1), device="cuda")

    def run(stream=None):
        for i in range(calls):
            plan.distill_topk(0, n, xt, V, ids, val, kl, ws, weight=w[i], loss=loss[i], stream=stream)
            plan.token_logprob(0, n, xt, V, tok, w[i], logp, ws2, loss=loss2[i], stream=stream)

    def check():
        torch.cuda.synchronize()
        # n / 1024 + 10 fp32 additions of a sum, and the roundings of a row's loss
        for got, row in ((loss, kl.double()), (loss2, -logp.double())):
            want = (w.double() * row).sum(1)
            bound = (n / 1024 + 14) * 2.0 ** -24 * (w.double() * row.abs()).sum(1)
            assert ((got[:, 0].double() - want).abs() <= bound + 1e-30).all()

    run()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(side)
    for s in (2.0, 0.5):
        w.mul_(s)
        xt.mul_(0.9)
        graph.replay()
        check()
    plan.sync()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("c", [1.0, 0.7])
def test_distill_gradient_of_far_logits(lib, c, tail):
    """Logits of 20,000 to 60,000: their exponents in base 2 are rounded by up to 2^-8, which the
    gradient takes out again to the last bit; counted twice it would be 2e-3 of every entry."""
    n, V, k = 40, 70, 4
    rng = np.random.default_rng(11)
    x = rng.normal(0, 2, (n, V)) + rng.uniform(20000, 60000, (n, 1))
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(n)]).astype(np.int32)
    val = (np.log(rng.dirichlet(np.ones(k + 1), n)[:, :k]) if tail else rng.normal(0, 2, (n, k))).astype(np.float32)
    check_distill(decode_plan(lib, n), x, "f32", ids, val, None, c, tail)


@pytest.mark.parametrize("c", [1.0, 0.7])
@pytest.mark.parametrize("V,k", [(20001, 0), (20001, 9), (300007, 0)])
def test_score_rising_far_logits(lib, V, k, c):
    """Rows that rise to the end, far from zero: every thread's reference moves again and again,
    by differences of rounded products."""
    n = 24
    rng = np.random.default_rng(V)
    x = np.linspace(0, 200, V)[None] + rng.uniform(20000, 60000, (n, 1)) + rng.normal(0, 0.1, (n, V))
    check_score(decode_plan(lib, n), np.arange(n), x, "f32", rng.integers(V - 100, V, n), k, c)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_distill_repeated_ids_are_one_class(lib, dtype, tail):
    """A list with ids repeated equals the list with their probabilities added up by hand, and the
    divergence from a student that has learnt it is 0."""
    N, V, m, c = 40, 1203, 6, 0.8
    plan = chain_plan(lib, N)
    rng = np.random.default_rng(21)
    x = rng.normal(0, 3, (N, V))
    one = np.stack([rng.choice(V, m, replace=False) for _ in range(N)]).astype(np.int32)
    parts = rng.dirichlet(np.ones(4 * m + 1), N)[:, :4 * m].reshape(N, m, 4)   # four shares of each id
    parts[:, 0, 1:] = 0.0                              # an id listed once
    parts[:, 1, 2] = 0.0                               # an entry that is empty
    q = np.repeat(one, 4, 1)
    with np.errstate(divide="ignore"):
        val = np.log(parts).reshape(N, 4 * m) / (1.0 if tail else c)
        whole = np.log(parts.sum(2)) / (1.0 if tail else c)
    mix = np.stack([rng.permutation(4 * m) for _ in range(N)])
    q, val = np.take_along_axis(q, mix, 1), np.take_along_axis(val, mix, 1).astype(np.float32)
    x[0] = -200.0                                      # the student is the teacher
    x[0, one[0]] = whole[0] / (c if tail else 1.0)
    if tail:
        rest = 1 - np.exp(whole[0]).sum()
        x[0, np.setdiff1d(np.arange(V), one[0])] = np.log(rest / (V - m)) / c
    xt, xr = rows_on_gpu(x, dtype)
    kl, _, d = run_distill(plan, xt, V, q, val, None, c, tail, "sep")
    kl1, _, d1 = run_distill(plan, xt, V, one, whole.astype(np.float32), None, c, tail, "sep")
    plan.sync()
    close(kl, kl1, "row_kl", scale=5.0)
    close(d[:, :V], d1[:, :V], "dlogits", dtype == "bf16", scale=2.0)
    assert (kl >= -5e-5).all() and (dtype == "bf16" or abs(kl[0]) < 5e-5)
    # by the formula, without the reference
    lp = xr * c - (xr * c).max(1, keepdims=True)
    lp = lp - np.log(np.exp(lp).sum(1, keepdims=True))
    P = parts.sum(2) if tail else parts.sum(2) / parts.sum((1, 2))[:, None]
    want = (P * (np.log(P) - np.take_along_axis(lp, one, 1))).sum(1)
    if tail:
        R, qR = 1 - P.sum(1), 1 - np.exp(np.take_along_axis(lp, one, 1)).sum(1)
        want = want + R * np.log(R / qR)
    close(kl, want, "row_kl by the formula", scale=5.0)


@pytest.mark.parametrize("dtype,fits,past", [("f32", 2900000, 2930000), ("bf16", 5800000, 5840000)])
def test_distill_rest_up_to_the_largest_vocabulary(lib, dtype, fits, past):
    """The rest class at the sizes that the header gives: the last that are taken, the first refused."""
    rng = np.random.default_rng(14)
    x = rng.normal(0, 3, (1, fits))
    ids, val = teacher(rng, 1, fits, 40, True)
    ids[0, :3] = [fits - 1, fits - 9, 0]
    plan = decode_plan(lib, 1)
    check_distill(plan, x, dtype, ids, val, None, 1.0, True)
    big, kl = torch.zeros((1, past), dtype=DT[dtype], device="cuda"), torch.zeros(1, device="cuda")
    with pytest.raises(lib.OctoError) as e:
        plan.distill_topk(0, 1, big, past, gpu(ids, torch.int32), gpu(val), kl, tail=True)
    assert e.value.code == lib.ENOTSUP
    plan.sync()
