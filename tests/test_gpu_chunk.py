"""GPU parity of octo_chunk_attn (whole contexts, sliding windows with sinks) against the oracle's
row contexts and a softmax in fp64, and a speculative step of the chunk calls together.

Tolerances, with A = sum p |v| of the row in fp64.  fp32: scores are inner products of at most 128
terms and exponents of at most ~40 (2^-24 each, relative), sums of at most some thousand positive
terms: below 2^-16 of A together, 2^-15 allowed.  bf16: besides, the probabilities are rounded before the product with V
(2^-8 of A) and the output once (2^-8 of it).  lse: an exponent's error, 2^-16 (1 + |lse|)."""
import math

import numpy as np
import pytest

import synth
from helpers import pool_pages_needed, replay_device

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


class Case:
    """An episode in the library's pool and in the oracle, and the rows of a chunk plan."""

    def __init__(self, lib, oracle_mod, ep, G, Hkv, d, dtype, seed=0, scale=1.0):
        self.lib, self.ep, self.G, self.Hkv, self.d, self.dtype = lib, ep, G, Hkv, d, dtype
        t = synth.make_tensors(ep, G * Hkv, Hkv, d, dtype, scale, seed, with_do=False)
        self.t, P = t, ep.page_size
        npages = pool_pages_needed(ep)
        self.kp = torch.zeros((npages, Hkv, P, d), dtype=DT[dtype], device="cuda")
        self.vp = torch.zeros_like(self.kp)
        self.pool = lib.Pool(npages, P, Hkv, d, lib.DTYPE_BF16 if dtype == "bf16" else lib.DTYPE_F32, self.kp, self.vp)
        replay_device(self.pool, ep, torch.from_numpy(t.K).cuda().to(DT[dtype]), torch.from_numpy(t.V).cuda().to(DT[dtype]))
        self.orc = oracle_mod.Oracle(P, npages, Hkv, d)
        self.orc.replay(ep, t.K.astype(np.float64), t.V.astype(np.float64))
        self.K, self.V = t.K.astype(np.float64), t.V.astype(np.float64)
        self.plan = self.orc.pack(ep.roots, 32)
        self.base = {int(s): int(b) for s, b in zip(self.plan.seg_order, self.plan.seg_row_base)}
        seg, idx = self.orc.token_owner()
        pos = {s: self.orc.seg_pos(s) for s in range(ep.n_segments)}
        self.tok_pos = np.array([pos[s][i] for s, i in zip(seg, idx)])

    def queries(self, cursors, n_new, seed):
        n = int(sum(n_new))
        q = np.random.default_rng(seed).standard_normal((n, self.G * self.Hkv, self.d)).astype(np.float32)
        return torch.from_numpy(q).cuda().to(DT[self.dtype])

    def reference(self, cursors, n_new, q, scale, window, sink):
        """out, lse and sum p |v| in fp64."""
        q = q.float().cpu().numpy().astype(np.float64)
        o, a, lse = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2])
        r = 0
        for c, n in zip(cursors, n_new):
            for i in range(self.ep.length[c] - n, self.ep.length[c]):
                row = self.base[c] + i
                tok, _ = self.plan.row_context(row)
                if window:
                    p = self.tok_pos[tok]
                    tok = tok[(p > self.plan.row_pos[row] - window) | (p < sink)]
                k, v = self.K[tok], self.V[tok]                      # [tokens][kv heads][d]
                x = scale * np.einsum("ghd,ngd->ghn", q[r].reshape(self.Hkv, self.G, -1), k)
                L = np.logaddexp.reduce(x, axis=2)
                w = np.exp(x - L[:, :, None])
                lse[r] = L.reshape(-1)
                o[r] = np.einsum("ghn,ngd->ghd", w, v).reshape(o[r].shape)
                a[r] = np.einsum("ghn,ngd->ghd", w, np.abs(v)).reshape(a[r].shape)
                r += 1
        return o, lse, a

    def run(self, plan, q, scale, **kw):
        out = torch.full_like(q, float("nan"))
        lse = torch.full(q.shape[:2], float("nan"), device="cuda")
        ws = torch.full((max(1, plan.chunk_attn_workspace_size()),), 255, dtype=torch.uint8, device="cuda")
        plan.chunk_attn(q, out, lse, scale, ws, **kw)
        plan.sync()
        return out, lse

    def check(self, cursors, n_new, window=0, sink=0, seed=1):
        scale = 1 / math.sqrt(self.d)
        q = self.queries(cursors, n_new, seed)
        plan = self.pool.chunk_plan(cursors, n_new, self.G * self.Hkv, window=window, n_sink=sink)
        assert plan.info["n_rows"] == sum(n_new) and plan.info["n_segments"] == len(cursors) and plan.info["is_decode"] == 2
        out, lse = self.run(plan, q, scale)
        o, L, a = self.reference(cursors, n_new, q, scale, window, sink)
        close(out, lse, o, L, a, self.dtype)
        return plan, q, out, lse


def close(out, lse, o, L, a, dtype):
    out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    tol = 2.0 ** -15 * a + 1e-7
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (a + np.abs(o))
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    assert np.all(np.abs(out - o) <= tol), "out: %g over" % (np.abs(out - o) - tol).max()
    assert np.all(np.abs(lse - L) <= 2.0 ** -16 * (1 + np.abs(L))), "lse: %g" % np.abs(lse - L).max()


def live(case):
    return [s for s in range(case.ep.n_segments) if case.ep.length[s] > 0 and not case.orc.seg_info(s)["flags"] & 16]


SHAPES = [  # group, kv heads, head_dim, page, type
    (4, 4, 128, 64, "bf16"), (1, 2, 128, 64, "bf16"), (8, 1, 64, 32, "bf16"), (3, 2, 128, 16, "bf16"), (5, 1, 64, 128, "bf16"),
    (2, 2, 64, 24, "bf16"), (3, 2, 64, 16, "f32"), (4, 1, 128, 64, "f32"), (1, 1, 64, 128, "f32"), (2, 1, 128, 48, "f32"),
    (16, 1, 64, 8, "f32"), (2, 1, 64, 100, "bf16"),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("window,sink", [(0, 0), (1, 0), (37, 0), (90, 70), (64, 5), (100000, 3)])
def test_random_trees(lib, oracle_mod, shape, window, sink):
    G, Hkv, d, P, dtype = shape
    seed = 100 * SHAPES.index(shape) + window % 97
    ep = synth.random_dag(seed, page_size=P, max_segments=12, max_len=220, n_roots=2)
    c = Case(lib, oracle_mod, ep, G, Hkv, d, dtype, seed)
    rng = np.random.default_rng(seed)
    cur = live(c)
    n_new = [int(rng.integers(0, min(ep.length[s], 150) + 1)) for s in cur]
    n_new[0] = ep.length[cur[0]]
    c.check(cur, n_new, window, sink, seed)


def chain(P, *lens):
    ep = synth.Episode(P)
    c = ep.root()
    for n in lens[:-1]:
        ep.append(c, n)
        c = ep.fork(c, 1)[0]
    ep.append(c, lens[-1])
    return ep, c


@pytest.mark.parametrize("dtype,P", [("bf16", 64), ("f32", 16)])
@pytest.mark.parametrize("n", [1, 2, 5, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_chunk_lengths(lib, oracle_mod, dtype, P, n):
    """Around the ends of tiles, query groups and blocks; the first token of a root alone."""
    ep, c = chain(P, n)
    Case(lib, oracle_mod, ep, 4, 2, 128, dtype).check([c], [n])
    ep, c = chain(P, 130, n)
    Case(lib, oracle_mod, ep, 4, 2, 128, dtype).check([c], [n], window=70, sink=3)


@pytest.mark.parametrize("G,Hkv,d,P,dtype", [(128, 1, 128, 64, "bf16"), (127, 1, 64, 32, "bf16"), (65, 1, 128, 128, "bf16"), (33, 2, 64, 16, "f32")])
def test_many_heads_a_kv_head(lib, oracle_mod, G, Hkv, d, P, dtype):
    """Tiles of one, two or three tokens."""
    ep, c = chain(P, 150, 9)
    case = Case(lib, oracle_mod, ep, G, Hkv, d, dtype)
    case.check([c, 0], [5, 3])
    case.check([c], [9], window=70, sink=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_context_is_split_and_joined(lib, oracle_mod, dtype):
    ep, c = chain(64, 5000, 1100, 7)
    case = Case(lib, oracle_mod, ep, 4, 1, 128, dtype)
    plan, q, out, lse = case.check([c], [7])
    assert plan.chunk_attn_workspace_size() > 0
    again, lse2 = case.run(plan, q, 1 / math.sqrt(128))      # a workspace of other content: the same bits
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mounts_inside_a_chunk(lib, oracle_mod, dtype):
    """Spans mounted between the chunk's own rows, also twice in one block, one at a longer position."""
    ep = synth.Episode(64)
    r = ep.root()
    ep.append(r, 50)
    a, b, e = ep.fork(r, 3)
    ep.append(a, 300)
    ep.append(e, 90)
    ep.append(b, 10)
    ep.mount(b, a, 3, 70)
    ep.append(b, 7)
    ep.mount(b, e, 0, 90)
    ep.append(b, 100)
    case = Case(lib, oracle_mod, ep, 4, 2, 128, dtype)
    for n in (117, 110, 107, 101, 100, 1):
        case.check([b], [n])
        case.check([b], [n], window=80, sink=20)
        case.check([b], [n], window=12)


def forest(P):
    """Two prompts; forks of forks, one before its parent went on and one after, a rewound one, a parent with a mount that only its
    later children see."""
    ep = synth.Episode(P)
    leaves = []
    for n in (600, 1300):
        r = ep.root()
        ep.append(r, n)
        kids = ep.fork(r, 3)
        for i, k in enumerate(kids):
            ep.append(k, 610 + 100 * i)
        early = ep.fork(kids[0], 2)
        ep.append(kids[0], 30)
        ep.mount(kids[0], kids[2], 20, 640)
        ep.append(kids[0], 9)
        late = ep.fork(kids[0], 3)
        for k in early + late + ep.fork(kids[1], 9):
            ep.append(k, 3 + k % 5)
            leaves.append(k)
        cont = ep.rewind(kids[2], 600)
        ep.append(cont, 4)
        leaves.append(cont)
    return ep, leaves


@pytest.mark.parametrize("dtype,P,G", [("bf16", 64, 4), ("f32", 16, 2), ("bf16", 16, 16)])
def test_shared_prefixes(lib, oracle_mod, dtype, P, G):
    """What neighbouring cursors share is read for all of them: every order of the cursors, chunks that fill a tile among short ones."""
    ep, leaves = forest(P)
    case = Case(lib, oracle_mod, ep, G, 1, 64, dtype)
    scale = 1 / 8
    rng = np.random.default_rng(1)
    for cursors in (leaves, leaves[::-1], [int(x) for x in rng.permutation(leaves)], leaves + leaves[:3] + [1, 1, 2, 0]):
        n_new = [min(ep.length[c], 1 + c % 4) if c > 2 else (200, 3, 90)[c] for c in cursors]
        n_new[3] = 0
        plan, _, _, _ = case.check(cursors, n_new)
        want = sum(len(case.plan.row_context(case.base[c] + i)[0]) for c, n in zip(cursors, n_new)
                   for i in range(ep.length[c] - n, ep.length[c]))
        assert plan.info["pairs"] == want
        case.check(cursors, n_new, window=700, sink=9)


@pytest.mark.parametrize("G,Hkv,d,P", [(4, 8, 128, 64), (1, 8, 64, 32), (3, 8, 128, 16), (8, 8, 64, 128)])
def test_long_chunks(lib, oracle_mod, G, Hkv, d, P):
    """Work for every SM: tiles of twice 128 rows, chunks that end in either half of one beside short ones and empty ones, mounts inside
    chunks, prefixes that short neighbours share, a window that ends inside tiles."""
    T = 128 // G
    ep = synth.Episode(P)
    r = ep.root()
    ep.append(r, 1500)
    leaves = []
    for i, n in enumerate((2 * T, 3 * T + 5, 7 * T - 1, 3, 4, 3 * T, 2 * T + 1, 5 * T)):
        c = ep.fork(r, 1)[0]
        ep.append(c, 40 + i)
        if leaves and i % 3 == 2:
            ep.append(c, n // 2)
            ep.mount(c, leaves[-1], 10, 100 if ep.length[leaves[-1]] >= 100 else ep.length[leaves[-1]])
            ep.append(c, n - n // 2)
        else:
            ep.append(c, n)
        leaves.append(c)
    case = Case(lib, oracle_mod, ep, G, Hkv, d, "bf16")
    n_new = [ep.length[c] - 40 - i for i, c in enumerate(leaves)]
    n_new[3] = 2
    plan, q, out, lse = case.check(leaves, n_new)
    assert plan.info["bm"] == 2 * T
    again, lse2 = case.run(plan, q, 1 / math.sqrt(d))
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    case.check(leaves + [0], n_new + [3 * T], window=1300, sink=70)
    case.check([0], [1500], window=T + 7)


def test_same_cursor_twice_and_empty_plans(lib, oracle_mod):
    ep, c = chain(64, 100, 40)
    case = Case(lib, oracle_mod, ep, 2, 2, 128, "bf16")
    case.check([c, c, 0], [40, 3, 100])
    for cur, n_new in (([], []), ([c], [0])):
        plan = case.pool.chunk_plan(cur, n_new, 4)
        assert plan.info["n_rows"] == 0 and plan.chunk_attn_workspace_size() == 0
        q = torch.zeros((0, 4, 128), dtype=torch.bfloat16, device="cuda")
        plan.chunk_attn(q, q.clone(), None, 1.0)
        plan.sync()


def test_large_scores_and_hidden_values(lib, oracle_mod):
    """Scores of some hundred, a row's maximum moving from block to block; slots that no row may see hold the type's largest values."""
    ep, c = chain(64, 700, 30)
    case = Case(lib, oracle_mod, ep, 4, 1, 128, "bf16")
    case.kp[:, :, :, :] *= 8
    case.K *= 8
    pages = case.pool.seg_pages(c)
    case.kp[pages[-1], :, 30:] = 3e38
    case.vp[pages[-1], :, 30:] = 3e38
    scale = 1 / math.sqrt(128)
    q = case.queries([c], [30], 5) * 4
    plan = case.pool.chunk_plan([c], [30], 4)
    out, lse = case.run(plan, q, scale)
    o, L, a = case.reference([c], [30], q, scale, 0, 0)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    # an exponent of size E = |s| + max |s| carries 2^-24 E per rounding, some eight of them
    s = np.abs(L).max()
    rel = 2.0 ** -20 * s + 2.0 ** -8
    assert np.all(np.abs(out - o) <= rel * (a + np.abs(o)) + 1e-6) and np.all(np.abs(lse - L) <= 2.0 ** -20 * s + 1e-5)


def test_other_stream_other_arrays_and_capture(lib, oracle_mod):
    """A plan used on another stream than it was built on, with arrays of another layer, and from a graph replayed on new queries;
    rows behind the plan's stay as they are."""
    ep, c = chain(64, 900, 12)
    case = Case(lib, oracle_mod, ep, 4, 2, 128, "bf16")
    scale = 1 / math.sqrt(128)
    plan = case.pool.chunk_plan([c], [12], 8)
    q = case.queries([c], [12], 3)
    want, lse_want = case.run(plan, q, scale)
    kp, vp = case.kp.clone(), case.vp.clone()
    case.kp.zero_()
    ws = torch.empty(plan.chunk_attn_workspace_size(), dtype=torch.uint8, device="cuda")
    out, lse = torch.full((14, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((14, 8), 7.0, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan.chunk_attn(q, out, lse, scale, ws, k_pool=kp, v_pool=vp, stream=side)
    side.synchronize()
    assert torch.equal(out[:12], want) and torch.equal(lse[:12], lse_want) and (out[12:] == 7).all() and (lse[12:] == 7).all()
    static = q.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.chunk_attn(static, out, lse, scale, ws, k_pool=kp, v_pool=vp)
    q2 = case.queries([c], [12], 4)
    static.copy_(q2)
    g.replay()
    torch.cuda.synchronize()
    first = out[:12].clone()
    plan.chunk_attn(q2, out, lse, scale, ws, k_pool=kp, v_pool=vp)
    plan.sync()
    assert torch.equal(first, out[:12]) and not torch.equal(first, want)


def test_refusals(lib, oracle_mod):
    ep, c = chain(64, 900, 12)
    case = Case(lib, oracle_mod, ep, 2, 2, 128, "bf16")
    plan = case.pool.chunk_plan([c], [12], 4)
    q = case.queries([c], [12], 3)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    need = plan.chunk_attn_workspace_size()
    assert need > 0
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    for bad in (None, ws[:need - 1].contiguous(), ws[1:]):
        with pytest.raises(lib.OctoError):
            plan.chunk_attn(q, out, lse, 1.0, bad)
    with pytest.raises(ValueError):
        plan.chunk_attn(q.float(), out, lse, 1.0, ws)
    with pytest.raises(ValueError):
        plan.chunk_attn(q[:11], out, lse, 1.0, ws)
    with pytest.raises(ValueError):
        plan.chunk_attn(q.transpose(0, 1), out, lse, 1.0, ws)
    with pytest.raises(ValueError):
        plan.chunk_attn(q, out, lse.half(), 1.0, ws)
    with pytest.raises(ValueError):
        plan.chunk_attn(q.cpu(), out, lse, 1.0, ws)
    with pytest.raises(ValueError):
        plan.chunk_attn(q, out, lse, 1.0, ws, k_pool=case.kp[:1])
    shifted = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    with pytest.raises(lib.OctoError):
        plan.chunk_attn(shifted, out, lse, 1.0, ws)
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        with pytest.raises(lib.OctoError):
            plan.chunk_attn(q, out, lse, scale, ws)
    # other plans and calls
    pack, dec = case.pool.pack_tree(ep.roots, 128), case.pool.decode_plan([c])
    assert pack.chunk_attn_workspace_size() == dec.chunk_attn_workspace_size() == 0
    for other in (pack, dec):
        with pytest.raises(lib.OctoError):
            other.chunk_attn(q, out, lse, 1.0, ws)
        with pytest.raises(lib.OctoError):
            other.verify_drafts_workspace_size(0, 1)
    lse_t = torch.empty((4, 12), device="cuda")
    for call in (lambda: plan.attn_fwd(4, q, out, lse_t, 1.0), lambda: plan.decode(4, q, out, lse, 1.0, ws),
                 lambda: plan.decode_noalloc(4, q, out, lse, 1.0), lambda: plan.advance(),
                 lambda: plan.rope_pool_grad(case.kp.float(), 1e4),
                 lambda: plan.recurrent_fwd(1, 128, *[torch.zeros(12 * 128, device="cuda")] * 6, ws)):
        with pytest.raises(lib.OctoError):
            call()
    got = plan.copy_out()
    assert got["seg_order"].tolist() == [c] and got["seg_row_base"].tolist() == [0] and len(got["entries"]) == 0
    assert np.array_equal(got["row_pos"], case.pool.seg_pos(c)) and got["tile_seg"].tolist() == [c] and got["tile_rows"].tolist() == [12]
    assert plan.recurrent_workspace_size(1, 128) == 0
    plan.sync()


def test_nan_queries_stay_in_their_rows(lib, oracle_mod):
    """A row of NaN beside others of its tile and a NaN key in one cursor's own tokens: the other rows are what they were."""
    ep, leaves = forest(64)
    case = Case(lib, oracle_mod, ep, 4, 1, 128, "bf16")
    cur = leaves[:6]
    n_new = [min(3, ep.length[c]) for c in cur]
    scale = 1 / math.sqrt(128)
    q = case.queries(cur, n_new, 7)
    plan = case.pool.chunk_plan(cur, n_new, 4)
    want, lse = case.run(plan, q, scale)
    q[4] = float("nan")
    out, lse2 = case.run(plan, q, scale)
    keep = torch.arange(len(q), device="cuda") != 4
    assert torch.isnan(out[4].float()).all() and torch.equal(out[keep], want[keep]) and torch.equal(lse2[keep], lse[keep])


def test_layers_of_a_step_share_a_plan_on_two_streams(lib, oracle_mod):
    """One plan, two calls under way at once on other arrays and workspaces."""
    ep, c = chain(64, 3000, 40)
    case = Case(lib, oracle_mod, ep, 4, 2, 128, "bf16")
    scale = 1 / math.sqrt(128)
    plan = case.pool.chunk_plan([c], [40], 8)
    qs = [case.queries([c], [40], k) for k in (1, 2)]
    want = [case.run(plan, q, scale)[0] for q in qs]
    outs = [torch.empty_like(q) for q in qs]
    ws = [torch.empty(max(1, plan.chunk_attn_workspace_size()), dtype=torch.uint8, device="cuda") for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for q, o, w, s in zip(qs, outs, ws, streams):
            plan.chunk_attn(q, o, None, scale, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_scores_of_a_chunk(lib):
    """octo_token_score on a chunk plan: row t leads to the token given for it."""
    pool = lib.Pool(8, 16, 1, 64, lib.DTYPE_BF16)
    r = pool.root()
    pool.append(r, 30)
    plan = pool.chunk_plan([r], [7], 1)
    V = 500
    x = torch.randn((7, 504), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids = torch.arange(7, dtype=torch.int32, device="cuda") * 60
    stat, logp = torch.empty((7, 2), device="cuda"), torch.empty(7, device="cuda")
    plan.token_score(0, 7, x, V, stat, ids=ids, logp=logp)
    plan.sync()
    ref = torch.log_softmax(x[:, :V].double(), 1)[torch.arange(7), ids.long()]
    assert torch.all((logp.double() - ref).abs() <= 1e-5 * (1 + ref.abs()))


def test_a_speculative_step(lib):
    """Drafts of a forked child checked and the accepted ones kept: prefill of the prompt in parts, then the drafts appended to a child of
    the cursor, attention of its rows, the target's tokens by greedy choice from a fixed read-out, the child released and the accepted
    tokens appended to the cursor.  The tokens are those of decoding one by one."""
    Hq, Hkv, d, P, V = 4, 2, 64, 32, 97
    g = torch.Generator(device="cuda").manual_seed(5)
    emb = torch.randn((V, Hkv * d * 2 + Hq * d), generator=g, device="cuda")
    read = torch.randn((Hq * d, V), generator=g, device="cuda")
    ld = 104
    scale = 1 / math.sqrt(d)

    def rows(ids):
        e = emb[torch.as_tensor(ids, device="cuda")].bfloat16()
        n = len(ids)
        return e[:, :Hkv * d].reshape(n, Hkv, d).contiguous(), e[:, Hkv * d:2 * Hkv * d].reshape(n, Hkv, d).contiguous(), \
            e[:, 2 * Hkv * d:].reshape(n, Hq, d).contiguous()

    def new_pool():
        kp = torch.zeros((64, Hkv, P, d), dtype=torch.bfloat16, device="cuda")
        return lib.Pool(64, P, Hkv, d, lib.DTYPE_BF16, kp, torch.zeros_like(kp))

    def attend(plan, q):
        q = q.clone()
        plan.rope_rows(Hq, q, 1e4)
        out = torch.empty_like(q)
        ws = torch.empty(max(1, plan.chunk_attn_workspace_size()), dtype=torch.uint8, device="cuda")
        plan.chunk_attn(q, out, None, scale, ws)
        x = torch.zeros((len(q), ld), device="cuda")
        x[:, :V] = out.float().reshape(len(q), -1) @ read
        return x

    prompt = [(7 * i) % V for i in range(150)]
    # one by one
    pool = new_pool()
    c = pool.root()
    k, v, _ = rows(prompt[:-1])
    pool.append_rope(c, len(prompt) - 1, k, v, 1e4)
    slow, last = [], prompt[-1]
    for _ in range(24):
        k, v, q = rows([last])
        pool.append_rope(c, 1, k, v, 1e4)
        last = int(attend(pool.chunk_plan([c], [1], Hq), q)[0, :V].argmax())
        slow.append(last)
    # with drafts: right ones for a while, then a wrong one
    pool = new_pool()
    c = pool.root()
    for part in (prompt[:100], prompt[100:-1]):        # read in in parts
        k, v, q = rows(part)
        pool.append_rope(c, len(part), k, v, 1e4)
        attend(pool.chunk_plan([c], [len(part)], Hq), q)
    fast, last, steps = [], prompt[-1], 0
    while len(fast) < 24:
        right = steps % 4
        ahead = slow[len(fast):len(fast) + 4]
        drafts = [t if i < right else (t + 1) % V for i, t in enumerate(ahead)] + [0] * (4 - len(ahead))
        ids = [last] + drafts
        child = pool.fork(c, 1)[0]
        k, v, q = rows(ids)
        pool.append_rope(child, len(ids), k, v, 1e4)
        plan = pool.chunk_plan([child], [len(ids)], Hq)
        x = attend(plan, q)
        acc, nxt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        ws = torch.empty(plan.verify_drafts_workspace_size(0, 1), dtype=torch.uint8, device="cuda")
        plan.verify_drafts(0, 1, x, V, torch.tensor(ids, dtype=torch.int32, device="cuda"), acc, nxt, ws)
        plan.sync()
        n = int(acc)
        plan.close()
        pool.release(child)
        pool.append_rope(c, n + 1, k[:n + 1], v[:n + 1], 1e4)
        fast += drafts[:n] + [int(nxt)]
        last = int(nxt)
        steps += 1
    assert fast[:24] == slow and steps < 24


def test_one_chunk_is_its_tokens_one_by_one(lib):
    """The rows of a chunk against octo_decode of the same tokens, each the newest of its cursor; rotary positions too."""
    Hq, Hkv, d, P, n = 8, 2, 128, 64, 9
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    kp = torch.zeros((40, Hkv, P, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    pool = lib.Pool(40, P, Hkv, d, lib.DTYPE_BF16, kp, vp)
    root = pool.root()
    pool.append_rope(root, 500, rnd(500, Hkv, d), rnd(500, Hkv, d), 1e4)
    a, b = pool.fork(root, 2)
    pool.append_rope(a, 77, rnd(77, Hkv, d), rnd(77, Hkv, d), 1e4)
    pool.mount(b, a, 5, 70)
    k, v, q = rnd(n, Hkv, d), rnd(n, Hkv, d), rnd(n, Hq, d)
    scale = 1 / math.sqrt(d)
    one = torch.empty_like(q)
    for t in range(n):
        pool.append_rope(b, 1, k[t:t + 1], v[t:t + 1], 1e4)
        plan = pool.decode_plan([b])
        qt, o = q[t:t + 1].clone(), one[t:t + 1]
        plan.rope_rows(Hq, qt, 1e4)
        ws = torch.empty(plan.decode_workspace_size(Hq), dtype=torch.uint8, device="cuda")
        plan.decode(Hq, qt, o, None, scale, ws)
        plan.sync()
    plan = pool.chunk_plan([b], [n], Hq)
    q_rot, out = q.clone(), torch.empty_like(q)
    plan.rope_rows(Hq, q_rot, 1e4)
    ws = torch.empty(max(1, plan.chunk_attn_workspace_size()), dtype=torch.uint8, device="cuda")
    plan.chunk_attn(q_rot, out, None, scale, ws)
    plan.sync()
    # both round P to at most bf16 and the output once: 2^-8 (|o| + A) each, A < 1 for means of randn
    assert torch.all((out.float() - one.float()).abs() <= 2.0 ** -7 * (one.float().abs() + 1))


@pytest.mark.parametrize("G,Hkv,d,P", [(4, 8, 128, 64), (2, 8, 64, 16)])
def test_pieces_of_one_and_two_slots_in_turn(lib, oracle_mod, G, Hkv, d, P):
    """CTAs that take short chunks behind long contexts (one slot of 128 rows) and long chunks of few blocks (two slots, one to a
    handful of blocks) one after the other, under a window in another order: each piece's barriers are made anew."""
    T = 128 // G
    ep = synth.Episode(P)
    cur, n_new = [], []
    for i in range(60):
        r = ep.root()
        long = i % 2
        n = (2 * T, 3 * T + 1, 6 * T - 2, T + 1)[i // 2 % 4] if long else 1 + i % T
        ep.append(r, n if long else 700 + 130 * (i % 5) + n)
        cur.append(r), n_new.append(n)
    case = Case(lib, oracle_mod, ep, G, Hkv, d, "bf16")
    plan, q, out, lse = case.check(cur, n_new)
    assert plan.info["bm"] == 2 * T and plan.info["max_tile_entries"] >= 19
    for _ in range(20):
        again, lse2 = case.run(plan, q, 1 / math.sqrt(d))
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    case.check(cur, n_new, window=T + 3, sink=2)
    case.check(cur[::-1], n_new[::-1], window=500)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("lens,n", [((100, 5), 5), ((5000, 7), 7), ((900, 5), 1), ((1500,), 1500)], ids=str)
def test_lse_of_a_nan_row(lib, oracle_mod, dtype, d, lens, n):
    """NaN, as octo_decode gives it, whether the row's tile is cut and joined or not; the other rows are what they were."""
    ep, c = chain(64, *lens)
    case = Case(lib, oracle_mod, ep, 4, 1, d, dtype)
    q = case.queries([c], [n], 8)
    for window in (0, 150):
        plan = case.pool.chunk_plan([c], [n], 4, window=window)
        want, lse = case.run(plan, q, 1 / math.sqrt(d))
        bad = q.clone()
        bad[n // 2, 1:3] = float("nan")
        out, lse2 = case.run(plan, bad, 1 / math.sqrt(d))
        is_bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
        is_bad[n // 2, 1:3] = True
        assert torch.isnan(out[is_bad]).all() and torch.isnan(lse2[is_bad]).all()
        assert torch.equal(out[~is_bad], want[~is_bad]) and torch.equal(lse2[~is_bad], lse[~is_bad])


@pytest.mark.parametrize("dtype,P,long", [("bf16", 64, False), ("bf16", 16, False), ("bf16", 64, True), ("f32", 64, False), ("f32", 16, False)])
@pytest.mark.parametrize("window", [0, 300])
def test_nan_keys_stay_with_who_sees_them(lib, oracle_mod, dtype, P, long, window):
    """A NaN key among one cursor's own new tokens: its rows from there on are NaN, their lse too; the rows before it and the other
    cursors', in shared tiles and two-slot ones as well, are what they were bit for bit."""
    ep, leaves = forest(P)
    cur = leaves[:8] + [leaves[0]]
    Hkv = 8 if long else 2
    if long:                                     # chunks of more than a tile beside them, work for every SM
        for i in range(12):
            r = ep.root()
            ep.append(r, 600 + 30 * i)
            cur.append(r)
    case = Case(lib, oracle_mod, ep, 4, Hkv, 128, dtype)
    n_new = [min(5, ep.length[c]) if c in leaves else ep.length[c] - 7 for c in cur]
    q = case.queries(cur, n_new, 9)
    plan = case.pool.chunk_plan(cur, n_new, 4 * Hkv, window=window)
    if long and not window:
        assert plan.info["bm"] == 64
    want, lse = case.run(plan, q, 1 / math.sqrt(128))
    row0 = np.concatenate([[0], np.cumsum(n_new)])
    for victim in (2, len(cur) - 1):
        c, n, L = cur[victim], n_new[victim], ep.length[cur[victim]]
        t = L - n + n // 2                       # own index of the token with the NaN key
        page = case.pool.seg_pages(c)[t // P]
        before = case.kp[page, 1, t % P].clone()
        case.kp[page, 1, t % P] = float("nan")
        out, lse2 = case.run(plan, q, 1 / math.sqrt(128))
        case.kp[page, 1, t % P] = before
        bad = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
        for i, x in enumerate(cur):
            if x == c:
                first = L - n_new[i]
                for k in range(n_new[i]):
                    if first + k >= t and not (window and first + k >= t + window):
                        bad[int(row0[i]) + k, 4:8] = True
        assert bad.any() and torch.isnan(out[bad]).all() and torch.isnan(lse2[bad]).all()
        assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse2[~bad], lse[~bad])


def test_training_calls_on_a_chunk(lib):
    """The gradient of the scores and a distillation over a chunk plan's rows, against autograd in 64 bits: terms of size at most 1 with a
    dozen fp32 roundings of exponents of at most 20, 1e-5 (1 + |ref|)."""
    pool = lib.Pool(16, 16, 1, 64, lib.DTYPE_BF16)
    a, b = pool.root(), pool.root()
    pool.append(a, 30), pool.append(b, 9)
    plan = pool.chunk_plan([a, b], [7, 4], 1)
    V, N, k = 500, 11, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    x = 2 * torch.randn((N, 504), generator=g, device="cuda")
    ids = (torch.arange(N, device="cuda") * 37 % V).int()
    stat, logp, H = torch.empty((N, 2), device="cuda"), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    gl, gH = (torch.rand(N, generator=g, device="cuda") for _ in range(2))
    dx = torch.empty_like(x)
    plan.token_score(0, N, x, V, stat, entropy=H, ids=ids, logp=logp, inv_temp=0.8)
    plan.token_score_bwd(0, N, x, V, stat, H, ids, gl, gH, dx, inv_temp=0.8)
    plan.sync()
    z = x[:, :V].double().requires_grad_()
    lp = torch.log_softmax(0.8 * z, 1)
    ref = (gl * lp[torch.arange(N), ids.long()] - gH * (lp.exp() * lp).sum(1)).sum()
    want, = torch.autograd.grad(ref, z)
    assert torch.all((dx[:, :V].double() - want).abs() <= 1e-5 * (1 + want.abs()))
    val, top = (2 * torch.randn((N, V), generator=g, device="cuda")).topk(k)
    w = torch.rand(N, generator=g, device="cuda")
    kl, dx2 = torch.empty(N, device="cuda"), torch.empty_like(x)
    plan.distill_topk(0, N, x, V, top.int().contiguous(), val.contiguous(), weight=w, row_kl=kl, dlogits=dx2)
    plan.sync()
    lq, P = torch.log_softmax(z, 1).gather(1, top), torch.softmax(val.double(), 1)
    d = (P * (P.log() - lq)).sum(1)
    want, = torch.autograd.grad((w * d).sum(), z)
    assert torch.all((kl.double() - d).abs() <= 1e-5 * (1 + d.abs())) and torch.all((dx2[:, :V].double() - want).abs() <= 1e-5 * (1 + want.abs()))
