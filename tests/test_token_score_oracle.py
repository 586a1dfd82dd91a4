"""Pins of the fp64 reference of token scoring and top-logit distillation, and the
refusals of the binding that need no GPU."""
import numpy as np
import pytest

from oracle.token_logprob import token_logprob
from oracle import token_score as ts


def _case(seed, N=7, V=13):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2, (N, V))
    pred = np.arange(-1, N - 1)
    pred[N - 2] = 1                                  # row 1 feeds two tokens, row N - 3 none
    return rng, x, rng.integers(0, V, N), pred


def test_equals_token_logprob_and_closed_forms():
    rng, x, ids, pred = _case(0)
    logp, stat, H, top, top_lp = ts.score(x, ids, pred, k=3)
    rlogp, rlse, _, rdx = token_logprob(x, ids, None, pred)
    assert np.allclose(logp, rlogp, atol=1e-13)
    assert np.allclose(stat.sum(axis=1), rlse, atol=1e-13)
    # the gradient of -sum logp is the loss gradient
    assert np.allclose(ts.score_bwd(x, ids, pred, -np.ones(len(x)), None), rdx, atol=1e-13)
    u = ts.score(np.full((2, 8), 5.0), np.zeros(2, int), np.arange(2), k=8)
    assert np.allclose(u[2], np.log(8)) and np.array_equal(u[3], np.tile(np.arange(8), (2, 1)))   # ties: lowest id
    m = np.array([[-np.inf, 1.0, -np.inf, 1.0], [-np.inf] * 4])
    logp, stat, H, top, top_lp = ts.score(m, np.array([1, 2]), np.arange(2), k=3)
    assert np.allclose(H, [np.log(2), 0.0]) and logp[1] == -np.inf and np.array_equal(top, [[1, 3, 0], [0, 1, 2]])


@pytest.mark.parametrize("c", [1.0, 0.6])
def test_score_gradient_against_differences(c):
    rng, x, ids, pred = _case(1)
    gl, gh = rng.normal(size=len(x)), rng.normal(size=len(x))

    def f(y):
        logp, _, H, _, _ = ts.score(y, ids, pred, c)
        return (gl * logp)[pred >= 0].sum() + (gh * H).sum()

    d = ts.score_bwd(x, ids, pred, gl, gh, c)
    h = 1e-6
    for r, v in [(0, 2), (1, 5), (3, 12), (6, 0), (4, 7)]:
        e = np.zeros_like(x)
        e[r, v] = h
        assert abs((f(x + e) - f(x - e)) / (2 * h) - d[r, v]) < 1e-7


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(tail):
    rng, x, _, _ = _case(2)
    N, V = x.shape
    ids = rng.integers(0, V, (N, 4))                 # repeated ids among them
    ids[2, 1:] = -1
    ids[3] = -1
    val = np.log(rng.uniform(0.02, 0.2, (N, 4))) if tail else rng.normal(size=(N, 4))
    w = rng.normal(size=N)
    w[5] = 0.0
    kl, loss, d = ts.distill(x, ids, val, w, 0.7, tail, 1.5)
    assert kl[5] == 0 and not d[5].any() and (kl[:5] >= -1e-12).all()
    if not tail:
        assert kl[3] == 0 and not d[3].any()
    h = 1e-6
    for r, v in [(0, 2), (1, ids[1, 0]), (2, ids[2, 0]), (4, ids[4, 3]), (6, 1)]:
        e = np.zeros_like(x)
        e[r, v] = h
        g = (ts.distill(x + e, ids, val, w, 0.7, tail)[1] - ts.distill(x - e, ids, val, w, 0.7, tail)[1]) / (2 * h)
        assert abs(1.5 * g - d[r, v]) < 1e-7


def test_distill_of_the_teacher_itself_is_zero():
    rng, x, ids, pred = _case(3)
    for k in (3, x.shape[1]):
        _, _, _, top, lp = ts.score(x, ids, pred, 0.8, k)
        kl, _, d = ts.distill(x, top, lp, None, 0.8, True)
        assert np.abs(kl).max() < 1e-12 and np.abs(d).max() < 1e-12
    # all entries listed: the renormalised form is the same divergence
    _, _, _, top, lp = ts.score(x[::-1], ids, pred, 1.0, x.shape[1])
    a, b = ts.distill(x, top, lp, None, 1.0, True), ts.distill(x, top, lp, None, 1.0, False)
    assert np.allclose(a[0], b[0], atol=1e-12) and np.allclose(a[2], b[2], atol=1e-12)


def test_binding_refuses_bad_tensors():
    torch = pytest.importorskip("torch")
    import packed_tree_attention_gb300 as pta
    p = pta.Plan.__new__(pta.Plan)
    p.info, p.h, p._L = {"n_rows": 4}, None, pta.load()
    x = torch.zeros((4, 16))
    f, i = torch.zeros(8), torch.zeros(8, dtype=torch.int32)
    for bad in (x.half(), x.t(), x[:3], torch.zeros(64), x[:, :9]):
        with pytest.raises(ValueError):
            p.token_score(0, 4, bad, 10, f)
        with pytest.raises(ValueError):
            p.distill_topk(0, 4, bad, 10, i.view(4, 2), f.view(4, 2), f)
    with pytest.raises(ValueError):                  # host memory
        p.token_score(0, 4, x, 10, f)
    dev = f.get_device()
    assert pta._vector(f, "float32", 8, dev, "logp") == f.data_ptr()
    for bad, n, where in ((i, 4, dev), (f[::2], 4, dev), (f, 9, dev), (f, 4, dev + 1)):
        with pytest.raises(ValueError):
            pta._vector(bad, "float32", n, where, "logp")


def test_binding_takes_one_row_of_any_pitch(monkeypatch):
    """Logits and gradient of one row need no common pitch, in tensors of one row or of several; of
    two rows they do."""
    torch = pytest.importorskip("torch")
    import packed_tree_attention_gb300 as pta
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    pta._torch()
    monkeypatch.setattr(pta, "_device", lambda: -1)
    p = pta.Plan.__new__(pta.Plan)
    p.info, p.h, p._L = {"n_rows": 4}, None, Lib()
    f, i = torch.zeros(8), torch.zeros(8, dtype=torch.int32)
    wide, narrow, one, odd = torch.zeros((4, 64)), torch.zeros((3, 56)), torch.zeros((1, 72)), torch.zeros((4, 51))

    def both(logits, grad, n):
        p.token_score_bwd(0, n, logits, 50, f, None, i, f, None, grad, stream=0)
        p.distill_topk(0, n, logits, 50, i.view(4, 2), f.view(4, 2), f, dlogits=grad, stream=0)

    for logits in (wide, narrow, one, odd):
        for grad in (wide, narrow, one, odd):
            both(logits, grad, 1)
            for name, a in calls[-2:]:
                assert a[3] == logits.data_ptr() and a[5] >= 50 and a[5] % 8 == 0
            assert grad.data_ptr() in calls[-2][1] and grad.data_ptr() in calls[-1][1]
    both(wide, torch.zeros((2, 64)), 2)
    assert [a[5] for _, a in calls[-2:]] == [64, 64]
    for logits, grad in ((wide, narrow), (narrow, wide), (wide, one)):
        with pytest.raises(ValueError):
            both(logits, grad, 2)


@pytest.mark.parametrize("tail", [False, True])
def test_repeated_ids_are_one_class(tail):
    """A list with an id repeated is the list with its probabilities added up: a divergence of
    distributions, 0 where the student is the teacher."""
    x = np.log([[0.4, 0.3, 0.2, 0.1], [0.1, 0.1, 0.1, 0.7]])
    ids, val = np.array([[0, 0, 1]] * 2), np.log([[0.15, 0.25, 0.3]] * 2)
    kl, loss, d = ts.distill(x, ids, val, tail=tail)
    one = ts.distill(x, np.array([[0, 1]] * 2), np.log([[0.4, 0.3]] * 2), tail=tail)
    assert np.allclose(kl, one[0], atol=1e-14) and np.allclose(d, one[2], atol=1e-14) and abs(loss - one[1]) < 1e-14
    if tail:                                            # P = (0.4, 0.3, rest 0.3) against the same and against (0.1, 0.1, 0.8)
        assert abs(kl[0]) < 1e-14
        assert abs(kl[1] - (0.4 * np.log(4) + 0.3 * np.log(3) + 0.3 * np.log(0.3 / 0.8))) < 1e-14
    else:                                               # (4/7, 3/7) against shares 0.4 and 0.3 of the whole
        assert abs(kl[0] - np.log(1 / 0.7)) < 1e-14
    rng = np.random.default_rng(1)
    ids = rng.integers(0, 4, (500, 9))
    val = np.log(rng.dirichlet(np.ones(10), 500)[:, :9])
    # by the log sum inequality at least T ln T, T the teacher's mass: 1, or what is listed where every
    # id is, so that the rest drops out
    T = np.exp(val).sum(1) if tail else np.ones(500)
    T[[len(set(i)) < 4 for i in ids]] = 1.0
    assert (T < 1).any() == tail
    assert (ts.distill(rng.normal(0, 1, (500, 4)), ids, val, tail=tail)[0] >= T * np.log(T) - 1e-14).all()


def test_binding_asks_again_for_a_gpu(monkeypatch):
    """A first call without a GPU says so and does not settle it."""
    torch = pytest.importorskip("torch")
    import packed_tree_attention_gb300 as pta
    monkeypatch.setattr(pta, "_T", {})
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    assert pta._device() == pta._device() == -2
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 40 + dev, raising=False)
    assert pta._device() == 3 and pta._current(None, 3) == 43
