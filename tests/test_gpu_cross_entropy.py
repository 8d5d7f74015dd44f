"""The vocabulary head's cross entropy and its gradient against the definition in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32) and h = 2^-8 (half a step of bf16):
  logits   products of two bf16 are exact in fp32; the tensor core adds 16 of them a step, each step rounding or cutting
           to at most 4 u of the magnitudes summed so far: (d / 16 + 2) 4u S, S = r sum_k |x_k w_k|. r (sum of squares,
           division, root) and log2(e) r are within 32 u.
  lse      moves by at most the largest logit error; its sum of exponentials (2^-22 each from the SFU, chains of at most
           16 + 4 adds a tile and half, then `parts` joins of three roundings) by (64 + 4 parts) u, its two final
           roundings by 4 u |lse|.
  loss     lse's error, the target logit's, and one rounding.
  dl       q = exp(l - lse) moves by q (error of l + 32 u |l| + 4 u |lse| + 4 u); minus one, times g, times r: 4 u.
  P        one rounding to bf16: h |P|.
  dW, dx   linear in P: sums of |error of P| |x| or |W|, plus the product's own (terms / 16 + 16) 4u sum |P| |.|, plus h.
           dx's second term adds |x| r^2/d times the error of c = sum dl l: (terms / 16 + 64) 4u sum |dl l|, what
           dl's and l's errors move it, and 8 u.
A half step more for bf16 outputs. Independent roundings add up far below these sums of magnitudes, so the gradients are
also held in norm: two roundings to bf16 (P and the output), each at most h / sqrt(3) in the mean square, give at most
0.0032; 2^-7 leaves room for the part that two factors share. The fp32 errors come on top, in norm at most the norm of
their own elementwise bound: with a single class dl = g (exp(l - lse) - 1) is nothing but the rounding of lse to fp32
(|l| u against a true value of 0), and no relative accuracy exists, so a bound relative to the gradient alone cannot hold
there whatever computes it."""

import numpy as np
import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn

pytestmark = pytest.mark.gpu

U, HB = 2.0 ** -24, 2.0 ** -8
EPS = 1e-6
SIZES = [
    (1, 8, 1), (1, 576, 49152), (3, 16, 5), (7, 64, 31), (16, 576, 33), (23, 576, 4099), (64, 136, 1000), (65, 1040, 257),
    (128, 64, 2049), (129, 576, 777), (257, 72, 3001), (300, 2056, 512), (517, 320, 8197),
    # many rows per class (a pass of its own finishes dW*), also over 2048 rows, and just above that vocabulary
    (2167, 280, 602), (2500, 64, 7), (1500, 2056, 130), (2600, 136, 2048), (2600, 136, 2056),
]


def _draw(M, d, V, seed, ignore=-100):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, d)) * np.exp(rng.uniform(-2.3, 2.3, (M, 1)))).to(torch.bfloat16)
    W = torch.from_numpy(rng.standard_normal((V, d)) * (2 / d ** 0.5)).to(torch.bfloat16)
    t = torch.from_numpy(rng.integers(0, V, M))
    if M > 2:
        t[rng.random(M) < 0.2] = ignore
        t[0], t[1], t[2] = 0, V - 1, ignore
    g = torch.from_numpy(rng.uniform(0.5, 1.5, M).astype(np.float32) / M)
    return x, W, t, g


def _forward(x, W, t, eps, ignore):
    """(loss, lse, their tolerances, and what the gradient needs) in float64."""
    x, W = x.double(), W.double()
    M, d = x.shape
    V = W.shape[0]
    r = 1 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + eps)
    l = (x * r) @ W.T
    el = (d / 16 + 2) * 4 * U * ((x * r).abs() @ W.abs().T) + 32 * U * l.abs()
    lse = torch.logsumexp(l, dim=1)
    parts = 2 * ((V + 31) // 32)
    e_lse = el.amax(dim=1) + (64 + 4 * parts) * U + 4 * U * lse.abs()
    live = t != ignore
    at = t.clamp(min=0)[:, None]
    loss = torch.where(live, lse - l.gather(1, at)[:, 0], 0.0)
    e_loss = torch.where(live, e_lse + el.gather(1, at)[:, 0] + 2 * U * (lse.abs() + loss.abs()), 0.0)
    return loss, lse, e_loss, e_lse, (x, W, r, l, el, live, at)


def _backward(g, lse, ctx):
    x, W, r, l, el, live, at = ctx
    M, d = x.shape
    V = W.shape[0]
    g = torch.where(live, g.double(), 0.0)[:, None]
    lse = lse.double()[:, None]
    q = torch.exp(l - lse)
    dq = q.scatter_add(1, at, torch.full_like(at, -1, dtype=torch.float64))
    dl = g * dq
    e_dl = g * (q * (el + 32 * U * l.abs() + 4 * U * lse.abs() + 4 * U) + 4 * U * dq.abs())
    P, e_P = r * dl, r * (e_dl + 32 * U * dl.abs())
    dW = P.T @ x
    f_dW = e_P.T @ x.abs() + (M / 16 + 16) * 4 * U * (P.abs().T @ x.abs())  # what fp32 costs
    t_dW = f_dW + HB * (P.abs().T @ x.abs())
    c = (dl * l).sum(dim=1, keepdim=True)
    k = r * r / d
    e_c = (e_dl * l.abs() + dl.abs() * el).sum(dim=1, keepdim=True) \
        + ((V / 16 + 64) * 4 * U) * (dl * l).abs().sum(dim=1, keepdim=True)
    dx = P @ W - x * k * c
    f_dx = e_P @ W.abs() + (V / 16 + 16) * 4 * U * (P.abs() @ W.abs()) + x.abs() * k * (e_c + 64 * U * c.abs())
    t_dx = f_dx + HB * (P.abs() @ W.abs())
    return dx, dW, (t_dx, f_dx), (t_dW, f_dW)


def _near(got, want, tols, what):
    tol, tol_f32 = tols
    got = got.double().cpu()
    half = torch.finfo(torch.bfloat16).eps / 2
    bad = (got - want).abs() > tol + half * want.abs() + 1e-38
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()))
    assert float((got - want).norm()) <= 2.0 ** -7 * float(want.norm()) + float(tol_f32.norm()), what


@pytest.mark.parametrize("M,d,V", SIZES)
def test_loss_matches_float64(M, d, V):
    x, W, t, _ = _draw(M, d, V, seed=M + d + V)
    loss, lse = fn.flashnorm_linear_cross_entropy(x.cuda(), W.cuda(), t.cuda(), EPS)
    want, want_lse, tol, tol_lse, _ = _forward(x, W, t, EPS, -100)
    assert loss.dtype == lse.dtype == torch.float32
    assert ((loss.double().cpu() - want).abs() <= tol).all()
    assert ((lse.double().cpu() - want_lse).abs() <= tol_lse).all()
    assert (loss.cpu()[t == -100] == 0).all()
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("M,d,V", SIZES)
def test_gradient_matches_float64(M, d, V):
    x, W, t, g = _draw(M, d, V, seed=M * 3 + d + V)
    _, lse, _, _, ctx = _forward(x, W, t, EPS, -100)
    lse = lse.float()
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), x.cuda(), W.cuda(), t.cuda(), lse.cuda(), EPS)
    want_dx, want_dW, t_dx, t_dW = _backward(g, lse, ctx)
    _near(dx, want_dx, t_dx, "dx")
    _near(dW, want_dW, t_dW, "dW")
    assert (dx.cpu()[t == -100] == 0).all()
    fn.flashnorm_check_device_error()


def test_pieces_of_the_vocabulary():
    """A vocabulary that takes two pieces, the second not a whole number of tiles: 64 bits on the GPU, in norm and row by
    row (a row or class left out, or counted twice, would be wholly wrong)."""
    M, d, V = 4200, 72, 9001
    x, W, t, g = _draw(M, d, V, seed=12)
    args = [v.cuda() for v in (x, W, t)]
    loss, lse = fn.flashnorm_linear_cross_entropy(*args, EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), *args, lse, EPS)
    xd, Wd, td = x.cuda().double(), W.cuda().double(), args[2]
    r = 1 / torch.sqrt((xd * xd).mean(dim=1, keepdim=True) + EPS)
    l = (xd * r) @ Wd.T
    live = td != -100
    want = torch.logsumexp(l, dim=1)
    assert (lse.double() - want).abs().max() < 1e-5  # |l| < 32: 100 roundings of 2^-24 |l| at most
    at = td.clamp(min=0)[:, None]
    assert (loss.double() - torch.where(live, want - l.gather(1, at)[:, 0], 0.0)).abs().max() < 2e-5
    dl = torch.exp(l - lse.double()[:, None]).scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    dl *= torch.where(live, g.cuda().double(), 0.0)[:, None]
    dn = dl @ Wd
    want_dx = r * (dn - xd * r * (dn * xd * r).mean(dim=1, keepdim=True))
    want_dW = dl.T @ (xd * r)
    for got, want in ((dx, want_dx), (dW, want_dW)):
        off, size = (got.double() - want).norm(dim=1), want.norm(dim=1)
        assert off.norm() <= 2.0 ** -7 * size.norm() and (off <= 2.0 ** -6 * size + 1e-7 * size.max()).all()


def test_gradient_matches_differences():
    """Directional derivatives of sum g loss, the definition's losses at +-h in 64 bits. Central differences with
    h = 1e-4 along a unit direction are off by h^2 / 6 of the third derivative and 2^-52 / h of the value, both
    far under the bound that the gradient's own tolerance gives for its product with the direction."""
    M, d, V = 37, 136, 515
    x, W, t, g = _draw(M, d, V, seed=8)
    _, lse, _, _, ctx = _forward(x, W, t, EPS, -100)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), x.cuda(), W.cuda(), t.cuda(), lse.float().cuda(), EPS)
    _, _, t_dx, t_dW = _backward(g, lse.float(), ctx)
    rng = np.random.default_rng(3)

    def total(x, W):
        return float((_forward(x, W, t, EPS, -100)[0] * g.double()).sum())

    for got, tol, like, at in ((dx, t_dx[0], x, 0), (dW, t_dW[0], W, 1)):
        v = torch.from_numpy(rng.standard_normal(tuple(like.shape)))
        v /= v.norm()
        h = 1e-4
        lo, hi = [x.double(), W.double()], [x.double(), W.double()]
        lo[at], hi[at] = lo[at] - h * v, hi[at] + h * v
        diff = (total(*hi) - total(*lo)) / (2 * h)
        got = got.double().cpu()
        assert abs(float((got * v).sum()) - diff) <= float(((tol + HB * got.abs()) * v.abs()).sum()) + 1e-8


def test_masked_rows_hold_anything():
    """Rows without a target (padding) may hold NaN or infinities: the others' losses and all gradients stay what they are
    without those rows; every row ignored gives zero gradients."""
    M, d, V = 75, 144, 1003
    x, W, t, g = _draw(M, d, V, seed=5)
    t[10:20] = -100
    keep = t != -100
    args = [v.cuda() for v in (x, W, t)]
    loss, lse = fn.flashnorm_linear_cross_entropy(*args, EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), *args, lse, EPS)
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        xb, gb = x.clone(), g.clone()
        xb[~keep], gb[~keep] = value, value
        bad = [v.cuda() for v in (xb, W, t)]
        lossb, lseb = fn.flashnorm_linear_cross_entropy(*bad, EPS)
        assert torch.equal(lossb, loss) and torch.equal(lseb[keep.cuda()], lse[keep.cuda()])
        dxb, dWb = fn.flashnorm_linear_cross_entropy_backward(gb.cuda(), *bad, lseb, EPS)
        assert torch.equal(dxb, dx) and torch.equal(dWb, dW)
    t[:] = -100
    loss, lse = fn.flashnorm_linear_cross_entropy(args[0], args[1], t.cuda(), EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), args[0], args[1], t.cuda(), lse, EPS)
    assert (loss == 0).all() and (dx == 0).all() and (dW == 0).all() and lse.isfinite().all()
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("every", [1, 2, 13])
@pytest.mark.parametrize("V", [1500, 5000])
def test_one_frequent_class(V, every):
    """Rows that share a class, as a frequent token's do: all, half, or two in most blocks of 32 (more than the 32 that one
    look lists); right whichever way dW* is finished."""
    M, d = 700, 200
    x, W, t, g = _draw(M, d, V, seed=11)
    t[::every] = 33
    _, lse, _, _, ctx = _forward(x, W, t, EPS, -100)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), x.cuda(), W.cuda(), t.cuda(), lse.float().cuda(), EPS)
    want_dx, want_dW, t_dx, t_dW = _backward(g, lse.float(), ctx)
    _near(dx, want_dx, t_dx, "dx")
    _near(dW, want_dW, t_dW, "dW")


def test_ignore_index_may_be_a_class():
    M, d, V = 40, 64, 300
    x, W, t, g = _draw(M, d, V, seed=6, ignore=7)
    want, want_lse, tol, _, ctx = _forward(x, W, t, EPS, 7)
    args = [v.cuda() for v in (x, W, t)]
    loss, lse = fn.flashnorm_linear_cross_entropy(*args, EPS, ignore_index=7)
    assert ((loss.double().cpu() - want).abs() <= tol).all() and (loss.cpu()[t == 7] == 0).all()
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), *args, want_lse.float().cuda(), EPS, ignore_index=7)
    want_dx, want_dW, t_dx, t_dW = _backward(g, want_lse.float(), ctx)
    _near(dx, want_dx, t_dx, "dx")
    _near(dW, want_dW, t_dW, "dW")


@pytest.mark.parametrize("bad", [-1, 300, 2 ** 40, -2 ** 62])
def test_bad_targets_are_reported(bad):
    """A target that is no class: NaN in its own row, reported, nothing else touched."""
    M, d, V = 20, 64, 300
    x, W, t, g = _draw(M, d, V, seed=7)
    t[4] = -100
    args = [v.cuda() for v in (x, W, t)]
    loss, lse = fn.flashnorm_linear_cross_entropy(*args, EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), *args, lse, EPS)
    t[4] = bad
    args[2] = t.cuda()
    lossb, lseb = fn.flashnorm_linear_cross_entropy(*args, EPS)
    with pytest.raises(fn.FlashNormError) as e:
        fn.flashnorm_check_device_error()
    assert e.value.status == fn.FN_ERR_INVALID_ARG and "target" in str(e.value)
    dxb, dWb = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), *args, lse, EPS)
    with pytest.raises(fn.FlashNormError):
        fn.flashnorm_check_device_error()
    rest = torch.arange(M, device="cuda") != 4
    assert lossb[4].isnan() and torch.equal(lossb[rest], loss[rest]) and torch.equal(lseb, lse)
    assert dxb[4].isnan().all() and torch.equal(dxb[rest], dx[rest]) and torch.equal(dWb, dW)


def test_extreme_logits():
    """Logits whose exponentials overflow or vanish without the running maximum; equal logits; a row of zeros."""
    M, d, V = 33, 64, 700
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((M, d))).to(torch.bfloat16)
    W = torch.from_numpy(rng.standard_normal((V, d)) * 40).to(torch.bfloat16)
    W[100:] = W[100:101]  # equal logits in every later tile
    x[5] = 0
    t = torch.from_numpy(rng.integers(0, V, M))
    g = torch.ones(M)
    want, want_lse, tol, tol_lse, ctx = _forward(x, W, t, EPS, -100)
    assert want_lse.abs().max() > 300
    args = [v.cuda() for v in (x, W, t)]
    loss, lse = fn.flashnorm_linear_cross_entropy(*args, EPS)
    assert ((loss.double().cpu() - want).abs() <= tol).all() and ((lse.double().cpu() - want_lse).abs() <= tol_lse).all()
    assert abs(float(lse[5]) - np.log(V)) < 1e-5
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), *args, want_lse.float().cuda(), EPS)
    want_dx, want_dW, t_dx, t_dW = _backward(g, want_lse.float(), ctx)
    half = HB
    assert ((dx.double().cpu() - want_dx).abs() <= t_dx[0] + half * want_dx.abs() + 1e-38).all()
    assert ((dW.double().cpu() - want_dW).abs() <= t_dW[0] + half * want_dW.abs() + 1e-38).all()


@pytest.mark.parametrize("M,d,V", [(5, 64, 300), (130, 136, 2100)])
def test_workspace_guards_and_determinism(M, d, V):
    x, W, t, g = (v.cuda() for v in _draw(M, d, V, seed=9))
    loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS)
    nf = fn.flashnorm_cross_entropy_workspace_bytes(M, d, V)
    nb = fn.flashnorm_cross_entropy_workspace_bytes(M, d, V, backward=True)
    ws = torch.full((max(nf, nb) + 4096,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    for _ in range(2):
        again = fn.flashnorm_linear_cross_entropy(x, W, t, EPS, workspace=ws[:nf])
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse) and (ws[nf:] == 0xFF).all()
        ws.fill_(0xFF)
        again = fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS, workspace=ws[:nb])
        assert torch.equal(again[0], dx) and torch.equal(again[1], dW) and (ws[nb:] == 0xFF).all()
        ws.fill_(0xFF)
    for call in (lambda w: fn.flashnorm_linear_cross_entropy(x, W, t, EPS, workspace=w[: nf - 16]),
                 lambda w: fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS, workspace=w[: nb - 16])):
        with pytest.raises(fn.FlashNormError) as e:
            call(ws)
        assert e.value.status == fn.FN_ERR_INVALID_ARG


def test_graphs_and_streams():
    """Two captured forward-backward pairs replayed on two streams at once, and eager calls between, give the eager bits."""
    sets = []
    for seed, (M, d, V) in enumerate([(9, 576, 5000), (140, 136, 2100)]):
        x, W, t, g = (v.cuda() for v in _draw(M, d, V, seed))
        sets.append((x, W, t, g))

    def step(x, W, t, g):
        loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
        return (loss, lse, *fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*s)
        graphs.append((graph, out))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for (graph, out), st in zip(graphs, streams):
            for o in out:
                o.zero_()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                graph.replay()
        eager = [step(*s) for s in sets]
        torch.cuda.synchronize()
        for w, (_, out), e in zip(want, graphs, eager):
            assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(w, out, e))
    call = fn.prepare(fn.flashnorm_linear_cross_entropy, *sets[0][:3], EPS)
    assert torch.equal(call()[0], want[0][0])
    fn.flashnorm_check_device_error()


def test_empty_and_refused():
    x, W, t, g = (v.cuda() for v in _draw(6, 64, 50, 0))
    loss, lse = fn.flashnorm_linear_cross_entropy(x[:0], W, t[:0], EPS)
    assert loss.shape == lse.shape == (0,)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g[:0], x[:0], W, t[:0], lse, EPS)
    assert dx.shape == (0, 64) and (dW == 0).all()
    ok = dict(x=x, Wstar=W, targets=t, eps=EPS)
    for bad in (dict(x=x.float()), dict(x=x[:, :60]), dict(Wstar=W[:, :8].contiguous()), dict(targets=t.int()),
                dict(targets=t[:-1]), dict(eps=float("nan")), dict(workspace=None), dict(workspace="no"),
                dict(targets=t.cpu())):
        with pytest.raises((TypeError, ValueError, fn.FlashNormError)):
            fn.flashnorm_linear_cross_entropy(**{**ok, **bad})
    lse = torch.zeros(6, device="cuda")
    ok = dict(grad_loss=g, lse=lse, **ok)
    for bad in (dict(grad_loss=g.double()), dict(lse=lse[:-1]), dict(grad_loss=g[0]), dict(Wstar=W.float())):
        with pytest.raises((TypeError, ValueError, fn.FlashNormError)):
            fn.flashnorm_linear_cross_entropy_backward(**{**ok, **bad})


@pytest.mark.parametrize("M,d", [(20, 4096), (32, 1024), (48, 4096), (40, 8192), (36, 520)])
def test_rows_predicted_well(M, d):
    """Rows whose target has probability 0.9 to 0.999, its weights along x so that every product of its logit has one sign.

    The target's entry of dl is g (exp(l - lse) - 1). Below l = 32 the forward rounds lse twice (2^-20 each: half a step), the
    gradient log2(e) lse once (2^-19 log2 units, 1.3e-6), the SFU's power of two is within 2^-22: together 3.5e-6, 0.35 % at
    1 - p = 1e-3. The target's logit itself must cancel, however d products are summed: the same sum in both calls, and
    within 2^-24 sqrt(d) of 64 bits' for a lse from there (1e-6 l at d = 8192 in the mean). The outputs' own roundings are at
    most 2^-8. So each row of dx and each target's row of dW* is within 1 % in norm. The loss, log(1 + the others' share),
    has that sum's roundings, 4 * 2^-24, beside the others' logits' errors, 1e-5 of itself: within 0.1 %."""
    V, miss = 2000, (1e-1, 1e-2, 1e-3)
    rng = np.random.default_rng(M + d)
    x = torch.from_numpy(rng.standard_normal((M, d))).to(torch.bfloat16)
    W = torch.from_numpy(rng.standard_normal((V, d)) * (2 / d ** 0.5)).to(torch.bfloat16)
    t = torch.from_numpy(rng.permutation(V)[:M])
    xd = x.double()
    r = 1 / torch.sqrt((xd * xd).mean(dim=1, keepdim=True) + EPS)
    base = torch.logsumexp((xd * r) @ W.double().T, dim=1)
    for m in range(M):
        q = miss[m % 3]
        W[t[m]] = (xd[m] * ((base[m] + np.log((1 - q) / q)) / (r[m] * xd[m].square().sum()))).to(torch.bfloat16)
    Wd = W.double()
    l = (xd * r) @ Wd.T
    lse = torch.logsumexp(l, dim=1)
    at = (torch.arange(M), t)
    others = torch.logsumexp(l.clone().index_put_(at, torch.tensor(-torch.inf, dtype=torch.float64)), dim=1)
    want = torch.nn.functional.softplus(others - l[at])  # lse - l_t without their difference
    left = -torch.expm1(-want)
    assert ((left > 0.7 * 1e-3) & (left < 0.2)).all() and lse.max() < 32
    loss, own = fn.flashnorm_linear_cross_entropy(x.cuda(), W.cuda(), t.cuda(), EPS)
    assert ((loss.double().cpu() - want).abs() <= 1e-3 * want).all()
    g = torch.ones(M)
    dl = torch.exp(l - lse[:, None])
    dl[at] = -left
    dn = dl @ Wd
    dx_w = r * (dn - xd * r * (dn * xd * r).mean(dim=1, keepdim=True))
    dW_w = (dl.T @ (xd * r))[t]
    for given in (own, lse.float().cuda()):
        dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), x.cuda(), W.cuda(), t.cuda(), given, EPS)
        for got, ref in ((dx.double().cpu(), dx_w), (dW.double().cpu()[t], dW_w)):
            assert ((got - ref).norm(dim=1) <= 0.01 * ref.norm(dim=1)).all()
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("M", [20, 75])
def test_shifted_labels_and_sliced_vectors(M):
    """Next-token labels are the tokens from the second on: a slice 8 bytes into its storage. It, and slices of g and lse that
    start 4 bytes in, give the bits of their aligned copies."""
    d, V = 72, 1003
    x, W, t, g = _draw(M, d, V, seed=4)
    x, W, t, g = (v.cuda() for v in (x, W, t, g))
    tokens = torch.cat([t[:1], t])[None]
    labels = tokens[:, 1:].contiguous().view(-1)
    assert labels.data_ptr() % 16 == 8
    loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
    again = fn.flashnorm_linear_cross_entropy(x, W, labels, EPS)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS)
    g1, lse1 = torch.cat([g[:1], g])[1:], torch.cat([lse[:1], lse])[1:]
    again = fn.flashnorm_linear_cross_entropy_backward(g1, x, W, labels, lse1, EPS)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dW)
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("what", ["neighbours", "equal rows", "crowd"])
def test_neighbouring_targets(what):
    """Targets that share a block of 32 rows and 32 classes: three different classes, each once; one class whose rows have the
    same norm, g and logit, so that their entries round the same way; and 20 rows of six classes. The target's entry may be
    rounded once, by 2^-8 of itself, and the output once: no element of dW* is further off than both, no row in norm
    than 2^-7, and the rows of lone targets, held in fp32, than the output's rounding: 2^-8."""
    M, d, V = 96, 136, 4096
    x, W, t, g = _draw(M, d, V, seed=21)
    t = torch.from_numpy(np.random.default_rng(2).permutation(np.arange(64, V, 32))[:M])  # one target in 32 classes
    g = torch.full((M,), 0.37)
    if what == "neighbours":
        t[[3, 9, 30]] = torch.tensor([5, 17, 31])
    elif what == "equal rows":
        x[:40] = x[0]
        t[:40] = 7
    else:
        t[40:60] = torch.arange(20) % 6
    _, lse, _, _, ctx = _forward(x, W, t, EPS, -100)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), x.cuda(), W.cuda(), t.cuda(), lse.float().cuda(), EPS)
    want_dx, want_dW, t_dx, t_dW = _backward(g, lse.float(), ctx)
    _near(dx, want_dx, t_dx, "dx")
    _near(dW, want_dW, t_dW, "dW")
    off = (dW.double().cpu() - want_dW).norm(dim=1)
    size, f32 = want_dW.norm(dim=1), t_dW[1].norm(dim=1)
    rows = t.unique()
    lone = rows[rows >= 64]
    assert (off[rows] <= 2.0 ** -7 * size[rows] + f32[rows]).all()
    # beside the target's entry a lone row has the others' entries, rounded too
    rest = HB * ((ctx[2] * torch.exp(ctx[3] - lse[:, None]) * g.double()[:, None]).scatter(1, t[:, None], 0.0).T @ ctx[0].abs()).norm(dim=1)
    assert (off[lone] <= HB * size[lone] + f32[lone] + rest[lone]).all()


@pytest.mark.parametrize("M,d,V", [(1, 1032, 300), (16, 4096, 2000), (17, 2056, 20000), (24, 3000, 700), (31, 1088, 19500),
                                   (32, 4096, 1000), (33, 4096, 1000), (32, 2048, 20100), (33, 2056, 20100)])
def test_loss_of_few_rows_with_several_accumulations(M, d, V):
    """More than 1024 k, so that a slab's sums are carried over several accumulations, the last one short; both sides of the
    row count where the kernel changes; vocabularies of more than 128 rows per SM, so that CTAs take several slabs."""
    x, W, t, g = _draw(M, d, V, seed=M + d)
    loss, lse = fn.flashnorm_linear_cross_entropy(x.cuda(), W.cuda(), t.cuda(), EPS)
    want, want_lse, tol, tol_lse, ctx = _forward(x, W, t, EPS, -100)
    assert ((loss.double().cpu() - want).abs() <= tol).all()
    assert ((lse.double().cpu() - want_lse).abs() <= tol_lse).all()
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g.cuda(), x.cuda(), W.cuda(), t.cuda(), lse, EPS)
    want_dx, want_dW, t_dx, t_dW = _backward(g, lse.cpu(), ctx)
    _near(dx, want_dx, t_dx, "dx")
    _near(dW, want_dW, t_dW, "dW")
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("M,d,V", [(8200, 64, 10000), (8200, 192, 10003)])
def test_three_pieces_of_the_vocabulary(M, d, V):
    """The second and third piece add to dx; operands of whole 64-column blocks. 64 bits on the GPU, in norm and row by row. A
    row's gradient has the roundings of P and of the output, 2^-8 each at most."""
    x, W, t, g = (v.cuda() for v in _draw(M, d, V, seed=13))
    loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS)
    xd, Wd = x.double(), W.double()
    r = 1 / torch.sqrt((xd * xd).mean(dim=1, keepdim=True) + EPS)
    l = (xd * r) @ Wd.T
    live = t != -100
    at = t.clamp(min=0)[:, None]
    dl = torch.exp(l - lse.double()[:, None]).scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    dl *= torch.where(live, g.double(), 0.0)[:, None]
    dn = dl @ Wd
    want_dx = r * (dn - xd * r * (dn * xd * r).mean(dim=1, keepdim=True))
    want_dW = dl.T @ (xd * r)
    for got, want in ((dx, want_dx), (dW, want_dW)):
        off, size = (got.double() - want).norm(dim=1), want.norm(dim=1)
        assert off.norm() <= 2.0 ** -7 * size.norm() and (off <= 2.0 ** -6 * size + 1e-7 * size.max()).all()
    fn.flashnorm_check_device_error()
