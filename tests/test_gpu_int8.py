"""The 8-bit integer projection against plain numpy in 64 bits.

The codes are integer decisions and have to be equal. Tolerances: the integer sum is exact (at most 127^2 * 131072 <
2^31). Its fp32 value, rho's two factors and their product, and the two products of the epilogue are one rounding each;
the fp32 sum of squares of at most 8192 elements runs in chains of at most 16 fused steps joined by at most 8 + 8 adds,
so 1/rms is within 16 + 4 half steps. Together under 32 * 2^-24 relative (F32 below), element by element, plus half a
step of the output type. SwiGLU: silu(g) moves by at most (1 + |g|) times g's relative error, its exponential's argument
is rounded twice more, and the SFU's exp2 and reciprocal are within 2^-22 each."""

import numpy as np
import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn
from tests.gpu_util import glu_dst_rows

pytestmark = pytest.mark.gpu

F32 = 32 * 2.0 ** -24


def _oracle_rows(x, eps, norm):
    """(codes, rho) in float64; a row that is not finite gets NaN."""
    a = np.abs(x).max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        # a quotient of bf16 values that is no tie is at least 2^-17 from one, so float64 decides exactly
        q = np.where(a > 0, np.rint(127.0 * x / np.where(a > 0, a, 1)), 0.0)
        rho = a[:, 0] / 127.0
        if norm:
            rho = rho / np.sqrt((x * x).mean(axis=1) + eps)
    bad = ~np.isfinite(x).all(axis=1)
    q[bad], rho[bad] = 0, np.nan
    return q, rho


def _oracle(x, Q, s, eps, norm, glu):
    q, rho = _oracle_rows(x, eps, norm)
    z = (q @ Q.astype(np.float64).T) * rho[:, None] * s.astype(np.float64)
    if not glu:
        return z, F32 * np.abs(z)
    z = z.reshape(len(z), -1, 2, 16)
    g, u = z[:, :, 0].reshape(len(z), -1), z[:, :, 1].reshape(len(z), -1)
    y = g / (1 + np.exp(-g)) * u
    return y, ((2 + np.abs(g)) * (F32 + 2 * 2.0 ** -24) + 2 * 2.0 ** -22) * np.abs(y)


def _draw(M, d, rows, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, d)) * np.exp(rng.uniform(-2.3, 2.3, (M, 1)))).to(torch.bfloat16)
    Q = torch.from_numpy(rng.integers(-127, 128, (rows, d)).astype(np.int8))
    s = torch.from_numpy((rng.uniform(0.5, 2.0, rows) / (127 * d ** 0.5)).astype(np.float32))
    return x, Q, s


def _check(y, x, Q, s, eps, norm, glu):
    ref, tol = _oracle(x.double().numpy(), Q.numpy(), s.numpy(), eps, norm, glu)
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    # below the smallest normal bf16 the step is absolute
    assert (np.abs(got - ref)[ok] <= (1.01 * tol + torch.finfo(y.dtype).eps / 2 * np.abs(ref) + 1e-38)[ok]).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,d,N,glu", [
    (1, 16, 8, False), (1, 576, 960, False), (4, 4096, 1544, False), (16, 8192, 136, False), (7, 144, 2064, False),
    (3, 64, 16, True), (16, 1040, 1008, True), (5, 576, 48, True),
    # K ranges of one to eight ranks, of which some re-read their part of x; token counts around 8; the two-launch kernel
    (8, 8192, 1032, False), (9, 2064, 8200, False), (13, 3088, 19000, False), (2, 12304, 256, False), (16, 8192, 40008, False),
    (16, 16384, 10000, True),
    (17, 16, 8, False), (64, 576, 960, False), (129, 208, 1000, False), (257, 4112, 312, False), (300, 128, 4104, False),
    (17, 32, 16, True), (130, 576, 496, True), (513, 272, 1040, True),
])
def test_int8_matches_float64(M, d, N, glu, out):
    rows = 2 * N if glu else N
    x, Q, s = _draw(M, d, rows, seed=M * 7 + d)
    xd, Qd, sd = x.cuda(), Q.cuda(), s.cuda()
    if glu:
        _check(fn.flashnorm_glu_int8(xd, Qd, sd, 1e-5, out_dtype=out), x, Q, s, 1e-5, True, True)
    else:
        for norm in (True, False):
            _check(fn.flashnorm_linear_int8(xd, Qd, sd, 1e-5, out_dtype=out, norm=norm), x, Q, s, 1e-5, norm, False)
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("d", [16, 1024, 1040, 4096, 4112, 8192, 8208])
def test_codes_are_equal(M, d):
    """Q = the unit matrix reads the codes back: rows full of ties, of one magnitude, with extreme scales, with one
    large element, of zeros; every row length of the row pass."""
    rng = np.random.default_rng(d)
    x = np.zeros((M, d))
    for m in range(M):
        k = m % 5
        if k == 0:  # largest 254: 127 x / 254 = x / 2, ties at every odd x
            x[m] = rng.integers(-254, 255, d)
            x[m, rng.integers(d)] = 254
        elif k == 1:
            x[m] = rng.standard_normal(d) * 10.0 ** rng.integers(-38, 37)
        elif k == 2:
            x[m] = rng.standard_normal(d)
            x[m, -1] = 300.0
        elif k == 3:
            x[m] = 1.5 * rng.choice([-1.0, 1.0], d)
    xb = torch.from_numpy(x).to(torch.bfloat16)
    n = min(d, 256)
    cols = np.sort(rng.choice(d, n, replace=False))
    cols[0], cols[-1] = 0, d - 1
    n = n // 8 * 8
    Q = torch.zeros(n, d, dtype=torch.int8)
    Q[torch.arange(n), torch.from_numpy(cols[-n:])] = 1
    y = fn.flashnorm_linear_int8(xb.cuda(), Q.cuda(), torch.ones(n).cuda(), 0.0, out_dtype=torch.float32, norm=False)
    q, rho = _oracle_rows(xb.double().numpy(), 0.0, False)
    got = y.double().cpu().numpy()
    want = q[:, cols[-n:]]
    live = rho > 1e-36  # where the row scale itself is a normal fp32 number
    assert live.any()
    assert np.array_equal(np.rint(got[live] / rho[live, None]), want[live])
    assert (got[rho == 0] == 0).all()


@pytest.mark.parametrize("M", [6, 33])
def test_rows_that_are_not_finite(M):
    x, Q, s = _draw(M, 576, 96, seed=1)
    x[1, 7], x[2, 575], x[3] = float("inf"), float("nan"), 0.0
    x[4, 0] = -float("inf")
    for norm in (True, False):
        y = fn.flashnorm_linear_int8(x.cuda(), Q.cuda(), s.cuda(), 1e-5, norm=norm)
        _check(y, x, Q, s, 1e-5, norm, False)
        assert y[[1, 2, 4]].isnan().all() and (y[3] == 0).all()
    y = fn.flashnorm_glu_int8(x.cuda(), Q.cuda(), s.cuda(), 1e-5)
    assert y[[1, 2, 4]].isnan().all() and (y[3] == 0).all() and y[[0, 5]].isfinite().all()


@pytest.mark.parametrize("d,N,glu", [(16, 8, False), (576, 960, False), (208, 96, True), (1040, 200, False)])
def test_fold_is_bitwise(d, N, glu):
    rng = np.random.default_rng(d)
    W = torch.from_numpy(rng.standard_normal((d, N)) / d ** 0.5).to(torch.bfloat16)
    W[:, 3] = 0
    g = torch.from_numpy(rng.uniform(0.5, 1.5, d)).to(torch.bfloat16)
    Q, s = fn.flashnorm_fold_weights_int8(W.cuda(), g.cuda(), glu=glu)
    w = (W.float() * g.float()[:, None]).numpy()  # exact
    amax = np.abs(w).max(axis=0)
    sc = np.where(amax > 0, amax / np.float32(127), np.float32(1)).astype(np.float32)
    codes = np.clip(np.rint(w / sc), -127, 127).astype(np.int8)
    rows = glu_dst_rows(N // 2) if glu else np.arange(N)
    assert np.array_equal(Q.cpu().numpy()[rows], codes.T) and np.array_equal(s.cpu().numpy()[rows], sc)


def test_folded_projection_near_the_definition():
    """Fold and projection together against RMSNorm(x) . W: what 8 bits cost. A code is off by at most half a step of
    max/127; for normal rows of 576 (largest near 3.3 sigma) that is a relative error of about 1 / (127 / 3.3 * sqrt(12))
    = 0.75 % per factor, 1.1 % for both, against sums of independent terms: 3 % leaves room."""
    rng = np.random.default_rng(4)
    M, d, N = 50, 576, 320
    x = torch.from_numpy(rng.standard_normal((M, d))).to(torch.bfloat16)
    W = torch.from_numpy(rng.standard_normal((d, N)) / d ** 0.5).to(torch.bfloat16)
    g = torch.from_numpy(rng.uniform(0.5, 1.5, d)).to(torch.bfloat16)
    Q, s = fn.flashnorm_fold_weights_int8(W.cuda(), g.cuda())
    y = fn.flashnorm_linear_int8(x.cuda(), Q, s, 1e-6, out_dtype=torch.float32).double().cpu()
    xd = x.double()
    ref = (xd / torch.sqrt((xd * xd).mean(dim=1, keepdim=True) + 1e-6) * g.double()) @ W.double()
    assert float((y - ref).norm() / ref.norm()) < 0.03


def test_guard_rows_and_workspace():
    """Nothing past the output or the stated workspace is written; the caller's workspace gives the same bits."""
    for M, d, N, glu in [(3, 576, 968, False), (16, 208, 80, True), (16, 16384, 19008, False), (70, 144, 104, False), (300, 64, 48, True)]:
        rows = 2 * N if glu else N
        x, Q, s = (t.cuda() for t in _draw(M, d, rows, seed=d))
        call = fn.flashnorm_glu_int8 if glu else fn.flashnorm_linear_int8
        want = call(x, Q, s, 1e-5)
        n = fn.flashnorm_int8_workspace_bytes(M, d, N, glu)
        ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        buf = torch.full((M * N + 512,), 3.0, dtype=torch.bfloat16, device="cuda")
        for _ in range(2):  # its contents do not matter
            call(x, Q, s, 1e-5, out=buf[: M * N].view(M, N), workspace=ws[:n])
        assert torch.equal(buf[: M * N].view(M, N), want) and (buf[M * N:] == 3).all() and (ws[n:] == 0xA5).all()
        if n:
            with pytest.raises(fn.FlashNormError) as e:
                call(x, Q, s, 1e-5, workspace=ws[: n - 16])
            assert e.value.status == fn.FN_ERR_INVALID_ARG


def test_streams_graphs_and_back_to_back():
    """Calls in flight on two streams, replays of two captured graphs between eager calls, and many calls without a host
    wait give the eager bits."""
    sets = []
    for seed, (M, d, N) in enumerate([(2, 576, 960), (16, 4096, 256), (200, 576, 960)]):
        x, Q, s = (t.cuda() for t in _draw(M, d, N, seed))
        sets.append((x, Q, s, fn.flashnorm_linear_int8(x, Q, s, 1e-5)))
    torch.cuda.synchronize()
    graphs = []
    for x, Q, s, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = fn.flashnorm_linear_int8(x, Q, s, 1e-5)
        graphs.append((graph, y))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = []
        for (x, Q, s, _), st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(fn.flashnorm_linear_int8(x, Q, s, 1e-5))
        for (graph, y), st in zip(graphs, reversed(streams)):
            y.zero_()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, _, want), y, (_, gy) in zip(sets, got, graphs):
            assert torch.equal(y, want) and torch.equal(gy, want)
    x, Q, s, want = sets[0]
    ys = [fn.flashnorm_linear_int8(x, Q, s, 1e-5) for _ in range(200)]
    assert all(torch.equal(y, want) for y in ys)
    step = fn.prepare(fn.flashnorm_linear_int8, x, Q, s, 1e-5)
    assert torch.equal(step(), want)
    fn.flashnorm_check_device_error()


def test_int8_refuses():
    x, Q, s = (t.cuda() for t in _draw(4, 64, 32, 0))
    for bad in (dict(x=x.float()), dict(Q=Q.view(torch.uint8)), dict(scales=s.double()), dict(scales=s[:-1]),
                dict(Q=Q[:, :-16]), dict(x=x.cpu()), dict(out_dtype=torch.float16), dict(workspace="no"),
                dict(workspace=None), dict(eps=-1.0), dict(out=torch.empty(4, 16, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises((TypeError, ValueError, fn.FlashNormError)):
            fn.flashnorm_linear_int8(**{**dict(x=x, Q=Q, scales=s, eps=1e-5), **bad})
    assert fn.flashnorm_linear_int8(x[:0], Q, s, 1e-5).shape == (0, 32)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("M", [3, 40])
def test_fold_of_weights_that_are_not_finite(M, glu, value):
    """A channel whose folded weights hold a NaN or an infinity has scale NaN and zero codes, its outputs are NaN, and the
    others keep their bits; a gain that is not finite is in every channel."""
    rng = np.random.default_rng(M)
    d, N = 208, 96
    W = torch.from_numpy(rng.standard_normal((d, N)) / d ** 0.5).to(torch.bfloat16)
    g = torch.from_numpy(rng.uniform(0.5, 1.5, d)).to(torch.bfloat16)
    x = torch.from_numpy(rng.standard_normal((M, d))).to(torch.bfloat16).cuda()
    call = fn.flashnorm_glu_int8 if glu else fn.flashnorm_linear_int8
    dst = glu_dst_rows(N // 2) if glu else np.arange(N)
    Q, s = fn.flashnorm_fold_weights_int8(W.cuda(), g.cuda(), glu=glu)
    want = call(x, Q, s, 1e-5)
    bad_n = [0, 37, N - 1]
    Wb = W.clone()
    for n, k in zip(bad_n, (0, 100, d - 1)):
        Wb[k, n] = value
    Qb, sb = fn.flashnorm_fold_weights_int8(Wb.cuda(), g.cuda(), glu=glu)
    rows = torch.zeros(N, dtype=torch.bool)
    rows[[int(dst[n]) for n in bad_n]] = True
    rows = rows.cuda()
    assert torch.equal(sb.isnan(), rows) and (Qb[rows] == 0).all()
    assert torch.equal(sb[~rows], s[~rows]) and torch.equal(Qb[~rows], Q[~rows])
    cols = torch.zeros(want.shape[1], dtype=torch.bool, device="cuda")
    cols[[n % want.shape[1] for n in bad_n]] = True  # GLU: columns of a gate or an up channel
    y = call(x, Qb, sb, 1e-5)
    assert y[:, cols].isnan().all() and torch.equal(y[:, ~cols], want[:, ~cols])
    gb = g.clone()
    gb[5] = value
    Qb, sb = fn.flashnorm_fold_weights_int8(W.cuda(), gb.cuda(), glu=glu)
    assert sb.isnan().all() and (Qb == 0).all() and call(x, Qb, sb, 1e-5).isnan().all()
    fn.flashnorm_check_device_error()
