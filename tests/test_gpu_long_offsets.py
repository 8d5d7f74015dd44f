"""Tensors of more than 2^31 elements: what lies past the 32-bit offsets is compared with calls on that part alone, whose kernels see
small offsets (and are tested against 64 bits elsewhere)."""

import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _bf16(rows, cols, scale=1.0, seed=0):
    """Normal values, made in parts (fp32 of the whole would take twice the room)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for part in out.split(max(1, (1 << 28) // cols)):
        part.copy_(torch.randn(part.shape, device="cuda", generator=gen) * scale)
    return out


def test_rope():
    M, H, hd = 270_000, 64, 128
    assert M * H * hd > 2 ** 31
    x = _bf16(M, H * hd).view(M, H, hd)
    cs = fn.flashnorm_rope_table_scaled(512, hd)
    pos = torch.arange(M, dtype=torch.int32, device="cuda") % 512
    keep = x[-300:].clone()
    want = fn.flashnorm_rope(keep, cs, pos[-300:], layout="half")
    y = fn.flashnorm_rope(x, cs, pos, layout="half")
    assert torch.equal(y[-300:], want)
    del y
    # heads before rows, in place: the head stride passes 2^31 bytes, the last head's offset 2^31 elements
    hx = x.view(H, M, hd).transpose(0, 1)
    last = hx[-300:].clone()
    want = fn.flashnorm_rope(last, cs, pos[-300:])
    fn.flashnorm_rope(hx, cs, pos, out=hx)
    assert torch.equal(hx[-300:], want)
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("M", [3, 40])
def test_int8_weights(M):
    d, N = 4096, 540_000
    assert d * N > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randint(-127, 128, (N, d), dtype=torch.int8, device="cuda", generator=gen)
    s = torch.rand(N, device="cuda", generator=gen) + 0.5
    x = _bf16(M, d, seed=2)
    y = fn.flashnorm_linear_int8(x, Q, s, EPS, out_dtype=torch.float32)
    want = fn.flashnorm_linear_int8(x, Q[-4096:].clone(), s[-4096:].clone(), EPS, out_dtype=torch.float32)
    # the two calls cut K into different numbers of ranges, which add the sum of squares in another order: each value is within 32
    # roundings of 2^-24 of the exact one (tests/test_gpu_int8.py), so they are within 64 of each other
    assert ((y[:, -4096:] - want).abs() <= 64 * 2.0 ** -24 * want.abs()).all()
    fn.flashnorm_check_device_error()


def test_int8_rows_and_outputs():
    M, d, N = 540_000, 4096, 64
    x = _bf16(M, d, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randint(-127, 128, (N, d), dtype=torch.int8, device="cuda", generator=gen)
    s = torch.rand(N, device="cuda", generator=gen) + 0.5
    y = fn.flashnorm_linear_int8(x, Q, s, EPS)
    assert torch.equal(y[-300:], fn.flashnorm_linear_int8(x[-300:].clone(), Q, s, EPS))
    del x, y, Q, s
    M, d, N = 70_000, 16, 32_000
    assert M * N > 2 ** 31
    x = _bf16(M, d, seed=3)
    Q = torch.randint(-127, 128, (N, d), dtype=torch.int8, device="cuda", generator=gen)
    s = torch.rand(N, device="cuda", generator=gen) + 0.5
    y = fn.flashnorm_linear_int8(x, Q, s, EPS)
    assert torch.equal(y[-300:], fn.flashnorm_linear_int8(x[-300:].clone(), Q, s, EPS))
    fn.flashnorm_check_device_error()


def test_int8_fold():
    d, N = 4096, 540_000
    W = _bf16(d, N, seed=5)
    g = _bf16(1, d, seed=6)[0]
    Q, s = fn.flashnorm_fold_weights_int8(W, g)
    Qp, sp = fn.flashnorm_fold_weights_int8(W[:, -4096:].contiguous(), g)
    assert torch.equal(Q[-4096:], Qp) and torch.equal(s[-4096:], sp)


@pytest.mark.parametrize("M", [20, 40])
def test_head_of_a_long_vocabulary(M):
    """Targets at the far end. The reference takes the logits a part at a time in fp32."""
    d, V = 4096, 540_000
    W = _bf16(V, d, 2 / d ** 0.5, seed=7)
    x = _bf16(M, d, seed=8)
    t = torch.arange(V - M, V, device="cuda")
    t[3] = 5
    loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
    xn = x.double() / (x.double().square().mean(dim=1, keepdim=True) + EPS).sqrt()
    parts = [xn @ w.double().T for w in W.split(20_000)]
    want = torch.logsumexp(torch.stack([torch.logsumexp(p, dim=1) for p in parts]), dim=0)
    lt = (xn * W[t].double()).sum(dim=1)
    # |l| < 16: 100 roundings of 2^-24 |l| at most
    assert (lse.double() - want).abs().max() < 1e-4 and (loss.double() - (want - lt)).abs().max() < 1e-4
    g = torch.full((M,), 1.0, device="cuda")
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS)
    # the far end of dW*, and dx
    dl = [torch.exp(p - lse.double()[:, None]) for p in parts]
    far = torch.cat(dl[-2:], dim=1)
    n0 = V - far.shape[1]
    rows = torch.arange(M, device="cuda")
    here = t >= n0
    far[rows[here], t[here] - n0] -= 1
    want_dW = far.T @ xn
    off, size = (dW[n0:].double() - want_dW).norm(dim=1), want_dW.norm(dim=1)
    assert (off <= 2.0 ** -6 * size + 1e-7 * size.max()).all()
    dn = torch.zeros(M, d, dtype=torch.float64, device="cuda")
    for w, q in zip(W.split(20_000), dl):
        dn += q @ w.double()
    dn -= W[t].double()
    r = 1 / (x.double().square().mean(dim=1, keepdim=True) + EPS).sqrt()
    want_dx = r * (dn - xn * (dn * xn).mean(dim=1, keepdim=True))
    assert ((dx.double() - want_dx).norm(dim=1) <= 2.0 ** -6 * want_dx.norm(dim=1)).all()
    fn.flashnorm_check_device_error()


def test_head_of_many_rows():
    M, d, V = 530_000, 4096, 72
    assert M * d > 2 ** 31
    x = _bf16(M, d, seed=9)
    W = _bf16(V, d, 2 / d ** 0.5, seed=10)
    t = torch.arange(M, device="cuda") % V
    t[::7] = -100
    loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
    n = 500
    xe, te = x[-n:].clone(), t[-n:].clone()
    le, lsee = fn.flashnorm_linear_cross_entropy(xe, W, te, EPS)
    assert torch.equal(loss[-n:], le) and torch.equal(lse[-n:], lsee)
    g = torch.rand(M, device="cuda")
    g[: M - n] = 0.0  # only the last rows reach dW*
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS)
    dxe, dWe = fn.flashnorm_linear_cross_entropy_backward(g[-n:].clone(), xe, W, te, lsee, EPS)
    half = 2.0 ** -8
    assert ((dx[-n:].double() - dxe.double()).abs() <= 2 * half * dxe.double().abs() + 1e-30).all()
    assert (dx[: M - n] == 0).all()
    assert ((dW.double() - dWe.double()).norm(dim=1) <= 2 * half * dWe.double().norm(dim=1)).all()
    fn.flashnorm_check_device_error()
