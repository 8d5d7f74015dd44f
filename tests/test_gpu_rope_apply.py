"""flashnorm_rope and flashnorm_rope_table_scaled against plain numpy in 64 bits.

Tolerances. y = a c - b s takes at most two fp32 roundings (one product, one fused multiply-add), each at most 2^-24 of
|a c| + |b s|, and one rounding to the output type: half a step, 2^-8 relative in bf16, 2^-24 in fp32. A table entry is
an angle in float64 (relative error a few 2^-53, so under 1e-9 absolute at the positions used here), rounded once to
fp32: 2^-24 of its size."""

import math

import numpy as np
import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn

pytestmark = pytest.mark.gpu


def _ref(x, cs, pos, n_rope, layout, backward):
    """(y, bound on the fp32 arithmetic) in float64; x [M, H, hd], cs [max_pos, rot/2, 2]."""
    rot = 2 * cs.shape[1]
    y, err = x.copy(), np.zeros_like(x)
    c, s = cs[pos, :, 0][:, None], cs[pos, :, 1][:, None]
    if backward:
        s = -s
    i = np.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
    a, b = x[:, :n_rope][:, :, ia], x[:, :n_rope][:, :, ib]
    h = np.arange(n_rope)
    y[:, h[:, None], ia], y[:, h[:, None], ib] = a * c - b * s, a * s + b * c
    err[:, h[:, None], ia] = np.abs(a * c) + np.abs(b * s)
    err[:, h[:, None], ib] = np.abs(a * s) + np.abs(b * c)
    return y, 2 * 2.0 ** -24 * err


def _inputs(M, H, hd, rot, max_pos, dtype, seed, extra=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H + extra, hd, generator=gen).to(dtype).cuda()[:, :H]
    pos = torch.randint(0, max_pos, (M,), generator=gen, dtype=torch.int32).cuda()
    return x, pos, fn.flashnorm_rope_table_scaled(max_pos, rot)


def _check(y, x, cs, pos, n_rope, layout, backward):
    xh, yh = x.double().cpu().numpy(), y.double().cpu().numpy()
    ref, err = _ref(xh, cs.double().cpu().numpy(), pos.cpu().numpy(), n_rope, layout, backward)
    assert (np.abs(yh - ref) <= torch.finfo(x.dtype).eps / 2 * np.abs(ref) + 1.01 * err).all()
    # what is not turned is carried over bit for bit
    rot = 2 * cs.shape[1]
    assert torch.equal(y[:, n_rope:], x[:, n_rope:]) and torch.equal(y[:, :, rot:], x[:, :, rot:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("M,H,hd,rot,n_rope,extra", [
    (1, 1, 2, 2, 1, 0),        # one pair
    (3, 5, 64, 64, 3, 0),      # whole heads, two of them carried over
    (17, 4, 128, 32, 4, 2),    # a part of the head, heads inside wider rows
    (5, 3, 80, 20, 2, 0),      # rot/2 no multiple of a 16-byte access
    (9, 2, 38, 34, 2, 1),      # head_dim and strides that only narrow accesses fit; rot/2 odd
    (11, 3, 44, 24, 3, 0), (11, 3, 44, 26, 2, 1), (4, 2, 46, 12, 2, 1), (6, 7, 210, 210, 5, 0),  # accesses of 4, 2 and 1 features
    (33, 2, 72, 36, 1, 0),     # rot_dim ends inside a wide access (interleaved)
    (700, 40, 128, 128, 33, 0),  # several heads per thread, the last set ragged
    (4, 2, 16, 16, 0, 0),      # nothing turned
])
def test_rope_matches_float64(M, H, hd, rot, n_rope, extra, layout, dtype):
    x, pos, cs = _inputs(M, H, hd, rot, 97, dtype, seed=M + hd, extra=extra)
    for backward in (False, True):
        y = fn.flashnorm_rope(x, cs, pos, n_rope_heads=n_rope, layout=layout, backward=backward)
        _check(y, x, cs, pos, n_rope, layout, backward)
        inp = x.clone()
        assert fn.flashnorm_rope(inp, cs, pos, n_rope_heads=n_rope, layout=layout, backward=backward, out=inp) is inp
        assert torch.equal(inp, y)  # in place: the same bits
    fn.flashnorm_check_device_error()


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_strided_output_and_misaligned_rows(layout):
    """Heads before rows ([H, M, hd] storage), an output inside a larger buffer whose rest stays as it was, and a base
    address that is aligned to its elements only."""
    M, H, hd, rot = 13, 3, 64, 48
    x, pos, cs = _inputs(M, H, hd, rot, 50, torch.bfloat16, seed=3)
    want = fn.flashnorm_rope(x, cs, pos, layout=layout)
    hx = x.transpose(0, 1).contiguous().transpose(0, 1)
    ho = torch.full((H + 2, M, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    fn.flashnorm_rope(hx, cs, pos, layout=layout, out=ho[1:-1].transpose(0, 1))
    assert torch.equal(ho[1:-1].transpose(0, 1), want)
    assert (ho[0] == 7).all() and (ho[-1] == 7).all()
    buf = torch.empty(M * H * hd + 1, dtype=torch.bfloat16, device="cuda")
    off = buf[1:].view(M, H, hd)
    off.copy_(x)
    assert torch.equal(fn.flashnorm_rope(off, cs, pos, layout=layout), want)
    one = x[:, :, :].expand(M, H, hd)[:, :1].expand(M, 4, hd)  # a broadcast input: head stride 0
    assert torch.equal(fn.flashnorm_rope(one, cs, pos, layout=layout)[:, 3], want[:, 0])


def test_rope_gradient_by_differences():
    """backward=True is the transpose: <v, R x> = <R^T v, x>, and the directional difference of R (linear, so exact up to
    rounding) agrees, with a scaled table too."""
    M, H, hd, rot = 20, 3, 48, 32
    gen = torch.Generator().manual_seed(9)
    x, v, dx = (torch.randn(M, H, hd, generator=gen).cuda() for _ in range(3))
    pos = torch.randint(0, 64, (M,), generator=gen, dtype=torch.int32).cuda()
    cs = fn.flashnorm_rope_table_scaled(64, rot, scaling="yarn", factor=4.0, original_max_pos=16)
    for layout in ("interleaved", "half"):
        gx = fn.flashnorm_rope(v, cs, pos, layout=layout, backward=True).double()
        f = lambda t: (v.double() * fn.flashnorm_rope(t, cs, pos, layout=layout).double()).sum()  # noqa: E731
        want = float(f(x + dx) - f(x - dx)) / 2
        got = float((gx * dx.double()).sum())
        # 2880 products, each a few fp32 roundings of terms near 1: 4 * 2^-24 * sum |v||dx| (about 2 * 2880)
        assert abs(want - got) <= 4 * 2.0 ** -24 * float((v.abs() * (dx.abs() + x.abs())).double().sum()) * 2


def test_rope_special_values_and_empty():
    cs = fn.flashnorm_rope_table_scaled(4, 4)
    x = torch.zeros(2, 2, 8, device="cuda")
    x[:, 1] = math.inf
    x[:, :, 6] = math.nan
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = fn.flashnorm_rope(x, cs, pos, n_rope_heads=1, layout="half")
    assert torch.equal(y[:, 1].isnan(), x[:, 1].isnan()) and torch.equal(y[:, 0, :4], x[:, 0, :4])
    assert y[:, 0, 6].isnan().all() and (y[:, 1, 4] == math.inf).all()  # infinities beside a turned pair stay
    assert fn.flashnorm_rope(x[:0], cs, pos[:0]).shape == (0, 2, 8)


def test_rope_position_outside_table():
    M, H, hd, rot = 6, 3, 32, 16
    x, pos, cs = _inputs(M, H, hd, rot, 10, torch.float32, seed=1)
    pos[2], pos[4] = 10, -1
    y = fn.flashnorm_rope(x, cs, pos, n_rope_heads=2, layout="half")
    with pytest.raises(fn.FlashNormError) as e:
        fn.flashnorm_check_device_error()
    assert e.value.status == fn.FN_ERR_INVALID_ARG
    bad = torch.tensor([2, 4], device="cuda")
    assert y[bad, :2, :rot].isnan().all()
    assert torch.equal(y[bad][:, :, rot:], x[bad][:, :, rot:]) and torch.equal(y[bad, 2], x[bad, 2])
    good = torch.tensor([0, 1, 3, 5], device="cuda")
    _check(y[good], x[good], cs, pos[good], 2, "half", False)
    fn.flashnorm_check_device_error()


def _table_ref(max_pos, rot, base, scaling, factor, original, alpha, beta, mscale):
    theta = base ** (-np.arange(0, rot, 2, dtype=np.longdouble) / rot)
    if scaling == "ntk":
        theta = (np.longdouble(base) * np.longdouble(factor) ** (np.longdouble(rot) / (rot - 2))) ** (
            -np.arange(0, rot, 2, dtype=np.longdouble) / rot)
    elif scaling == "linear":
        theta = theta / factor
    elif scaling == "yarn":
        k = np.clip((original * theta / (2 * np.pi) - alpha) / (beta - alpha), 0, 1)
        theta = theta * (k + (1 - k) / factor)
    ang = np.arange(max_pos, dtype=np.longdouble)[:, None] * theta
    return (np.stack([np.cos(ang), np.sin(ang)], axis=-1) * mscale).astype(np.float64)


@pytest.mark.parametrize("max_pos,rot", [(1, 2), (3, 4), (64, 10), (257, 128), (70001, 64)])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_scaled_table(max_pos, rot, scaling):
    if scaling == "ntk" and rot < 4:
        with pytest.raises(fn.FlashNormError):
            fn.flashnorm_rope_table_scaled(max_pos, rot, scaling="ntk", factor=2.0)
        return
    cs = fn.flashnorm_rope_table_scaled(max_pos, rot, 10000.0, scaling=scaling, factor=8.0, original_max_pos=2048,
                                        alpha=1.0, beta=32.0)
    m = 0.1 * math.log(8.0) + 1 if scaling == "yarn" else 1.0
    ref = _table_ref(max_pos, rot, 10000.0, scaling, 8.0, 2048, 1.0, 32.0, m)
    assert np.max(np.abs(cs.cpu().numpy().astype(np.float64) - ref)) <= m * 2.0 ** -24 + 1e-9
    if scaling == "none":
        old = fn.flashnorm_rope_table(max_pos, rot, 10000.0)
        assert (cs - old).abs().max() <= 2.0 ** -23  # two roundings of the same value


def test_rope_refuses():
    x, pos, cs = _inputs(4, 2, 32, 16, 8, torch.bfloat16, seed=2)
    for bad in (dict(x=x[0]), dict(x=x.half()), dict(x=x.cpu()), dict(rope_cs=cs.double()), dict(rope_cs=cs[..., :1]),
                dict(positions=pos.long()), dict(positions=pos[:3]), dict(layout="pairs"), dict(out=x.float()),
                dict(out=torch.empty(4, 2, 16, dtype=torch.bfloat16, device="cuda")), dict(n_rope_heads=3),
                dict(n_rope_heads=-1), dict(x=x[..., ::2], rope_cs=cs[:, :4].contiguous()),
                dict(rope_cs=fn.flashnorm_rope_table_scaled(8, 64))):
        with pytest.raises((TypeError, ValueError, fn.FlashNormError)):
            fn.flashnorm_rope(**{**dict(x=x, rope_cs=cs, positions=pos), **bad})
    with pytest.raises(fn.FlashNormError):  # an output whose heads share their place
        fn.flashnorm_rope(x, cs, pos, out=torch.empty(4, 1, 32, dtype=torch.bfloat16, device="cuda").expand(4, 2, 32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hd,rot,layout", [(20, 20, "half"), (18, 12, "interleaved"), (36, 36, "half"), (24, 16, "interleaved")])
def test_rotations_in_place_back_to_back(hd, rot, layout, dtype):
    """Each call starts while the one before still writes the same buffer; rows are no multiples of a cache line, so blocks share
    lines. Forty rotations, the table written again before each fourth, give the bits of the same calls with a wait between."""
    M, H = 3001, 5
    x, pos, _ = _inputs(M, H, hd, rot, 61, dtype, seed=hd)
    cs = torch.empty(61, rot // 2, 2, device="cuda")

    def turn(y, between):
        for i in range(40):
            if i % 4 == 0:
                fn.flashnorm_rope_table_scaled(61, rot, base=10000.0 + 100 * i, out=cs)
                between()
            fn.flashnorm_rope(y, cs, pos, n_rope_heads=H - i % 2, layout=layout, backward=i % 3 == 2, out=y)
            between()
        return y

    want = turn(x.clone(), torch.cuda.synchronize)
    for _ in range(5):
        assert torch.equal(turn(x.clone(), lambda: None), want)
