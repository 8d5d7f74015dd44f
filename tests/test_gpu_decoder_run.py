"""The operators around the folded projections one after the other, as a decoder layer and its head use them: 8-bit q/k/v
projection, rotary positions in place on its query and key heads, 8-bit output projection without a norm, residual,
8-bit SwiGLU, the head's loss and its gradient, and back through the rotation. Each step is compared with the definition in
64 bits from that step's actual inputs, so errors do not pile up; then the whole run is captured and replayed.

Tolerances: a value rounded to bf16 is off by at most half a step, 2^-8 of itself, and its fp32 part by less than 2^-18 of
the magnitudes in it (32 roundings for the projections, 4 for the rotation); SwiGLU moves by (2 + |gate|) times that. The
loss is held to 1e-5 (its terms are below 32 and carry at most 100 roundings of 2^-24 each); the gradients, whose own tests
derive elementwise bounds, in norm to the two bf16 roundings in their path, 2^-7."""

import numpy as np
import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _weights(rng, d, F, V, dev):
    def w(rows, cols):
        return torch.from_numpy(rng.standard_normal((rows, cols)) / rows ** 0.5).to(torch.bfloat16).to(dev)

    g = torch.from_numpy(rng.uniform(0.5, 1.5, d)).to(torch.bfloat16).to(dev)
    one = torch.ones(d, dtype=torch.bfloat16, device=dev)
    return dict(qkv=fn.flashnorm_fold_weights_int8(w(d, 3 * d), g), out=fn.flashnorm_fold_weights_int8(w(d, d), one),
                glu=fn.flashnorm_fold_weights_int8(w(d, 2 * F), g, glu=True), head=fn.flashnorm_fold_weights(w(d, V), g))


def _run(x, p, cs, pos, t, gl, H, hd):
    M, d = x.shape
    qkv = fn.flashnorm_linear_int8(x, *p["qkv"], EPS).view(M, 3 * H, hd)
    before = qkv.clone()
    fn.flashnorm_rope(qkv, cs, pos, n_rope_heads=2 * H, layout="half", out=qkv)
    v = qkv[:, 2 * H:].reshape(M, d).contiguous()
    o = fn.flashnorm_linear_int8(v, *p["out"], 0.0, out_dtype=torch.float32, norm=False)
    h = (x.float() + o).to(torch.bfloat16)
    ff = fn.flashnorm_glu_int8(h, *p["glu"], EPS)
    loss, lse = fn.flashnorm_linear_cross_entropy(h, p["head"], t, EPS)
    dx, dW = fn.flashnorm_linear_cross_entropy_backward(gl, h, p["head"], t, lse, EPS)
    back = fn.flashnorm_rope(dx.view(M, H, hd), cs, pos, layout="half", backward=True)
    return dict(before=before, qkv=qkv, v=v, o=o, h=h, ff=ff, loss=loss, lse=lse, dx=dx, dW=dW, back=back)


def _int8(x, Q, s, norm):
    x, a = x.double(), x.double().abs().amax(dim=1, keepdim=True)
    rho = a / 127
    if norm:
        rho = rho / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    return torch.round(127 * x / a) @ Q.double().T * rho * s.double()


def _turn(x, cs, pos, heads, sign):
    x = x.double().clone()
    half = cs.shape[1]
    c, s = cs.double()[pos.long(), None, :, 0], sign * cs.double()[pos.long(), None, :, 1]
    a, b = x[:, :heads, :half].clone(), x[:, :heads, half:2 * half].clone()
    x[:, :heads, :half], x[:, :heads, half:2 * half] = a * c - b * s, a * s + b * c
    return x


def _near(got, want, scale, what):
    half = torch.finfo(got.dtype).eps / 2
    assert ((got.double() - want).abs() <= 1.01 * half * want.abs() + 2.0 ** -18 * scale + 1e-38).all(), what


@pytest.mark.parametrize("M", [1, 16, 17, 150])
def test_a_decoder_run(M):
    rng = np.random.default_rng(M)
    H, hd, F, V = 6, 32, 272, 1112  # the fold takes multiples of 8
    d = H * hd
    dev = torch.device("cuda")
    p = _weights(rng, d, F, V, dev)
    x = torch.from_numpy(rng.standard_normal((M, d)) * np.exp(rng.uniform(-2, 2, (M, 1)))).to(torch.bfloat16).to(dev)
    cs = fn.flashnorm_rope_table_scaled(4096, hd // 2, 10000.0, scaling="yarn", factor=4.0, original_max_pos=1024)
    pos = torch.from_numpy(rng.integers(0, 4096, M).astype(np.int32)).to(dev)
    t = torch.from_numpy(rng.integers(0, V, M)).to(dev)
    t[M // 2:M // 2 + M // 8] = -100
    gl = torch.full((M,), 1.0 / M, device=dev)
    r = _run(x, p, cs, pos, t, gl, H, hd)

    qkv = _int8(x, *p["qkv"], True)
    _near(r["before"].view(M, -1), qkv, qkv.abs(), "qkv")
    turned = _turn(r["before"], cs, pos, 2 * H, 1)
    assert torch.equal(r["qkv"][:, 2 * H:], r["before"][:, 2 * H:])
    assert torch.equal(r["qkv"][:, :, hd // 2:], r["before"][:, :, hd // 2:])
    _near(r["qkv"], turned, r["before"].double().abs().amax(dim=2, keepdim=True), "rope")
    o = _int8(r["v"], *p["out"], False)
    _near(r["o"], o, o.abs(), "out")
    z = _int8(r["h"], *p["glu"], True).view(M, -1, 2, 16)
    gate, up = z[:, :, 0].reshape(M, -1), z[:, :, 1].reshape(M, -1)
    ff = gate * torch.sigmoid(gate) * up
    _near(r["ff"], ff, (2 + gate.abs()) * ff.abs(), "glu")

    h, W = r["h"].double(), p["head"].double()
    ri = 1 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    logits = (h * ri) @ W.T
    live = t != -100
    lse = torch.logsumexp(logits, dim=1)
    loss = torch.where(live, lse - logits.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    assert (r["loss"].double() - loss).abs().max() < 1e-5 and (r["lse"].double() - lse).abs().max() < 1e-5
    dl = torch.exp(logits - lse[:, None])
    dl[torch.arange(M, device=dev)[live], t[live]] -= 1
    dl *= (gl.double() * live)[:, None]
    dn = dl @ W
    dx = ri * (dn - h * ri * (dn * h * ri).mean(dim=1, keepdim=True))
    dW = dl.T @ (h * ri)
    for got, want, what in ((r["dx"], dx, "dx"), (r["dW"], dW, "dW")):
        assert float((got.double() - want).norm()) <= 2.0 ** -7 * float(want.norm()), what
    back = _turn(r["dx"].view(M, H, hd), cs, pos, H, -1)
    _near(r["back"], back, r["dx"].double().view(M, H, hd).abs().amax(dim=2, keepdim=True), "back")

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        again = _run(x, p, cs, pos, t, gl, H, hd)
    for _ in range(3):
        for k, v in again.items():
            if k != "h":
                v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(again[k], r[k]) for k in r)
    fn.flashnorm_check_device_error()
