"""The 8-bit projection, the rotation and the head's loss and gradient with producers right before them and from two host threads:
calls follow each other without a host wait, each starts while the one before still writes its inputs, and the bits are those of the
same calls with a wait between."""

import threading

import numpy as np
import pytest
import torch

import rmsnorm_linear_projection_fold_b200 as fn

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("M", [5, 16, 32, 48, 300])
def test_operands_written_right_before(M):
    """Folds, tables and rows made new in the same buffers before every round."""
    rng = np.random.default_rng(M)
    d, V, hd = 576, 2048, 64
    Ws = [_bf16(rng, d, V, scale=1 / 24) for _ in range(3)]
    xs = [_bf16(rng, M, d) for _ in range(3)]
    g = torch.from_numpy(rng.uniform(0.5, 1.5, d)).to(torch.bfloat16).cuda()
    t = torch.from_numpy(rng.integers(0, V, M)).cuda()
    gl = torch.rand(M, device="cuda")
    pos = torch.from_numpy(rng.integers(0, 128, M).astype(np.int32)).cuda()
    x, head = torch.empty_like(xs[0]), torch.empty(V, d, dtype=torch.bfloat16, device="cuda")
    cs = torch.empty(128, hd // 2, 2, device="cuda")

    def rounds(between):
        out = []
        for i in range(6):
            x.copy_(xs[i % 3])
            between()
            fn.flashnorm_rope_table_scaled(128, hd, base=1000.0 * (i + 1), out=cs)
            between()
            fn.flashnorm_rope(x.view(M, d // hd, hd), cs, pos, layout="half", out=x.view(M, d // hd, hd))
            between()
            fn.flashnorm_fold_weights(Ws[i % 3], g, out=head)
            between()
            loss, lse = fn.flashnorm_linear_cross_entropy(x, head, t, EPS)
            between()
            dx, dW = fn.flashnorm_linear_cross_entropy_backward(gl, x, head, t, lse, EPS)
            between()
            Q, s = fn.flashnorm_fold_weights_int8(Ws[i % 3], g)
            between()
            y = fn.flashnorm_linear_int8(x, Q, s, EPS)
            between()
            z = fn.flashnorm_linear_int8(dx, Q, s, EPS, norm=False, out_dtype=torch.float32)
            between()
            out += [x.clone(), loss, lse, dx, dW, Q, s, y, z]
        return out

    want = rounds(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(rounds(lambda: None), want))
    fn.flashnorm_check_device_error()


def test_two_host_threads():
    rng = np.random.default_rng(0)
    sets = []
    for M, d, V in ((24, 576, 5000), (150, 320, 3001)):
        x, W = _bf16(rng, M, d), _bf16(rng, V, d, scale=2 / d ** 0.5)
        Q, s = fn.flashnorm_fold_weights_int8(_bf16(rng, d, 960, scale=1 / 24), torch.ones(d, dtype=torch.bfloat16, device="cuda"))
        t = torch.from_numpy(rng.integers(0, V, M)).cuda()
        sets.append((x, W, t, torch.rand(M, device="cuda"), Q, s))

    def step(x, W, t, g, Q, s):
        loss, lse = fn.flashnorm_linear_cross_entropy(x, W, t, EPS)
        return (loss, lse, *fn.flashnorm_linear_cross_entropy_backward(g, x, W, t, lse, EPS), fn.flashnorm_linear_int8(x, Q, s, EPS))

    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(100):
                    got = step(*sets[k])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                        wrong.append(k)
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
    fn.flashnorm_check_device_error()
