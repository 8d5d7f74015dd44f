"""Operators of the decoder around the folded projections: what is timed, on which inputs, and their plain forms.

Three operators, at the places where a decoder built on the folded projections calls them:

  int8     the W8A8 projection: each row of x is quantized to 8-bit integers with one scale (its RMSNorm rides in
           that scale), the folded weight has one scale per output channel, and the product is exact in integers;
           linear and SwiGLU forms
  rope     rotary positions on the projected heads, and the (cos, sin) table scaled for long contexts
  head     final norm -> vocabulary projection -> softmax cross entropy, without keeping the logits, and its
           gradient

`own` False computes the plain form (elementary torch operations in 32 bits, rounded once); `own` True makes the
library's calls. `exact` gives the same results from the definitions in 64 bits.
"""

import math

import numpy as np
import torch

own = False

IGNORE = -100  # target of a row that carries no loss (padding, prompt tokens)


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token through a small model's fused q/k/v projection: latency is all that counts
        dict(name="int8_decode_small", op="int8", M=1, d=576, N=960, glu=False, norm=True, out="bf16"),
        # four sequences, one token each, through a 7B-width q/k/v projection: bound by the 50 MB of weights
        dict(name="int8_decode_wide", op="int8", M=4, d=4096, N=12288, glu=False, norm=True, out="bf16"),
        # a ragged prefill through a projection that no norm precedes (attention output), fp32 residual
        dict(name="int8_ragged_no_norm", op="int8", M=333, d=4096, N=4096, glu=False, norm=False, out="f32"),
        # a 2048-token prefill through the 7B-width gated feed-forward: the largest 8-bit product
        dict(name="int8_glu_prefill", op="int8", M=2048, d=4096, N=11008, glu=True, norm=True, out="bf16"),
        # 16 decoded tokens far into their sequences, half layout, query and key heads of one fused row
        dict(name="rope_decode", op="rope", M=16, H=96, rot_heads=64, hd=128, rot=128, max_pos=32768, layout="half",
             backward=False, extra=0, dtype="bf16"),
        # an 8192-token prefill of the 7B width, adjacent pairs
        dict(name="rope_prefill", op="rope", M=8192, H=96, rot_heads=64, hd=128, rot=128, max_pos=8192,
             layout="interleaved", backward=False, extra=0, dtype="bf16"),
        # the gradient of a partial rotation (a quarter of the head), fp32, heads inside wider rows, odd row count
        dict(name="rope_partial_backward", op="rope", M=1023, H=9, rot_heads=9, hd=64, rot=16, max_pos=4096,
             layout="half", backward=True, extra=6, dtype="f32"),
        # the table of a model whose context is stretched by 32, frequency by frequency
        dict(name="rope_table_long", op="table", max_pos=131072, rot=128, base=500000.0, scaling="yarn", factor=32.0,
             original=4096),
        # scoring a short answer with a small model
        dict(name="head_loss_small", op="head", M=23, d=576, V=49152, backward=False),
        # scoring a 2048-token batch at the 7B width
        dict(name="head_loss_wide", op="head", M=2048, d=4096, V=32000, backward=False),
        # gradient of a ragged batch, a vocabulary that no tile divides
        dict(name="head_grad_ragged", op="head", M=517, d=576, V=50257, backward=True),
        # gradient of a 2048-token batch at the 7B width: the largest case
        dict(name="head_grad_wide", op="head", M=2048, d=4096, V=32000, backward=True),
    ]


def _log_int(rng, lo, hi, step=1):
    """A whole number between lo and hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["int8", "int8", "rope", "table", "head", "head"])
    if op == "int8":
        while True:
            glu = rng.random() < 0.4
            M, d = _log_int(rng, 1, 4096), _log_int(rng, 64, 8192, 16)
            N = _log_int(rng, 64, 16384, 16 if glu else 8)
            if M * d * N * (2 if glu else 1) <= 2048 * 4096 * 22016 and d * N <= 4096 * 22016:
                break
        return dict(op=op, M=M, d=d, N=N, glu=glu, norm=glu or rng.random() < 0.7, out=rng.choice(["bf16", "f32"]))
    if op == "rope":
        while True:
            hd = 2 * rng.randint(8, 128)
            H, M = _log_int(rng, 1, 96), _log_int(rng, 1, 16384)
            if M * H * hd <= 8192 * 96 * 128:
                break
        rot = hd if rng.random() < 0.5 else 2 * rng.randint(1, hd // 2)
        return dict(op=op, M=M, H=H, rot_heads=rng.randint(1, H), hd=hd, rot=rot, max_pos=_log_int(rng, 256, 65536),
                    layout=rng.choice(["half", "interleaved"]), backward=rng.random() < 0.4,
                    extra=rng.choice([0, 0, 1, 6]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "table":
        rot = 2 * rng.randint(8, 64)
        return dict(op=op, max_pos=_log_int(rng, 128, 131072), rot=rot, base=rng.choice([10000.0, 500000.0, 1e6]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=float(rng.choice([2, 4, 8, 32])),
                    original=rng.choice([2048, 4096, 8192]))
    while True:
        M, d, V = _log_int(rng, 1, 4096), _log_int(rng, 64, 4096, 8), _log_int(rng, 128, 65536)
        if M * d * V <= 2048 * 4096 * 32000:
            break
    return dict(op=op, M=M, d=d, V=V, backward=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------ inputs
def _rows(M, d, gen):
    """Activations: normal, each row with a scale of its own between 0.1 and 10 (a residual stream's rows)."""
    scale = torch.exp(torch.rand(M, 1, device="cuda", generator=gen) * math.log(100.0) + math.log(0.1))
    return (torch.randn(M, d, device="cuda", generator=gen) * scale).to(torch.bfloat16)


def _interleave(a, F):
    """Rows [gate 0..F | up 0..F] in the library's order: 16 gate rows, the matching 16 up rows, and so on."""
    return a.view(2, F // 16, 16, *a.shape[1:]).transpose(0, 1).reshape(a.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    if op == "int8":
        M, d, N = case["M"], case["d"], case["N"]
        rows = 2 * N if case["glu"] else N
        st["x"] = _rows(M, d, gen)
        w = torch.randn(rows, d, device="cuda", generator=gen) / math.sqrt(d)
        w *= 0.5 + torch.rand(d, device="cuda", generator=gen)  # the folded norm gain
        if case["glu"]:
            w = _interleave(w, N)
        big = w.abs().amax(dim=1)
        st["s"] = big / 127
        st["Q"] = torch.round(w * 127 / big[:, None]).to(torch.int8)
        st["eps"] = 1e-6
    elif op == "rope":
        M, H, hd, rot = case["M"], case["H"], case["hd"], case["rot"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["x"] = torch.randn(M, H + case["extra"], hd, device="cuda", generator=gen).to(dt)[:, :H]
        st["pos"] = torch.randint(0, case["max_pos"], (M,), device="cuda", generator=gen, dtype=torch.int32)
        theta = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * theta
        st["cs"] = torch.stack([ang.cos(), ang.sin()], dim=-1).float()
    elif op == "table":
        # the only inputs are numbers; a base of its own for each seed keeps one pass's table from being another's
        st["base"] = case["base"] * (1 + 1e-3 * float(torch.rand(1, device="cuda", generator=gen)))
    else:
        M, d, V = case["M"], case["d"], case["V"]
        st["x"] = _rows(M, d, gen)
        # logits of a standard deviation near 2, as a trained head's
        st["W"] = (torch.randn(V, d, device="cuda", generator=gen) * (2.0 / math.sqrt(d))).to(torch.bfloat16)
        t = torch.randint(0, V, (M,), device="cuda", generator=gen)
        skip = torch.rand(M, device="cuda", generator=gen) < 0.1
        t[skip] = IGNORE
        st["t"] = t
        st["eps"] = 1e-6
        if case["backward"]:
            z = st["x"].float()
            l = (z @ st["W"].float().T) * torch.rsqrt(z.square().mean(dim=1, keepdim=True) + st["eps"])
            st["lse"] = torch.logsumexp(l, dim=1)  # the forward pass's, in hand when the gradient is asked for
            st["g"] = torch.full((M,), 1.0 / M, device="cuda") * (0.5 + torch.rand(M, device="cuda", generator=gen))
    return st


# ------------------------------------------------------------------------------------------------ the calls
def run(st):
    op = st["op"]
    if own:
        import rmsnorm_linear_projection_fold_b200 as fn

        if op == "int8":
            dt = torch.bfloat16 if st["out"] == "bf16" else torch.float32
            if st["glu"]:
                return fn.flashnorm_glu_int8(st["x"], st["Q"], st["s"], st["eps"], out_dtype=dt)
            return fn.flashnorm_linear_int8(st["x"], st["Q"], st["s"], st["eps"], out_dtype=dt, norm=st["norm"])
        if op == "rope":
            return fn.flashnorm_rope(st["x"], st["cs"], st["pos"], n_rope_heads=st["rot_heads"], layout=st["layout"],
                                     backward=st["backward"])
        if op == "table":
            return fn.flashnorm_rope_table_scaled(st["max_pos"], st["rot"], st["base"], scaling=st["scaling"],
                                                  factor=st["factor"], original_max_pos=st["original"])
        if st["backward"]:
            return fn.flashnorm_linear_cross_entropy_backward(st["g"], st["x"], st["W"], st["t"], st["lse"],
                                                              st["eps"], ignore_index=IGNORE)
        return fn.flashnorm_linear_cross_entropy(st["x"], st["W"], st["t"], st["eps"], ignore_index=IGNORE)
    return {"int8": _int8, "rope": _rope, "table": _table, "head": _head}[op](st)


def _int8(st):
    x = st["x"].float()
    big = x.abs().amax(dim=1, keepdim=True)
    q = torch.round(x * 127 / big)
    scale = big / 127
    if st["norm"]:
        scale = scale * torch.rsqrt(x.square().mean(dim=1, keepdim=True) + st["eps"])
    y = (q @ st["Q"].float().T) * scale * st["s"]
    if st["glu"]:
        y = y.view(y.shape[0], -1, 2, 16)
        gate, up = y[:, :, 0], y[:, :, 1]
        y = (gate / (1 + torch.exp(-gate)) * up).reshape(y.shape[0], -1)
    return y.to(torch.bfloat16) if st["out"] == "bf16" else y


def _rope(st):
    x, half = st["x"].float(), st["rot"] // 2
    cs = st["cs"][st["pos"].long()][:, None]  # [M, 1, rot / 2, 2]
    c, s = cs[..., 0], cs[..., 1]
    if st["backward"]:
        s = -s
    h = st["rot_heads"]
    y = x.clone()
    if st["layout"] == "half":
        a, b = x[:, :h, :half], x[:, :h, half:2 * half]
        y[:, :h, :half], y[:, :h, half:2 * half] = a * c - b * s, a * s + b * c
    else:
        a, b = x[:, :h, 0:2 * half:2], x[:, :h, 1:2 * half:2]
        y[:, :h, 0:2 * half:2], y[:, :h, 1:2 * half:2] = a * c - b * s, a * s + b * c
    return y.to(st["x"].dtype)


def _table(st):
    D, base, s = st["rot"], st["base"], st["factor"]
    if st["scaling"] == "ntk":
        base = base * s ** (D / (D - 2))
    theta = base ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    m = 1.0
    if st["scaling"] == "linear":
        theta = theta / s
    elif st["scaling"] == "yarn":
        # a frequency that turns more than 32 times within the original context stays, one that turns less than
        # once is divided by the factor, and those between are blended
        keep = ((st["original"] * theta / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / s)
        m = 0.1 * math.log(s) + 1
    ang = torch.arange(st["max_pos"], device="cuda", dtype=torch.float64)[:, None] * theta
    return (torch.stack([ang.cos(), ang.sin()], dim=-1) * m).float()


def _head(st):
    x, W, t = st["x"].float(), st["W"].float(), st["t"]
    r = torch.rsqrt(x.square().mean(dim=1, keepdim=True) + st["eps"])
    l = (x @ W.T) * r
    live = t != IGNORE
    at = t.clamp(min=0)[:, None]
    if not st["backward"]:
        top = l.amax(dim=1, keepdim=True)
        lse = (l - top).exp().sum(dim=1).log() + top[:, 0]
        return torch.where(live, lse - l.gather(1, at)[:, 0], torch.zeros_like(lse)), lse
    p = torch.exp(l - st["lse"][:, None])
    p.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
    p *= torch.where(live, st["g"], torch.zeros_like(st["g"]))[:, None]
    # l = r x . W, r = (mean(x^2) + eps)^(-1/2): the norm's own share of the gradient is -x r^2/d sum_n p_n l_n
    dx = r * (p @ W) - x * (r.square() / x.shape[1]) * (p * l).sum(dim=1, keepdim=True)
    dW = (p * r).T @ x
    return dx.to(torch.bfloat16), dW.to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "int8":
        M, d, N = case["M"], case["d"], case["N"]
        rows = 2 * N if case["glu"] else N
        return {"bytes": 2 * M * d + rows * d + 4 * rows + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * d * rows}
    if op == "rope":
        n = case["M"] * case["H"] * case["hd"] * (2 if case["dtype"] == "bf16" else 4)
        turned = case["M"] * case["rot_heads"] * case["rot"]
        return {"bytes": 2 * n + 4 * case["M"] + 4 * case["rot"] * min(case["M"], case["max_pos"]), "flops": 3 * turned}
    if op == "table":
        n = case["max_pos"] * case["rot"]
        return {"bytes": 4 * n, "flops": 20 * n}
    M, d, V = case["M"], case["d"], case["V"]
    if case["backward"]:
        return {"bytes": 4 * M * d + 4 * V * d + 16 * M, "flops": 6 * M * d * V}
    return {"bytes": 2 * M * d + 2 * V * d + 16 * M, "flops": 2 * M * d * V}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"int8": _exact_int8, "rope": _exact_rope, "table": _exact_table, "head": _exact_head}[case["op"]](st)


def _exact_int8(st):
    x, Q = st["x"].double(), st["Q"].double()
    big, _ = x.abs().max(dim=1)
    codes = torch.round(x.mul(127.0).div(big.unsqueeze(1)))
    z = torch.einsum("mk,nk->mn", codes, Q)
    z = z * (st["s"].double() * 1.0).unsqueeze(0) * (big / 127.0).unsqueeze(1)
    if st["norm"]:
        z = z / torch.sqrt((x * x).sum(dim=1) / x.shape[1] + st["eps"]).unsqueeze(1)
    if not st["glu"]:
        return z
    rows = torch.arange(z.shape[1], device=z.device)
    gate, up = z[:, (rows // 16) % 2 == 0], z[:, (rows // 16) % 2 == 1]
    return gate * torch.sigmoid(gate) * up


def _exact_rope(st):
    x, rot = st["x"].double(), st["rot"]
    turn = torch.view_as_complex(st["cs"].double()[st["pos"].long()]).unsqueeze(1)
    if st["backward"]:
        turn = turn.conj()
    head, tail = x[..., :rot], x[..., rot:]
    if st["layout"] == "half":
        pairs = head.reshape(*head.shape[:-1], 2, rot // 2).transpose(-1, -2)
    else:
        pairs = head.reshape(*head.shape[:-1], rot // 2, 2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    if st["layout"] == "half":
        turned = turned.transpose(-1, -2)
    y = torch.cat([turned.reshape(head.shape), tail], dim=-1)
    keep = torch.arange(x.shape[1], device=x.device) >= st["rot_heads"]
    return torch.where(keep[None, :, None], x, y)


def _exact_table(st):
    L = np.longdouble
    D, s = st["rot"], L(st["factor"])
    base, kind = L(st["base"]), st["scaling"]
    if kind == "ntk":
        base = base * s ** (L(D) / L(D - 2))
    freq = np.exp(-np.log(base) * np.arange(0, D, 2).astype(L) / L(D))
    if kind == "linear":
        freq = freq / s
    if kind == "yarn":
        turns = L(st["original"]) * freq / (2 * L(math.pi))
        mix = np.minimum(np.maximum((turns - 1) / L(31), L(0)), L(1))
        freq = (1 - mix) * freq / s + mix * freq
    ang = np.outer(np.arange(st["max_pos"]).astype(L), freq)
    size = L(1) + L("0.1") * np.log(s) if kind == "yarn" else L(1)
    ang = ang.astype(np.float64)
    return torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], axis=-1) * float(size))


def _exact_head(st):
    x, W, t = st["x"].double(), st["W"].double(), st["t"]
    ms = (x * x).sum(dim=1) / x.shape[1] + st["eps"]
    logits = torch.einsum("mk,nk->mn", x / ms.sqrt().unsqueeze(1), W)
    rows = torch.arange(len(t), device=t.device)
    live = t >= 0
    if not st["backward"]:
        lse = torch.logsumexp(logits, dim=1)
        loss = lse - logits[rows, t.clamp(min=0)]
        loss[~live] = 0
        return loss, lse
    d_logits = torch.exp(logits - st["lse"].double().unsqueeze(1))
    d_logits[rows[live], t[live]] -= 1
    d_logits *= (st["g"].double() * live).unsqueeze(1)
    xn = x / ms.sqrt().unsqueeze(1)
    d_xn = d_logits @ W
    dx = (d_xn - xn * (d_xn * xn).mean(dim=1, keepdim=True)) / ms.sqrt().unsqueeze(1)
    return dx, d_logits.T @ xn
