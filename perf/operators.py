"""The training and serving operators around the W4A8 linear layer, as cases to
be timed: a plain form of each in elementary torch operations, and the call a
user makes of this package.

  norm_fwd    residual addition + RMS norm + block rotation + per-token int8
  norm_bwd    its gradient (the rotation's and the norm's backward, dgamma)
  rotate      the block rotation alone, bf16 to bf16 (its own backward)
  ffn_bwd     gradient of a gated (SwiGLU) layer: both projections recomputed
              from the packed codes, the activation's gradient, the input's
  ce_fwd      softmax cross entropy over the outputs of a W4A8 head
  ce_bwd      the gradient of that loss with respect to the head's input

A case's "op" is one of these names.  M is rows (tokens), K the layer's input
width (a multiple of 256, the rotation block), F the gated layer's width, V the
vocabulary.  The int8 activations of norm_fwd are returned as the bf16 values
they stand for (xq * xs).
"""
import math

import torch

own = False

ROT, GROUP, QMAX, IGNORE, EPS = 256, 16, 127, -100, 1e-6

# 16 sorted levels of a 4-bit codebook for normalised Gaussian groups
LEVELS = (-0.980602, -0.794529, -0.638165, -0.500986, -0.377321, -0.263187, -0.155210, -0.050720,
          0.052541, 0.156985, 0.265284, 0.379533, 0.502636, 0.638953, 0.794876, 0.980671)


def listed():
    return [
        # one decode step of a batch of eight sequences: the norm before a projection
        {"name": "norm decode 8x4096", "op": "norm_fwd", "M": 8, "K": 4096, "residual": True, "gamma": "bf16"},
        # the largest prefill batch of the benchmark
        {"name": "norm prefill 16384x8192", "op": "norm_fwd", "M": 16384, "K": 8192, "residual": True, "gamma": "bf16"},
        # a short ragged fine-tuning batch, no gradient on the residual path (the last norm), fp32 weight
        {"name": "norm bwd 100x1280", "op": "norm_bwd", "M": 100, "K": 1280, "residual": False, "gamma": "f32"},
        # a training batch of 4096-wide layers
        {"name": "norm bwd 8192x4096", "op": "norm_bwd", "M": 8192, "K": 4096, "residual": True, "gamma": "bf16"},
        # the gradient of a down projection's input for a few tokens
        {"name": "rotate 33x12288", "op": "rotate", "M": 33, "K": 12288},
        # the same for the benchmark's MLP pair
        {"name": "rotate 4096x12288", "op": "rotate", "M": 4096, "K": 12288},
        # a small adapter run with a ragged last batch
        {"name": "ffn bwd 333x1280", "op": "ffn_bwd", "M": 333, "F": 1412, "K": 1280, "bias": True},
        # a training step of the benchmark's MLP (12288 rows: gate and up interleaved)
        {"name": "ffn bwd 4096x4096", "op": "ffn_bwd", "M": 4096, "F": 6144, "K": 4096, "bias": False},
        # scoring one next token for eight sequences
        {"name": "ce score 8x32768", "op": "ce_fwd", "M": 8, "V": 32768, "K": 4096, "ignored": 0.0, "bias": False},
        # evaluation loss on a batch with padding, odd vocabulary
        {"name": "ce fwd 2048x50021", "op": "ce_fwd", "M": 2048, "V": 50021, "K": 2048, "ignored": 0.2, "bias": False},
        # a small training batch, odd vocabulary, half of it prompt tokens without a loss
        {"name": "ce bwd 500x10007", "op": "ce_bwd", "M": 500, "V": 10007, "K": 1024, "ignored": 0.5, "bias": True},
        # a training batch against a large vocabulary
        {"name": "ce bwd 4096x65536", "op": "ce_bwd", "M": 4096, "V": 65536, "K": 4096, "ignored": 0.1, "bias": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "rotate", "ffn_bwd", "ce_fwd", "ce_bwd"))
    if op in ("norm_fwd", "norm_bwd", "rotate"):
        K = ROT * _log_int(rng, 1, 128)
        M = _log_int(rng, 1, min(32768, 16384 * 8192 // K))
        if op == "rotate":
            return {"op": op, "M": M, "K": K}
        return {"op": op, "M": M, "K": K, "residual": rng.random() < 0.7, "gamma": rng.choice(("bf16", "f32"))}
    K = ROT * _log_int(rng, 1, 32)
    if op == "ffn_bwd":
        F = 4 * _log_int(rng, 16, 4096)
        M = _log_int(rng, 1, min(8192, 4096 * 6144 * 4096 // (F * K)))
        return {"op": op, "M": M, "F": F, "K": K, "bias": rng.random() < 0.3}
    V = _log_int(rng, 500, min(131072, 65536 * 4096 // K))
    M = _log_int(rng, 1, min(8192, 4096 * 65536 * 4096 // (V * K), 4096 * 65536 // V))
    return {"op": op, "M": M, "V": V, "K": K, "ignored": rng.choice((0.0, 0.1, 0.5)), "bias": rng.random() < 0.3}


# ---------------------------------------------------------------- inputs

def _hidden(g, M, K):
    """Hidden states: N(0, 1) with one percent of the channels twenty times larger."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 20
    return x.to(torch.bfloat16)


def _quantised(g, M, K):
    """Rotated int8 activations as the layer makes them: Gaussian rows whose largest value is 127."""
    z = torch.randn(M, K, generator=g, device="cuda")
    xq = (z * (QMAX / z.abs().amax(1, keepdim=True))).round().to(torch.int8)
    return xq, torch.rand(M, generator=g, device="cuda") * 0.04 + 0.03


def _layer(g, N, K, bias):
    """A packed layer: uniform codes, group scales U[32, 128], channel scales U[1e-4, 5e-4]."""
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(N, K // GROUP, generator=g, device="cuda") * 96 + 32).to(torch.float8_e4m3fn).view(torch.uint8)
    c = torch.rand(N, generator=g, device="cuda") * 4e-4 + 1e-4
    b = torch.randn(N, generator=g, device="cuda") * 0.1 if bias else None
    return {"qdata": q, "srel": s, "codebook": torch.tensor(LEVELS, device="cuda"), "s_channel": c, "bias": b}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    st = {"op": op}
    if op in ("norm_fwd", "norm_bwd"):
        gamma = 1 + 0.1 * torch.randn(K, generator=g, device="cuda")
        st["gamma"] = gamma.to(torch.bfloat16) if case["gamma"] == "bf16" else gamma
    if op == "norm_fwd":
        st["x"] = _hidden(g, M, K)
        st["residual"] = _hidden(g, M, K) if case["residual"] else None
        st["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    elif op == "norm_bwd":
        st["h"] = _hidden(g, M, K)
        st["rs"] = (st["h"].double().square().mean(1) + EPS).rsqrt().float()
        st["dr"] = (0.01 * torch.randn(M, K, generator=g, device="cuda")).to(torch.bfloat16)
        st["dres"] = (0.01 * torch.randn(M, K, generator=g, device="cuda")).to(torch.bfloat16) if case["residual"] else None
    elif op == "rotate":
        st["x"] = (0.01 * torch.randn(M, K, generator=g, device="cuda")).to(torch.bfloat16)
    elif op == "ffn_bwd":
        st.update(_layer(g, 2 * case["F"], K, case["bias"]))
        st["xq"], st["xs"] = _quantised(g, M, K)
        st["dout"] = (0.01 * torch.randn(M, case["F"], generator=g, device="cuda")).to(torch.bfloat16)
    else:
        V = case["V"]
        st.update(_layer(g, V, K, case["bias"]))
        st["xq"], st["xs"] = _quantised(g, M, K)
        t = torch.randint(0, V, (M,), generator=g, device="cuda")
        skip = torch.rand(M, generator=g, device="cuda") < case["ignored"]
        skip[0] = False  # a batch has at least one row with a loss
        st["targets"] = t.masked_fill(skip, IGNORE)
        if op == "ce_bwd":
            valid = (st["targets"] != IGNORE).sum().clamp(min=1)
            st["dloss"] = (1.0 / valid).float().expand(M).contiguous()
            st["lse"] = _lse(_logits(st))
    return st


# ---------------------------------------------------------------- plain forms

def _hadamard(dtype):
    h4 = 1 - 2 * torch.eye(4, dtype=dtype, device="cuda").flip(1)
    h = torch.kron(h4, h4)
    return torch.kron(h, h) / 16


def _rotated(v):
    M, K = v.shape
    return (v.reshape(M, K // ROT, ROT) @ _hadamard(v.dtype)).reshape(M, K)


def _decoded(st):
    """The layer's int8 grid as fp32 values [N, K]."""
    q = st["qdata"]
    N, half = q.shape
    codes = torch.stack([q & 15, q >> 4], dim=2).reshape(N, 2 * half)
    s = st["srel"].view(torch.float8_e4m3fn).float()
    w = (st["codebook"][codes.int()].reshape(N, -1, GROUP) * s[:, :, None]).reshape(N, 2 * half)
    return w.round_().clamp_(-128, 127)


def _logits(st, w8=None):
    """The layer's fp32 outputs."""
    w8 = _decoded(st) if w8 is None else w8
    y = st["xq"].float() @ w8.T
    y *= st["xs"][:, None] * st["s_channel"]
    return y if st["bias"] is None else y.add_(st["bias"])


def _lse(logits):
    m = logits.amax(1)
    return m + (logits - m[:, None]).exp_().sum(1).log()


def _gradient_weight(st, w8):
    """The straight-through backward's weight: the grid times the bf16 channel scale, in bf16."""
    return (w8 * st["s_channel"].to(torch.bfloat16).float()[:, None]).to(torch.bfloat16).float()


def _plain(st):
    op = st["op"]
    if op == "norm_fwd":
        h = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(torch.bfloat16)
        rs = (1 / (h.double().square().mean(1) + EPS).sqrt()).float()
        r = _rotated(h.float() * rs[:, None] * st["gamma"].float())
        xs = r.abs().amax(1) / QMAX
        xs = torch.where(xs > 0, xs, torch.ones_like(xs))
        xq = (r / xs[:, None]).round().clamp(-QMAX, QMAX)
        return {"values": (xq * xs[:, None]).to(torch.bfloat16), "xs": xs, "h": h, "rs": rs}
    if op == "norm_bwd":
        dv = _rotated(st["dr"].float())
        xh = st["h"].float() * st["rs"][:, None]
        gr = dv * st["gamma"].float()
        dx = (gr - xh * (gr * xh).mean(1, keepdim=True)) * st["rs"][:, None]
        if st["dres"] is not None:
            dx = dx + st["dres"].float()
        return {"dx": dx.to(torch.bfloat16), "dgamma": (dv * xh).sum(0)}
    if op == "rotate":
        return _rotated(st["x"].float()).to(torch.bfloat16)
    w8 = _decoded(st)
    z = _logits(st, w8)
    if op == "ffn_bwd":
        gate, up, do = z[:, 0::2], z[:, 1::2], st["dout"].float()
        s = 1 / (1 + (-gate).exp())
        dz = torch.stack([do * up * s * (1 + gate * (1 - s)), do * gate * s], dim=2).reshape(z.shape)
        return {"dx": (dz @ _gradient_weight(st, w8)).to(torch.bfloat16), "dz": dz.to(torch.bfloat16)}
    t, valid = st["targets"].clamp(min=0), st["targets"] != IGNORE
    if op == "ce_fwd":
        lse = _lse(z)
        return {"loss": torch.where(valid, lse - z.gather(1, t[:, None])[:, 0], torch.zeros_like(lse)), "lse": lse}
    d = z.sub_(st["lse"][:, None]).exp_()
    d[torch.arange(len(t), device=t.device), t] -= 1
    d *= torch.where(valid, st["dloss"], torch.zeros_like(st["dloss"]))[:, None]
    return (d @ _gradient_weight(st, w8)).to(torch.bfloat16)


# ---------------------------------------------------------------- this package

def _package(st):
    import w4a8_codebook_quantized_b200 as cr
    op = st["op"]
    if op == "norm_fwd":
        xq, xs, h, rs = cr.cr_rmsnorm_quant_act(st["x"], st["gamma"], EPS, residual=st["residual"])
        return {"values": torch.mul(xq, xs[:, None], out=st["values"]), "xs": xs, "h": h, "rs": rs}
    if op == "norm_bwd":
        dx, dgamma = cr.cr_rmsnorm_backward(st["dr"], st["h"], st["gamma"], st["rs"], dres=st["dres"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "rotate":
        return cr.cr_rotate(st["x"])
    layer = (st["qdata"], st["srel"], st["codebook"], st["s_channel"])
    if op == "ffn_bwd":
        dx, dz = cr.cr_w4a8_swiglu_backward(st["dout"], st["xq"], st["xs"], *layer, bias=st["bias"])
        return {"dx": dx, "dz": dz}
    if op == "ce_fwd":
        loss, lse = cr.cr_w4a8_cross_entropy(st["xq"], st["xs"], *layer, st["targets"], bias=st["bias"],
                                             ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    return cr.cr_w4a8_cross_entropy_backward(st["xq"], st["xs"], *layer, st["targets"], st["lse"], st["dloss"],
                                             bias=st["bias"], ignore_index=IGNORE)


def run(state):
    if own:
        return _package(state)
    return _plain(state)


# ---------------------------------------------------------------- floors

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "norm_fwd":
        ins = 4 if case["residual"] else 2
        return {"bytes": M * K * (ins + (2 if case["residual"] else 0) + 1) + 8 * M + 2 * K, "flops": 20 * M * K}
    if op == "norm_bwd":
        return {"bytes": M * K * (8 if case["residual"] else 6) + 4 * M + 6 * K, "flops": 20 * M * K}
    if op == "rotate":
        return {"bytes": 4 * M * K, "flops": 11 * M * K}
    N = 2 * case["F"] if op == "ffn_bwd" else case["V"]
    layer = N * K // 2 + N * K // GROUP + 4 * N
    if op == "ffn_bwd":
        return {"bytes": layer + M * K + 4 * M + M * N + 2 * M * N + 2 * M * K, "flops": 4 * M * N * K}
    if op == "ce_fwd":
        return {"bytes": layer + M * K + 20 * M, "flops": 2 * M * N * K}
    return {"bytes": layer + 3 * M * K + 20 * M, "flops": 4 * M * N * K}


# ---------------------------------------------------------------- 64-bit values

def _blocks64(v):
    """Each block of 256 as a 4 x 4 x 4 x 4 tensor; along every axis, the sum minus twice the mirrored value."""
    t = v.reshape(v.shape[0], -1, 4, 4, 4, 4)
    for axis in (2, 3, 4, 5):
        t = t.sum(axis, keepdim=True) - 2 * t.flip(axis)
    return (t / 16).reshape(v.shape)


def _grid64(st):
    """The int8 grid from a table over (scale byte, code)."""
    scales = torch.arange(256, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    table = (scales[:, None] * st["codebook"][None, :]).nan_to_num(0.0).round().clamp(-128, 127).to(torch.int8)
    N, half = st["qdata"].shape
    codes = torch.empty(N, 2 * half, dtype=torch.int32, device="cuda")
    codes[:, 0::2] = st["qdata"] % 16
    codes[:, 1::2] = st["qdata"] // 16
    codes += 16 * st["srel"].int().repeat_interleave(GROUP, dim=1)
    return table.reshape(-1)[codes]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        h = st["x"]
        if st["residual"] is not None:
            h = (st["x"].double() + st["residual"].double()).to(torch.bfloat16)  # h is defined as rounded to bf16
        h64 = h.double()
        rs = 1 / torch.sqrt((h64 * h64).sum(1) / case["K"] + EPS)
        r = _blocks64(h64 * rs[:, None] * st["gamma"].double())
        xs = r.abs().max(1).values / QMAX
        return {"values": torch.round(r / xs[:, None]) * xs[:, None], "xs": xs, "h": h64, "rs": rs}
    if op == "norm_bwd":
        h, rs, gamma = st["h"].double(), st["rs"].double()[:, None], st["gamma"].double()
        dv = _blocks64(st["dr"].double())
        gr, n = dv * gamma, h * rs
        dx = rs * gr - h * rs * rs * ((gr * n).sum(1) / case["K"])[:, None]
        if st["dres"] is not None:
            dx += st["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("mk,mk->k", dv, n)}
    if op == "rotate":
        return _blocks64(st["x"].double())
    grid = _grid64(st)
    wd = grid.double()
    l64 = torch.matmul(st["xq"].double(), wd.t()) * st["xs"].double()[:, None] * st["s_channel"].double()
    if st["bias"] is not None:
        l64 += st["bias"].double()
    # the gradient's weight is defined as rounded to bf16
    wg = (grid.float() * st["s_channel"].to(torch.bfloat16).float()[:, None]).to(torch.bfloat16)
    if op == "ffn_bwd":
        del wd
        a, b, do = l64[:, 0::2], l64[:, 1::2], st["dout"].double()
        sig = torch.sigmoid(a)
        dz = torch.empty_like(l64)
        dz[:, 0::2] = do * b * (sig + a * sig * (1 - sig))
        dz[:, 1::2] = do * a * sig
        return {"dx": torch.matmul(dz, wg.double()), "dz": dz}
    keep = st["targets"] >= 0
    if op == "ce_fwd":
        lse = torch.logsumexp(l64, 1)
        rows = torch.nonzero(keep)[:, 0]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - l64[rows, st["targets"][rows]]
        return {"loss": loss, "lse": lse}
    del wd
    l64 -= st["lse"].double()[:, None]
    l64.exp_()
    rows = torch.nonzero(keep)[:, 0]
    l64[rows, st["targets"][rows]] -= 1
    l64 *= (st["dloss"].double() * keep)[:, None]
    return torch.matmul(l64, wg.double())
