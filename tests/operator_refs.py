"""Plain restatements of the operators around the W4A8 layer (norm, rotation,
gated layer's gradient, cross entropy) for their tests: numpy, 64 bits, except
where the definition itself rounds to 32 or 16 bits."""
import numpy as np
import torch

import oracle

F32 = np.float32


def bf16_round(v):
    """To bf16 (nearest even) and back, as float64."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def to_bf16(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float64)).to(torch.bfloat16)


def f64(t):
    """A torch tensor (any float type, any device) as float64 numpy."""
    return t.detach().cpu().double().numpy()


def hadamard():
    """H_256 in float64: the four-fold Kronecker power of h4 over 16."""
    h4 = 1.0 - 2.0 * np.eye(4)[::-1]
    h = np.kron(np.kron(h4, h4), np.kron(h4, h4))
    return h / 16.0


def rotate64(v):
    M, K = v.shape
    return (v.reshape(M, K // 256, 256) @ hadamard()).reshape(M, K)


def rotate32(v):
    """The rotation in fp32, in its defined order: digits of stride 1, 4, 16,
    64; a quadruple becomes ((v0 + v1) + (v2 + v3)) - 2 v[3 - a]; then / 16."""
    M, K = v.shape
    t = v.astype(F32).reshape(M, K // 256, 4, 4, 4, 4)  # strides 64, 16, 4, 1
    for axis in (5, 4, 3, 2):
        q = [np.take(t, i, axis=axis) for i in range(4)]
        s = (q[0] + q[1]) + (q[2] + q[3])
        t = np.stack([s - F32(2) * q[3 - a] for a in range(4)], axis=axis)
    assert t.dtype == F32
    return (t * F32(0.0625)).reshape(M, K)


def norm_quant(x, gamma, eps, residual=None, mp=None, qmax=127):
    """cr_rmsnorm_quant_act bit for bit.  x, residual: float64 holding bf16
    values; gamma: float32.  Returns (xq, xs, h, rs)."""
    M, K = x.shape
    mp = M if mp is None else mp
    h = x if residual is None else bf16_round((x.astype(F32) + residual.astype(F32)).astype(np.float64))
    rs = (1.0 / np.sqrt((h * h).sum(1) / K + eps)).astype(F32)
    with np.errstate(under="ignore"):
        r = rotate32((h.astype(F32) * rs[:, None]) * gamma[None, :])
    amax = np.abs(r).max(1) if K else np.zeros(M, F32)
    xs = np.ones(mp, F32)
    xs[:M] = np.where(amax > 0, amax / F32(qmax), F32(1))
    xq = np.zeros((mp, K), np.int8)
    xq[:M] = np.clip(np.rint(r / xs[:M, None]), -qmax, qmax).astype(np.int8)
    return xq, xs, h, rs


def norm_backward(dr, h, gamma, rs, dres=None):
    """The gradient in float64, and the sums of magnitudes that bound fp32
    rounding: (dx, dgamma, bound of dx's fp32 error / 2^-24, the same of dgamma)."""
    M, K = dr.shape
    dv = rotate64(dr)
    av = np.abs(dr).reshape(M, K // 256, 256).sum(2).repeat(256, 1) / 16  # sum |dr| over the block
    xh = h * rs[:, None]
    g = dv * gamma
    c = (g * xh).mean(1, keepdims=True)
    dx = rs[:, None] * (g - xh * c)
    # dv carries 12 roundings (8 additions, 4 products by 2 fused with them, the
    # 1/16 exact) of at most av each; products and the final sum 6 more; c is a
    # sum in chains of at most K / 64 + 64 terms.
    ac = (np.abs(gamma) * av * np.abs(xh)).mean(1, keepdims=True)
    e_dx = np.abs(rs[:, None]) * (18 * np.abs(gamma) * av + (K / 64 + 64 + 18) * np.abs(xh) * ac)
    if dres is not None:
        dx = dx + dres
        e_dx = e_dx + np.abs(dx) + np.abs(dres)
    dgamma = (dv * xh).sum(0)
    e_dg = ((M + 18) * av * np.abs(xh)).sum(0)
    return dx, dgamma, e_dx, e_dg


def assert_bf16_near(got, ref, e32, what="", extra=0.0):
    """got (bf16 tensor) is ref rounded once, after fp32 arithmetic whose
    error is at most e32 * 2^-24 (and `extra` more)."""
    g = f64(got)
    e = e32 * 2.0 ** -24 + extra
    bad = np.abs(g - ref) > 2.0 ** -8 * (np.abs(ref) + e) + e + 2.0 ** -133
    assert not bad.any(), f"{what}: {int(bad.sum())} of {g.size} off, worst {np.abs(g - ref)[bad].max()}"


def grid(layer):
    """The int8 grid of a layer (inputs.Layer) as float64."""
    return oracle.decode_w8(layer.qdata, layer.srel, layer.codebook).astype(np.float64)


def logits64(layer, xq, xs):
    """The layer's outputs in float64 from int8 activations."""
    y = (xq.astype(np.float64) @ grid(layer).T) * xs.astype(np.float64)[:, None] * layer.s_channel.astype(np.float64)
    return y if layer.bias is None else y + layer.bias.astype(np.float64)


def gradient_weight(layer):
    """w[n, k] = bf16(w8 * bf16(s_channel)), as float64."""
    return bf16_round(grid(layer) * bf16_round(layer.s_channel)[:, None])


def swiglu_backward(layer, xq, xs, dout):
    """(dx, dz, bound of dz's fp32 error / 2^-24, bound of dx's error) of a
    gated layer with interleaved rows, float64."""
    z = logits64(layer, xq, xs)
    g, u = z[:, 0::2], z[:, 1::2]
    s = 0.5 * (1 + np.tanh(0.5 * g))
    dz = np.empty_like(z)
    dz[:, 0::2] = dout * u * s * (1 + g * (1 - s))
    dz[:, 1::2] = dout * g * s
    # g and u carry 4 roundings each (float(acc), two products, the bias), with
    # the bias's share bounded by |y| + |bias|; the derivatives of the three
    # factors are at most 1 + |g| in size; exp, the fast division and the
    # products add about 16 more.
    b = 0.0 if layer.bias is None else 2 * np.abs(layer.bias)
    eg, eu = 4 * (np.abs(g) + (b if np.isscalar(b) else b[0::2])), 4 * (np.abs(u) + (b if np.isscalar(b) else b[1::2]))
    e = np.empty_like(z)
    e[:, 0::2] = np.abs(dout) * (np.abs(u) * (1 + np.abs(g)) * (16 + eg) + eu * (1 + np.abs(g)))
    e[:, 1::2] = np.abs(dout) * (np.abs(g) * 16 + eg * (1 + np.abs(g)))
    w = gradient_weight(layer)
    # dz is rounded to bf16 (2^-8) before the contraction; fp32 accumulation
    # of N terms
    e_dx = (2.0 ** -8 * np.abs(dz) + 2.0 ** -23 * e) @ np.abs(w) + z.shape[1] * 2.0 ** -24 * (np.abs(dz) @ np.abs(w))
    return dz @ w, dz, e, e_dx


def cross_entropy(layer, xq, xs, targets, ignore=-100):
    """(loss, lse, logits) in float64."""
    y = logits64(layer, xq, xs)
    m = y.max(1)
    base = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        lse = base + np.log(np.exp(y - base[:, None]).sum(1))
    ok = targets != ignore
    loss = np.zeros(len(lse))
    valid = ok & (targets >= 0) & (targets < y.shape[1])
    loss[valid] = lse[valid] - y[valid, targets[valid]]
    loss[ok & ~valid] = np.nan
    return loss, lse, y


def cross_entropy_backward(layer, xq, xs, targets, lse, dloss, ignore=-100):
    """(dx, bound of its error before the last rounding) in float64."""
    y = logits64(layer, xq, xs)
    p = np.exp(y - lse[:, None])
    hot = np.zeros_like(p)
    ok = targets != ignore
    hot[ok, targets[ok]] = 1.0
    d = np.where(ok, dloss, 0.0)[:, None] * (p - hot)
    assert np.isfinite(d).all()
    w = gradient_weight(layer)
    # an exponential: its argument's fp32 error (logit, lse and product, 2^-24
    # of each magnitude, 4 roundings) and 2^-22 of the unit's own; then bf16
    ay = np.where(p > 0, np.abs(y), 0.0)  # a masked entry has no error
    e = np.where(ok, np.abs(dloss), 0.0)[:, None] * p * (4 * (ay + np.abs(lse)[:, None]) + 8) * 2.0 ** -24
    e_dx = (2.0 ** -8 * np.abs(d) + 2 * e + 2.0 ** -133) @ np.abs(w)
    e_dx = e_dx + y.shape[1] * 2.0 ** -24 * (np.abs(d) @ np.abs(w))
    return d @ w, e_dx
