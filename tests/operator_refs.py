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


def silence_targets(layer, entries):
    """Zero group scales, so zero weights, in a head's rows `entries`: as targets
    they leave only the softmax part of the gradient, which the target's -1
    otherwise outweighs by far."""
    layer.srel[entries] = 0
    return layer


def softmax_gradient(layer, xq, xs, lse, dloss, device="cpu", drop=None, columns=8192):
    """The cross entropy's input gradient of rows whose targets have zero
    weights, and the size of its error: (dx, sigma) float64 tensors, sigma the
    root of the sum of the squares of its terms, computed `columns` vocabulary
    entries at a time.  drop = (a, b): without the entries a .. b - 1 (a planted
    mistake)."""
    t64 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.float64), device=device)
    x, scale, base, d = t64(xq), t64(xs)[:, None], t64(lse)[:, None], t64(dloss)[:, None]
    dx, sq = torch.zeros_like(x), torch.zeros_like(x)
    for a in range(0, layer.N, columns):
        s = slice(a, min(a + columns, layer.N))
        w8 = t64(oracle.decode_w8(layer.qdata[s], layer.srel[s], layer.codebook))
        ch = torch.as_tensor(layer.s_channel[s], device=device)
        y = (x @ w8.T) * scale * ch.double()
        if layer.bias is not None:
            y += t64(layer.bias[s])
        p = torch.exp(y - base) * d
        if drop is not None:
            p[:, max(0, drop[0] - a):max(0, drop[1] - a)] = 0
        w = (w8 * ch.to(torch.bfloat16).double()[:, None]).to(torch.bfloat16).double()
        dx += p @ w
        sq += (p * p) @ (w * w)
    return dx, sq.sqrt()


def assert_sum_of_random_terms(got, ref, sigma, terms, rel=0.0, what=""):
    """got (bf16) is ref, a sum of `terms` products of signs that are
    independent of the errors, each factor rounded to bf16 once at most
    (2^-8), added up in fp32 in any order, rounded once.

    A sum of terms a_i e_i with |e_i| <= 2^-8 and random signs is beyond 7 *
    2^-8 * sigma, sigma^2 = sum a_i^2, with a probability of 2 exp(-49 / 2) =
    5e-11 (Hoeffding).  The sum's own roundings: terms / 16 additions of the
    tensor core's groups (and some 64 of a split's joining), each cut off by at
    most 2^-23 of a partial sum, which is below 7 sigma by the same bound (plus
    the mean's share, below |ref|).  rel: an error all terms have in common."""
    g = got.double().cpu()
    r, s = ref.cpu(), sigma.cpu()
    add = (terms / 16 + 64) * 2.0 ** -23 * (7 * s + r.abs())
    inner = 7 * 2.0 ** -8 * s + add + rel * r.abs()
    bad = (g - r).abs() > 2.0 ** -8 * (r.abs() + inner) + inner + 2.0 ** -133
    assert not bad.any(), f"{what}: {int(bad.sum())} of {g.numel()} off"
