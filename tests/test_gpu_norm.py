"""The norm with int8 output, its gradient, and the rotation alone, on the GPU
against 64-bit restatements (bit for bit where the definition fixes every
rounding)."""
import numpy as np
import pytest
import torch

import w4a8_codebook_quantized_b200 as cr
from w4a8_codebook_quantized_b200 import inputs

from gpu_util import Guarded, bf16_dev, dev, host
from operator_refs import (assert_bf16_near, bf16_round, f64, norm_backward, norm_quant, rotate32, to_bf16)

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cr.lib()
    yield
    cr.cr_check_device_error()


def _bf16(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _gamma(K, seed, dtype):
    g = 1 + 0.1 * np.random.default_rng([seed, 77]).standard_normal(K)
    if dtype == torch.bfloat16:
        return bf16_round(g).astype(np.float32)
    return g.astype(np.float32)


def _check_forward(xb, rb, gamma, gdt, MP, eps=EPS, qmax=127, alias=None):
    M, K = xb.shape
    x = bf16_dev(xb)
    r = None if rb is None else bf16_dev(rb)
    g = dev(gamma).to(gdt)
    xq, xs, rs = Guarded((MP, K), torch.int8), Guarded((MP,), torch.float32), Guarded((M,), torch.float32)
    hg = Guarded((M, K), torch.bfloat16)
    h = None if rb is None else {"x": x, "residual": r, None: hg.tensor}[alias]
    _, _, h_out, _ = cr.cr_rmsnorm_quant_act(x, g, eps, residual=r, mp=MP, act_qmax=qmax, h=h, xq=xq.tensor,
                                             xs=xs.tensor, rs=rs.tensor)
    torch.cuda.synchronize()
    assert xq.intact() and xs.intact() and rs.intact() and hg.intact()
    q_ref, s_ref, h_ref, rs_ref = norm_quant(_bf16(xb), gamma, eps, None if rb is None else _bf16(rb), MP, qmax)
    assert np.array_equal(f64(h_out), h_ref)
    assert np.array_equal(host(rs.tensor), rs_ref)
    assert np.array_equal(host(xs.tensor), s_ref)
    assert np.array_equal(host(xq.tensor), q_ref)


@pytest.mark.parametrize("M,K,MP", [(1, 256, 1), (3, 1024, 4), (8, 4096, 8), (5, 4096, 8), (2, 8192, 2), (4, 12288, 4),
                                    (2, 16384, 2), (2, 20480, 2), (1, 65536, 1), (33, 768, 33), (100, 256, 100),
                                    (40, 1280, 40), (17, 4096, 40), (24, 12288, 24), (17, 16384, 17), (20, 24576, 20),
                                    (17, 40960, 17), (300, 4096, 300), (17, 131072, 17), (17, 256, 27), (45, 512, 45),
                                    (19, 1024, 30), (21, 768, 21), (18, 32768, 18), (27, 1280, 34), (19, 1536, 19),
                                    (40, 2560, 40), (20, 3328, 20), (30, 5120, 31), (20, 6912, 20), (18, 10240, 18),
                                    (18, 13824, 18)])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
def test_norm_quant_shapes(M, K, MP, gdt):
    """Every CTA size and holding depth of both forms, with a residual for
    every other shape, padding rows, and both types of the weight."""
    res = (M + K // 256) % 2 == 0
    xb = inputs.activations(M, K, M + K)
    rb = inputs.activations(M, K, M + K + 1) if res else None
    _check_forward(xb, rb, _gamma(K, M, gdt), gdt, MP)


@pytest.mark.parametrize("M,K", [(2, 20480), (3, 512), (20, 24576), (20, 768)])
@pytest.mark.parametrize("alias", ["x", "residual"])
def test_norm_quant_updates_the_residual_in_place(M, K, alias):
    xb, rb = inputs.activations(M, K, 3), inputs.activations(M, K, 4)
    _check_forward(xb, rb, _gamma(K, 5, torch.float32), torch.float32, M, alias=alias)


@pytest.mark.parametrize("reps", [1, 4])
@pytest.mark.parametrize("qmax,eps", [(127, 1e-6), (7, 1e-5), (127, 1e-30), (1, 1.0)])
def test_norm_quant_degenerate_rows(reps, qmax, eps):
    """Zero rows, rows of one value, one-hot rows, rows whose squares pass
    fp32 at both ends, and a weight with zeros and a large entry."""
    K = 768
    rows = np.zeros((7, K))
    rows[1, :7] = 2.0 ** -100
    rows[2] = np.linspace(-2.0 ** 100, 2.0 ** 100, K)
    rows[3, 300] = -1.0
    rows[4] = 1.0
    rows[5, 5] = 2.0 ** -126
    rows[6] = np.where(np.arange(K) % 2, 2.0 ** 90, -2.0 ** -60)
    rows = np.tile(rows, (reps, 1))
    xb = to_bf16(rows).view(torch.int16).numpy().view(np.uint16)
    gamma = _gamma(K, 9, torch.float32)
    gamma[:3] = 0.0
    gamma[10] = 1000.0
    mp = 8 if reps == 1 else rows.shape[0]
    _check_forward(xb, None, gamma, torch.float32, mp, eps, qmax)
    _check_forward(xb, np.ascontiguousarray(xb[::-1]), gamma, torch.float32, mp, eps, qmax)


def test_norm_quant_feeds_the_layer():
    """The int8 activations are those the layer's own rotate + quantise makes
    of the same values, when the normed values are exact in bf16."""
    M, K, N = 6, 512, 96
    rng = np.random.default_rng(0)
    xb = to_bf16(rng.choice([-1.0, 1.0], size=(M, K))).view(torch.int16).numpy().view(np.uint16)
    gamma = torch.full((K,), 0.5)
    # h = +-1: mean square 1, rs = 1 / sqrt(1 + 2^-60) rounds to 1, v = +-0.5
    xq, xs, _, rs = cr.cr_rmsnorm_quant_act(bf16_dev(xb), gamma.cuda(), 2.0 ** -60, mp=8)
    assert (rs == 1).all()
    xq2, xs2 = cr.cr_rotate_quant_act(bf16_dev(xb) * 0.5, 8)
    assert torch.equal(xq, xq2) and torch.equal(xs, xs2)
    ly = inputs.layer(N, K, 3)
    w = [dev(a) for a in (ly.qdata, ly.srel, ly.codebook, ly.s_channel)]
    assert torch.equal(cr.cr_w4a8_gemv(xq, xs, *w, m=M), cr.cr_w4a8_linear(bf16_dev(xb) * 0.5, *w))


# ---------------------------------------------------------------- rotation

@pytest.mark.parametrize("M,K", [(1, 256), (3, 768), (33, 12288), (5, 131072), (700, 2048)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rotate(M, K, in_place):
    xb = inputs.activations(M, K, 11)
    x = bf16_dev(xb)
    out = Guarded((M, K), torch.bfloat16)
    got = cr.cr_rotate(x, out=x if in_place else out.tensor)
    torch.cuda.synchronize()
    assert out.intact()
    assert np.array_equal(f64(got), bf16_round(rotate32(_bf16(xb)).astype(np.float64)))


# ---------------------------------------------------------------- gradient

def _grad_inputs(M, K, seed, gdt, dres):
    rng = np.random.default_rng([seed, M, K])
    dr = to_bf16(0.01 * rng.standard_normal((M, K)))
    h = torch.from_numpy(inputs.activations(M, K, seed).view(np.int16)).view(torch.bfloat16)
    gamma = _gamma(K, seed, gdt)
    rs = (1 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).astype(np.float32)
    dd = to_bf16(0.01 * rng.standard_normal((M, K))) if dres else None
    return dr, h, gamma, rs, dd


@pytest.mark.parametrize("M,K", [(1, 256), (2, 512), (37, 1024), (100, 1280), (64, 2048), (450, 4096), (9, 4352),
                                 (200, 8192), (160, 12288), (5, 16384), (150, 16640), (3, 131072), (1500, 256),
                                 (1, 512), (9000, 256), (3001, 512), (77, 768), (400, 8448), (90, 32768), (60, 33024),
                                 (170, 49152), (40, 65536), (200, 66048), (1600, 1536), (450, 2560), (450, 2816),
                                 (310, 5120), (150, 9728), (170, 10240)])
@pytest.mark.parametrize("gdt,dres", [(torch.bfloat16, True), (torch.float32, False)])
def test_norm_backward(M, K, gdt, dres):
    dr, h, gamma, rs, dd = _grad_inputs(M, K, 21, gdt, dres)
    dx, dg = Guarded((M, K), torch.bfloat16), Guarded((K,), torch.float32)
    need = cr.lib().cr_rmsnorm_backward_work_bytes(M, K)
    work = Guarded((need,), torch.uint8)
    args = (dr.cuda(), h.cuda(), dev(gamma).to(gdt), dev(rs))
    dd_d = None if dd is None else dd.cuda()
    cr.cr_rmsnorm_backward(*args, dres=dd_d, dx=dx.tensor, dgamma=dg.tensor, work=work.tensor)
    torch.cuda.synchronize()
    assert dx.intact() and dg.intact() and work.intact()
    rx, rg, ex, eg = norm_backward(f64(dr), f64(h), gamma.astype(np.float64), rs.astype(np.float64),
                                   None if dd is None else f64(dd))
    assert_bf16_near(dx.tensor, rx, ex, "dx")
    assert (np.abs(f64(dg.tensor) - rg) <= eg * 2.0 ** -24).all()
    # again, with fresh buffers, without dgamma, and in place: the same bits
    dx2, dg2 = cr.cr_rmsnorm_backward(*args, dres=dd_d)
    assert torch.equal(dx2, dx.tensor) and torch.equal(dg2, dg.tensor)
    dx3, none = cr.cr_rmsnorm_backward(*args, dres=dd_d, with_dgamma=False)
    assert none is None and torch.equal(dx3, dx.tensor)
    over = args[0].clone()
    assert torch.equal(cr.cr_rmsnorm_backward(over, *args[1:], dres=dd_d, dx=over)[0], dx.tensor)
    if dd is not None:
        over = dd_d.clone()
        assert torch.equal(cr.cr_rmsnorm_backward(*args, dres=over, dx=over)[0], dx.tensor)


@pytest.mark.parametrize("M,K", [(19, 256), (19, 512), (19, 768), (19, 4352), (19, 12288), (19, 16640), (19, 33024)])
@pytest.mark.parametrize("dres", [False, True])
def test_norm_backward_of_large_and_small_rows(M, K, dres):
    """Rows of every size the norm takes: rs is their inverse, and its square
    leaves fp32 at both ends (rs * rs * 1e25^2 is not what the formula has)."""
    dr, h, gamma, _, dd = _grad_inputs(M, K, 71, torch.float32, dres)
    scale = 10.0 ** np.array([25, 33, -14, 0, 20, 23, 30, 34, -10, 28, 22, 19, 18, 32, 5, -5, 10, 24, 26])[:M]
    h = to_bf16(f64(h) / 20 * scale[:, None])  # inputs.activations has values up to about 100
    dr = to_bf16(f64(dr) * np.minimum(scale, 1.0)[:, None])  # dx stays a normal number
    if dd is not None:
        dd = to_bf16(f64(dd) / np.maximum(scale, 1.0)[:, None])
    eps = 1e-30
    rs = (1 / np.sqrt((f64(h) ** 2).mean(1) + eps)).astype(np.float32)
    g = gamma.astype(np.float64)
    dx, dg = cr.cr_rmsnorm_backward(dr.cuda(), h.cuda(), dev(gamma), dev(rs), dres=None if dd is None else dd.cuda())
    rx, rg, ex, eg = norm_backward(f64(dr), f64(h), g, rs.astype(np.float64), None if dd is None else f64(dd))
    assert_bf16_near(dx, rx, ex, "dx")
    assert (np.abs(f64(dg) - rg) <= eg * 2.0 ** -24).all()


def test_norm_backward_against_differences():
    """The gradient against central differences of the forward's real-valued
    function: sum(dr * R(norm(h) * gamma)), in float64."""
    from operator_refs import rotate64
    M, K = 2, 256
    dr, h, gamma, _, _ = _grad_inputs(M, K, 31, torch.float32, False)
    h64, g64, dr64 = f64(h), gamma.astype(np.float64), f64(dr)

    def loss(hh, gg):
        return (dr64 * rotate64(hh / np.sqrt((hh ** 2).mean(1, keepdims=True) + EPS) * gg)).sum()

    rs = 1 / np.sqrt((h64 ** 2).mean(1) + EPS)
    dx, dg = cr.cr_rmsnorm_backward(dr.cuda(), h.cuda(), dev(gamma), dev(rs.astype(np.float32)))
    dx, dg = f64(dx), f64(dg)
    step = 1e-5
    for m, k in ((0, 0), (0, 17), (1, 255), (1, 100)):
        e = np.zeros_like(h64)
        e[m, k] = step
        d = (loss(h64 + e, g64) - loss(h64 - e, g64)) / (2 * step)
        # bf16 output (2^-8), the difference's own error (step^2) far below it
        assert abs(dx[m, k] - d) <= 2.0 ** -8 * abs(d) + 1e-6 * np.abs(dx).max()
    for k in (0, 99, 255):
        e = np.zeros_like(g64)
        e[k] = step
        d = (loss(h64, g64 + e) - loss(h64, g64 - e)) / (2 * step)
        assert abs(dg[k] - d) <= 1e-5 * np.abs(dg).max()


def test_norm_backward_of_no_rows():
    K = 512
    z = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    dx, dg = cr.cr_rmsnorm_backward(z, z, torch.ones(K, device="cuda"), torch.empty(0, device="cuda"),
                                    dgamma=torch.full((K,), 7.0, device="cuda"))
    assert dx.shape == (0, K) and (dg == 0).all()
    assert cr.cr_rotate(z).shape == (0, K)
    xq, xs, h, rs = cr.cr_rmsnorm_quant_act(z, torch.ones(K, device="cuda"), mp=4)
    assert (xq == 0).all() and (xs == 1).all() and rs.shape == (0,)


# ---------------------------------------------------------------- streams, graphs, refusals

def test_norm_on_another_stream_and_in_a_graph():
    M, K = 40, 1024
    dr, h, gamma, rs, dd = _grad_inputs(M, K, 41, torch.float32, True)
    x, r, g = h.cuda(), dd.cuda(), dev(gamma)

    def step(**kw):
        xq, xs, hh, rr = cr.cr_rmsnorm_quant_act(x, g, EPS, residual=r, **kw)
        dx, dg = cr.cr_rmsnorm_backward(dr_d, hh, g, rr, dres=r, **kw)
        return xq, xs, hh, rr, dx, dg, cr.cr_rotate(dx, **kw)

    dr_d = dr.cuda()
    ref = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for kw in ({"stream": s}, {"stream": s.cuda_stream}):
        got = step(**kw)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        x.copy_(bf16_dev(inputs.activations(M, K, seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(), out))


def _shifted(t):
    """The same values 16 bytes past a 512-byte boundary: rows that are not
    aligned to 32 bytes."""
    raw = torch.empty(t.numel() * t.element_size() + 16, dtype=torch.uint8, device="cuda")
    out = raw[16:].view(t.dtype).view(t.shape)
    out.copy_(t)
    assert out.data_ptr() % 32 == 16
    return out


@pytest.mark.parametrize("M,K", [(3, 1024), (3, 20480), (40, 768), (40, 36864), (200, 2048)])
def test_norm_of_rows_aligned_to_16_bytes_only(M, K):
    dr, h, gamma, rs, dd = _grad_inputs(M, K, 51, torch.float32, True)
    dr, x, g, rs, r = dr.cuda(), h.cuda(), dev(gamma), dev(rs), dd.cuda()
    ref = [*cr.cr_rmsnorm_quant_act(x, g, EPS, residual=r), *cr.cr_rmsnorm_backward(dr, x, g, rs, dres=r),
           cr.cr_rotate(x)]
    sx, sr, sdr = _shifted(x), _shifted(r), _shifted(dr)
    got = [*cr.cr_rmsnorm_quant_act(sx, _shifted(g), EPS, residual=sr, h=_shifted(x)),
           *cr.cr_rmsnorm_backward(sdr, sx, _shifted(g), rs, dres=sr, dx=_shifted(x)),
           cr.cr_rotate(sx, out=_shifted(x))]
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_norm_of_more_than_two_to_the_31_elements():
    """Offsets past 32 bits: the last rows of a batch of 2.4e9 elements equal
    those computed alone."""
    M, K = 295_000, 8192
    x = torch.randn(1000, K, device="cuda").to(torch.bfloat16).repeat(M // 1000, 1)
    x[-3:] *= 3
    g = torch.rand(K, device="cuda") + 0.5
    xq, xs, h, rs = cr.cr_rmsnorm_quant_act(x, g, EPS, residual=x)
    tail = x[-40:].clone()
    tq, ts, th, trs = cr.cr_rmsnorm_quant_act(tail, g, EPS, residual=tail)
    assert torch.equal(xq[-40:], tq) and torch.equal(xs[-40:], ts) and torch.equal(h[-40:], th)
    assert torch.equal(rs[-40:], trs)
    del xq, xs
    dx, dg = cr.cr_rmsnorm_backward(x, h, g, rs, dres=x)
    assert torch.equal(dx[-40:], cr.cr_rmsnorm_backward(tail, th, g, trs, dres=tail)[0])
    assert torch.isfinite(dg).all()
    del dx
    assert torch.equal(cr.cr_rotate(x, out=h)[-40:], cr.cr_rotate(tail))


def test_norm_from_two_threads():
    import threading
    M, K = 64, 4096
    sets = [_grad_inputs(M, K, s, torch.float32, True) for s in (61, 62)]
    args = [(dr.cuda(), h.cuda(), dev(g), dev(rs)) for dr, h, g, rs, _ in sets]
    refs = [cr.cr_rmsnorm_backward(*a) for a in args]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                dx, dg = cr.cr_rmsnorm_backward(*args[i])
                s.synchronize()
                if not (torch.equal(dx, refs[i][0]) and torch.equal(dg, refs[i][1])):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_norm_refusals():
    K = 512
    x = torch.zeros(4, K, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(K, device="cuda")
    rs = torch.ones(4, device="cuda")
    for bad in (0.0, -1e-6, float("nan"), float("inf"), 1e-40):
        with pytest.raises(cr.CrError):
            cr.cr_rmsnorm_quant_act(x, g, bad)
    with pytest.raises(TypeError):
        cr.cr_rmsnorm_quant_act(x.float(), g)
    with pytest.raises(TypeError):
        cr.cr_rmsnorm_quant_act(x, g.half())
    with pytest.raises(ValueError):
        cr.cr_rmsnorm_quant_act(x, g[:256])
    with pytest.raises(ValueError):
        cr.cr_rmsnorm_quant_act(x, g, residual=x[:2])
    with pytest.raises(ValueError):
        cr.cr_rmsnorm_quant_act(x.t(), g)
    with pytest.raises(ValueError):
        cr.cr_rmsnorm_quant_act(x, g, h=torch.empty_like(x))  # no residual: h is x
    with pytest.raises(cr.CrError):
        cr.cr_rmsnorm_quant_act(x, g, mp=2)
    with pytest.raises(cr.CrError):
        cr.cr_rotate(torch.zeros(2, 384, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        cr.cr_rmsnorm_backward(x, x, g, rs, work=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        cr.cr_rmsnorm_backward(x, x, g, rs[:2])
    big = torch.zeros(5, K, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cr.CrError):  # a shifted overlap
        cr.cr_rotate(big[:4], out=big[1:])
    with pytest.raises(cr.CrError):
        cr.cr_rmsnorm_backward(x, big[:4], g, rs, dx=big[:4])
    with pytest.raises(ValueError):
        cr.cr_rotate(x.cpu())
