"""The gradients' contractions over large vocabularies and wide gated layers,
checked so closely that one tile or piece of the reduction could not be missing
or wrong: targets whose weights are zero leave the softmax part of the cross
entropy's gradient alone, and the gated layer's dx is compared with the
contraction of the dz that the call returns.  (tests/test_operators.py shows
that the comparison sees a missing tile.)"""
import numpy as np
import pytest
import torch

import w4a8_codebook_quantized_b200 as cr
from w4a8_codebook_quantized_b200 import inputs

from gpu_util import Guarded, dev
from operator_refs import (assert_sum_of_random_terms, f64, gradient_weight, silence_targets, softmax_gradient, to_bf16)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cr.lib()
    yield
    cr.cr_check_device_error()


def _quantised(M, K, seed):
    rng = np.random.default_rng([seed, M, K])
    z = rng.standard_normal((M, K))
    xq = np.rint(z * (127 / np.abs(z).max(1, keepdims=True))).astype(np.int8)
    return xq, rng.uniform(0.02, 0.05, M).astype(np.float32)


# Decoded on the way: one tile of rows against one and several pieces, and
# several tiles of rows; decoded first: short and long pieces, split reductions;
# rows gathered.  The last has a last piece of one entry, whose single block of
# terms leaves one of the two ranges of the split reduction empty.
@pytest.mark.parametrize("M,V,K", [(20, 65549, 2048), (40, 20001, 256), (1, 50021, 512), (128, 30001, 512),
                                   (300, 1900, 1024), (300, 9000, 2048), (16, 5000, 8192), (200, 70001, 1024),
                                   (900, 20011, 1024), (3000, 33000, 512), (8192, 262145, 256)])
def test_every_tile_of_the_cross_entropy_gradient(M, V, K):
    ly = inputs.layer(V, K, 81)
    at = np.array([0, V // 3, V // 2, V - 2])
    silence_targets(ly, at)
    xq, xs = _quantised(M, K, 82)
    rng = np.random.default_rng(83)
    t = at[rng.integers(0, len(at), M)]
    t[1::5] = -100
    w = [dev(a) for a in (ly.qdata, ly.srel, ly.codebook, ly.s_channel)]
    args = (dev(xq), dev(xs), *w, dev(t))
    _, lse = cr.cr_w4a8_cross_entropy(*args)
    dloss = rng.uniform(0.5, 1, M).astype(np.float32)
    work = Guarded((cr.lib().cr_w4a8_cross_entropy_backward_work_bytes(M, V, K),), torch.uint8)
    work.tensor.fill_(0xFF)
    dx = Guarded((M, K), torch.bfloat16)
    cr.cr_w4a8_cross_entropy_backward(*args, lse, dev(dloss), dx=dx.tensor, work=work.tensor)
    assert work.intact() and dx.intact()
    del work
    lse = f64(lse)
    ref, sigma = softmax_gradient(ly, xq, xs, lse, np.where(t < 0, 0.0, dloss), device="cuda", columns=8192)
    # what the terms of a row have in common: lse's product with log2 e, rounded,
    # and the row's factor and scales
    rel = 2.0 ** -24 * (2 * np.abs(lse).max() + 8)
    assert_sum_of_random_terms(dx.tensor, ref, sigma, V, rel, "dx")


@pytest.mark.parametrize("M,N,K", [(1, 4096, 512), (17, 12288, 1024), (33, 19208, 256), (128, 8320, 768),
                                   (333, 2824, 1280), (300, 6000, 2048), (700, 6400, 256), (3900, 3200, 1280)])
def test_every_tile_of_the_gated_gradient(M, N, K):
    ly = inputs.layer(N, K, 91)
    xq, xs = _quantised(M, K, 92)
    dout = to_bf16(np.random.default_rng(93).standard_normal((M, N // 2))).cuda()
    w = [dev(a) for a in (ly.qdata, ly.srel, ly.codebook, ly.s_channel)]
    dx, dz = cr.cr_w4a8_swiglu_backward(dout, dev(xq), dev(xs), *w)
    g = dev(gradient_weight(ly))
    z = dz.double()
    # dz is what the call contracted: no term has an error, only the sum's additions
    ref, sigma = z @ g, ((z * z) @ (g * g)).sqrt()
    add = (N / 16 + 64) * 2.0 ** -23 * (7 * sigma + ref.abs())
    bad = (dx.double() - ref).abs() > 2.0 ** -8 * (ref.abs() + add) + add + 2.0 ** -133
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"
