"""The operators around the layer without a GPU: argument checks of the C ABI
(nothing is launched on these paths), and the restatements the GPU tests use
against each other and against the oracle."""
import ctypes
import glob
import os
import re

import numpy as np
import pytest
import torch

import oracle
import w4a8_codebook_quantized_b200 as cr
from w4a8_codebook_quantized_b200 import build, inputs

from operator_refs import (assert_sum_of_random_terms, cross_entropy, gradient_weight, hadamard, norm_backward,
                           norm_quant, rotate32, rotate64, silence_targets, softmax_gradient)

A, B, C = 0x10000, 0x4000000, 0x8000000  # aligned stand-in addresses far apart; never dereferenced
MIS = 0x10008
OK, INVALID, UNSUPPORTED, ALIGNMENT = (cr.CR_OK, cr.CR_ERR_INVALID_ARG, cr.CR_ERR_UNSUPPORTED, cr.CR_ERR_ALIGNMENT)
NO_DEVICE = cr.CR_ERR_NO_DEVICE


@pytest.fixture(scope="module")
def L():
    build.build()
    return cr.lib()


def test_norm_quant_validation(L):
    def call(x=A, res=None, gamma=A, gdt=1, eps=1e-6, M=4, K=256, MP=4, qmax=127, h=None, xq=B, xs=A, rs=A):
        return L.cr_rmsnorm_quant_act(x, res, gamma, gdt, eps, M, K, MP, qmax, h, xq, xs, rs, None)

    assert call(M=-1) == INVALID and call(MP=3) == INVALID and call(qmax=0) == INVALID and call(qmax=128) == INVALID
    assert call(gdt=2) == INVALID
    for eps in (0.0, -1.0, 1e-31, 1e31, float("nan"), float("inf")):
        assert call(eps=eps) == INVALID
    assert call(K=384) == UNSUPPORTED and call(K=0) == UNSUPPORTED and call(K=131072 + 256) == UNSUPPORTED
    assert call(M=1, MP=2 ** 31) == UNSUPPORTED
    assert call(x=None) == INVALID and call(gamma=None) == INVALID and call(xq=None) == INVALID
    assert call(res=C) == INVALID                       # a residual needs h
    assert call(res=C, h=A + 512) == INVALID            # h overlaps x without being x
    assert call(res=C, h=C + 512) == INVALID
    assert call(xq=A + 1024) == INVALID                 # xq overlaps x
    assert call(res=C, h=0x9000000, xq=C) == INVALID and call(res=C, h=B, xq=B) == INVALID
    for name in ("x", "gamma", "xq", "xs", "rs"):
        assert call(**{name: MIS}) == ALIGNMENT
    assert call(res=MIS, h=B) == ALIGNMENT and call(res=C, h=MIS) == ALIGNMENT
    assert call(M=0, MP=0, x=None, gamma=None, xq=None, xs=None, rs=None) == OK


def test_norm_backward_validation(L):
    need = L.cr_rmsnorm_backward_work_bytes(4, 256)
    assert need == 256 * 4 and L.cr_rmsnorm_backward_work_bytes(4, 1280) == 4 * 1280 * 4
    assert L.cr_rmsnorm_backward_work_bytes(0, 256) == 0 and L.cr_rmsnorm_backward_work_bytes(4, 300) == 0

    def call(dr=A, h=B, gamma=A, gdt=0, rs=A, dres=None, M=4, K=256, dx=C, dg=A, work=A, wb=need):
        return L.cr_rmsnorm_backward(dr, h, gamma, gdt, rs, dres, M, K, dx, dg, work, wb, None)

    assert call(M=-1) == INVALID and call(gdt=5) == INVALID and call(K=300) == UNSUPPORTED
    assert call(M=2 ** 31) == UNSUPPORTED
    for name in ("dr", "h", "gamma", "rs", "dx"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: MIS}) == ALIGNMENT
    assert call(dres=MIS) == ALIGNMENT and call(dg=MIS) == ALIGNMENT and call(work=MIS) == ALIGNMENT
    assert call(wb=need - 1) == INVALID and call(work=None) == INVALID
    assert call(dx=B) == INVALID and call(dx=A + 512) == INVALID
    assert call(M=0, dr=None, h=None, gamma=None, rs=None, dx=None, dg=None, work=None, wb=0) == OK


def test_rotate_validation(L):
    f = L.cr_rotate
    assert f(A, -1, 256, B, None) == INVALID and f(A, 2, 384, B, None) == UNSUPPORTED
    assert f(None, 2, 256, B, None) == INVALID and f(A, 2, 256, None, None) == INVALID
    assert f(MIS, 2, 256, B, None) == ALIGNMENT and f(A, 2, 256, MIS, None) == ALIGNMENT
    assert f(A, 2, 256, A + 512, None) == INVALID
    assert f(A, 2 ** 31, 256, B, None) == UNSUPPORTED
    assert f(None, 0, 256, None, None) == OK


def test_rotation_restatements_agree():
    """H is symmetric and its own inverse; the fp32 order against the matrix
    (8 additions and as many roundings, each at most the block's sum of
    magnitudes over 16)."""
    H = hadamard()
    assert np.array_equal(H, H.T) and np.allclose(H @ H, np.eye(256), atol=1e-12)
    v = np.random.default_rng(0).standard_normal((3, 512))
    v32 = v.astype(np.float32).astype(np.float64)
    bound = 12 * 2.0 ** -24 * np.abs(v32).reshape(3, 2, 256).sum(2).repeat(256, 1) / 16
    assert (np.abs(rotate32(v32) - rotate64(v32)) <= bound).all()
    assert np.allclose(rotate64(rotate64(v)), v, atol=1e-12)


def test_norm_restatement_quantises_as_the_oracle():
    """With a unit weight and rows of mean square 1 the norm changes nothing,
    and its int8 activations are the oracle's of the same rows."""
    rng = np.random.default_rng(1)
    x = rng.choice([-1.0, 1.0], size=(5, 512))
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    xq, xs, h, rs = norm_quant(x, np.ones(512, np.float32), 2.0 ** -60, mp=8)
    q_ref, s_ref = oracle.rotate_quant_act(bits, 8, 127)
    assert (rs == 1).all() and np.array_equal(h, x)
    assert np.array_equal(xq, q_ref) and np.array_equal(xs, s_ref)


def test_norm_gradient_formula_against_differences():
    rng = np.random.default_rng(2)
    M, K, eps = 3, 512, 1e-5
    h, dr, gamma = rng.standard_normal((M, K)), rng.standard_normal((M, K)), 1 + 0.1 * rng.standard_normal(K)

    def loss(hh, gg):
        return (dr * rotate64(hh / np.sqrt((hh ** 2).mean(1, keepdims=True) + eps) * gg)).sum()

    rs = 1 / np.sqrt((h ** 2).mean(1) + eps)
    dx, dg, _, _ = norm_backward(dr, h, gamma, rs)
    step = 1e-6
    for m, k in ((0, 0), (1, 300), (2, 511)):
        e = np.zeros_like(h)
        e[m, k] = step
        assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / (2 * step) - dx[m, k]) < 1e-6
    for k in (0, 200, 511):
        e = np.zeros(K)
        e[k] = step
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * step) - dg[k]) < 1e-6


def test_swiglu_backward_validation(L):
    need = L.cr_w4a8_swiglu_backward_work_bytes(4, 8, 256)
    assert need >= 3 * 8 * 256 and L.cr_w4a8_swiglu_backward_work_bytes(4, 8, 300) == 0

    def call(ptrs=(A,) * 8, M=4, N=8, K=256, dx=B, dz=C, work=A, wb=need):  # dout at A, apart from dx and dz
        return L.cr_w4a8_swiglu_backward(*ptrs, M, N, K, dx, dz, work, wb, None)

    assert call(M=-1) == INVALID and call(M=2 ** 31) == UNSUPPORTED and call(N=-8) == INVALID
    assert call(N=12) == UNSUPPORTED and call(K=320) == UNSUPPORTED
    for i in range(7):  # dout, xq, xs, qdata, srel, codebook, s_channel; the bias is optional
        assert call(ptrs=tuple(None if j == i else A for j in range(8))) == INVALID
    for i in range(8):
        assert call(ptrs=tuple(MIS if j == i else A for j in range(8))) == ALIGNMENT
    assert call(dx=None) == INVALID and call(dz=None) == INVALID and call(work=None) == INVALID
    assert call(dx=MIS) == ALIGNMENT and call(dz=MIS) == ALIGNMENT and call(work=MIS) == ALIGNMENT
    assert call(wb=need - 1) == INVALID
    assert call(dz=B) == INVALID and call(dz=A) == INVALID and call(dx=A) == INVALID  # overlapping buffers
    assert call(ptrs=(None,) * 8, M=0, dx=None, dz=None, work=None, wb=0) == OK


@pytest.mark.parametrize("backward", [False, True])
def test_cross_entropy_validation(L, backward):
    name = "cr_w4a8_cross_entropy" + ("_backward" if backward else "")
    need = getattr(L, name + "_work_bytes")(16, 8, 256)
    assert need > 0 and getattr(L, name + "_work_bytes")(16, 0, 256) == 0

    def call(ptrs=(A,) * 8, M=16, V=8, K=256, two=(B, C), dx=0x9000000, work=A, wb=need):
        f = getattr(L, name)
        if backward:
            return f(*ptrs, -100, *two, M, V, K, dx, work, wb, None)
        return f(*ptrs, -100, M, V, K, *two, work, wb, None)

    assert call(M=-1) == INVALID and call(V=-1) == INVALID and call(V=0) == INVALID and call(K=320) == UNSUPPORTED
    assert call(M=2 ** 31) == UNSUPPORTED and call(V=2 ** 31) == UNSUPPORTED
    for i in (0, 1, 2, 3, 4, 5, 7):  # xq, xs, the layer, targets; the bias (6) is optional
        assert call(ptrs=tuple(None if j == i else A for j in range(8))) == INVALID
    for i in range(8):
        assert call(ptrs=tuple(MIS if j == i else A for j in range(8))) == ALIGNMENT
    for two in ((None, C), (B, None)):
        assert call(two=two) == INVALID
    for two in ((MIS, C), (B, MIS)):
        assert call(two=two) == ALIGNMENT
    if backward:
        assert call(dx=None) == INVALID and call(dx=MIS) == ALIGNMENT
        assert call(dx=A) == INVALID        # over xq
    else:
        assert call(two=(B, B)) == INVALID  # loss and lse in one place
    assert call(work=None) == INVALID and call(work=MIS) == ALIGNMENT and call(wb=need - 1) == INVALID
    assert call(ptrs=(None,) * 8, M=0, two=(None, None), dx=None, work=None, wb=0) == OK


def test_work_sizes_are_bounded(L):
    """The cross entropy's buffers do not grow with the vocabulary or with the
    rows beyond one block, but for the 8 bytes per 256 outputs."""
    f, b = L.cr_w4a8_cross_entropy_work_bytes, L.cr_w4a8_cross_entropy_backward_work_bytes
    assert b(8192, 262144, 4096) <= 600 << 20
    assert b(1 << 20, 262144, 4096) == b(8192, 262144, 4096)
    assert f(2048, 262144, 4096) <= (64 << 20) + (2048 * 1024 * 8) + (1 << 20)
    assert f(1 << 20, 131072, 4096) == f(32768, 131072, 4096)


def test_written_buffers_overlap_nothing(L):
    """Any written buffer over another of the call's buffers is refused.  The
    addresses below (16 MB apart) belong to nothing, so this runs only where a
    call that is not refused ends at the missing device."""
    if torch.cuda.is_available():
        pytest.skip("the good calls would run")
    at = [0x10000000 + (i << 24) for i in range(16)]

    def pairs(call, written, read):
        for w in written:
            for o in [o for o in written if o != w] + read:
                assert call({w: o}) == INVALID, (w, o)
        assert call({}) == NO_DEVICE

    def norm(same):
        a = lambda i: at[same.get(i, i)]
        return L.cr_rmsnorm_quant_act(a(0), a(1), a(2), 1, 1e-6, 4, 256, 4, 127, a(3), a(4), a(5), a(6), None)

    pairs(norm, [4, 5, 6], [0, 1, 2, 3])
    assert norm({3: 2}) == INVALID

    def norm_backward(same):
        a = lambda i: at[same.get(i, i)]
        return L.cr_rmsnorm_backward(a(0), a(1), a(2), 0, a(3), a(4), 4, 256, a(5), a(6), a(7), 4 * 4 * 256, None)

    pairs(norm_backward, [6, 7], [0, 1, 2, 3, 4, 5])
    for o in (1, 2, 3, 6, 7):
        assert norm_backward({5: o}) == INVALID
    assert norm_backward({5: 0}) == NO_DEVICE and norm_backward({5: 4}) == NO_DEVICE  # in place

    def swiglu(same):
        a = lambda i: at[same.get(i, i)]
        need = L.cr_w4a8_swiglu_backward_work_bytes(4, 8, 256)
        return L.cr_w4a8_swiglu_backward(*(a(i) for i in range(8)), 4, 8, 256, a(8), a(9), a(10), need, None)

    pairs(swiglu, [8, 9, 10], list(range(8)))

    def ce(same):
        a = lambda i: at[same.get(i, i)]
        need = L.cr_w4a8_cross_entropy_work_bytes(16, 8, 256)
        return L.cr_w4a8_cross_entropy(*(a(i) for i in range(8)), -100, 16, 8, 256, a(8), a(9), a(10), need, None)

    pairs(ce, [8, 9, 10], list(range(8)))

    def ce_backward(same):
        a = lambda i: at[same.get(i, i)]
        need = L.cr_w4a8_cross_entropy_backward_work_bytes(16, 8, 256)
        return L.cr_w4a8_cross_entropy_backward(*(a(i) for i in range(8)), -100, a(8), a(9), 16, 8, 256, a(10), a(11),
                                                need, None)

    pairs(ce_backward, [10, 11], list(range(10)))


def test_shared_arrays_written_in_wide_words_say_their_alignment():
    """A shared array of bytes, words or floats that a kernel accesses in words
    of 8 or 16 bytes declares the alignment: its element type alone promises 1
    to 4 bytes, and a misaligned access is a fault."""
    wide = r"(?:store_partial\(\s*&?|reinterpret_cast<(?:const )?(?:uint4|uint2|float4|float2|ulonglong2|uint64_t) \*>\(\s*&?)"
    declared = 0
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cuh"))):
        for kernel in re.split(r"__global__", open(path).read())[1:]:
            for line, name in re.findall(r"(__shared__[^;]*?\b(\w+)(?:\[[^;]*\])+;)", kernel):
                if not re.search(r"\b(float|int|uint32_t|int32_t|uint16_t|uint8_t|int8_t)\b", line):
                    continue
                declared += 1
                used = {name} | set(re.findall(r"\*(\w+) = &?%s\b" % name, kernel))
                for n in used:
                    if re.search(wide + n + r"\b", kernel):
                        assert "__align__" in line, f"{os.path.basename(path)}: {line}"
    assert declared > 20


def test_gradient_work_holds_no_weight_that_is_decoded_on_the_way(L):
    """The cross entropy's gradient of few rows keeps the bf16 weight of a piece
    but not its int8 grid, unless a piece (the short last one too) needs it."""
    f = L.cr_w4a8_cross_entropy_backward_work_bytes
    slack = 1 << 20
    for M, V, K in ((64, 8192, 4096), (1, 16384, 4096), (40, 20001, 1024)):  # one piece: bf16 weight, dl, fp32 sums, copies
        copies = 20 << 20
        assert f(M, V, K) <= 2 * V * K + 2 * (V + 8) * M + 4 * M * K + copies + slack
    assert f(64, 32768, 4096) <= 2 * 16384 * 4096 + 2 * 16384 * 64 + 4 * 64 * 4096 + (20 << 20) + slack  # two pieces
    assert f(64, 2048, 8192) >= 3 * 2048 * 8192   # fewer columns than terms: decoded first
    assert f(300, 9000, 2048) >= 3 * 9000 * 2048  # three tiles of rows, long reduction
    assert f(900, 20011, 1024) >= 3 * 20011 * 1024  # rows gathered
    assert f(20, 128 * 32768 + 1, 2048) >= 3 * 32768 * 2048  # 129 pieces, the last of one entry


@pytest.mark.parametrize("M,V,K", [(20, 20011, 256), (3, 6000, 512), (300, 5000, 256)])
def test_gradient_comparison_sees_a_missing_tile(M, V, K):
    """The comparison that the GPU tests of every tile use: it passes the
    formula with dl rounded to bf16 and fp32 sums, and fails it without one tile
    of 64 or 128 entries, or a ragged last one of 13, of the reduction."""
    ly = inputs.layer(V, K, 5)
    at = np.array([0, V // 3, V // 2, V - 2])
    silence_targets(ly, at)
    rng = np.random.default_rng([M, V, K])
    z = rng.standard_normal((M, K))
    xq = np.rint(z * (127 / np.abs(z).max(1, keepdims=True))).astype(np.int8)
    xs = rng.uniform(0.02, 0.05, M).astype(np.float32)
    t = at[rng.integers(0, len(at), M)]
    _, lse, y = cross_entropy(ly, xq, xs, t)
    lse32, dloss = lse.astype(np.float32), rng.uniform(0.5, 1, M).astype(np.float32)
    dl = torch.exp(torch.from_numpy(y).float() - torch.from_numpy(lse32)[:, None])
    dl[torch.arange(M), torch.from_numpy(t)] -= 1
    w = torch.from_numpy(gradient_weight(ly)).float()
    got = ((dl.to(torch.bfloat16).float() @ w) * torch.from_numpy(dloss)[:, None]).to(torch.bfloat16)
    rel = 2.0 ** -24 * (2 * np.abs(lse).max() + 8)

    def check(drop=None):
        ref, sigma = softmax_gradient(ly, xq, xs, lse32, dloss, drop=drop, columns=4096)
        assert_sum_of_random_terms(got, ref, sigma, V, rel)

    check()
    for drop in ((1, 129), (256, 320), (V // 2 // 64 * 64 - 64, V // 2 // 64 * 64), (4096 - 64, 4096), (V - 15, V)):
        with pytest.raises(AssertionError):
            check(drop)
