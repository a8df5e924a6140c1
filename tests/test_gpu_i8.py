"""serq_linear_i8 against exact integer sums, at the sizes where its kernels
change over and end.

Tolerance: the sum is exact; float(sum) is off by at most half a step (2^-24 of
it), the two products by one rounding each: 3 * 2^-24 (1 + small) of |y|, below
2^-22, then the output type's rounding (2^-8 for bf16)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a4_linear_layers_amd as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


def sums(x, w):
    """Exact: sums of at most 2^17 products of 8 bits are whole numbers below 2^53."""
    return (x.double() @ w.double().t()).to(torch.int64)


def run(M, K, N, dtype, *, seed=1, low=-128, high=128):
    g = torch.Generator()
    g.manual_seed(seed + M + 7 * N)
    x = torch.randint(low, high, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(low, high, (N, K), generator=g, dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g) + 0.1, torch.randn(N, generator=g)
    layer = S.I8Layer(K=K, N=N, s_hat_inv=None, Wq=w.to(DEV), sw=sw.to(DEV))
    guard = torch.full((M + 2, N), 7.0, dtype=dtype, device=DEV)
    pad = -(-N * (2 if dtype == torch.bfloat16 else 4) // 16) * 16 // (2 if dtype == torch.bfloat16 else 4)
    flat = torch.full((pad + M * N + 64,), 7.0, dtype=dtype, device=DEV)
    out = flat[pad:pad + M * N].view(M, N)
    y, acc = S.linear_i8(x.to(DEV), sx.to(DEV), layer, out=out, debug=True)
    torch.cuda.synchronize()
    want = sums(x, w)
    assert torch.equal(acc.cpu().long(), want), S.i8_kernel_name(M, K, N)
    exact = sx.double()[:, None] * sw.double() * want
    tol = exact.abs() * (2.0 ** -22 + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24))
    assert ((y.cpu().double() - exact).abs() <= tol).all()
    assert (flat[:pad] == 7).all() and (flat[pad + M * N:] == 7).all()
    again = S.linear_i8(x.to(DEV), sx.to(DEV), layer, out_dtype=dtype)
    assert torch.equal(again, y)
    del guard


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [
    (1, 16, 1), (1, 4096, 320), (2, 272, 33), (16, 256, 16), (17, 2064, 50), (33, 4112, 100), (49, 1040, 65), (64, 2048, 64),
    (5, 1024, 16400), (64, 528, 16385),                             # two tiles of rows to a workgroup
    (65, 16, 1), (65, 64, 130), (128, 128, 128), (129, 80, 127), (200, 4096, 96), (66, 16384, 40), (130, 2064, 260),
    (300, 320, 5000), (1000, 1040, 700), (1100, 528, 2050), (130, 12304, 260), (257, 80, 4500), (65, 64, 20000),
    (4096, 64, 4096), (3600, 272, 4000), (3585, 528, 4097), (2050, 1088, 7001),      # 256 x 256
    (1, 15, 3), (7, 131, 70), (70, 33, 300), (3, 20000 + 2, 5),      # no whole 16 bytes
])
def test_linear(dtype, M, K, N):
    run(M, K, N, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N", [
    (8, 1040, 16401), (9, 1040, 16401), (16, 2576, 16384), (17, 528, 16390), (32, 16, 20001),      # tokens in one part or two
    (33, 2064, 4096), (33, 2064, 4097), (48, 528, 4111), (49, 4624, 5000), (64, 16, 4112), (64, 3088, 7003),
    (300, 64, 28600), (513, 80, 16385), (2305, 16, 8192),                     # rounds of the larger tiles or of the smaller
    (520, 80, 8200), (129, 336, 20001), (1100, 528, 4100), (1025, 64, 4096), (1030, 2000, 4098),     # 256 x 128
])
def test_linear_where_the_tiles_change(dtype, M, K, N):
    run(M, K, N, dtype)


def test_largest_sums():
    """Every product 2^14 at the longest K: sums just below 2^31."""
    K = 131056
    for M in (1, 70):
        x = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
        w = torch.full((20, K), -128, dtype=torch.int8, device=DEV)
        one = torch.ones(128, device=DEV)
        layer = S.I8Layer(K=K, N=20, s_hat_inv=None, Wq=w, sw=one[:20].contiguous())
        y, acc = S.linear_i8(x, one[:M].contiguous(), layer, out_dtype=torch.float32, debug=True)
        assert (acc == K * 16384).all() and (y == float(np.float32(K * 16384))).all()


def test_quantized_layer_end_to_end():
    """A calibrated layer with its quantizer: against the product of the values that codes and scales stand for, and
    near the unquantized product (a code is off by half a step: relative error of each side's noise below 1 / 127)."""
    g = np.random.default_rng(3)
    K, N, M = 512, 384, 77
    W = (0.02 * g.standard_normal((K, N))).astype(np.float32)
    x = g.standard_normal((M, K)).astype(np.float32)
    x[:, 5] *= 30
    layer = S.calibrate_i8(W, np.abs(x).max(0)).to(DEV)
    xq, sx = S.quant_act(torch.from_numpy(x).to(DEV), layer.s_hat_inv, a_bits=8)
    y = S.linear_i8(xq, sx, layer, out_dtype=torch.float32).cpu().double()
    values = (xq.cpu().double() * sx.cpu().double()[:, None]) @ (layer.Wq.cpu().double() * layer.sw.cpu().double()[:, None]).t()
    assert ((y - values).abs() <= 2.0 ** -21 * (xq.cpu().double().abs() * sx.cpu().double()[:, None]) @ (layer.Wq.cpu().double().abs() * layer.sw.cpu().double()[:, None]).t()).all()
    full = x.astype(np.float64) @ W.astype(np.float64)
    assert np.linalg.norm(y.numpy() - full) / np.linalg.norm(full) < 2 / 127


def test_mlp_in_8_bits():
    """silu(g) * u straight into the 8-bit down layer."""
    g = torch.Generator()
    g.manual_seed(2)
    M, K, N = 19, 256, 128
    gu = torch.randn(M, 2 * K, generator=g).to(torch.bfloat16).to(DEV)
    layer = S.calibrate_i8(torch.randn(K, N, generator=g) * 0.05).to(DEV)
    xq, sx = S.silu_mul_quant_act(gu[:, :K], gu[:, K:], layer.s_hat_inv, a_bits=8)
    y, acc = S.linear_i8(xq, sx, layer, out_dtype=torch.float32, debug=True)
    assert torch.equal(acc.cpu().long(), sums(xq.cpu(), layer.Wq.cpu()))
    h = torch.nn.functional.silu(gu[:, :K].float()) * gu[:, K:].float()
    want = h.double().cpu() @ (layer.Wq.cpu().double() * layer.sw.cpu().double()[:, None]).t()
    step = sx.cpu().double()[:, None] / 2 * 1.01          # half a code, and fp32's silu
    assert ((y.cpu().double() - want).abs() <= step * (layer.Wq.cpu().double().abs().sum(1) * layer.sw.cpu().double())).all()


def test_streams_graphs_and_refusals():
    M, K, N = 100, 16384, 256                      # K in parts, through a workspace
    g = torch.Generator()
    g.manual_seed(4)
    x = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8).to(DEV)
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).to(DEV)
    sx, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    layer = S.I8Layer(K=K, N=N, s_hat_inv=None, Wq=w, sw=sw)
    need = S.linear_i8_workspace(M, K, N)
    assert need > 0
    want = S.linear_i8(x, sx, layer, out_dtype=torch.float32)
    out, ws = torch.empty(M, N, device=DEV), torch.empty(need, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        S.linear_i8(x, sx, layer, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    with torch.cuda.graph(graph):
        S.linear_i8(x, sx, layer, out=out, workspace=ws)
    for i in range(3):
        x.copy_(x.roll(1, 0))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.roll(i + 1, 0))
    for bad in (dict(out=out.t()), dict(workspace=ws[:-1]), dict(out=out[:, :-1]), dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            S.linear_i8(x, sx, layer, **bad)
    for args in ((x.float(), sx), (x[:, :-1], sx), (x, sx[:-1]), (x.cpu(), sx), (x.t(), sx)):
        with pytest.raises(ValueError):
            S.linear_i8(*args, layer)
    assert S.linear_i8(x[:0], sx[:0], layer).shape == (0, N)
