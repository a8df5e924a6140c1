"""The outputs of serq_linear_i8 are defined bit for bit: sx (sw sum) in fp32, in
that order, rounded once to the output's type (ties to even). All kernels, with
and without the sums asked for, and channels that fill no whole vector."""

from __future__ import annotations

import pytest
import torch

import w4a4_linear_layers_amd as S

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,kernel", [
    (1, 512, 4096, "stream"), (16, 272, 333, "stream"), (17, 4096, 64, "stream"), (40, 528, 4100, "stream"), (64, 1040, 20001, "stream"),
    (9, 64, 16388, "stream"), (33, 96, 130, "stream"), (70, 1024, 256, "tile64x64"), (130, 80, 127, "tile64x64"), (300, 512, 4096, "tile64x128"),
    (321, 80, 4102, "tile64x128"), (700, 512, 4096, "tile128x128"), (700, 80, 4094, "tile128x128"), (70, 14336, 4096, "tile128x128"),
    (100, 12304, 131, "tile128x128"), (1024, 512, 8192, "tile256x128"), (1030, 80, 4098, "tile256x128"), (4096, 512, 4096, "tile256x256"),
    (4000, 80, 4100, "tile256x256"), (3590, 96, 4097, "tile256x256"), (5, 15, 9, "generic"), (300, 33, 70, "generic")])
def test_outputs(dtype, M, K, N, kernel):
    assert S.i8_kernel_name(M, K, N) == kernel
    g = torch.Generator(DEV).manual_seed(M + N)
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8, device=DEV)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8, device=DEV)
    sx, sw = torch.rand(M, generator=g, device=DEV) + 0.01, torch.randn(N, generator=g, device=DEV)
    sums = (x.double() @ w.double().t()).to(torch.int32)       # whole numbers below 2^31
    want = (sx[:, None] * (sw * sums.float())).to(dtype)
    layer = S.I8Layer(K=K, N=N, s_hat_inv=None, Wq=w, sw=sw)
    y, acc = S.linear_i8(x, sx, layer, out_dtype=dtype, debug=True)
    assert torch.equal(acc, sums) and torch.equal(y, want)
    around = torch.full((64 + M * N + 64,), 7.0, dtype=dtype, device=DEV)
    out = around[64:64 + M * N].view(M, N)
    assert torch.equal(S.linear_i8(x, sx, layer, out=out), want)
    assert (around[:64] == 7).all() and (around[64 + M * N:] == 7).all()


def test_ties_go_to_even():
    """Sums of 2^8 and more that lie half way between two bf16 numbers."""
    K, sums = 64, [257, 259, 261, 511, -257, -259, 256, 258, 514, 518, 1028, 1036]
    w = torch.zeros(len(sums), K, dtype=torch.int8)
    for n, s in enumerate(sums):
        a, b = divmod(abs(s), 100)
        w[n, :a], w[n, a] = (100, b) if s > 0 else (-100, -b)
    layer = S.I8Layer(K=K, N=len(sums), s_hat_inv=None, Wq=w.to(DEV), sw=torch.ones(len(sums), device=DEV))
    want = torch.tensor(sums, dtype=torch.float32).to(torch.bfloat16)
    assert want.tolist() == [256, 260, 260, 512, -256, -260, 256, 258, 512, 520, 1024, 1040]
    for M in (1, 70, 4096):
        y = S.linear_i8(torch.ones(M, K, dtype=torch.int8, device=DEV), torch.ones(M, device=DEV), layer)
        assert torch.equal(y.cpu(), want.expand(M, -1))
