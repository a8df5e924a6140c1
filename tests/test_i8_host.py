"""The linear in 8-bit integers without a GPU: calibration bit for bit against
its formulas, refusals, workspace sizes and the choice of kernel."""

from __future__ import annotations

import numpy as np
import pytest

import w4a4_linear_layers_amd as S
from synth import make_layer
from w4a4_linear_layers_amd import _lib

A = 0x100000          # an aligned fake device address, never dereferenced
OK, EINVAL, EALIGN = _lib.SERQ_OK, _lib.SERQ_EINVAL, _lib.SERQ_EALIGN
BF16, F32 = _lib.SERQ_BF16, _lib.SERQ_F32


def plain(W, amax, alpha):
    """Steps of the definition, each one fp32 operation but for s (64 bits, rounded once)."""
    K, N = W.shape
    s = np.ones(K, np.float32)
    if amax is not None:
        a, w = np.maximum(amax.astype(np.float64), 1e-5), np.maximum(np.abs(W).max(1).astype(np.float64), 1e-5)
        s = (np.sqrt(a) / np.sqrt(w) if alpha == 0.5 else a ** np.float64(np.float32(alpha)) / w ** (1 - np.float64(np.float32(alpha)))).astype(np.float32)
    v = s[:, None] * W
    m = np.abs(v).max(0)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.float32(127) / m
    zero = ~(inv <= np.finfo(np.float32).max)
    scale = np.where(zero, np.float32(0), m / np.float32(127)).astype(np.float32)
    inv = np.where(zero, np.float32(0), inv).astype(np.float32)
    return np.float32(1) / s, np.clip(np.rint(v * inv), -127, 127).astype(np.int8).T, scale


@pytest.mark.parametrize("K,N,alpha,smooth", [(64, 40, 0.5, True), (33, 200, 0.5, False), (96, 7, 0.5, True), (1, 1, 0.5, True)])
def test_calibrate(K, N, alpha, smooth):
    li = make_layer(K, N, 1, n_out=min(2, K), factor=20.0, seed=3, tag=K)
    W = li.W.copy()
    if N > 5:
        W[:, 3] = 0                       # a channel of zeros
        W[:, 4] = 1e-45
    amax = li.act_absmax if smooth else None
    L = S.calibrate_i8(W, amax, alpha=alpha)
    shi, Wq, sw = plain(W, amax, alpha)
    assert np.array_equal(L.s_hat_inv, shi) and np.array_equal(L.Wq, Wq) and np.array_equal(L.sw, sw)
    assert np.abs(L.Wq.astype(int)).max() <= 127
    if N > 5:
        assert not L.Wq[3].any() and L.sw[3] == 0


@pytest.mark.parametrize("K,N", [(16, 255), (5, 256), (7, 257), (3, 4100), (2, 16 * 256 + 17), (40, 1000)])
def test_calibrate_over_blocks_of_columns_and_threads(K, N):
    W = np.random.default_rng(N).standard_normal((K, N)).astype(np.float32)
    L = S.calibrate_i8(W, None)
    shi, Wq, sw = plain(W, None, 0.5)
    assert np.array_equal(L.s_hat_inv, shi) and np.array_equal(L.Wq, Wq) and np.array_equal(L.sw, sw)


def test_calibrate_other_exponents_and_types():
    li = make_layer(64, 48, 1, n_out=2, factor=20.0, seed=5, tag=1)
    for alpha in (0.0, 0.25, 1.0):
        L = S.calibrate_i8(li.W, li.act_absmax, alpha=alpha)
        v = (1 / L.s_hat_inv.astype(np.float64))[:, None] * li.W
        assert np.abs(L.Wq.T * L.sw.astype(np.float64) - v).max() <= 0.5001 * L.sw.max()
    bits = (li.W.view(np.uint32) >> 16).astype(np.uint16)
    a, b = S.calibrate_i8(bits, None), S.calibrate_i8((bits.astype(np.uint32) << 16).view(np.float32), None)
    assert np.array_equal(a.Wq, b.Wq) and np.array_equal(a.sw, b.sw)
    for bad in (dict(alpha=-0.1), dict(alpha=1.5), dict(alpha=float("nan"))):
        with pytest.raises(S.SerqError):
            S.calibrate_i8(li.W, li.act_absmax, **bad)
    with pytest.raises(ValueError):
        S.calibrate_i8(li.W, li.act_absmax[:-1])


def lin(xq=A, sx=A, wq=A, sw=A, M=4, K=64, N=32, y=A, dt=BF16, acc=None, ws=None, size=0):
    return _lib.lib.serq_linear_i8(xq, sx, wq, sw, M, K, N, y, dt, acc, ws, size, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), EINVAL), (dict(M=-1), EINVAL), (dict(K=0), EINVAL), (dict(K=-16), EINVAL), (dict(K=1 << 17), EINVAL),
    (dict(N=0), EINVAL), (dict(N=(1 << 26) + 1), EINVAL), (dict(M=1 << 20, N=(1 << 17) + 1), EINVAL),
    (dict(xq=None), EINVAL), (dict(sx=None), EINVAL), (dict(wq=None), EINVAL), (dict(sw=None), EINVAL), (dict(y=None), EINVAL),
    (dict(xq=A + 8), EALIGN), (dict(sx=A + 4), EALIGN), (dict(wq=A + 1), EALIGN), (dict(sw=A + 8), EALIGN), (dict(y=A + 2), EALIGN),
    (dict(acc=A + 4), EALIGN), (dict(ws=A + 4, size=1 << 40), EALIGN),
    (dict(M=100, K=16384, N=256), EINVAL), (dict(M=100, K=16384, N=256, ws=A, size=100), EINVAL),      # a workspace is needed
    (dict(M=0), OK), (dict(M=0, xq=None, sx=None, y=None), OK), (dict(M=0, wq=None), EINVAL),
])
def test_refusals(kw, code):
    assert lin(**kw) == code


def test_plans():
    w, name = _lib.lib.serq_linear_i8_workspace, S.i8_kernel_name
    assert w(-1, 64, 64) == -1 and w(1, 1 << 17, 64) == -1 and w(0, 64, 64) == 0 and name(1, 0, 1) is None
    assert name(4096, 8192, 8192) == "tile256x256" and name(1, 4096, 4096) == "stream" and name(1, 4090, 8) == "generic"
    assert name(1024, 8192, 8192) == "tile256x128" and name(1100, 528, 4100) == "tile256x128"
    assert name(100, 4096, 4096) == "tile64x64" and name(400, 4096, 4096) == "tile64x128"
    assert name(1000, 4096, 4096) == "tile128x128" and w(1000, 4096, 4096) == 0 and name(100, 14336, 4096) == "tile128x128"
    assert w(100, 14336, 4096) > 0
    for M in (1, 16, 64, 65, 100, 128, 500, 2000, 5000, 1 << 20):
        for K, N in ((16, 1), (64, 64), (4096, 4096), (14336, 4096), (131056, 300), (4096, 128256)):
            assert 0 <= w(M, K, N) < 1 << 28, (M, K, N)
