"""Host-side checks of the attention calls (no GPU needed): refusals, which
come before anything is launched; workspace sizes; the rotary table against
its formulas; the validators and the table under the compiler's sanitizers."""

from __future__ import annotations

import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import w4a4_linear_layers_amd as S
from w4a4_linear_layers_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a4_linear_layers_amd", "csrc")
A = 0x100000          # an aligned fake device address, never dereferenced
OK, EINVAL, EALIGN, EUNSUP = _lib.SERQ_OK, _lib.SERQ_EINVAL, _lib.SERQ_EALIGN, _lib.SERQ_EUNSUPPORTED
BF16, F32 = _lib.SERQ_BF16, _lib.SERQ_F32


def append(QKV=A, dt=BF16, ld=768, M=4, Hq=4, Hkv=1, D=128, qn=A, kn=A, eps=1e-5, table=A, rot=128, max_pos=10,
           layout=0, pos=A, slot=A, Q=A, ldq=512, Kc=A, Vc=A, n_pages=4, page=16):
    return _lib.lib.serq_rope_append(QKV, dt, ld, M, Hq, Hkv, D, qn, kn, eps, table, rot, max_pos, layout, pos, slot, Q,
                                     ldq, Kc, Vc, n_pages, page, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), EINVAL), (dict(layout=2), EINVAL), (dict(layout=-1), EINVAL), (dict(M=-1), EINVAL),
    (dict(Hq=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(Hq=3, Hkv=2), EINVAL), (dict(Hq=20000, ld=1 << 30), EINVAL),
    (dict(D=0), EINVAL), (dict(D=96), EUNSUP), (dict(D=256, ld=1 << 20, ldq=1 << 20), EUNSUP), (dict(page=0), EINVAL),
    (dict(page=8), EUNSUP), (dict(page=24), EUNSUP), (dict(page=2048), EUNSUP), (dict(n_pages=0), EINVAL),
    (dict(n_pages=1 << 27), EINVAL), (dict(ld=767), EINVAL), (dict(ldq=511), EINVAL), (dict(rot=-2), EINVAL),
    (dict(rot=3), EINVAL), (dict(rot=130), EINVAL), (dict(table=None), EINVAL), (dict(max_pos=0), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=math.nan), EINVAL), (dict(eps=math.inf), EINVAL), (dict(Kc=None), EINVAL),
    (dict(Vc=None), EINVAL), (dict(QKV=None), EINVAL), (dict(slot=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(Q=None), EINVAL), (dict(Kc=A + 8), EALIGN), (dict(Vc=A + 2), EALIGN), (dict(table=A + 4), EALIGN),
    (dict(qn=A + 4), EALIGN), (dict(kn=A + 8), EALIGN), (dict(QKV=A + 1), EALIGN), (dict(Q=A + 1), EALIGN),
    (dict(dt=F32, QKV=A + 2), EALIGN), (dict(pos=A + 2), EALIGN), (dict(slot=A + 1), EALIGN),
    (dict(M=0), OK), (dict(M=0, QKV=None, slot=None, pos=None, Q=None), OK),
    (dict(M=0, Hq=0, ld=256, Q=None, ldq=0), OK), (dict(M=0, rot=0, table=None, max_pos=0), OK),
    (dict(M=0, qn=None, kn=None, eps=-1.0), OK),
])
def test_append_refusals(kw, code):
    assert append(**kw) == code


def prefill(Q=A, dt=BF16, ldq=512, cu=A, B=2, T=9, Hq=4, Hkv=1, D=128, K=A, V=A, n_pages=4, page=16, table=A,
            max_pages=4, kv=A, max_len=64, scale=0.1, O=A, ldo=512, ws=None, size=0):
    return _lib.lib.serq_attn_prefill(Q, dt, ldq, cu, B, T, Hq, Hkv, D, K, V, n_pages, page, table, max_pages, kv,
                                      max_len, scale, O, ldo, ws, size, None)


def decode(Q=A, dt=BF16, ldq=512, B=2, Hq=4, Hkv=1, D=128, K=A, V=A, n_pages=4, page=16, prefix=A, prefix_len=20,
           table=A, max_pages=4, kv=A, max_len=64, scale=0.1, O=A, ldo=512, ws=A, size=1 << 30):
    return _lib.lib.serq_attn_decode(Q, dt, ldq, B, Hq, Hkv, D, K, V, n_pages, page, prefix, prefix_len, table,
                                     max_pages, kv, max_len, scale, O, ldo, ws, size, None)


SHARED = [
    (dict(dt=7), EINVAL), (dict(B=-1), EINVAL), (dict(Hq=0), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(Hq=3, Hkv=2), EINVAL), (dict(Hq=16385, Hkv=1, ldq=1 << 30, ldo=1 << 30), EINVAL), (dict(D=0), EINVAL),
    (dict(D=80), EUNSUP), (dict(page=0), EINVAL), (dict(page=17), EUNSUP), (dict(n_pages=0), EINVAL),
    (dict(max_pages=-1), EINVAL), (dict(max_len=-1), EINVAL), (dict(max_len=(1 << 30) + 1), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(ldq=504), EINVAL), (dict(ldo=504), EINVAL),
    (dict(ldq=516), EALIGN), (dict(ldo=516), EALIGN), (dict(dt=F32, ldq=514), EALIGN), (dict(K=None), EINVAL),
    (dict(V=None), EINVAL), (dict(Q=None), EINVAL), (dict(O=None), EINVAL), (dict(kv=None), EINVAL),
    (dict(table=None), EINVAL), (dict(K=A + 8), EALIGN), (dict(V=A + 8), EALIGN), (dict(Q=A + 8), EALIGN),
    (dict(O=A + 4), EALIGN), (dict(kv=A + 2), EALIGN), (dict(table=A + 1), EALIGN),
    (dict(B=0), OK), (dict(B=0, Q=None, O=None, kv=None, table=None), OK),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(T=-1), EINVAL), (dict(cu=None), EINVAL), (dict(cu=A + 2), EALIGN), (dict(T=1 << 30), EINVAL),
    (dict(T=0), OK), (dict(max_len=100000, max_pages=1 << 20), EINVAL),      # a workspace is needed
    (dict(max_len=100000, ws=A, size=1000), EINVAL), (dict(max_len=100000, ws=A + 8, size=1 << 40), EALIGN),
])
def test_prefill_refusals(kw, code):
    assert prefill(**kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(prefix_len=-1), EINVAL), (dict(prefix_len=(1 << 30) + 1), EINVAL), (dict(prefix=None), EINVAL),
    (dict(prefix=A + 1), EALIGN), (dict(ws=None), EINVAL), (dict(size=64), EINVAL), (dict(ws=A + 4), EALIGN),
])
def test_decode_refusals(kw, code):
    assert decode(**kw) == code


def test_workspace_sizes():
    p, d = _lib.lib.serq_attn_prefill_workspace, _lib.lib.serq_attn_decode_workspace
    assert p(BF16, 0, 0, 4, 1, 128, 100) == 0 and d(BF16, 0, 4, 1, 128, 0, 100) == 0
    assert p(BF16, 1, 4, 4, 3, 128, 100) == -1 and p(5, 1, 4, 4, 1, 128, 100) == -1 and p(BF16, 1, 4, 4, 1, 96, 1) == -1
    assert d(BF16, 1, 4, 1, 128, -1, 100) == -1 and d(BF16, -1, 4, 1, 128, 0, 100) == -1
    assert d(BF16, 1, 4, 1, 128, 0, (1 << 30) + 1) == -1 and p(BF16, 1 << 29, 4, 4, 1, 128, 10) == -1
    assert p(BF16, 1, 4096, 32, 8, 128, 4096) == 0           # enough rows: no parts
    assert p(BF16, 1, 16, 32, 8, 128, 32768) > 0
    assert d(BF16, 1, 32, 8, 128, 0, 16) == 0                # one part
    assert d(F32, 9, 16, 16, 64, 777, 0) > 0
    for b in (1, 3, 64, 500):
        for n in (0, 1, 127, 128, 129, 5000, 1 << 20, 1 << 30):
            assert 0 <= d(BF16, b, 64, 8, 128, n, n) < 1 << 33


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (64, 10000.0), (128, 500000.0)])
def test_rope_table(rot, theta):
    """Each entry is the double value rounded once; sine and cosine of a
    double differ between libraries by a unit in its last place or so."""
    n = 300
    i = np.arange(rot // 2)
    f = theta ** (-2.0 * i / rot)

    def want(f, m=1.0):
        a = np.arange(n)[:, None] * f[None, :]
        return np.concatenate([m * np.cos(a), m * np.sin(a)], 1)

    def close(got, ref):
        # a unit of roundoff in f moves the angle by n 2^-51 at most
        assert got.dtype == np.float32 and np.abs(got - ref).max() <= 2.0 ** -24 * 1.5 + n * 2.0 ** -50

    close(S.rope_table(rot, n, theta=theta), want(f))
    close(S.rope_table(rot, n, theta=theta, scaling="linear", factor=8.0), want(f / 8.0))
    if rot > 2:
        close(S.rope_table(rot, n, theta=theta, scaling="base", factor=4.0),
              want((theta * 4.0 ** (rot / (rot - 2))) ** (-2.0 * i / rot)))
    turns = 128 * f / (2 * np.pi)
    g = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
    m = 0.1 * math.log(16.0) + 1
    close(S.rope_table(rot, n, theta=theta, scaling="bands", factor=16.0, orig_len=128, low=1.0, high=4.0, mscale=m),
          want((1 - g) * f / 16.0 + g * f, m))


def test_rope_table_bands_keep_high_and_interpolate_low_frequencies():
    plain = S.rope_table(128, 5000, theta=500000.0)
    bands = S.rope_table(128, 5000, theta=500000.0, scaling="bands", factor=8.0, orig_len=8192, low=1.0, high=4.0)
    line = S.rope_table(128, 5000, theta=500000.0, scaling="linear", factor=8.0)
    assert np.array_equal(plain[:, 0], bands[:, 0]) and np.array_equal(line[:, 63], bands[:, 63])
    assert not np.array_equal(line[:, 0], bands[:, 0])


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=65538), dict(max_pos=0), dict(theta=0.0),
    dict(theta=math.nan), dict(mscale=math.inf), dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=math.nan),
    dict(rot_dim=2, scaling="base", factor=2.0), dict(scaling="bands", factor=2.0),
    dict(scaling="bands", factor=2.0, orig_len=100, low=4.0, high=4.0),
])
def test_rope_table_refusals(kw):
    with pytest.raises(S.SerqError) as e:
        S.rope_table(**{**dict(rot_dim=8, max_pos=4), **kw})
    assert e.value.status == EINVAL


def test_rope_table_unknown_scaling():
    with pytest.raises(ValueError):
        S.rope_table(8, 4, scaling="cubic")


def test_python_refusals_on_host_tensors():
    import torch
    t = torch.zeros(1, 1, 16, 64)
    with pytest.raises(ValueError):
        S.KvCache(t, t)
    with pytest.raises(ValueError):
        S.KvCache(t, t[0])


@pytest.mark.parametrize("flags", [["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]])
def test_host_code_under_sanitizers(tmp_path, flags):
    if shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("g++ and the ROCm headers are needed")
    exe = str(tmp_path / "driver")
    src = [os.path.join(ROOT, "tests", "host", "attention_driver.cpp"), os.path.join(CSRC, "attn_abi.cpp"),
           os.path.join(CSRC, "rope_table.cpp")]
    b = subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer"] + flags +
                       ["-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I",
                        CSRC] + src + ["-o", exe], capture_output=True, text=True, timeout=300)
    assert b.returncode == 0, b.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1:verify_asan_link_order=0")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and "all checks passed" in r.stdout, (r.stdout[-2000:], r.stderr[-4000:])
