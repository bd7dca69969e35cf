"""Host side of the 8-bit projection and of rotary positions, without a GPU: argument checks
(each rejected call has a defect that the host finds before the first CUDA call; the
addresses are never read), workspace sizes, launch counts and the frequency tables."""
import ctypes
import math

import numpy as np
import pytest

import adapter_gemv_sgmv_b200 as L
from adapter_gemv_sgmv_b200 import build as B

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 32
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _quant(lib, X=FAKE, dtype=0, ldx=64, Q=FAKE, ldq=64, S=FAKE, N=0, d=64):
    return lib.lora_quant_i8(X, dtype, ldx, Q, ldq, S, N, d, None)


@pytest.mark.parametrize("kw,want", [
    ({}, OK),
    (dict(N=-1), INVALID), (dict(d=0), INVALID), (dict(ldx=56), INVALID), (dict(ldq=48), INVALID),
    (dict(N=4, X=None), INVALID), (dict(N=4, Q=None), INVALID), (dict(N=4, S=None), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(d=60), UNSUPPORTED),
    (dict(ldx=68), UNSUPPORTED), (dict(ldq=72), UNSUPPORTED), (dict(X=FAKE + 8), UNSUPPORTED),
    (dict(Q=FAKE + 8), UNSUPPORTED), (dict(S=FAKE + 2), UNSUPPORTED),
])
def test_quant_validates(lib, kw, want):
    assert _quant(lib, **kw) == want


def _linear(lib, Q=FAKE, ldq=64, Sx=FAKE, W=FAKE, ldw=64, Sw=FAKE, Y=FAKE, dtype=0, ldy=32, N=4, d_in=64, d_out=32,
            ws=None, nb=0):
    return lib.lora_linear_i8(Q, ldq, Sx, W, ldw, Sw, Y, dtype, ldy, N, d_in, d_out, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    ({}, WORKSPACE), (dict(ws=FAKE, nb=255), WORKSPACE), (dict(ws=FAKE + 8, nb=256), WORKSPACE),
    (dict(N=0, ws=FAKE, nb=256), OK),
    (dict(N=-1), INVALID), (dict(Q=None), INVALID), (dict(Sx=None), INVALID), (dict(W=None), INVALID),
    (dict(Sw=None), INVALID), (dict(Y=None), INVALID), (dict(ldq=48), INVALID), (dict(ldw=48), INVALID),
    (dict(ldy=24), INVALID), (dict(d_in=0), INVALID), (dict(d_out=-8), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(d_in=60), UNSUPPORTED), (dict(d_out=28), UNSUPPORTED),
    (dict(ldq=72), UNSUPPORTED), (dict(ldw=72), UNSUPPORTED), (dict(ldy=36), UNSUPPORTED),
    (dict(Q=FAKE + 8), UNSUPPORTED), (dict(W=FAKE + 8), UNSUPPORTED), (dict(Y=FAKE + 8), UNSUPPORTED),
    (dict(Sx=FAKE + 2), UNSUPPORTED),
    (dict(d_in=65544, ldq=65552, ldw=65552), UNSUPPORTED),
])
def test_linear_i8_validates(lib, kw, want):
    assert _linear(lib, **kw) == want


def _pool(**kw):
    d = dict(A=FAKE, B=FAKE, A_off=FAKE, B_off=FAKE, rank=FAKE, A_elems=1 << 20, B_elems=1 << 20,
             n_adapters=4, d_in=64, d_out=32, max_rank=16)
    d.update(kw)
    return L.LoraPoolStruct(**d)


def _sgmv(lib, Q=FAKE, ldq=64, Sx=FAKE, X=FAKE, ldx=64, W=FAKE, ldw=64, Sw=FAKE, Y=FAKE, ldy=32, pool=_pool(),
          off=FAKE, ad=FAKE, n_seg=2, N=4, ws=None, nb=0):
    return lib.lora_linear_i8_sgmv(Q, ldq, Sx, X, ldx, W, ldw, Sw, Y, ldy,
                                   ctypes.byref(pool) if pool is not None else None, off, ad, n_seg, N, 1.0, ws, nb,
                                   None)


@pytest.mark.parametrize("kw,want", [
    ({}, WORKSPACE), (dict(N=0, ws=FAKE, nb=1 << 20), OK), (dict(n_seg=0, ws=FAKE, nb=1 << 20), OK),
    (dict(pool=None), INVALID), (dict(pool=_pool(A=0)), INVALID), (dict(pool=_pool(max_rank=12)), UNSUPPORTED),
    (dict(X=None), INVALID), (dict(ldx=32), INVALID), (dict(X=FAKE + 2), UNSUPPORTED), (dict(off=None), INVALID),
    (dict(ad=None), INVALID), (dict(n_seg=-1), INVALID), (dict(Q=None), INVALID), (dict(ldq=72), UNSUPPORTED),
    (dict(Y=None), INVALID), (dict(ldy=16), INVALID), (dict(Sw=None), INVALID),
    (dict(pool=_pool(d_in=65544), ldq=65552, ldw=65552, ldx=65552), UNSUPPORTED),
])
def test_linear_i8_sgmv_validates(lib, kw, want):
    assert _sgmv(lib, **kw) == want


def test_workspaces_and_launches(lib):
    assert L.lora_workspace_size(L.OP_LINEAR_I8, 256, 1, 4096, 4096, 8) == 256
    assert L.lora_workspace_size(L.OP_LINEAR_I8, 256, 1, 65544, 4096, 8) == 0
    a = L.lora_workspace_size(L.OP_LINEAR_I8_SGMV, 1000, 64, 4096, 14336, 64, 8)
    assert a == L.lora_workspace_size(L.OP_LINEAR, 1000, 64, 4096, 14336, 64, 8) and a >= 1000 * 2 * 64 * 2
    assert L.lora_workspace_size(L.OP_LINEAR_I8_SGMV, 1000, 64, 65544, 14336, 64, 8) == 0
    assert L.lora_kernel_launches(L.OP_LINEAR_I8, 256, 1, 4096) == 1
    assert L.lora_kernel_launches(L.OP_LINEAR_I8, 0, 1, 4096) == 0
    assert L.lora_kernel_launches(L.OP_LINEAR_I8_SGMV, 1000, 64, 4096, 8) == 3


def _mat(x=FAKE, y=FAKE + 4096, xt=256, xh=64, yt=256, yh=64, heads=4):
    return L.LoraRopeMat(x, y, xt, xh, yt, yh, heads)


def _rope(lib, mats=None, n=None, dtype=0, pos=FAKE, pb=4, freq=FAKE, N=4, dim=64, rot=64):
    ms = [_mat()] if mats is None else mats
    arr = (L.LoraRopeMat * max(len(ms), 1))(*ms)
    return lib.lora_rope(arr, len(ms) if n is None else n, dtype, pos, pb, freq, N, dim, rot, 0, 0, 1.0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), OK), (dict(N=0, mats=[_mat(x=FAKE, y=FAKE)]), OK),
    (dict(n=0), INVALID), (dict(N=-1), INVALID), (dict(rot=0), INVALID), (dict(rot=63), INVALID),
    (dict(rot=66), INVALID), (dict(pb=2), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(mats=[_mat(x=0)]), INVALID), (dict(mats=[_mat(y=0)]), INVALID), (dict(mats=[_mat(heads=0)]), INVALID),
    # in place with other strides; two outputs in one place; heads or tokens that run into each other
    (dict(mats=[_mat(x=FAKE, y=FAKE, yt=512)]), INVALID),
    (dict(mats=[_mat(), _mat(x=FAKE + 8192)]), INVALID),
    (dict(mats=[_mat(yh=32)]), INVALID), (dict(mats=[_mat(yt=192)]), INVALID), (dict(mats=[_mat(yt=0)]), INVALID),
    (dict(mats=[_mat(xt=-256)]), INVALID),
    (dict(dtype=3), UNSUPPORTED), (dict(dim=1026, rot=64, mats=[_mat(yt=8192, yh=1026)]), UNSUPPORTED),
    (dict(pos=FAKE + 2), UNSUPPORTED), (dict(freq=FAKE + 4), UNSUPPORTED), (dict(mats=[_mat(x=FAKE + 1)]), UNSUPPORTED),
    (dict(mats=[_mat(y=FAKE + 4096 * (i + 1)) for i in range(5)]), UNSUPPORTED),
    (dict(N=0, mats=[_mat(heads=5000, yh=64, yt=64 * 5000)]), UNSUPPORTED),
])
def test_rope_validates(lib, kw, want):
    assert _rope(lib, **kw) == want


def test_rope_outputs_may_be_head_major(lib):
    """Tokens 64 apart, heads a whole sequence apart: as distinct as the other order."""
    assert _rope(lib, N=0, mats=[_mat(yt=64, yh=4 * 64)]) == OK
    # validated as such before the launch: with one token too few between heads it is refused
    assert _rope(lib, N=5, mats=[_mat(yt=64, yh=4 * 64)]) == INVALID


# ------------------------------------------------------------------ frequencies
def test_freqs_plain_linear_and_ntk():
    f, m = L.lora_rope_freqs(128, 10000.0)
    want = 10000.0 ** (-np.arange(64) / 64)
    assert m == 1.0 and np.allclose(f.numpy(), want, rtol=1e-14, atol=0)
    g, m = L.lora_rope_freqs(128, 10000.0, "linear", factor=4.0)
    assert m == 1.0 and np.allclose(g.numpy(), want / 4, rtol=1e-14, atol=0)
    h, m = L.lora_rope_freqs(128, 10000.0, "ntk", factor=4.0)
    # the first pair is untouched, the last is stretched by the factor exactly
    assert m == 1.0 and h[0] == 1.0 and math.isclose(float(h[63]), want[63] / 4, rel_tol=1e-13)
    one, _ = L.lora_rope_freqs(2, 10000.0, "ntk", factor=4.0)
    assert one.tolist() == [1.0]


def test_freqs_bands():
    f, m = L.lora_rope_freqs(128, 500000.0, "bands", factor=8.0, low=1.0, high=4.0, original=8192)
    plain = 500000.0 ** (-np.arange(64) / 64)
    turns = 8192 * plain / (2 * math.pi)
    assert m == 1.0
    for got, p, t in zip(f.tolist(), plain, turns):
        if t >= 4:
            want = p
        elif t <= 1:
            want = p / 8
        else:
            s = (t - 1) / 3
            want = (1 - s) * p / 8 + s * p
        assert math.isclose(got, want, rel_tol=1e-13)
    assert np.all(np.diff(f.numpy()) < 0)


def test_freqs_yarn():
    f, m = L.lora_rope_freqs(128, 10000.0, "yarn", factor=16.0, low=1.0, high=32.0, original=4096)
    plain = 10000.0 ** (-np.arange(64) / 64)
    assert math.isclose(m, 0.1 * math.log(16) + 1, rel_tol=1e-15)

    def pair(turns):
        return 128 * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    lo, hi = math.floor(pair(32)), math.ceil(pair(1))
    assert 0 < lo < hi < 63
    assert np.allclose(f.numpy()[:lo + 1], plain[:lo + 1], rtol=1e-14, atol=0)
    assert np.allclose(f.numpy()[hi:], plain[hi:] / 16, rtol=1e-14, atol=0)
    mid = (lo + hi) // 2
    r = (mid - lo) / (hi - lo)
    assert math.isclose(float(f[mid]), plain[mid] * (1 - r) + plain[mid] / 16 * r, rel_tol=1e-13)
    _, m1 = L.lora_rope_freqs(128, 10000.0, "yarn", factor=1.0, low=1.0, high=32.0, original=4096)
    assert m1 == 1.0


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), INVALID), (dict(rot=7), INVALID), (dict(rot=64, base=1.0), INVALID),
    (dict(rot=64, base=float("nan")), INVALID), (dict(rot=64, scaling="linear", factor=0.0), INVALID),
    (dict(rot=64, scaling="ntk", factor=float("inf")), INVALID),
    (dict(rot=64, scaling="bands", factor=8.0, low=4.0, high=4.0, original=8192), INVALID),
    (dict(rot=64, scaling="yarn", factor=8.0), INVALID),
    (dict(rot=64, scaling="other"), UNSUPPORTED),
])
def test_freqs_refusals(kw, code):
    with pytest.raises(L.LoraError) as e:
        L.lora_rope_freqs(**kw)
    assert e.value.code == code


# --------------------------------------------------------------- native binding
def test_native_binding_refuses_on_the_host(lib):
    """Loaded without a GPU, it refuses what is no CUDA tensor before any CUDA call, as LoraError."""
    import torch
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2)
    for call in (lambda: L.lora_quant_i8(x, q, s), lambda: L.lora_quant_i8(None, q, s),
                 lambda: L.lora_linear_i8(q, s, q, s, x), lambda: L.lora_rope([x], [x], s, s),
                 lambda: L.lora_rope([], [], s, s), lambda: L.lora_rope([x, x], [x], s, s)):
        with pytest.raises(L.LoraError) as e:
            call()
        assert e.value.code == INVALID
    with pytest.raises(L.LoraError) as e:
        L.lora_rope([x] * 5, [x] * 5, s, s)
    assert e.value.code == UNSUPPORTED
    with pytest.raises(TypeError):
        L.lora_rope(3, [x], s, s)
