"""Rotary positions (lora_rope) against the definition in 64 bits, its gradient against the
formula's transpose and against differences, and the q/k/v run it belongs to.

Tolerance, from the roundings: the reduced angle in turns is rounded to fp32 (at most 2^-25
of a turn, pi 2^-24 radian), sincospif is within 2 units in the last place (2^-23 at 1), the
factor rounds once (2^-24): cos and sin are off by at most 6.2 * 2^-24 of mscale; the two
products and their sum add 2 * 2^-24 each of |a| + |b|.  So |error| <= (|a| + |b|) mscale *
9 * 2^-24, plus half a step of the output type.  The 64-bit reference's own angle is off by
2^-52 of pos * freq."""
import math

import numpy as np
import pytest
import torch

import adapter_gemv_sgmv_b200 as L
from helpers import DevPool, rand_host_pool

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _ref(x, pos, freqs, interleaved, m, inverse):
    """(rotated in 64 bits, |a| + |b| of each element's pair, 0 where it is copied)."""
    rot = 2 * freqs.numel()
    v = x.double()
    t = pos.double()[:, None] * freqs.double()
    c, s = torch.cos(t)[:, None] * m, torch.sin(t)[:, None] * m
    if inverse:
        s = -s
    if interleaved:
        ia, ib = torch.arange(0, rot, 2, device=x.device), torch.arange(1, rot, 2, device=x.device)
    else:
        ia, ib = torch.arange(rot // 2, device=x.device), torch.arange(rot // 2, rot, device=x.device)
    a, b = v[..., ia], v[..., ib]
    y, size = v.clone(), torch.zeros_like(v)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def _check(y, x, pos, freqs, interleaved, m, inverse, what=""):
    want, size = _ref(x, pos, freqs, interleaved, m, inverse)
    rot = 2 * freqs.numel()
    t = y.dtype
    far = float((pos.double().abs().max() if pos.numel() else 0) * freqs.abs().max()) * 2.0 ** -51
    tol = size * m * (9 * 2.0 ** -24 + far)
    if t != torch.float32:
        tol[..., :rot] += want[..., :rot].abs() * torch.finfo(t).eps / 2 * (1 + 2.0 ** -10)
        if t == torch.float16:
            tol[..., :rot] += 2.0 ** -25
    err = (y.double() - want).abs()
    assert float((err - tol).max()) <= 0, f"{what}: off by {float(err.max())}, tolerance {float(tol.max())}"
    assert torch.equal(y[..., rot:], x[..., rot:]), f"{what}: dimensions past rot"


def _freqs(rot, base=10000.0):
    f, m = L.lora_rope_freqs(rot, base)
    return f.to(DEV), m


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,dim,rot", [(1, 32, 8, 128, 128), (3, 1, 1, 2, 2), (17, 4, 2, 64, 32),
                                             (33, 5, 1, 72, 18), (100, 20, 20, 80, 40), (257, 3, 3, 96, 96),
                                             (5, 2, 1, 1024, 1024), (9, 7, 1, 26, 14), (64, 1, 1, 16, 16),
                                             (2, 300, 1, 128, 64)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_definition(t, interleaved, n, hq, hk, dim, rot, inverse):
    g = torch.Generator(device=DEV)
    g.manual_seed(n + dim + rot)
    q = torch.randn(n, hq, dim, generator=g, device=DEV).to(t)
    k = torch.randn(n, hk, dim, generator=g, device=DEV).to(t)
    pos = torch.randint(0, 100000, (n,), generator=g, device=DEV)
    f, _ = _freqs(rot)
    yq, yk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    L.lora_rope([q, k], [yq, yk], pos, f, interleaved=interleaved, mscale=1.25, inverse=inverse)
    _check(yq, q, pos, f, interleaved, 1.25, inverse, "q")
    _check(yk, k, pos, f, interleaved, 1.25, inverse, "k")
    # in place: the same bits
    L.lora_rope([q, k], [q, k], pos, f, interleaved=interleaved, mscale=1.25, inverse=inverse)
    assert torch.equal(q, yq) and torch.equal(k, yk)


@pytest.mark.parametrize("pt", [torch.int32, torch.int64])
def test_rope_far_and_negative_positions(pt):
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 7, -2 ** 20, 2 ** 31 - 1, -2 ** 31, 123456789], device=DEV).to(pt)
    x = torch.randn(8, 4, 128, device=DEV)
    f, _ = _freqs(128)
    y = torch.empty_like(x)
    L.lora_rope([x], [y], pos, f)
    _check(y, x, pos, f, False, 1.0, False, "far positions")
    assert torch.equal(y[0], x[0])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_rope_strides(t, interleaved):
    """Columns of a fused projection, heads before tokens, odd strides, one token read for all."""
    n, d = 37, 64
    pos = torch.arange(n, device=DEV)
    f, _ = _freqs(48)
    qkv = torch.randn(n, (8 + 2 * 2) * d, device=DEV).to(t)
    keep = qkv.clone()
    q, k = qkv[:, :8 * d].view(n, 8, d), qkv[:, 8 * d:10 * d].view(n, 2, d)
    L.lora_rope([q, k], [q, k], pos, f, interleaved=interleaved)
    _check(q, keep[:, :8 * d].view(n, 8, d), pos, f, interleaved, 1.0, False, "fused q")
    _check(k, keep[:, 8 * d:10 * d].view(n, 2, d), pos, f, interleaved, 1.0, False, "fused k")
    assert torch.equal(qkv[:, 10 * d:], keep[:, 10 * d:])
    # [heads, tokens, dim] seen as [tokens, heads, dim]
    hm = torch.randn(6, n, d, device=DEV).to(t).transpose(0, 1)
    out = torch.empty(6, n, d, device=DEV, dtype=t).transpose(0, 1)
    L.lora_rope([hm], [out], pos, f, interleaved=interleaved)
    _check(out, hm, pos, f, interleaved, 1.0, False, "head major")
    # addresses and strides that no 16-byte access fits
    odd = torch.randn(n, 3, d + 3, device=DEV).to(t)
    dst = torch.full((n, 3, d + 5), 9.0, device=DEV, dtype=t)
    L.lora_rope([odd[..., 1:d + 1]], [dst[..., 3:d + 3]], pos, f, interleaved=interleaved)
    _check(dst[..., 3:d + 3], odd[..., 1:d + 1], pos, f, interleaved, 1.0, False, "odd strides")
    assert torch.all(dst[..., :3] == 9) and torch.all(dst[..., d + 3:] == 9)
    # a broadcast input: its gradient is the sum over what was read, here of inverse turns
    one = torch.randn(1, 1, d, device=DEV).to(t)
    y = torch.empty(n, 3, d, device=DEV, dtype=t)
    L.lora_rope([one.expand(n, 3, d)], [y], pos, f, interleaved=interleaved)
    _check(y, one.expand(n, 3, d), pos, f, interleaved, 1.0, False, "broadcast")


def test_rope_four_tensors_and_rows_behind_are_left():
    n = 65
    pos = torch.randint(0, 4096, (n,), device=DEV, dtype=torch.int32)
    f, _ = _freqs(32)
    xs = [torch.randn(n + 3, h, 32, device=DEV).bfloat16() for h in (1, 2, 5, 16)]
    ys = [torch.full_like(x, 5.0) for x in xs]
    L.lora_rope([x[:n] for x in xs], [y[:n] for y in ys], pos, f)
    for x, y in zip(xs, ys):
        _check(y[:n], x[:n], pos, f, False, 1.0, False)
        assert torch.all(y[n:] == 5)


def test_rope_non_finite_values_stay_in_their_pair():
    x = torch.ones(4, 2, 64, device=DEV)
    x[1, 0, 3] = float("nan")
    x[2, 1, 40] = float("inf")
    f, _ = _freqs(64)
    y = torch.empty_like(x)
    L.lora_rope([x], [y], torch.tensor([3, 4, 5, 6], device=DEV), f)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, [3, 35]] = True
    want[2, 1, [8, 40]] = True
    assert torch.equal(bad, want)


def test_rope_no_tokens():
    f, _ = _freqs(64)
    x = torch.empty(0, 2, 64, device=DEV)
    L.lora_rope([x], [torch.empty_like(x)], torch.empty(0, dtype=torch.int64, device=DEV), f)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """<g, J d> for a random direction d: by differences of the call itself in fp32 and by the
    inverse call on g; both against the 64-bit formula."""
    n, h, dim, rot, m = 11, 3, 40, 24, 1.5
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    x, d, g = (torch.randn(n, h, dim, generator=gen, device=DEV) for _ in range(3))
    pos = torch.randint(0, 1000, (n,), generator=gen, device=DEV)
    f, _ = _freqs(rot)

    def call(v, inverse=False):
        y = torch.empty_like(v)
        L.lora_rope([v], [y], pos, f, interleaved=interleaved, mscale=m, inverse=inverse)
        return y
    # the call is linear: a difference over a step of 1 has no truncation error, only the
    # roundings of the two calls and of x + d and x - d
    diff = (call(x + d) - call(x - d)).double() / 2
    by_diff = float((g.double() * diff).sum())
    grad = call(g, inverse=True)
    # past rot the forward copies, and so does the gradient
    by_grad = float((grad.double() * d.double()).sum())
    y, _ = _ref(d, pos, f, interleaved, m, False)
    want = float((g.double() * y).sum())
    # each of the n h dim terms: inputs of |x| + |d| rounded (2^-24) and 9 * 2^-24 in the call
    size = float(((x.abs() + d.abs()).double().sum()) * 2 * m) * float(g.abs().max())
    assert abs(by_diff - want) <= 12 * 2.0 ** -24 * size
    assert abs(by_grad - want) <= 12 * 2.0 ** -24 * size
    # the transpose itself, element by element
    _check(grad, g, pos, f, interleaved, m, True, "gradient")
    # and a turn undone (m^2 remains)
    back = call(call(x), inverse=True)
    ref = x.double().clone()
    ref[..., :rot] *= m * m
    assert float((back.double() - ref).abs().max()) <= 40 * 2.0 ** -24 * m * m * float(x.abs().max())


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("bands", dict(base=500000.0, factor=8.0, low=1.0, high=4.0, original=8192)),
                                        ("yarn", dict(factor=16.0, low=1.0, high=32.0, original=4096))])
def test_rope_stretched_contexts(scaling, kw):
    f, m = L.lora_rope_freqs(64, scaling=scaling, **kw)
    f = f.to(DEV)
    x = torch.randn(50, 4, 80, device=DEV).bfloat16()
    pos = torch.randint(0, 131072, (50,), device=DEV)
    y = torch.empty_like(x)
    L.lora_rope([x], [y], pos, f, mscale=m)
    _check(y, x, pos, f, False, float(np.float32(m)), False, scaling)


def test_rope_captured_and_replayed():
    x = torch.randn(33, 8, 64, device=DEV).bfloat16()
    pos = torch.zeros(33, dtype=torch.int64, device=DEV)
    f, _ = _freqs(64)
    y = torch.empty_like(x)
    L.lora_rope([x], [y], pos, f)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        L.lora_rope([x], [y], pos, f)
    for step in range(3):
        pos.fill_(1000 * step + 1)
        x.copy_(torch.randn(33, 8, 64, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        _check(y, x, pos, f, False, 1.0, False, f"replay {step}")


def test_adapted_qkv_with_positions():
    """The run these operators make together: a prompt batch quantised once, q, k and v through
    8-bit weights with each segment's adapter, q and k rotated in place -- against 64 bits on
    the same 8-bit weights and bf16 tokens."""
    rng = np.random.default_rng(77)
    d, heads, kv, hd = 512, 8, 2, 64
    lens = [130, 1, 77, 200]
    ads = [1, -1, 0, 2]
    off = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    N = int(off[-1])
    x = torch.randn(N, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).bfloat16()
    Q = torch.empty(N, d, dtype=torch.int8, device=DEV)
    Sx = torch.empty(N, device=DEV)
    L.lora_quant_i8(x, Q, Sx)
    xd = x.double()
    top = xd.abs().amax(1, keepdim=True)
    q64 = torch.round(127 * xd / top)
    qkv = torch.zeros(N, (heads + 2 * kv) * hd, dtype=torch.bfloat16, device=DEV)
    seg_off, seg_ad = (torch.tensor(a, dtype=torch.int32, device=DEV) for a in (off, ads))
    want, col = [], 0
    for i, h in enumerate((heads, kv, kv)):
        d_out = h * hd
        W = torch.randn(d_out, d, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2 + i)) / d ** 0.5
        Wq = torch.empty(d_out, d, dtype=torch.int8, device=DEV)
        Sw = torch.empty(d_out, device=DEV)
        L.lora_quant_i8(W, Wq, Sw)
        hp = rand_host_pool(rng, [16, 64, 24], d, d_out)
        pool = DevPool(hp)
        Y = qkv[:, col:col + d_out]
        ws = L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, seg_off, seg_ad, 0.5)
        assert L.lora_get_error(ws) == 0
        y = (q64 @ Wq.double().t()) * (top / 127) * Sw.double()
        for k, a in enumerate(ads):
            if a >= 0:
                r, ao, bo = int(hp.rank[a]), int(hp.A_off[a]), int(hp.B_off[a])
                A = pool.A[ao:ao + r * d].view(r, d).double()
                B = pool.B[bo:bo + r * d_out].view(d_out, r).double()
                rows = slice(int(off[k]), int(off[k + 1]))
                y[rows] += 0.5 * (xd[rows] @ A.t()) @ B.t()
        want.append(y)
        col += d_out
    pos = torch.cat([torch.arange(n) for n in lens]).to(DEV)
    f, _ = _freqs(hd)
    views = [qkv[:, :heads * hd].view(N, heads, hd), qkv[:, heads * hd:(heads + kv) * hd].view(N, kv, hd)]
    L.lora_rope(views, views, pos, f)
    for v, y, h in zip(views, want, (heads, kv)):
        exact, size = _ref(y.view(N, h, hd), pos, f, False, 1.0, False)
        # two bf16 roundings: of the projection (each of the pair's two values) and of the turn;
        # fp32 sums of 512 + 128 products below 2^-12 of the pair's size
        tol = size * (2.0 ** -8 + 2.0 ** -12) + exact.abs() * 2.0 ** -8 + 1e-3
        assert float(((v.double() - exact).abs() - tol).max()) <= 0
    v_err = (qkv[:, (heads + kv) * hd:].double() - want[2]).abs() - want[2].abs() * 2.0 ** -8 - 1e-3
    assert float(v_err.max()) <= 0


def test_rope_beyond_two_to_the_31_elements():
    n, h, d = 131_100, 130, 128
    x = torch.empty(n, h, d, dtype=torch.bfloat16, device=DEV).normal_()
    ends = [slice(0, 20), slice(n // 2, n // 2 + 20), slice(n - 20, n)]
    before = [x[e].clone() for e in ends]
    pos = torch.arange(n, device=DEV)
    f, _ = _freqs(d)
    L.lora_rope([x], [x], pos, f)
    for e, b in zip(ends, before):
        _check(x[e].clone(), b, pos[e], f, False, 1.0, False, f"rows {e}")
