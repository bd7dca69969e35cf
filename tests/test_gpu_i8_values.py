"""Deltas of lora_linear_i8_sgmv at the end of the number range, against the definition in 64
bits: s V beyond bf16's largest value, beyond fp32's, infinite and NaN.

The factors are chosen so that each value of V is one exact sum of powers of two; what an
output then takes is the two bf16 parts of V (2^-17 of it, their rounding), fp32 sums (2^-23
each of three products and the base) and the store's half step, 2^-8."""
import numpy as np
import pytest
import torch

import adapter_gemv_sgmv_b200 as L
from helpers import DevPool, rand_host_pool

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def _i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


# (few tokens, CTA pairs) x (a rank that is gathered, one with a view)
@pytest.mark.parametrize("N", [24, 8193])
@pytest.mark.parametrize("rank", [24, 64])
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("what", ["past bf16", "past fp32", "infinite A", "NaN in A"])
def test_delta_at_the_end_of_the_range(N, rank, scale, what):
    rng = np.random.default_rng(rank + N)
    d_in, d_out = 128, 72
    hp = rand_host_pool(rng, [rank, 16], d_in, d_out)
    pool = DevPool(hp)
    A = pool.A[:rank * d_in].view(rank, d_in)
    B = pool.B[:rank * d_out].view(d_out, rank)
    A.zero_()
    x = torch.randn(N, d_in, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)).bfloat16()
    off, ads = [0, 5, 9, N], [1, 0, -1]
    sign = torch.tensor([1.0, -1.0, 1.0, -1.0], device=DEV)
    x[5:9] = 0
    if what == "past bf16":              # 2^127 (2 - 2^-10): below fp32's end, rounded to bf16 it would be infinite
        x[5:9, 7] = x[5:9, 70] = 2.0 ** 100 * sign
        A[3, 7], A[3, 70] = 2.0 ** 27 * 255 / 128, 2.0 ** 27 * 7 / 1024
        B *= 2.0 ** -12
    elif what == "past fp32":
        x[5:9, 7] = 2.0 ** 100 * sign
        A[3, 7] = 2.0 ** 100             # (times the smallest B, 2^-14, still past bf16's largest value)
    else:
        x[5:9, 7] = sign
        A[3, 7] = INF if what == "infinite A" else float("nan")
    B[B == 0] = 2.0 ** -14
    Q, Sx = torch.empty(N, d_in, dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    Wq, Sw = torch.empty(d_out, d_in, dtype=torch.int8, device=DEV), torch.empty(d_out, device=DEV)
    L.lora_quant_i8(x, Q, Sx)
    L.lora_quant_i8(torch.randn(d_out, d_in, device=DEV) / 16, Wq, Sw)
    Y = torch.zeros(N, d_out, dtype=torch.bfloat16, device=DEV)
    ws = L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, _i32(off), _i32(ads), scale)
    assert L.lora_get_error(ws) == 0
    base = (Q.double() @ Wq.double().t()) * Sx.double()[:, None] * Sw.double()
    got = Y[5:9].double()
    if what == "NaN in A":
        assert torch.all(torch.isnan(got))
    elif what == "past bf16":
        V = scale * 2.0 ** 127 * (2 - 2.0 ** -10) * sign.double()[:, None]
        want = base[5:9] + V * B[:, 3].double()
        tol = want.abs() * 2.0 ** -8 + (V * B[:, 3].double()).abs() * (2.0 ** -17 + 4 * 2.0 ** -23) + 2.0 ** 80
        assert float(((got - want).abs() - tol).max()) <= 0
    else:
        assert torch.equal(got, scale * sign.double()[:, None] * torch.sign(B[:, 3].double()) * INF)
    # the other segments' tokens know nothing of it
    r1 = 16
    A1, B1 = pool.A[rank * d_in:].view(r1, d_in).double(), pool.B[rank * d_out:].view(d_out, r1).double()
    want = base.clone()
    want[:5] += scale * (x[:5].double() @ A1.t()) @ B1.t()
    rest = torch.cat([torch.arange(5), torch.arange(9, N)]).to(DEV)
    size = base[rest].abs() + (x[rest].double().abs() @ A1.abs().t()) @ B1.abs().t()
    err = (Y[rest].double() - want[rest]).abs() - want[rest].abs() * 2.0 ** -8 - size * 2.0 ** -15
    assert float(err.max()) <= 0
