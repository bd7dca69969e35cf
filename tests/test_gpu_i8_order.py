"""Memory order of lora_linear_i8_sgmv: every operand rewritten in place by the launches just
before the call, nothing waited for, against the definition in 64 bits (tolerances as in
test_gpu_i8.py: the parity bound, and at least 99 % of the outputs the correctly rounded bf16)."""
import dataclasses

import numpy as np
import pytest
import torch

import adapter_gemv_sgmv_b200 as L
import oracle
from helpers import DevPool, check_parity, check_rounded, dev_bf16, rand_host_pool, rand_x, widen
from workloads import to_host

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


@pytest.mark.parametrize("d_in", [64, 1024])
@pytest.mark.parametrize("N", [5, 40, 120])
def test_adapted_scales_and_tables_rewritten_between_calls(N, d_in):
    """Few tokens: their product starts beside the shrink, before it has waited for anything
    itself.  Scales, segments' adapters and the pool's tables stand at the same addresses in
    every round and hold other values, so a line kept from the round before would show."""
    rng = np.random.default_rng(N + d_in)
    d_out, kinds, rounds = 1032, 4, 48
    hp = rand_host_pool(rng, [64, 24, 16, 128], d_in, d_out)
    pool = DevPool(hp)
    perms = [rng.permutation(4) for _ in range(kinds)]
    hps = [dataclasses.replace(hp, A_off=hp.A_off[p].copy(), B_off=hp.B_off[p].copy(), rank=hp.rank[p].copy())
           for p in perms]
    off = np.array([0, 1, 1, N // 2, N - 1, N], np.int32)
    ads = [rng.permutation([0, 1, 2, 3, -1]).astype(np.int32) for _ in range(kinds)]
    # (scales that differ by more than any tolerance from one round to the next)
    X = [rand_x(rng, N, d_in) for _ in range(kinds)]
    xs = [dev_bf16(a) for a in X]
    Ws = [torch.randn(d_out, d_in, device=DEV) * (4.0 ** v) / d_in ** 0.5 for v in range(kinds)]
    tables = [(torch.tensor(h.A_off, device=DEV), torch.tensor(h.B_off, device=DEV), _i32(h.rank)) for h in hps]
    ads_dev = [_i32(a) for a in ads]
    Q, Sx = torch.empty(N, d_in, dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    Wq, Sw = torch.empty(d_out, d_in, dtype=torch.int8, device=DEV), torch.empty(d_out, device=DEV)
    wants = []
    for v in range(kinds):
        L.lora_quant_i8(xs[v], Q, Sx)
        L.lora_quant_i8(Ws[v], Wq, Sw)
        base = (Q.double() @ Wq.double().t()) * Sx.double()[:, None] * Sw.double()
        wants.append(base.cpu().numpy() + oracle.linear_sgmv(X[v], np.zeros((d_out, d_in), np.uint16), hps[v], off,
                                                             ads[v], 0.5))
    x, seg_off, seg_ad = torch.empty_like(xs[0]), _i32(off), torch.empty_like(ads_dev[0])
    Ys = [torch.zeros(N, d_out, dtype=torch.bfloat16, device=DEV) for _ in range(rounds)]
    torch.cuda.synchronize()
    for i, Y in enumerate(Ys):
        v = i % kinds
        x.copy_(xs[v])
        seg_ad.copy_(ads_dev[v])
        for dst, src in zip((pool.A_off, pool.B_off, pool.rank), tables[v]):
            dst.copy_(src)
        L.lora_quant_i8(Ws[v], Wq, Sw)
        L.lora_quant_i8(x, Q, Sx)
        ws = L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, seg_off, seg_ad, 0.5)
    torch.cuda.synchronize()
    assert L.lora_get_error(ws) == 0
    for v in range(kinds):
        check_parity(widen(to_host(Ys[v])), wants[v], f"kind {v}")
        check_rounded(widen(to_host(Ys[v])), wants[v], f"kind {v}")
        for i in range(v, rounds, kinds):
            assert torch.equal(Ys[i], Ys[v]), f"round {i} differs from round {v}"


@pytest.mark.parametrize("d_out", [136, 1032])
def test_gathered_adapter_rows_rewritten_between_calls(d_out):
    """Behind 8192 rows pairs of CTAs run, in tiles of 128 outputs (136) and of 256 (1032).  B rows
    of a rank without a tensor map, or off its grid, are gathered by both CTAs, each its half of
    the tile, and one thread multiplies both halves: a half that came too late would leave the
    round before's rows."""
    rng = np.random.default_rng(d_out)
    d_in, N, kinds, rounds = 64, 8193, 3, 18
    hps = [rand_host_pool(rng, [24, 40, 120, 8, 104], d_in, d_out) for _ in range(kinds)]
    pools = [DevPool(h) for h in hps]
    pool = DevPool(hps[0])
    cuts = np.sort(rng.choice(np.arange(1, N), 90, replace=False))
    off = np.r_[0, cuts, N].astype(np.int32)
    ads = (np.arange(91) % 5).astype(np.int32)
    X = rand_x(rng, N, d_in)
    x = dev_bf16(X)
    Q, Sx = torch.empty(N, d_in, dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    Wq, Sw = torch.empty(d_out, d_in, dtype=torch.int8, device=DEV), torch.empty(d_out, device=DEV)
    L.lora_quant_i8(x, Q, Sx)
    L.lora_quant_i8(torch.randn(d_out, d_in, device=DEV) / d_in ** 0.5, Wq, Sw)
    base = ((Q.double() @ Wq.double().t()) * Sx.double()[:, None] * Sw.double()).cpu().numpy()
    seg_off, seg_ad = _i32(off), _i32(ads)
    Ys = [torch.zeros(N, d_out, dtype=torch.bfloat16, device=DEV) for _ in range(rounds)]
    torch.cuda.synchronize()
    for i, Y in enumerate(Ys):
        pool.B.copy_(pools[i % kinds].B)
        pool.A.copy_(pools[i % kinds].A)
        ws = L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, seg_off, seg_ad, 0.5)
    torch.cuda.synchronize()
    assert L.lora_get_error(ws) == 0
    for v in range(kinds):
        want = base + oracle.linear_sgmv(X, np.zeros((d_out, d_in), np.uint16), hps[v], off, ads, 0.5)
        check_parity(widen(to_host(Ys[v])), want, f"kind {v}")
        check_rounded(widen(to_host(Ys[v])), want, f"kind {v}")
        for i in range(v, rounds, kinds):
            assert torch.equal(Ys[i], Ys[v]), f"round {i} differs from round {v}"
