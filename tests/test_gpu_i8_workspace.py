"""Workspaces of the 8-bit projections: ones the caller made, in the wrong place; the library's
own, of a stream whose handle another stream had before."""
import ctypes

import numpy as np
import pytest
import torch

import adapter_gemv_sgmv_b200 as L
from helpers import DevPool, rand_host_pool

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(a):
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def _operands(N=20, d_in=64, d_out=32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(N, d_in, device=DEV, generator=g).bfloat16()
    Q, Sx = torch.empty(N, d_in, dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    Wq, Sw = torch.empty(d_out, d_in, dtype=torch.int8, device=DEV), torch.empty(d_out, device=DEV)
    L.lora_quant_i8(x, Q, Sx)
    L.lora_quant_i8(torch.randn(d_out, d_in, device=DEV, generator=g) / d_in ** 0.5, Wq, Sw)
    return x, Q, Sx, Wq, Sw


class _Bare:
    """What the calls ask of a workspace, over some memory."""

    def __init__(self, address, nbytes):
        self.address, self.nbytes = address, nbytes

    def ptr(self):
        return self.address


@pytest.mark.parametrize("bare", [False, True])
@pytest.mark.parametrize("adapted", [False, True])
def test_workspace_in_host_memory_is_refused(adapted, bare):
    x, Q, Sx, Wq, Sw = _operands()
    pool = DevPool(rand_host_pool(np.random.default_rng(1), [8, 16], 64, 32))
    Y = torch.ones((20, 32), dtype=torch.bfloat16, device=DEV)
    buf = torch.zeros(1 << 20, dtype=torch.uint8)
    ws = L.Workspace(1 << 20, device="cpu")
    if bare:
        ws = _Bare((buf.data_ptr() + 255) // 256 * 256, (1 << 20) - 256)
    with pytest.raises(L.LoraError) as e:
        if adapted:
            L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, _i32([0, 10, 20]), _i32([0, 1]), 1.0, ws=ws)
        else:
            L.lora_linear_i8(Q, Sx, Wq, Sw, Y, ws=ws)
    assert e.value.code == 1
    torch.cuda.synchronize()
    assert torch.all(Y == 1)


@pytest.mark.parametrize("bare", [False, True])
def test_workspace_on_the_device_is_taken(bare):
    x, Q, Sx, Wq, Sw = _operands()
    pool = DevPool(rand_host_pool(np.random.default_rng(1), [8, 16], 64, 32))
    Y, Z = (torch.ones((20, 32), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    own = L.Workspace(1 << 20)
    ws = _Bare(own.ptr(), own.nbytes) if bare else own
    segs = _i32([0, 10, 20]), _i32([0, 1])
    assert L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, *segs, 1.0, ws=ws) is ws
    assert L.lora_get_error(ws) == 0
    L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Z, pool, *segs, 1.0)
    assert torch.equal(Y, Z)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_workspace_of_another_gpu_is_refused():
    x, Q, Sx, Wq, Sw = _operands()
    Y = torch.ones((20, 32), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(L.LoraError):
        L.lora_linear_i8(Q, Sx, Wq, Sw, Y, ws=L.Workspace(256, device="cuda:1"))


def _cudart():
    """The runtime that torch uses (its streams and this test's are of one kind)."""
    for line in open("/proc/self/maps"):
        if "libcudart.so" in line:
            return ctypes.CDLL(line.split()[-1])
    pytest.skip("torch's CUDA runtime is not a shared library")


def test_streams_destroyed_with_work_in_flight():
    """Streams made and destroyed one after another, each with calls queued when it goes: a new
    stream may come at the handle of an old one, whose work still uses the workspace kept for it."""
    rt = _cudart()
    d_in, d_out, N = 1024, 1032, 600
    pool = DevPool(rand_host_pool(np.random.default_rng(2), [64, 24], d_in, d_out))
    sets = [_operands(N, d_in, d_out, seed) for seed in range(2)]
    segs = [(_i32([0, 200, N]), _i32([0, 1])), (_i32([0, 450, N]), _i32([1, 0]))]
    want = []
    for (x, Q, Sx, Wq, Sw), (off, ad) in zip(sets, segs):
        Y = torch.zeros(N, d_out, dtype=torch.bfloat16, device=DEV)
        L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, off, ad, 0.5)
        want.append(Y)
    torch.cuda.synchronize()
    handles, done = [], []
    for i in range(12):
        h = ctypes.c_void_p()
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0
        handles.append(h.value)
        s = torch.cuda.ExternalStream(h.value)
        (x, Q, Sx, Wq, Sw), (off, ad) = sets[i % 2], segs[i % 2]
        Ys = [torch.zeros(N, d_out, dtype=torch.bfloat16, device=DEV) for _ in range(30)]
        torch.cuda.current_stream().synchronize()
        for Y in Ys:
            ws = L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, off, ad, 0.5, stream=s)
        done.append((i % 2, Ys, ws))
        assert rt.cudaStreamDestroy(h) == 0
    torch.cuda.synchronize()
    for kind, Ys, ws in done:
        assert L.lora_get_error(ws) == 0
        for Y in Ys:
            assert torch.equal(Y, want[kind])
    print(f"{len(set(handles))} handles for {len(handles)} streams")
