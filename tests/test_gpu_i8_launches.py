"""The launches of an adapted 8-bit projection, counted in a captured graph, are the header's:
two up to 128 segments, three above, and never more than lora_kernel_launches says."""
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


def _cudart():
    for line in open("/proc/self/maps"):
        if "libcudart.so" in line:
            return ctypes.CDLL(line.split()[-1])
    pytest.skip("torch's CUDA runtime is not a shared library")


def _kernels(graph):
    rt, raw = _cudart(), ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    assert rt.cudaGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert rt.cudaGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    kinds = []
    for node in nodes:
        k = ctypes.c_int(-1)
        assert rt.cudaGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(k)) == 0
        kinds.append(k.value)
    return kinds.count(0)                                    # cudaGraphNodeTypeKernel


@pytest.mark.parametrize("N", [300, 8200])
@pytest.mark.parametrize("n_seg,launches", [(1, 2), (8, 2), (128, 2), (129, 3), (200, 3)])
def test_adapted_launches(N, n_seg, launches):
    d_in, d_out = 64, 40
    pool = DevPool(rand_host_pool(np.random.default_rng(1), [8, 16], d_in, d_out))
    x = torch.zeros(N, d_in, dtype=torch.bfloat16, device=DEV)
    Q, Sx = torch.zeros(N, d_in, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV)
    Wq, Sw = torch.zeros(d_out, d_in, dtype=torch.int8, device=DEV), torch.ones(d_out, device=DEV)
    Y = torch.zeros(N, d_out, dtype=torch.bfloat16, device=DEV)
    off, ad = _i32(np.linspace(0, N, n_seg + 1)), _i32(np.arange(n_seg) % 2)
    ws = L.Workspace(L.lora_workspace_size(L.OP_LINEAR_I8_SGMV, N, 2, d_in, d_out, 16, n_seg))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        L.lora_linear_i8_sgmv(Q, Sx, x, Wq, Sw, Y, pool, off, ad, 1.0, ws=ws)
    assert _kernels(g) == launches <= L.lora_kernel_launches(L.OP_LINEAR_I8_SGMV, N, 2, d_in, n_seg)
