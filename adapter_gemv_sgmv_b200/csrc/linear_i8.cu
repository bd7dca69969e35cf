// The projection with an 8-bit weight and 8-bit tokens (lora_linear_i8), and the same
// with the segments' LoRA deltas (lora_linear_i8_sgmv):
//
//     y[n][o] = s_x[n] s_w[o] sum_i q[n][i] w[o][i]  (+ s sum_j B[a][o][j] v[n][j])
//
// The sum of integer products is exact in 32 bits (d_in <= 65536: at most 2^30).
//
// Simple form: 64 x 64 output tiles through shared memory, four products an
// instruction on the CUDA cores; the delta is read from the shrink's high and low
// bf16 parts.

#include "lora_internal.cuh"

#include <cuda_fp16.h>

namespace lora {
namespace {

constexpr int kST = 64;     // rows and outputs per tile
constexpr int kSK = 64;     // bytes of the reduction per step

__device__ __forceinline__ void store_as(void *Y, int32_t dtype, int64_t i, float v)
{
    if (dtype == LORA_BF16)
        static_cast<__nv_bfloat16 *>(Y)[i] = __float2bfloat16_rn(v);
    else if (dtype == LORA_F16)
        static_cast<__half *>(Y)[i] = __float2half_rn(v);
    else
        static_cast<float *>(Y)[i] = v;
}

__global__ void __launch_bounds__(256) k_i8_simple(const I8Args p)
{
    __shared__ int a[kST][kSK / 4 + 1], b[kST][kSK / 4 + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int n0 = blockIdx.y * kST, rows = min(kST, p.N - n0), ad = -1, r = 0;
    int64_t ao = 0, bo = 0;
    if (p.groups) {
        const int tile = blockIdx.y / 2, part = blockIdx.y & 1;
        if (tile >= p.hdr->n_groups)
            return;
        const Group g = p.groups[tile];
        n0 = g.p0 + part * kST;
        rows = min(kST, g.cnt - part * kST);
        ad = p.seg_ad[g.item];
        if (ad != -1 && !pool_adapter_ok(p.pool, ad, &r, &ao, &bo)) {
            if (threadIdx.x == 0)
                atomicOr(p.err, (uint32_t)LORA_ERR_BAD_ADAPTER);
            r = 0;
        }
    }
    if (rows <= 0)
        return;
    const int o0 = blockIdx.x * kST, outs = min(kST, p.d_out - o0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.d_in; k0 += kSK) {
        for (int e = threadIdx.x; e < kST * kSK / 4; e += 256) {
            const int i = e / (kSK / 4), c = e % (kSK / 4), k = k0 + 4 * c;
            a[i][c] = i < rows && k < p.d_in ? *reinterpret_cast<const int *>(p.Q + (int64_t)(n0 + i) * p.ldq + k) : 0;
            b[i][c] = i < outs && k < p.d_in ? *reinterpret_cast<const int *>(p.W + (int64_t)(o0 + i) * p.ldw + k) : 0;
        }
        __syncthreads();
        for (int c = 0; c < kSK / 4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __dp4a(a[ty + 16 * i][c], b[tx + 16 * j][c], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int n = ty + 16 * i, o = tx + 16 * j;
            if (n >= rows || o >= outs)
                continue;
            float v = p.Sx[n0 + n] * p.Sw[o0 + o] * (float)acc[i][j];
            if (r) {
                const __nv_bfloat16 *vb = p.Vb + (int64_t)(n0 + n) * p.ldvb;
                const __nv_bfloat16 *B = p.pool.B + bo + (int64_t)(o0 + o) * r;
                float d = 0.f;
                for (int k = 0; k < r; ++k)
                    d += ((float)vb[k] + (float)vb[p.kv + k]) * (float)B[k];
                v += d;
            }
            store_as(p.Y, p.dtype, (int64_t)(n0 + n) * p.ldy + o0 + o, v);
        }
}

}  // namespace

cudaError_t launch_linear_i8(const I8Args &a, int max_tiles, cudaStream_t s)
{
    const int rows = a.groups ? 2 * max_tiles : (a.N + kST - 1) / kST;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.d_out + kST - 1) / kST, rows);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_i8_simple, a);
}

}  // namespace lora
