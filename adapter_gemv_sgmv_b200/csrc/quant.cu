// lora_quant_i8: rows of activations (or of a weight) as 8-bit integers with one
// scale a row, the form lora_linear_i8 multiplies.
//
//     s[n] = max_i |x[n][i]| / 127        q[n][i] = round(127 x[n][i] / max |x[n]|)
//
// with the quotient rounded as the exact real number is, halves to even: an integer
// result has no rounding error to hide in, so every reader of this formula gets the
// same bytes.  A division for each element would cost more than the memory traffic.
// Instead t = x * (127 / max) is rounded, which is off by at most 127.5 * 2 * 2^-24 <
// 2^-15; where t lies that near a half, the sign of 127 x - h max decides, h the half:
// 127 x splits into two fp32 parts without error, h has 8 bits, so the fused
// multiply-add that subtracts h max is exact there and the sign is the true one.
//
// Bound: HBM, one read of x and one write of q.  A block takes a row and holds it in
// registers between the two passes (maximum, rounding), so x is read once.

#include "lora_internal.cuh"

#include <cuda_fp16.h>

namespace lora {
namespace {

constexpr int kQVec = 8;            // elements per load unit (16 bytes of bf16/fp16, 32 of fp32)
constexpr float kNear = 0.5f - 3.1e-5f;    // |t - round(t)| above this: within 2^-15 of a half
constexpr float kMagic = 12582912.f;       // 1.5 * 2^23: adding it rounds to an integer, ties to even

template <class T> struct Vec8;                      // 8 elements as loaded
template <> struct Vec8<float> { uint4 a, b; };
template <> struct Vec8<__nv_bfloat16> { uint4 a; };
template <> struct Vec8<__half> { uint4 a; };

template <class T> __device__ __forceinline__ Vec8<T> load8(const T *p)
{
    Vec8<T> v;
    v.a = __ldg(reinterpret_cast<const uint4 *>(p));
    if constexpr (sizeof(T) == 4)
        v.b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    return v;
}

// max |x| as an unsigned bit pattern of fp32: ordered like the value, with inf and
// every NaN above all finite ones
template <class T> __device__ __forceinline__ uint32_t absmax8(const Vec8<T> &v)
{
    if constexpr (sizeof(T) == 4) {
        uint32_t m = v.a.x & 0x7fffffffu;
        m = max(m, v.a.y & 0x7fffffffu);
        m = max(m, v.a.z & 0x7fffffffu);
        m = max(m, v.a.w & 0x7fffffffu);
        m = max(m, v.b.x & 0x7fffffffu);
        m = max(m, v.b.y & 0x7fffffffu);
        m = max(m, v.b.z & 0x7fffffffu);
        return max(m, v.b.w & 0x7fffffffu);
    } else {
        uint32_t m = __vmaxu2(__vmaxu2(v.a.x & 0x7fff7fffu, v.a.y & 0x7fff7fffu),
                              __vmaxu2(v.a.z & 0x7fff7fffu, v.a.w & 0x7fff7fffu));
        return max(m & 0xffffu, m >> 16);            // 16-bit pattern, widened once per row
    }
}

template <class T> __device__ __forceinline__ uint32_t widen_bits(uint32_t m)
{
    if constexpr (sizeof(T) == 4)
        return m;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return m << 16;
    else
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

template <class T> __device__ __forceinline__ void unpack8(const Vec8<T> &v, float (&x)[8])
{
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
    if constexpr (sizeof(T) == 4) {
        const uint32_t u[4] = {v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(w[i]);
            x[4 + i] = __uint_as_float(u[i]);
        }
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// The exact rounding where t = x * (127 / top) lies next to a half: q is round(t) as an
// integer-valued float, d = t - q with |d| about 1/2.
__device__ __forceinline__ float settle(float x, float top, float q, float d)
{
    const float step = d > 0.f ? 1.f : -1.f;
    const float h = q + 0.5f * step;                 // the half between q and q + step
    const float p = x * 127.f;
    const float lo = fmaf(x, 127.f, -p);             // 127 x = p + lo
    const float r = (fmaf(-h, top, p) + lo) * step;  // > 0: beyond the half, towards q + step
    if (r > 0.f)
        return q + step;
    if (r == 0.f && (((int)q) & 1))
        return q + step;                             // a tie: the even neighbour
    return q;
}

// 8 elements -> 8 bytes.  `pre` is a power of two that keeps 127 x and 127 / top in range.
__device__ __forceinline__ uint2 round8(float (&x)[8], float inv, float top, float pre)
{
    uint32_t bits[8];
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] *= pre;
        const float m = fmaf(x[i], inv, kMagic);
        const float q = m - kMagic;
        worst = fmaxf(worst, fabsf(fmaf(x[i], inv, -q)));
        bits[i] = __float_as_uint(m);                // low byte: the integer in two's complement
    }
    if (worst > kNear) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __uint_as_float(bits[i]) - kMagic;
            const float d = fmaf(x[i], inv, -q);
            if (fabsf(d) > kNear)
                bits[i] = __float_as_uint(settle(x[i], top, q, d) + kMagic);
        }
    }
    const uint32_t a = __byte_perm(bits[0], bits[1], 0x0040), b = __byte_perm(bits[2], bits[3], 0x0040);
    const uint32_t c = __byte_perm(bits[4], bits[5], 0x0040), e = __byte_perm(bits[6], bits[7], 0x0040);
    return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, e, 0x5410));
}

struct QuantArgs {
    const void *X;
    int64_t ldx;
    int8_t *Q;
    int64_t ldq;
    float *S;
    int32_t d;
};

// One block per row.  VPT units of 8 elements a thread stay in registers; a row longer
// than the block holds (WIDE) is read a second time, from L2.
template <class T, int VPT, bool WIDE>
__global__ void __launch_bounds__(1024) k_quant_rows(const QuantArgs p)
{
    __shared__ uint32_t part[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t n = blockIdx.x;
    const T *x = static_cast<const T *>(p.X) + n * p.ldx;
    int8_t *q = p.Q + n * p.ldq;
    const int units = p.d / kQVec, tid = threadIdx.x, nt = blockDim.x;

    Vec8<T> v[VPT];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (tid + j * nt < units)
            v[j] = load8(x + (int64_t)(tid + j * nt) * kQVec);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (tid + j * nt < units)
            m = max(m, absmax8<T>(v[j]));
    if constexpr (WIDE)
        for (int u = tid + VPT * nt; u < units; u += nt)
            m = max(m, absmax8<T>(load8(x + (int64_t)u * kQVec)));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0)
        part[tid >> 5] = m;
    __syncthreads();
    m = part[0];
    for (int w = 1; w < (nt >> 5); ++w)
        m = max(m, part[w]);
    const uint32_t bits = widen_bits<T>(m);
    const bool bad = bits >= 0x7f800000u;            // inf or NaN in the row
    float top = __uint_as_float(bits);
    if (tid == 0)
        p.S[n] = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(top, 127.f);
    const float pre = top < 0x1p-80f ? 0x1p90f : (top > 0x1p100f ? 0x1p-40f : 1.f);
    top *= pre;
    const float inv = bad || bits == 0 ? 0.f : 127.f / top;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        if (tid + j * nt < units) {
            float f[8];
            unpack8<T>(v[j], f);
            const uint2 o = bad ? make_uint2(0, 0) : round8(f, inv, top, pre);
            *reinterpret_cast<uint2 *>(q + (int64_t)(tid + j * nt) * kQVec) = o;
        }
    }
    if constexpr (WIDE)
        for (int u = tid + VPT * nt; u < units; u += nt) {
            float f[8];
            unpack8<T>(load8(x + (int64_t)u * kQVec), f);
            *reinterpret_cast<uint2 *>(q + (int64_t)u * kQVec) = bad ? make_uint2(0, 0) : round8(f, inv, top, pre);
        }
}

template <class T> cudaError_t launch_quant(const QuantArgs &a, int32_t N, cudaStream_t s)
{
    constexpr int VPT = sizeof(T) == 4 ? 2 : 4;
    const int units = a.d / kQVec;
    int threads = ((units + VPT - 1) / VPT + 31) & ~31;
    const bool wide = threads > 1024;
    if (wide)
        threads = 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(N);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return wide ? cudaLaunchKernelEx(&cfg, k_quant_rows<T, VPT, true>, a)
                : cudaLaunchKernelEx(&cfg, k_quant_rows<T, VPT, false>, a);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" lora_status lora_quant_i8(const void *X, int32_t dtype, int64_t ldx, int8_t *Q, int64_t ldq, float *S,
                                     int32_t N, int32_t d, void *stream)
{
    if (N < 0 || d <= 0 || ldx < d || ldq < d || (N > 0 && (!X || !Q || !S)))
        return LORA_ERR_INVALID_ARG;
    if (dtype < LORA_BF16 || dtype > LORA_F32)
        return LORA_ERR_UNSUPPORTED;
    if ((d & 7) || (ldx & 7) || (ldq & 15) || ((uintptr_t)X & 15) || ((uintptr_t)Q & 15) || ((uintptr_t)S & 3))
        return LORA_ERR_UNSUPPORTED;
    if (N == 0)
        return LORA_OK;
    QuantArgs a = {X, ldx, Q, ldq, S, d};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = dtype == LORA_BF16 ? launch_quant<__nv_bfloat16>(a, N, s)
                  : dtype == LORA_F16 ? launch_quant<__half>(a, N, s)
                                      : launch_quant<float>(a, N, s);
    return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}
