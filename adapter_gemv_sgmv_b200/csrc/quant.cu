// lora_quant_i8: rows of activations (or of a weight) as 8-bit integers with one
// scale a row, the form lora_linear_i8 multiplies.
//
//     s[n] = max_i |x[n][i]| / 127        q[n][i] = round(127 x[n][i] / max |x[n]|)
//
// with the quotient rounded as the exact real number is, halves to even: an integer
// result has no rounding error to hide in, so every reader of this formula gets the
// same bytes.  A division for each element would cost more than the memory traffic.
// Instead t = x * (127 / max) is rounded, which is off by at most 127.5 * 2^-23 <
// 2^-15; where t lies that near a half, the sign of 127 x - h max decides, h the half:
// 127 x splits into two fp32 parts without error, h has 8 bits, so the fused
// multiply-add that subtracts h max is exact there and the sign is the true one.
//
// Bound: HBM, one read of x and one write of q; in bf16 the instructions come close
// behind (17389 x 4096: 38.5 us, 5.5 TB/s; the exact comparison inlined for every element
// near a half, ties at half the maximum among them, cost 62).

#include "lora_internal.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace lora {
namespace {

constexpr int kQVec = 8;            // elements per load unit (16 bytes of bf16/fp16, 32 of fp32)
constexpr float kNear = 0.5f - 3.1e-5f;    // |t - round(t)| above this: within 2^-15 of a half
constexpr float kMagic = 12582912.f;       // 1.5 * 2^23: adding it rounds to an integer, ties to even

template <class T> struct Vec8;                      // 8 elements as loaded
template <> struct Vec8<float> { uint4 a, b; };
template <> struct Vec8<__nv_bfloat16> { uint4 a; };
template <> struct Vec8<__half> { uint4 a; };

// (from L2: the kernel before this one may still be writing x when this one starts, so
// nothing read here may come from a cache that it does not reach)
template <class T> __device__ __forceinline__ Vec8<T> load8(const T *p)
{
    Vec8<T> v;
    v.a = __ldcg(reinterpret_cast<const uint4 *>(p));
    if constexpr (sizeof(T) == 4)
        v.b = __ldcg(reinterpret_cast<const uint4 *>(p) + 1);
    return v;
}

// Running max |x|: an fp32 bit pattern, or a pair of 16-bit values; NaN wins.
template <class T> __device__ __forceinline__ uint32_t absmax8(const Vec8<T> &v, uint32_t m)
{
    if constexpr (sizeof(T) == 4) {
        // as integers: ordered like the magnitudes, with inf and every NaN above
        m = max(max(m, v.a.x & 0x7fffffffu), v.a.y & 0x7fffffffu);
        m = max(max(m, v.a.z & 0x7fffffffu), v.a.w & 0x7fffffffu);
        m = max(max(m, v.b.x & 0x7fffffffu), v.b.y & 0x7fffffffu);
        return max(max(m, v.b.z & 0x7fffffffu), v.b.w & 0x7fffffffu);
    } else {
        using T2 = std::conditional_t<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>;
        T2 h = *reinterpret_cast<T2 *>(&m);
        const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h = __hmax2_nan(h, __habs2(*reinterpret_cast<const T2 *>(&w[i])));
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

// The running maximum as an fp32 bit pattern that orders like it
template <class T> __device__ __forceinline__ uint32_t max_bits(uint32_t m)
{
    if constexpr (sizeof(T) == 4) {
        return m;
    } else {
        const uint32_t k = max(m & 0x7fffu, (m >> 16) & 0x7fffu);
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return k << 16;
        else
            return __float_as_uint(__half2float(__ushort_as_half((unsigned short)k))) & 0x7fffffffu;
    }
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

// two fp32 operations an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return d;
}

// 8 elements -> 8 bytes.  `pre` is a power of two that keeps 127 x and 127 / top in range.
// SHORT: the elements came from a 16-bit type.  There the one half that turns up often is
// x = top / 2 (a thousandth of normal data in bf16), t = 63.5, rounded to the even 64: `inv`
// is rounded up, so it comes out as 64 already, and no other 16-bit x comes within 2^-15 of
// that half (it stays 1 / (8 * 2047) away).
template <bool SHORT>
__device__ __forceinline__ uint2 round8(float (&x)[8], float inv, float top, float pre, float near)
{
    uint32_t bits[8];
    float d[8], worst = 0.f;
    if (pre != 1.f) {                                // (the same for the whole row)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] *= pre;
    }
    const float2 inv2 = make_float2(inv, inv), magic2 = make_float2(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 v = make_float2(x[i], x[i + 1]);
        const float2 m = fma2(v, inv2, magic2);
        const float2 nq = add2(magic2, make_float2(-m.x, -m.y));     // -q
        const float2 r = fma2(v, inv2, nq);
        d[i] = r.x;
        d[i + 1] = r.y;
        worst = fmaxf(worst, fmaxf(fabsf(r.x), fabsf(r.y)));
        bits[i] = __float_as_uint(m.x);              // low byte: the integer in two's complement
        bits[i + 1] = __float_as_uint(m.y);
    }
    if (worst > near) {
        bool open = !SHORT;
        if (SHORT) {
            const float half = 0.5f * top;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                open |= fabsf(d[i]) > near && fabsf(x[i]) != half;
        }
        if (open) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (fabsf(d[i]) > near)
                    bits[i] = __float_as_uint(settle(x[i], top, __uint_as_float(bits[i]) - kMagic, d[i]) + kMagic);
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
    int32_t N, d;
};

// What a row's maximum gives for rounding it.
struct RowScale {
    float top, inv, pre;
    float near;                     // |t - round(t)| from which the exact comparison decides
    bool bad;                       // inf or NaN in the row

    __device__ RowScale(uint32_t bits, float *s)
    {
        bad = bits >= 0x7f800000u;
        top = __uint_as_float(bits);
        if (s)
            *s = bad ? __uint_as_float(0x7fffffffu) : __fdiv_rn(top, 127.f);
        pre = top < 0x1p-80f ? 0x1p90f : (top > 0x1p100f ? 0x1p-40f : 1.f);
        top *= pre;
        inv = bad || bits == 0 ? 0.f : __fdiv_ru(127.f, top);
        // 127 / top a value of fp32 (top = 127 * 2^k, whose bf16 rows are full of halves): x * inv
        // is t itself, and its one rounding is the definition's
        near = fmaf(inv, top, -127.f) == 0.f ? 1.f : kNear;
    }
    template <class T> __device__ void unit(const Vec8<T> &w, int8_t *q) const
    {
        float f[8];
        unpack8<T>(w, f);
        *reinterpret_cast<uint2 *>(q) = bad ? make_uint2(0, 0) : round8<sizeof(T) == 2>(f, inv, top, pre, near);
    }
};

// Many rows: a warp holds a whole row (VPT units of 8 elements a lane), 4 rows a block; the
// rows' latencies overlap across the 16 and more warps of an SM.
constexpr int kRowWarps = 4;
template <class T, int VPT>
__global__ void __launch_bounds__(32 * kRowWarps) k_quant_warp(const QuantArgs p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int units = p.d / kQVec, lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    if (n >= p.N)
        return;
    const T *x = static_cast<const T *>(p.X) + n * p.ldx + lane * kQVec;
    int8_t *q = p.Q + n * p.ldq + lane * kQVec;
    Vec8<T> v[VPT];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (lane + 32 * j < units)
            v[j] = load8(x + 32 * kQVec * j);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (lane + 32 * j < units)
            m = absmax8<T>(v[j], m);
    const RowScale r(__reduce_max_sync(0xffffffffu, max_bits<T>(m)), lane == 0 ? p.S + n : nullptr);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (lane + 32 * j < units)
            r.unit<T>(v[j], q + 32 * kQVec * j);
}

// Few rows, or long ones: a block holds a row; a row longer than that (WIDE) is read a second
// time, from L2.  (Blocks of up to 512 threads, several to an SM, so that one block's waits
// are another's work: 2011 rows of 14336 took 28 us with 896 threads a row.)
constexpr int kRowThreads = 512;
template <class T, int VPT, bool WIDE>
__global__ void __launch_bounds__(kRowThreads, VPT == 1 ? 4 : 2) k_quant_block(const QuantArgs p)
{
    __shared__ uint32_t part[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int units = p.d / kQVec, tid = threadIdx.x, nt = blockDim.x;
    const int64_t n = blockIdx.x;
    const T *x = static_cast<const T *>(p.X) + n * p.ldx;
    int8_t *q = p.Q + n * p.ldq;
    Vec8<T> v[VPT];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (tid + j * nt < units)
            v[j] = load8(x + (int64_t)(tid + j * nt) * kQVec);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (tid + j * nt < units)
            m = absmax8<T>(v[j], m);
    if constexpr (WIDE)
        for (int u = tid + VPT * nt; u < units; u += nt)
            m = absmax8<T>(load8(x + (int64_t)u * kQVec), m);
    m = __reduce_max_sync(0xffffffffu, max_bits<T>(m));
    if ((tid & 31) == 0)
        part[tid >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, (tid & 31) < (nt >> 5) ? part[tid & 31] : 0u);
    const RowScale r(m, tid == 0 ? p.S + n : nullptr);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
        if (tid + j * nt < units)
            r.unit<T>(v[j], q + (int64_t)(tid + j * nt) * kQVec);
    if constexpr (WIDE)
        for (int u = tid + VPT * nt; u < units; u += nt)
            r.unit<T>(load8(x + (int64_t)u * kQVec), q + (int64_t)u * kQVec);
}

cudaError_t launch_rows(void (*kernel)(QuantArgs), const QuantArgs &a, int grid, int threads, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <class T> cudaError_t launch_quant(const QuantArgs &a, cudaStream_t s)
{
    const int units = a.d / kQVec;
    // A warp a row wastes no time on block-wide waits and little on the row's own arithmetic,
    // but leaves few rows to few slow warps: 4096 bf16, 256 rows 4.1 us against 2.4 for a block a
    // row, 1024 rows 4.7 for both, 2048 rows 6.8 against 7.8, 17389 rows 38.5 against 64.  fp32
    // rows above 2048 do not fit its registers.  fp16 needs more rows: one in 150 has a maximum
    // of 127 times a small odd number, halves everywhere, and 10 us for its warp (2048 rows of
    // 4096 13.7 against 7.9, 17389 rows 44 against 60).
    const int per_lane = (units + 31) / 32;
    const int many = std::is_same<T, __half>::value ? 4096 : 1024;
    if (a.N >= many && per_lane <= (sizeof(T) == 4 ? 8 : 16)) {
        void (*k)(QuantArgs);
        if (per_lane <= 2)
            k = k_quant_warp<T, 2>;
        else if (per_lane <= 5)
            k = k_quant_warp<T, 5>;
        else if (per_lane <= 8)
            k = k_quant_warp<T, 8>;
        else if constexpr (sizeof(T) == 4)
            return cudaErrorInvalidValue;            // (not reached)
        else
            k = k_quant_warp<T, 16>;
        return launch_rows(k, a, (int)(((int64_t)a.N + kRowWarps - 1) / kRowWarps), 32 * kRowWarps, s);
    }
    auto threads = [&](int vpt) { return ((units + vpt - 1) / vpt + 31) & ~31; };
    if (threads(1) <= kRowThreads)
        return launch_rows(k_quant_block<T, 1, false>, a, a.N, threads(1), s);
    if (threads(2) <= kRowThreads)
        return launch_rows(k_quant_block<T, 2, false>, a, a.N, threads(2), s);
    if (threads(4) <= kRowThreads)
        return launch_rows(k_quant_block<T, 4, false>, a, a.N, threads(4), s);
    return launch_rows(k_quant_block<T, 4, true>, a, a.N, kRowThreads, s);
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
    QuantArgs a = {X, ldx, Q, ldq, S, N, d};
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = dtype == LORA_BF16 ? launch_quant<__nv_bfloat16>(a, s)
                  : dtype == LORA_F16 ? launch_quant<__half>(a, s)
                                      : launch_quant<float>(a, s);
    return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}
