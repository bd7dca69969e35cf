// lora_rope: rotary positions on the heads of projections that share their tokens
// (q and k right after their adapted projection).  With t = pos[n] * freq[j], the pair
// (a, b) of a head's first rot dimensions becomes
//
//     a' = m (a cos t - b sin t),   b' = m (b cos t + a sin t)
//
// (inverse: t -> -t, the transpose, which is the gradient), pair j being dimensions
// (j, j + rot/2) or, interleaved, (2j, 2j + 1); dimensions past rot are copied.
//
// The angle is what needs care: at position 10^6 a frequency of 1 turns 160 000 times,
// and fp32 would leave an error of several hundredths of a radian.  So the turns
// u = pos * (freq / 2 pi) are formed and reduced to [-1/2, 1/2] in fp64, the factor in two
// parts (one alone is off by up to 1.6 * 2^-53: 2e-6 of a radian at 2^31 turns), and only the
// reduced angle goes to sincospif in fp32.  cos and sin carry m; the products are fp32, each
// output is rounded to its type once.
//
// Bound: HBM, one read and one write per element.  A block takes up to 8 tokens: their
// cos / sin come out once, in shared memory, for all heads, while the first loads of x
// are in flight.  17389 tokens of 32 + 8 heads of 128 in bf16 (356 MB): 62 us, 5.8 TB/s;
// with one token a block, its angles' latency in every token's way, 113 us.

#include "lora_internal.cuh"

#include <cuda_fp16.h>

#include <cmath>

namespace lora {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeHold = 2;        // items a thread has in flight
constexpr double kInv2Pi = 0x1.45f306dc9c883p-3, kInv2PiLow = -0x1.6b01ec5417056p-57;    // 1 / 2 pi

struct RopeMat {
    const void *x;
    void *y;
    int64_t xs, xh, ys, yh;         // token and head strides, elements
    int32_t first;                  // this matrix's first head among the token's heads
    int32_t pad;
};

struct RopeArgs {
    RopeMat mat[LORA_MAX_PROJ];
    int32_t n_mat;
    const void *pos;
    int32_t pos64;
    const double *freq;
    int32_t N, dim, half;           // half = rot / 2
    int32_t heads;                  // of a token, all matrices
    int32_t rot_items, head_items;  // items of a head that rotate; all of them
    int32_t cols, slots;            // threads along a head's items, and along heads
    int32_t tokens;                 // per block
    float m;
    float sign;                     // -1: inverse
};

// V elements as loaded: 16, 8 or 4 bytes in one access, or one element
template <int BYTES> struct Words;
template <> struct Words<16> { using type = uint4; };
template <> struct Words<8> { using type = uint2; };
template <> struct Words<4> { using type = uint32_t; };
template <class T, int V> struct Raw { typename Words<V * sizeof(T)>::type u; };
template <class T> struct Raw<T, 1> { T u; };

template <class T, int V> __device__ __forceinline__ void get(const T *p, Raw<T, V> &r)
{
    r.u = *reinterpret_cast<const decltype(r.u) *>(p);
}

template <class T, int V> __device__ __forceinline__ void widen(const Raw<T, V> &r, float *f)
{
    if constexpr (V == 1) {
        f[0] = (float)r.u;
    } else {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&r.u);
#pragma unroll
        for (int i = 0; i < (int)(V * sizeof(T) / 4); ++i) {
            if constexpr (std::is_same<T, float>::value) {
                f[i] = __uint_as_float(w[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                f[2 * i] = h.x;
                f[2 * i + 1] = h.y;
            }
        }
    }
}

template <class T, int V> __device__ __forceinline__ void put(T *p, const float *f)
{
    Raw<T, V> r;
    if constexpr (V == 1) {
        if constexpr (std::is_same<T, float>::value)
            r.u = f[0];
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            r.u = __float2bfloat16_rn(f[0]);
        else
            r.u = __float2half_rn(f[0]);
    } else {
        uint32_t *w = reinterpret_cast<uint32_t *>(&r.u);
#pragma unroll
        for (int i = 0; i < (int)(V * sizeof(T) / 4); ++i) {
            if constexpr (std::is_same<T, float>::value) {
                w[i] = __float_as_uint(f[i]);
            } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    *reinterpret_cast<decltype(r.u) *>(p) = r.u;
}

// An item is V pairs of one head (two runs of V elements half a rotation apart;
// interleaved: one run of V elements, or a single pair where V is 1), or, past rot, a run
// of V elements that is copied.  A thread keeps its place c along a head's items and
// walks the block's (token, head) list, so no index is divided on the way; kRopeHold
// items are in flight at a time, the first ones while the angles are worked out.  (Five
// blocks to an SM in 16 bits, 48 registers a thread: 61.6 us against 65.8 with four for the
// case above; in fp32 four, 56.4 against 57.7 for 8190 tokens.)
template <class T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 ? 5 : 4) k_rope(const __grid_constant__ RopeArgs p)
{
    extern __shared__ float2 cs[];                   // [tokens][half]
    constexpr bool kTwo = !INTER || V == 1;          // an item has a second run
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x;
    const int n0 = blockIdx.x * p.tokens;
    const int n_tok = min(p.tokens, p.N - n0);
    const int slot = tid / p.cols, c_first = tid - slot * p.cols;
    const int dt = p.slots / p.heads, dh = p.slots - dt * p.heads;    // a step along the list

    struct Item {
        T *y;
        int t;                                       // token of the block, -1: no item
        Raw<T, V> a, b;
    };
    auto fetch = [&](Item &it, int t, int h, int e, bool two) {
        it.t = t < n_tok ? t : -1;
        if (t >= n_tok)
            return;
        int q = 0;
#pragma unroll
        for (int j = 1; j < LORA_MAX_PROJ; ++j)
            if (j < p.n_mat && h >= p.mat[j].first)
                q = j;
        const RopeMat &m = p.mat[q];
        const int64_t n = n0 + t, hh = h - m.first;
        const T *x = static_cast<const T *>(m.x) + n * m.xs + hh * m.xh + e;
        it.y = static_cast<T *>(m.y) + n * m.ys + hh * m.yh + e;
        get<T, V>(x, it.a);
        if (kTwo && two)
            get<T, V>(x + (INTER ? 1 : p.half), it.b);
    };
    auto finish = [&](const Item &it, int pair, bool rotate) {
        if (it.t < 0)
            return;
        float a[V], b[V], oa[V], ob[V];
        widen<T, V>(it.a, a);
        if (!rotate) {
            put<T, V>(it.y, a);
            return;
        }
        const float2 *w = cs + it.t * p.half + pair;
        if constexpr (kTwo) {
            widen<T, V>(it.b, b);
#pragma unroll
            for (int u = 0; u < V; ++u) {
                oa[u] = a[u] * w[u].x - b[u] * w[u].y;
                ob[u] = b[u] * w[u].x + a[u] * w[u].y;
            }
            put<T, V>(it.y, oa);
            put<T, V>(it.y + (INTER ? 1 : p.half), ob);
        } else {
#pragma unroll
            for (int u = 0; u < V; u += 2) {
                oa[u] = a[u] * w[u / 2].x - a[u + 1] * w[u / 2].y;
                oa[u + 1] = a[u + 1] * w[u / 2].x + a[u] * w[u / 2].y;
            }
            put<T, V>(it.y, oa);
        }
    };

    bool angles = false;
    for (int c = c_first; c < p.head_items || !angles; c += p.cols) {
        const bool on = slot < p.slots && c < p.head_items, rotate = c < p.rot_items;
        // first element of the item in its head, first pair in the token's angles
        const int e = rotate ? (INTER && V == 1 ? 2 * c : c * V) : 2 * p.half + (c - p.rot_items) * V;
        const int pair = INTER ? e / 2 : e;
        int t = slot / p.heads, h = slot - t * p.heads;
        auto step = [&] {
            t += dt;
            h += dh;
            if (h >= p.heads) {
                h -= p.heads;
                ++t;
            }
        };
        Item it[kRopeHold];
        bool more = on && t < n_tok;
        auto fetch_all = [&] {
#pragma unroll
            for (int j = 0; j < kRopeHold; ++j) {
                fetch(it[j], t, h, e, rotate);
                step();
            }
        };
        if (more)
            fetch_all();
        if (!angles) {
            for (int i = tid; i < n_tok * p.half; i += blockDim.x) {
                const int tt = i / p.half, j = i - tt * p.half;
                const double at = p.pos64 ? (double)static_cast<const int64_t *>(p.pos)[n0 + tt]
                                          : (double)static_cast<const int32_t *>(p.pos)[n0 + tt];
                // f + fl = freq / 2 pi to 2^-104 of itself (the second constant is what the first
                // leaves of 1 / 2 pi); at * f less its whole turns is exact but for one rounding
                // below 1
                const double f = p.freq[j] * kInv2Pi, fl = fma(p.freq[j], kInv2Pi, -f) + p.freq[j] * kInv2PiLow;
                const double u = fma(at, fl, fma(at, f, -rint(at * f)));
                float s, co;
                sincospif(2.f * (float)u, &s, &co);
                cs[i] = make_float2(co * p.m, s * p.m * p.sign);
            }
            __syncthreads();
            angles = true;
        }
        while (more) {
#pragma unroll
            for (int j = 0; j < kRopeHold; ++j)
                finish(it[j], pair, rotate);
            more = t < n_tok;
            if (more)
                fetch_all();
        }
    }
}

template <class T, bool INTER, int V> cudaError_t launch_rope_v(RopeArgs &a, bool copy, cudaStream_t s)
{
    const int rot = 2 * a.half;
    a.rot_items = INTER ? (V > 1 ? rot / V : a.half) : a.half / V;
    a.head_items = a.rot_items + (copy ? (a.dim - rot) / V : 0);
    a.cols = a.head_items < kRopeThreads ? a.head_items : kRopeThreads;
    a.slots = kRopeThreads / a.cols;
    // tokens a block: as many as leave every SM four blocks, up to 8 (their angles cost the
    // block one wait, and it is spread over all of them), and at least half the threads' worth
    const int64_t per_tok = (int64_t)a.heads * a.cols;
    a.tokens = 1;
    while (a.tokens < 8 && ((int64_t)a.N >= 2 * 4 * 148 * (int64_t)a.tokens || a.tokens * per_tok < kRopeThreads / 2))
        a.tokens *= 2;
    if (a.slots > (int64_t)a.tokens * a.heads)
        a.slots = a.tokens * a.heads;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.N + a.tokens - 1) / a.tokens));
    cfg.blockDim = dim3((a.cols * a.slots + 31) & ~31);
    cfg.dynamicSmemBytes = sizeof(float2) * a.tokens * a.half;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_rope<T, V, INTER>, a);
}

// v: elements an access may move (a power of two, at most 16 bytes)
template <class T, bool INTER> cudaError_t launch_rope_t(RopeArgs &a, int v, bool copy, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2)
        if (v == 8)
            return launch_rope_v<T, INTER, 8>(a, copy, s);
    return v >= 4 ? launch_rope_v<T, INTER, 4>(a, copy, s)
         : v == 2 ? launch_rope_v<T, INTER, 2>(a, copy, s)
                  : launch_rope_v<T, INTER, 1>(a, copy, s);
}

template <class T> cudaError_t launch_rope(RopeArgs &a, bool inter, int v, bool copy, cudaStream_t s)
{
    return inter ? launch_rope_t<T, true>(a, v, copy, s) : launch_rope_t<T, false>(a, v, copy, s);
}

}  // namespace
}  // namespace lora

using namespace lora;

namespace {

// Distinct (token, head) of a tensor lie in distinct elements: tokens hold whole heads
// apart, or heads hold whole tokens apart.
bool apart(int64_t token, int64_t head, int32_t N, int32_t heads, int32_t dim)
{
    const __int128 t = token, h = head;
    const bool by_token = (heads == 1 || h >= dim) && (N == 1 || t >= (__int128)(heads - 1) * h + dim);
    const bool by_head = (N == 1 || t >= dim) && (heads == 1 || h >= (__int128)(N - 1) * t + dim);
    return by_token || by_head;
}

}  // namespace

extern "C" lora_status lora_rope(const lora_rope_mat *mats, int32_t n_mats, int32_t dtype, const void *pos,
                                 int32_t pos_bytes, const double *freq, int32_t N, int32_t dim, int32_t rot,
                                 int32_t interleaved, int32_t inverse, float mscale, void *stream)
{
    if (!mats || n_mats < 1 || N < 0 || dim < 2 || rot < 2 || rot > dim || (rot & 1) || (N > 0 && (!pos || !freq)) ||
        (pos_bytes != 4 && pos_bytes != 8))
        return LORA_ERR_INVALID_ARG;
    if (n_mats > LORA_MAX_PROJ || dim > LORA_MAX_ROPE_DIM || dtype < LORA_BF16 || dtype > LORA_F32)
        return LORA_ERR_UNSUPPORTED;
    const int es = dtype == LORA_F32 ? 4 : 2;
    if (((uintptr_t)pos & (pos_bytes - 1)) || ((uintptr_t)freq & 7))
        return LORA_ERR_UNSUPPORTED;
    RopeArgs a = {};
    // elements an access moves, v: every run of v starts on a boundary of its own size.  (A head of
    // 72 with 36 rotating allows 4, with 18 none; one element at a time costs 2 to 3 times as much.)
    uint64_t steps = (interleaved ? rot : rot / 2) | rot | dim, at = 0;
    bool copy = false;
    for (int i = 0; i < n_mats; ++i) {
        const lora_rope_mat &m = mats[i];
        if (N > 0 && (!m.x || !m.y))
            return LORA_ERR_INVALID_ARG;
        if (m.heads < 1 || m.x_token < 0 || m.x_head < 0 || !apart(m.y_token, m.y_head, N, m.heads, dim))
            return LORA_ERR_INVALID_ARG;
        const bool same = m.x == m.y;
        if (same && (m.x_token != m.y_token || m.x_head != m.y_head))
            return LORA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (N > 0 && mats[j].y == m.y)
                return LORA_ERR_INVALID_ARG;
        if (((uintptr_t)m.x | (uintptr_t)m.y) & (es - 1))
            return LORA_ERR_UNSUPPORTED;
        copy |= !same && rot < dim;
        steps |= (uint64_t)(m.x_token | m.x_head | m.y_token | m.y_head);
        at |= (uintptr_t)m.x | (uintptr_t)m.y;
        a.mat[i] = {m.x, m.y, m.x_token, m.x_head, m.y_token, m.y_head, a.heads, 0};
        if (m.heads > LORA_MAX_ROPE_HEADS || (a.heads += m.heads) > LORA_MAX_ROPE_HEADS)
            return LORA_ERR_UNSUPPORTED;
    }
    if (N == 0)
        return LORA_OK;
    a.n_mat = n_mats;
    a.pos = pos;
    a.pos64 = pos_bytes == 8;
    a.freq = freq;
    a.N = N;
    a.dim = dim;
    a.half = rot / 2;
    a.m = mscale;
    a.sign = inverse ? -1.f : 1.f;
    cudaStream_t s = (cudaStream_t)stream;
    const bool inter = interleaved != 0;
    int v = 16 / es;
    while (v > 1 && ((steps & (v - 1)) || (at & (v * es - 1))))
        v /= 2;
    const cudaError_t e = dtype == LORA_BF16 ? launch_rope<__nv_bfloat16>(a, inter, v, copy, s)
                        : dtype == LORA_F16 ? launch_rope<__half>(a, inter, v, copy, s)
                                            : launch_rope<float>(a, inter, v, copy, s);
    return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

extern "C" lora_status lora_rope_freqs(int32_t scaling, int32_t rot, double base, double factor, double low,
                                       double high, double original, double *freq, double *mscale)
{
    if (!freq || !mscale || rot < 2 || (rot & 1) || !(base > 1.0) || !std::isfinite(base))
        return LORA_ERR_INVALID_ARG;
    if (scaling < LORA_ROPE_NONE || scaling > LORA_ROPE_YARN)
        return LORA_ERR_UNSUPPORTED;
    if (scaling != LORA_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor)))
        return LORA_ERR_INVALID_ARG;
    const bool ramps = scaling == LORA_ROPE_BANDS || scaling == LORA_ROPE_YARN;
    if (ramps && (!(low > 0.0) || !(high > low) || !std::isfinite(high) || !(original > 0.0) || !std::isfinite(original)))
        return LORA_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586477;
    if (scaling == LORA_ROPE_NTK && rot > 2)
        base *= std::pow(factor, (double)rot / (rot - 2));
    double first = 0, last = 0;      // yarn: the ramp's pairs
    if (scaling == LORA_ROPE_YARN) {
        // the pair that makes `turns` turns over the original length
        const double per = rot / (2.0 * std::log(base));
        first = std::fmax(std::floor(per * std::log(original / (high * two_pi))), 0.0);
        last = std::fmin(std::ceil(per * std::log(original / (low * two_pi))), rot - 1.0);
    }
    for (int j = 0; j < rot / 2; ++j) {
        double f = std::pow(base, -2.0 * j / rot);
        double stretched = 0;        // share of the frequency that is divided by factor
        if (scaling == LORA_ROPE_LINEAR)
            stretched = 1;
        else if (scaling == LORA_ROPE_BANDS)
            stretched = 1 - (original * f / two_pi - low) / (high - low);
        else if (scaling == LORA_ROPE_YARN)
            stretched = (j - first) / std::fmax(last - first, 0.001);
        stretched = std::fmin(std::fmax(stretched, 0.0), 1.0);
        freq[j] = f * (1 - stretched) + f / factor * stretched;
        if (stretched == 0)
            freq[j] = f;
    }
    *mscale = scaling == LORA_ROPE_YARN && factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return LORA_OK;
}
