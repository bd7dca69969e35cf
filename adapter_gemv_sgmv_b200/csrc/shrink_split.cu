// s V = s A[a] x for the segments' tiles, as bf16 high and low parts (lora_linear_i8_sgmv):
//
//     v[n][j] = s sum_i A[a][j][i] x[n][i],   hi = bf16(v), lo = bf16(v - hi)
//
// At the end of the range: a finite v that bf16 would round to infinity has hi = bf16's largest
// value (lo holds the rest), and where v is infinite or NaN so are both parts (inf - inf would
// make a NaN of every infinity).
//
// A tile is at most 128 rows of one segment, its product [128 x d_in] x [d_in x rank].
// Few tiles leave most SMs idle, and a single CTA takes d_in / 64 k-blocks in a row (44 us
// for 23 segments of 1535 tokens at d_in 4096), so the reduction is split over the CTAs of
// a cluster: each multiplies its share (tcgen05, fp32 in tensor memory), leaves its sums in
// its shared memory, and finishes a share of the rows from all of them, added in the order
// of the CTAs.  Bound: the reads of x (from HBM for long prompts), and for short ones the
// chain launch - first loads - exchange - store: 8 us for the case above.
//
// 192 threads: warp 0 loads (TMA; A rows at offsets no view reaches with 16-byte copies),
// warp 1 issues the MMAs, warps 2-5 empty the accumulator.

#include "lora_internal.cuh"
#include "tc_ptx.cuh"

namespace lora {
namespace {

constexpr int kVThreads = 192;
// A stage is an x box of 128 rows x 64 columns and as many A rows as the pool's ranks reach;
// as many stages as leave two CTAs to an SM (3 at rank 128, 4 at 64, 6 at 16): a tile's loads
// are a chain of round trips, and rank 64 with 3 stages took 48 us for 17389 tokens.
constexpr int kVMaxStages = 6;
constexpr int kVRing = 110 * 1024;

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}

__device__ __forceinline__ float4 ld_remote(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// The tile's rows and segment, *n_tiles in all (-1: bad offsets).  Every warp asks for itself:
// a lane holds four segments, and a scan over the lanes numbers their tiles.  It saves the
// plan kernel in front: 19.5 us for 22.6 (16 rows in one segment, 1024 -> 1024), and with
// all 128 segments 70.2 for 73.2 (512 rows, 4096 -> 4096); more would need a loop.
__device__ __forceinline__ Group find_tile(const SplitShrinkArgs &p, int tile, int lane, int *n_tiles)
{
    static_assert(kSplitShrinkSegs == 32 * 4, "four segments a lane");
    int off[5], pre[5];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 5; ++i)
        off[i] = p.seg_off[min(4 * lane + i, p.n_seg)];   // (empty ones behind the last)
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= off[i] < 0 || off[i + 1] < off[i] || off[i + 1] > p.N;
    Group g = {};
    *n_tiles = -1;
    if (__any_sync(0xffffffffu, bad))
        return g;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sum += (int)(((unsigned)(off[i + 1] - off[i]) + 127u) / 128u);
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        incl += lane >= d ? o : 0;
    }
    *n_tiles = __shfl_sync(0xffffffffu, incl, 31);
    pre[0] = incl - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pre[i + 1] = pre[i] + (int)(((unsigned)(off[i + 1] - off[i]) + 127u) / 128u);
        if (tile >= pre[i] && tile < pre[i + 1]) {
            g.p0 = off[i] + (tile - pre[i]) * 128;
            g.cnt = min(128, off[i + 1] - g.p0);
            g.item = 4 * lane + i;
        }
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, g.cnt > 0)) - 1;   // (none: lane 31, nothing)
    g.p0 = __shfl_sync(0xffffffffu, g.p0, owner & 31);
    g.cnt = __shfl_sync(0xffffffffu, g.cnt, owner & 31);
    g.item = __shfl_sync(0xffffffffu, g.item, owner & 31);
    return g;
}

// The parts of a value whose rounding to bf16 is no finite number (others' stay).
constexpr float kBf16Max = 0x1.fep127f;
__device__ __forceinline__ void end_of_range(float v, __nv_bfloat16 &hi, float &lo)
{
    if (!(fabsf(v) <= 3.402823466e38f)) {            // infinite or NaN
        lo = v;
    } else if (fabsf(__bfloat162float(hi)) > kBf16Max) {
        hi = __float2bfloat16_rz(v);
        lo = v - __bfloat162float(hi);
    }
}

__global__ void __launch_bounds__(kVThreads) k_split_shrink(const __grid_constant__ SplitShrinkArgs p)
{
    extern __shared__ __align__(1024) unsigned char sm_dyn[];
    unsigned char *sm = sm_dyn + ((1024 - (smem_u32(sm_dyn) & 1023)) & 1023);
    __shared__ __align__(8) uint64_t full_bar[kVMaxStages], empty_bar[kVMaxStages], acc_full, mma_drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_stages = p.stages, stage = p.stage;
    const int split = p.split, rank = blockIdx.x % split, tile = blockIdx.x / split;
    int issued = 0;

    if (tid == 0) {
        for (int s = 0; s < n_stages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&mma_drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        tmem_alloc(&tmem_base, 128);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();                                      // the tiles are planned, the workspace is free
    pdl_trigger();
    // what ends here ends for the whole cluster: it works on one tile
    Group g = {};
    int32_t a = -1, r = 0;
    int64_t aoff = 0, boff = 0;
    int n_tiles;
    if (p.groups) {
        n_tiles = p.hdr->n_groups;
        if (tile < n_tiles)
            g = p.groups[tile];
    } else {
        g = find_tile(p, tile, lane, &n_tiles);
        if (blockIdx.x == 0 && tid == 0) {
            p.hdr->n_groups = max(n_tiles, 0);
            if (n_tiles < 0)
                atomicOr(p.err, (uint32_t)LORA_ERR_BAD_SEGMENT);
        }
    }
    if (tile < n_tiles) {
        a = p.seg_ad[g.item];
        if (a != -1 && !pool_adapter_ok(p.pool, a, &r, &aoff, &boff)) {
            if (tid == 0)
                atomicOr(p.err, (uint32_t)LORA_ERR_BAD_ADAPTER);
            r = 0;
        }
    }
    if (r == 0) {
        if (warp == 1)
            tmem_dealloc(tmem, 128);
        return;
    }
    const int d_in = p.pool.d_in, n_kb = (d_in + kBK - 1) / kBK, r16 = (r + 15) & ~15;
    const int k0 = rank * n_kb / split, k1 = (rank + 1) * n_kb / split;
    // (one 64-bit division: 200 instructions, and in the load loop it took longer than a load)
    const int64_t a_row = aoff / d_in;
    const bool view = p.a_tma && a_row * d_in == aoff && a_row + r <= 0x7fffffffLL;

    if (warp == 0) {
        const uint64_t pol_x = policy_evict_first(), pol_a = policy_evict_last();
        // (one thread: a warp that waits together took 0.35 us a k-block, this takes 0.29)
        if (view && lane == 0 && !p.test_stall) {
            const int row = (int)a_row;
            int s = 0;
            uint32_t ph = 1;
            for (int k = k0; k < k1; ++k, ++issued) {
                if (!mbar_wait(&empty_bar[s], ph, &abort_flag, p.err, p.wait_ns))
                    break;
                unsigned char *xs = sm + s * stage, *as = xs + kAtom;
                mbar_arrive_expect_tx(&full_bar[s], kAtom + r * 128);
                tma_load_2d_hint(xs, &p.map_x, &full_bar[s], k * kBK, g.p0, pol_x);
                // a box for every binary digit of the rank (each costs 60 ns a k-block: 24 loads
                // of 8 rows more took 1.7 us of 21 at d_in 14336)
                int j = 0;
#pragma unroll
                for (int m = 0; m < 5; ++m)
                    if (r & (128 >> m)) {
                        tma_load_2d_hint(as + j * 128, &p.map_a[m], &full_bar[s], k * kBK, row + j, pol_a);
                        j += 128 >> m;
                    }
                if (++s == n_stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        } else if (!view) {
            int s = 0;
            uint32_t ph = 1;
            for (int k = k0; k < k1 && !p.test_stall; ++k, ++issued) {
                if (!warp_wait(&empty_bar[s], ph, &abort_flag, p.err, p.wait_ns))
                    break;
                unsigned char *xs = sm + s * stage, *as = xs + kAtom;
                for (int idx = lane; idx < r * 8; idx += 32) {
                    const int j = idx >> 3, c = idx & 7, col = k * kBK + c * 8;
                    const bool ok = col < d_in;
                    cp_async16(smem_u32(as) + sw128_off(j, c), p.pool.A + aoff + (ok ? (int64_t)j * d_in + col : 0), ok);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full_bar[s], kAtom);
                    tma_load_2d_hint(xs, &p.map_x, &full_bar[s], k * kBK, g.p0, pol_x);
                }
                __syncwarp();
                if (++s == n_stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        __syncwarp();
        issued = __shfl_sync(0xffffffffu, issued, 0);
    } else if (warp == 1) {
        if (lane == 0) {
            // (rows r .. r16 - 1 of the A tile hold whatever was there: columns nobody reads)
            const uint32_t idesc = idesc_bf16(128, r16);
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int k = k0; k < k1; ++k) {
                if (!(ok = mbar_wait(&full_bar[s], ph, &abort_flag, p.err, p.wait_ns)))
                    break;
                tc_fence_after();
                const uint32_t xs = smem_u32(sm + s * stage), as = xs + kAtom;
#pragma unroll
                for (int i = 0; i < kBK / 16; ++i)
                    tc_mma(tmem, sw128_desc(xs + i * 32), sw128_desc(as + i * 32), idesc, (k > k0 || i > 0) ? 1u : 0u);
                tc_commit(&empty_bar[s]);
                if (++s == n_stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (ok)
                tc_commit(&acc_full);
        }
    } else {
        // sums to shared memory as [4 ranks][128 rows][4], in the ring's place: every fill has
        // been multiplied when the accumulator is full
        const int q = warp & 3, row = q * 32 + lane;
        if (warp_wait(&acc_full, 0, &abort_flag, p.err, p.wait_ns)) {
            tc_fence_after();
            for (int c = 0; c < r16; c += 32) {      // (128 columns are allocated)
                float v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (c + i < r16)
                        st_shared_v4(smem_u32(sm) + ((c + i) / 4 * 128 + row) * 16, __float_as_uint(v[i]),
                                     __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    if (warp == 0)
        drain_fills(full_bar, n_stages, issued, p.err, p.wait_ns);
    if (warp == 1 && lane == 0)
        drain_mma(&mma_drain, 0, p.err, p.wait_ns);
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
    __syncwarp();
    cluster_sync();
    bool whole = true;                               // a CTA that gave up has no sums to offer
    for (int c = 0; c < split; ++c) {
        int f;
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(f) : "r"(map_rank(smem_u32(&abort_flag), c)));
        whole &= f == 0;
    }
    if (whole) {
        // 8 ranks of a row at a time, zeros from the rank to the next multiple of 16
        for (int i = rank * kVThreads + tid; i < 16 * r16; i += split * kVThreads) {
            const int row = i & 127, o = i >> 7;
            if (row >= g.cnt)
                continue;
            const uint32_t at = smem_u32(sm) + (o * 256 + row) * 16;
            float v[8] = {};
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < split) {
                    const float4 x = ld_remote(map_rank(at, c)), y = ld_remote(map_rank(at + 128 * 16, c));
                    v[0] += x.x;
                    v[1] += x.y;
                    v[2] += x.z;
                    v[3] += x.w;
                    v[4] += y.x;
                    v[5] += y.y;
                    v[6] += y.z;
                    v[7] += y.w;
                }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float s0 = o * 8 + j < r ? p.scale * v[j] : 0.f, s1 = o * 8 + j + 1 < r ? p.scale * v[j + 1] : 0.f;
                __nv_bfloat162 h = __floats2bfloat162_rn(s0, s1);
                const float2 back = __bfloat1622float2(h);
                float l0 = s0 - back.x, l1 = s1 - back.y;
                if (!(fabsf(l0) <= kBf16Max && fabsf(l1) <= kBf16Max)) {
                    end_of_range(s0, h.x, l0);
                    end_of_range(s1, h.y, l1);
                }
                const __nv_bfloat162 l = __floats2bfloat162_rn(l0, l1);
                hi[j / 2] = *reinterpret_cast<const uint32_t *>(&h);
                lo[j / 2] = *reinterpret_cast<const uint32_t *>(&l);
            }
            __nv_bfloat16 *v_row = p.Vb + (int64_t)(g.p0 + row) * p.ldvb + o * 8;
            *reinterpret_cast<uint4 *>(v_row) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(v_row + p.vb_lo) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    __syncwarp();
    cluster_sync();                                  // (its sums are read: a CTA may go)
}

}  // namespace

cudaError_t launch_split_shrink(const SplitShrinkArgs &a_in, const void *X, int64_t ldx, int32_t N, int max_tiles,
                                cudaStream_t s, bool *ok)
{
    SplitShrinkArgs a = a_in;
    const int d_in = a.pool.d_in;
    *ok = encode_box(&a.map_x, X, N, d_in, ldx, 128);
    if (!*ok)
        return cudaSuccess;
    const int64_t rows = a.pool.A_elems / d_in;
    a.a_tma = rows >= 1 && rows <= 0x7fffffffLL;
    for (int m = 0; m < 5 && a.a_tma; ++m)
        a.a_tma = 128 >> m > a.pool.max_rank ||
                  encode_box(&a.map_a[m], a.pool.A, rows, d_in, d_in, 128 >> m);
    // as many CTAs as two to an SM hold at once, each with eight k-blocks at least
    const int n_kb = (d_in + kBK - 1) / kBK;
    a.split = 1;
    while (a.split < 8 && 2 * a.split * max_tiles <= 2 * sm_count() && n_kb >= 16 * a.split)
        a.split *= 2;
    // (the sums that take the ring's place need 512 bytes a rank)
    const int r16 = (a.pool.max_rank + 15) & ~15;
    a.stage = kAtom + r16 * 128;
    a.stages = kVRing / a.stage < kVMaxStages ? kVRing / a.stage : kVMaxStages;
    const int smem = a.stages * a.stage + 1024;
    a.wait_ns = wait_bound_ns();
    a.test_stall = test_stall_mode();
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if ((e = cudaFuncSetAttribute(k_split_shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, kVRing + 1024)) != cudaSuccess)
            return e;
        if (dev >= 0 && dev < 64)
            attr_set[dev] = true;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(max_tiles * a.split);
    cfg.blockDim = dim3(kVThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_split_shrink, a);
}

}  // namespace lora
