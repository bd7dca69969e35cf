// The projection with an 8-bit weight and 8-bit tokens (lora_linear_i8), and the same
// with the segments' LoRA deltas (lora_linear_i8_sgmv):
//
//     y[n][o] = s_x[n] s_w[o] sum_i q[n][i] w[o][i]  (+ s sum_j B[a][o][j] v[n][j])
//
// The sum of integer products is exact in 32 bits (d_in <= 65536: at most 2^30); it is
// widened to fp32, scaled, joined by the delta's fp32 sum and rounded once.
//
// k_i8_pair, long token runs: a pair of CTAs (cluster of 2, tcgen05 cta_group::2) owns a
// tile of 256 rows x BN outputs; each CTA holds 128 rows in its tensor memory and loads
// 128 token rows and half of the tile's weight rows per 128-byte k-block, so a weight
// byte crosses from L2 once per 256 rows and a token byte once per BN outputs.
// Persistent, 320 threads a CTA, with adapters 640:
//   warp 0        producer: TMA boxes into a ring; both CTAs' boxes complete on the
//                 leader's barrier;
//   warp 1        (leader) one thread issues tcgen05.mma kind::i8 (M = 256, K = 32);
//                 (other CTA, with adapters) tells the leader of the B rows gathered there;
//   warps 2-9     epilogue: tensor memory -> scale -> y (with adapters warps 2-17);
//   warps 18, 19  (with adapters) share the producer's gathers of B rows.
// Without adapters two integer accumulators alternate, so a tile's epilogue runs under
// the next one's products.  The delta (LORA) takes the second half of tensor memory as an
// fp32 accumulator: bf16 k-blocks of (s v) high and low parts against the adapter's B
// columns, after the base's.  The epilogue takes the integers into registers while those
// run and hands their accumulator to the next tile, then the fp32 sums while that one
// starts.  (160 columns, which leave room for two integer accumulators beside the fp32
// one, were slower: a tile of 256 x BN reads (256 + BN) / (256 BN) bytes a product.)
// B rows of a rank with a tensor map come by TMA.  Others are gathered, 16 bytes at a time, by
// the producer and two helpers: request_bar[s] lets the helpers into stage s, gather_bar[s] says
// that all three are done (the producer then sends the box of s V, whose barrier the leader's MMA
// thread waits for), and the other CTA's share reaches that thread through peer_bar[s].
// A tile's rows may belong to different adapters.  Each run of rows with one adapter has
// k-blocks of its own, multiplied with every other row of the accumulator masked: a row
// must not meet another adapter's B even with factors of zero, for that B may hold an
// infinity.

#include "lora_internal.cuh"
#include "tc_ptx.cuh"

#include <cuda_fp16.h>

namespace lora {
namespace {

constexpr int kPNsBlock = 16;           // output slices per block of the tile order
constexpr int kKB = 128;                // bytes of the reduction per k-block

// -------------------------------------------------------------- pair PTX glue
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// (orders tensor memory accesses only, through the tcgen05 fences around it: a release
// at cluster scope would wait for the epilogue's stores)
__device__ __forceinline__ void remote_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// (what this thread knows of shared memory comes with it: a waiter with CLUSTER sees it)
__device__ __forceinline__ void remote_arrive_release(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A box into this CTA's shared memory, completing on a barrier of the pair's leader.
__device__ __forceinline__ void tma_load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                              uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;"
        ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// The rows of D that a delta's MMAs leave alone: bit l of word l / 32, rows 0 - 127 in the
// leader's tensor memory, 128 - 255 in the other's.
struct RowMask {
    uint32_t off[8];
    __device__ RowMask(int r0, int r1)               // rows outside [r0, r1)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int lo = min(max(r0 - 32 * i, 0), 32), hi = min(max(r1 - 32 * i, 0), 32);
            off[i] = ~(uint32_t)((1ull << hi) - (1ull << min(lo, hi)));
        }
    }
};

__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                              const RowMask &m)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(m.off[0]), "r"(m.off[1]), "r"(m.off[2]), "r"(m.off[3]),
          "r"(m.off[4]), "r"(m.off[5]), "r"(m.off[6]), "r"(m.off[7])
        : "memory");
}

__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrive on the barrier at this offset in both CTAs when the MMAs issued so far complete.
__device__ __forceinline__ void commit_pair(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_u32(bar)), "h"((uint16_t)3)
        : "memory");
}

// Signed 8-bit A and B, 32-bit integer D, both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ------------------------------------------------------------------ the tiles
template <bool LORA_, int BN_> struct PairCfg {
    static constexpr bool LORA = LORA_;
    static constexpr int BN = BN_;                       // outputs of a tile
    static constexpr int stage = kAtom + BN / 2 * 128;   // token box, half of the weight box
    static constexpr int stages = LORA ? (BN == 256 ? 5 : 6) : 6;
    static constexpr int buffers = LORA ? 1 : 2;         // integer accumulators
    static constexpr int epi_warps = LORA ? 16 : 8, help_warps = LORA ? 2 : 0;
    static constexpr int box_bytes = LORA ? 64 : 128;    // of a row in an epilogue warp's staged box
    static constexpr int threads = 64 + 32 * (epi_warps + help_warps);
    static constexpr int smem = stages * stage + epi_warps * 32 * box_bytes + 1024;
};

struct PairTc {
    I8Args a;
    CUtensorMap map_q;       // tokens [N, d_in], boxes 128 bytes x 128 rows, 128-byte swizzle
    CUtensorMap map_w;       // weight [d_out, d_in], boxes 128 bytes x BN / 2 rows
    CUtensorMap map_y;       // y [N, d_out], boxes of 64 or 128 bytes x 32 rows (written)
    CUtensorMap map_v;       // LORA: s V as bf16 parts [N, 2 kv], boxes 64 columns x 128 rows
    CUtensorMap map_b[4];    // LORA: B pool as [B_elems / r, r], r = 16 << m, boxes of min(r, 64) x BN / 2 rows
    int32_t b_tma;
    int32_t sw_vec;          // the channel scales may be read 16 bytes at a time
    unsigned long long wait_ns;
    int32_t test_stall;
};

struct PairTile {
    int pair, ns;
};

// Tile u in the blocked order: block k holds every row pair against slices 16k .. 16k + 15,
// row-major inside, so the tiles in flight share a few MB of tokens and weights in L2.
// (32 bits: 2^31 tiles would be 2^47 outputs; the 64-bit divisions of every tile took
// the producer longer than a stage)
__device__ __forceinline__ PairTile pair_tile(uint32_t u, uint32_t n_pairs, uint32_t n_ns)
{
    const uint32_t per_blk = n_pairs * kPNsBlock;
    const uint32_t blk = u / per_blk, rem = u - blk * per_blk;
    const uint32_t nsb = min((uint32_t)kPNsBlock, n_ns - blk * kPNsBlock);
    const uint32_t pair = rem / nsb;
    return {(int)pair, (int)(blk * kPNsBlock + rem - pair * nsb)};
}

// ------------------------------------------------------------- segments (LORA)
// A tile is 256 consecutive rows, whatever segments they belong to: the base product does
// not ask.  The delta does: it walks the tile in runs of rows with one adapter.
// The segments' bounds and adapters are looked up once, by all threads, when the CTA
// starts: four dependent loads from global memory each, which every role would otherwise
// wait for in every tile.
struct __align__(16) SegAd {
    int64_t boff;    // the adapter's B
    int32_t a;       // adapter
    int16_t r;       // rank, 0: no delta
    int16_t m;       // B view, -1: rows gathered
};
constexpr int kSegTable = 512;          // segments in shared memory; more are looked up as they come

struct SegTable {
    SegAd ad[kSegTable];
    int32_t off[kSegTable + 1];
};

__device__ SegAd seg_lookup(const PairTc &p, int k, bool report)
{
    SegAd x = {0, -1, 0, -1};
    const int32_t a = p.a.seg_ad[k];
    int32_t r = 0;
    int64_t ao = 0, bo = 0;
    if (a == -1)
        return x;
    if (!pool_adapter_ok(p.a.pool, a, &r, &ao, &bo)) {
        if (report)
            atomicOr(p.a.err, (uint32_t)LORA_ERR_BAD_ADAPTER);
        return x;
    }
    // (the view's row index of the last box has to fit 32 bits)
    int m = b_map(r);
    if (m >= 0 && (!((p.b_tma >> m) & 1) || (bo & (r - 1)) || (bo >> (4 + m)) + p.a.d_out + 512 > 0x7fffffffLL))
        m = -1;
    x.boff = bo;
    x.a = a;
    x.r = (int16_t)r;
    x.m = (int16_t)m;
    return x;
}

struct Segments {
    const PairTc &p;
    const SegTable *tab;
    bool in_tab;

    __device__ int start(int k) const { return in_tab ? tab->off[k] : p.a.seg_off[k]; }
    __device__ SegAd ad(int k) const { return in_tab ? tab->ad[k] : seg_lookup(p, k, false); }
    // the segment of a row (start(0) <= row < start(n_seg)): the last one that starts at or before it
    __device__ int of_row(int row) const
    {
        int lo = 0, hi = p.a.n_seg;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start(mid) <= row)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    }
};

// The runs of rows with one adapter in a tile, in order.
struct Runs {
    const Segments &sg;
    int k, end;          // next segment; the tile's end
    int r0, r1;          // the run
    SegAd ad;

    __device__ Runs(const Segments &sg_, int row0, int end_) : sg(sg_), k(sg_.of_row(row0)), end(end_), r0(0), r1(0)
    {
        ad.r = 0;
    }
    __device__ bool next()
    {
        for (; k < sg.p.a.n_seg; ++k) {
            r0 = sg.start(k);
            if (r0 >= end)
                break;
            r1 = sg.start(k + 1);
            if (r1 == r0)
                continue;
            ad = sg.ad(k);
            if (ad.r == 0)
                continue;
            for (++k; k < sg.p.a.n_seg && r1 < end; ++k) {           // more of the same adapter
                const int e = sg.start(k + 1);
                if (e != r1 && sg.ad(k).a != ad.a)
                    break;
                r1 = e;
            }
            return true;
        }
        ad.r = 0;
        return false;
    }
    // bf16 k-blocks: high and low parts of every 64 rank columns
    __device__ int kblocks() const { return 2 * ((ad.r + 63) >> 6); }
};

__device__ __forceinline__ void tmem_ld16_raw(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld8_raw(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// N consecutive columns (a multiple of 16) of this thread's lane, not yet waited for
template <int N> __device__ __forceinline__ void tmem_ld16s(uint32_t taddr, uint32_t (&r)[N])
{
#pragma unroll
    for (int c = 0; c < N; c += 16)
        tmem_ld16_raw(taddr + c, *reinterpret_cast<uint32_t(*)[16]>(&r[c]));
}

// (a compiler-visible dependence keeps the registers' first use behind the wait)
template <int N> __device__ __forceinline__ void tmem_wait(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i)
        asm volatile("" : "+r"(r[i]));
}

// two results as T, packed (fp32: the bits of one)
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// byte offset of 16-byte chunk c (0..3) of row i inside a 64-byte-swizzled box
__device__ __forceinline__ uint32_t sw64_off(int i, int c) { return (uint32_t)(i * 64 + ((c ^ ((i >> 1) & 3)) << 4)); }

// a b, two at a time
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&d))
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return d;
}

// sums i, j of outputs with channel scales a, b, in fp32
__device__ __forceinline__ float2 scaled(uint32_t i, uint32_t j, float sx, float a, float b)
{
    return mul2(make_float2((float)(int)i, (float)(int)j), mul2(make_float2(sx, sx), make_float2(a, b)));
}

// channel scales of outputs o .. o + N - 1 (past d_out, a multiple of 8, some others':
// those outputs are not written).  All loads leave together: with a branch and a wait for
// every 16 of them they took a microsecond of each tile.
template <int N> __device__ __forceinline__ void load_sw(const PairTc &p, int o, float (&sw)[N])
{
    if (p.sw_vec) {
#pragma unroll
        for (int g = 0; g < N; g += 8) {
            const float4 *s = reinterpret_cast<const float4 *>(p.a.Sw + min(o + g, p.a.d_out - 8));
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 v = s[i / 4];
                sw[g + i] = v.x;
                sw[g + i + 1] = v.y;
                sw[g + i + 2] = v.z;
                sw[g + i + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int g = 0; g < N; g += 8)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sw[g + i] = p.a.Sw[min(o + g, p.a.d_out - 8) + i];
    }
}

// A warp's box of 32 rows in shared memory to y; the box may be written again
// after box_free().
__device__ __forceinline__ void box_store(const CUtensorMap *map, const void *box, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(map), "r"(smem_u32(box)), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void box_free() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void box_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <class C, class T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(C::threads, 1) k_i8_pair(const __grid_constant__ PairTc p)
{
    constexpr bool LORA = C::LORA;
    constexpr int BN = C::BN, kStages = C::stages;
    constexpr int kStage = C::stage;
    constexpr int kF = BN;                           // LORA: first column of the fp32 accumulator
    constexpr int NB = C::buffers;                   // integer accumulators
    constexpr int kEpiWarps = C::epi_warps, kHelp = C::help_warps, kThreads = C::threads;
    constexpr int kCols = BN / (kEpiWarps / 4);      // columns an epilogue warp takes
    constexpr int kBox = 32 * C::box_bytes, kBoxCols = C::box_bytes / sizeof(T);    // staged: 32 rows
    extern __shared__ __align__(1024) unsigned char sm_dyn[];
    // (the two CTAs' buffers must lie at the same offset: the launch gives both the same base)
    unsigned char *sm = sm_dyn + ((1024 - (smem_u32(sm_dyn) & 1023)) & 1023);
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], f_full, f_empty, mma_drain, tab_full;
    // a gather into a stage is asked for; it is in; (leader) the other CTA's is: its rows come by
    // plain copies, which no byte count of full_bar stands for
    __shared__ __align__(8) uint64_t request_bar[LORA ? kStages : 1], gather_bar[LORA ? kStages : 1],
        peer_bar[LORA ? kStages : 1];
    __shared__ std::conditional_t<LORA, SegTable, int> tab;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int G = gridDim.x / 2, c0 = blockIdx.x / 2;
    const int n_kb = (p.a.d_in + kKB - 1) / kKB;
    const int n_ns = (p.a.d_out + BN - 1) / BN;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full_bar[s], 1);              // leader's expect_tx, for both CTAs' boxes
            mbar_init(&empty_bar[s], 1);
        }
        if constexpr (LORA)
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&request_bar[s], 1);
                mbar_init(&gather_bar[s], 1 + kHelp);
                mbar_init(&peer_bar[s], 1);
            }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpiWarps);
        }
        mbar_init(&f_full, 1);
        mbar_init(&tab_full, kThreads - 32);
        mbar_init(&f_empty, 2 * kEpiWarps);
        mbar_init(&mma_drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();
    pdl_trigger();
    // rows: all of them, or what the segments cover (nothing where the plan found them bad)
    const int row_begin = LORA ? p.a.seg_off[0] : 0;
    const int row_end = LORA ? (p.a.hdr->n_groups ? p.a.seg_off[p.a.n_seg] : row_begin) : p.a.N;
    const int n_pairs = (row_end - row_begin + 255) / 256;
    const uint32_t n_units = (uint32_t)n_pairs * n_ns;
    int issued = 0;
    const SegTable *seg_tab = nullptr;
    if constexpr (LORA) {
        seg_tab = &tab;
        // (the producer warp does not look, and starts with the base's loads; whoever reads the
        // table waits for tab_full first)
        for (int k = tid - 32; k <= p.a.n_seg && n_pairs && warp; k += kThreads - 32) {
            const int r0 = p.a.seg_off[k];
            if (k <= kSegTable)
                tab.off[k] = r0;
            if (k < p.a.n_seg) {
                const bool report = blockIdx.x == 0 && p.a.seg_off[k + 1] > r0;
                if (k < kSegTable)
                    tab.ad[k] = seg_lookup(p, k, report);
                else if (report)
                    seg_lookup(p, k, true);
            }
        }
        if (warp)
            mbar_arrive(&tab_full);
    }
    const Segments segs = {p, seg_tab, p.a.n_seg <= kSegTable};

    if (warp == 0 || warp >= 2 + kEpiWarps) {
        // ------------------------------------------------ producer (both CTAs) and its helpers
        // (the last warps share the gathers of B rows and follow the ring for that only)
        const bool lead = warp == 0;
        const int share = lead ? 0 : warp - 1 - kEpiWarps;
        if (p.test_stall)
            goto done;
        const uint64_t pol_x = policy_evict_first(), pol_w = policy_evict_last();
        int s = 0;
        uint32_t ph = 1, gathers = 0;                // bit s: parity of stage s's next gather
        bool alive = true;
        // the next stage, free: its token (or s V) box, its weight (or B) box, the pair's barrier
        unsigned char *as = nullptr, *bs = nullptr;
        uint32_t bar = 0;
        // (a helper follows the lead's requests, not the ring: a barrier's parity tells only two
        // neighbouring rounds apart, and between gathers it may be any number of them away)
        auto stage = [&](bool gather = false) {
            if (lead) {
                alive = warp_wait(&empty_bar[s], ph, &abort_flag, p.a.err, p.wait_ns);
                if (gather && lane == 0)
                    mbar_arrive(&request_bar[s]);
            } else if (gather) {
                alive = warp_wait(&request_bar[s], (gathers >> s) & 1, &abort_flag, p.a.err, p.wait_ns);
            }
            as = sm + s * kStage;
            bs = as + kAtom;
            bar = map_rank(smem_u32(&full_bar[s]), 0);
            return alive;
        };
        auto sent = [&] {
            __syncwarp();
            ++issued;
            if (++s == kStages) {
                s = 0;
                ph ^= 1;
            }
        };
        for (uint32_t u = c0; u < n_units && alive; u += G) {
            const PairTile un = pair_tile(u, n_pairs, n_ns);
            const int tile0 = row_begin + un.pair * 256, row = tile0 + (int)rank * 128;
            const int o0 = un.ns * BN + (int)rank * (BN / 2);
            // a run's k-blocks: part j % 2 (high, low) of rank columns 64 (j / 2) ..; the low
            // part is multiplied with the B rows that came with the high part
            auto delta = [&](const Runs &run) {
                const SegAd &ad = run.ad;
                for (int j = 0; j < run.kblocks(); ++j) {
                    const bool with_b = (j & 1) == 0, gather = with_b && ad.m < 0;
                    if (!stage(gather))
                        return;
                    const int c = j >> 1, w = ad.r < 64 ? ad.r : 64;
                    if (gather) {
                        // no view of this rank: the CTA's BN / 2 output rows x 64 rank columns
                        // (128-byte swizzle), 16 bytes at a time; past r and past d_out zeros
                        for (int idx = share * 32 + lane; idx < BN / 2 * 8; idx += 32 * (1 + kHelp)) {
                            const int o = idx >> 3, cc = idx & 7, col = c * 64 + cc * 8;
                            const bool ok = o0 + o < p.a.d_out && col < ad.r;
                            const __nv_bfloat16 *src =
                                ok ? p.a.pool.B + ad.boff + (int64_t)(o0 + o) * ad.r + col : p.a.pool.B;
                            cp_async16(smem_u32(bs) + sw128_off(o, cc), src, ok);
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&gather_bar[s]);
                        if (lead)
                            alive = warp_wait(&gather_bar[s], (gathers >> s) & 1, &abort_flag, p.a.err, p.wait_ns);
                        gathers ^= 1u << s;
                        if (!alive)
                            return;
                    }
                    if (lead && lane == 0) {
                        // (the leader's own gather is in before it arrives on full_bar)
                        const uint32_t b_bytes = with_b && !gather ? BN / 2 * w * 2 : 0;
                        if (rank == 0)
                            mbar_arrive_expect_tx(&full_bar[s], 2 * (kAtom + b_bytes));
                        tma_load_pair(as, &p.map_v, bar, (j & 1) * p.a.kv + c * 64, row, pol_x);
                        if (b_bytes)
                            tma_load_pair(bs, &p.map_b[ad.m], bar, c * 64, (int)(ad.boff >> (4 + ad.m)) + o0, pol_w);
                    }
                    sent();
                }
            };
            auto base = [&] {
                for (int kb = 0; kb < n_kb && stage(); ++kb) {
                    if (lead && lane == 0) {
                        if (rank == 0)
                            mbar_arrive_expect_tx(&full_bar[s], 2 * kStage);
                        tma_load_pair(as, &p.map_q, bar, kb * kKB, row, pol_x);
                        tma_load_pair(bs, &p.map_w, bar, kb * kKB, o0, pol_w);
                    }
                    sent();
                }
            };
            base();
            if constexpr (LORA) {
                if (u == c0 && alive)
                    alive = warp_wait(&tab_full, 0, &abort_flag, p.a.err, p.wait_ns);
                if (!alive)
                    break;
                for (Runs run(segs, tile0, min(tile0 + 256, row_end)); alive && run.next();)
                    delta(run);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader, one thread)
        // The loop is what feeds the tensor cores: with a warp-wide wait and addresses worked
        // out per k-block it took 650 cycles for the 512 that a k-block's products take.
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = idesc_i8(256, BN), idesc_f = idesc_bf16(256, BN);
            const uint64_t a0 = sw128_desc(smem_u32(sm)), b0 = sw128_desc(smem_u32(sm) + kAtom);
            int s = 0, t = 0, n_delta = 0;
            uint32_t ph = 0, gathers = 0;            // bit s: parity of stage s's next gather
            bool alive = true;
            auto next = [&] {
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            };
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                alive = mbar_wait(bar, parity, &abort_flag, p.a.err, p.wait_ns);
                tc_fence_after();
                return alive;
            };
            auto delta = [&](const Runs &run, int tile0) {
                const int r = run.ad.r, m = run.ad.m;
                const RowMask mask(run.r0 - tile0, run.r1 - tile0);
                int s_b = 0;                         // the stage that holds the B rows
                for (int j = 0; j < run.kblocks() && wait(&full_bar[s], ph); ++j) {
                    if ((j & 1) == 0) {
                        s_b = s;
                        if (m < 0) {                 // gathered: the other CTA's half, too
                            alive = mbar_wait<true>(&peer_bar[s], (gathers >> s) & 1, &abort_flag, p.a.err, p.wait_ns);
                            if (!alive)
                                return;
                            tc_fence_after();
                            gathers ^= 1u << s;
                        }
                    }
                    const uint32_t as = smem_u32(sm + s * kStage), bs = smem_u32(sm + s_b * kStage) + kAtom;
                    const int left = r - (j >> 1) * 64;
                    const int steps = ((left < 64 ? left : 64) + 15) >> 4;
                    for (int i = 0; i < steps; ++i) {
                        // B columns in their view's swizzle
                        const uint64_t bd = r >= 64 || m < 0 ? sw128_desc(bs + i * 32)
                                          : (r == 32 ? sw64_desc(bs + i * 32) : sw32_desc(bs));
                        mma_bf16_pair(tmem + kF, sw128_desc(as + i * 32), bd, idesc_f, (j > 0 || i > 0) ? 1u : 0u, mask);
                    }
                    if (j & 1) {
                        commit_pair(&empty_bar[s_b]);
                        commit_pair(&empty_bar[s]);
                    }
                    next();
                }
            };
            auto base = [&] {
                const int b = t % NB;
                if (!wait(&acc_empty[b], ((t / NB) & 1) ^ 1))
                    return;
                const uint32_t d = tmem + b * BN;
                for (int kb = 0; kb < n_kb && wait(&full_bar[s], ph); ++kb) {
                    const uint64_t at = (uint64_t)(s * (kStage >> 4));
#pragma unroll
                    for (int i = 0; i < kKB / 32; ++i)
                        mma_i8_pair(d, a0 + at + i * 2, b0 + at + i * 2, idesc, (kb > 0 || i > 0) ? 1u : 0u);
                    commit_pair(&empty_bar[s]);
                    next();
                }
                if (alive)
                    commit_pair(&acc_full[b]);
            };
            for (uint32_t u = c0; u < n_units && alive; u += G, ++t) {
                base();
                if constexpr (LORA) {
                    if (!alive || (u == c0 && !wait(&tab_full, 0)))
                        break;
                    const int tile0 = row_begin + pair_tile(u, n_pairs, n_ns).pair * 256;
                    Runs run(segs, tile0, min(tile0 + 256, row_end));
                    if (!run.next())
                        continue;
                    if (!wait(&f_empty, (n_delta & 1) ^ 1))
                        break;
                    ++n_delta;
                    do
                        delta(run, tile0);
                    while (alive && run.next());
                    if (alive)
                        commit_pair(&f_full);
                }
            }
        } else if (LORA && lane == 0 && !p.test_stall) {
            // The other CTA's thread tells the leader of every gather here.  (By the producer, whose
            // next loads then wait for the release, 2048 rows with 16 adapters of rank 24, 4096 ->
            // 4096, take 56.4 us, and 55.2 so.)
            uint32_t gathers = 0;
            int s = 0;
            bool alive = mbar_wait(&tab_full, 0, &abort_flag, p.a.err, p.wait_ns);
            for (uint32_t u = c0; u < n_units && alive; u += G) {
                const int tile0 = row_begin + pair_tile(u, n_pairs, n_ns).pair * 256;
                s = (s + n_kb) % kStages;
                for (Runs run(segs, tile0, min(tile0 + 256, row_end)); alive && run.next();)
                    for (int j = 0; j < run.kblocks() && alive; ++j) {
                        if ((j & 1) == 0 && run.ad.m < 0) {
                            alive = mbar_wait(&gather_bar[s], (gathers >> s) & 1, &abort_flag, p.a.err, p.wait_ns);
                            gathers ^= 1u << s;
                            if (alive)
                                remote_arrive_release(map_rank(smem_u32(&peer_bar[s]), 0));
                        }
                        if (++s == kStages)
                            s = 0;
                    }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue (both CTAs)
        const int q = warp & 3;                      // TMEM lane quarter
        const int part = (warp - 2) >> 2;            // columns [part * kCols, + kCols)
        const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16) + part * kCols;
        unsigned char *const box = sm + kStages * kStage + (warp - 2) * kBox;    // 32 rows
        int t = 0, n_delta = 0;
        if constexpr (LORA)
            if (!warp_wait(&tab_full, 0, &abort_flag, p.a.err, p.wait_ns))
                goto done;
        for (uint32_t u = c0; u < n_units; u += G, ++t) {
            const PairTile un = pair_tile(u, n_pairs, n_ns);
            const int tile0 = row_begin + un.pair * 256;
            const int row0 = tile0 + (int)rank * 128 + q * 32, row = row0 + lane;    // the warp's first, this lane's
            const bool valid = row < row_end;
            const float sx = valid ? p.a.Sx[row] : 0.f;
            const int o0 = un.ns * BN + part * kCols, b = t % NB;
            const uint32_t acc = lane_base + b * BN;
            if constexpr (LORA) {
                const bool tile_delta = Runs(segs, tile0, min(tile0 + 256, row_end)).next();
                const bool delta = valid && segs.ad(segs.of_row(row)).r;             // this row's
                if (!warp_wait(&acc_full[b], (t / NB) & 1, &abort_flag, p.a.err, p.wait_ns))
                    goto done;
                tc_fence_after();
                uint32_t w[kCols];
                tmem_ld16s(acc, w);
                tmem_wait(w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    remote_arrive(map_rank(smem_u32(&acc_empty[b]), 0));
                if (tile_delta) {
                    if (!warp_wait(&f_full, n_delta & 1, &abort_flag, p.a.err, p.wait_ns))
                        goto done;
                    ++n_delta;
                    tc_fence_after();
                }
                const bool any_delta = __any_sync(0xffffffffu, delta);
                uint32_t out[kCols / 2];             // bf16 pairs
#pragma unroll
                for (int c = 0; c < kCols; c += 8) {
                    uint32_t f[8] = {};
                    float sw[8];
                    if (any_delta)
                        tmem_ld8_raw(lane_base + kF + c, f);
                    load_sw(p, o0 + c, sw);
                    tmem_wait(f);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        float2 v = scaled(w[c + i], w[c + i + 1], sx, sw[i], sw[i + 1]);
                        if (delta) {                 // (another row's sums may be anything)
                            v.x += __uint_as_float(f[i]);
                            v.y += __uint_as_float(f[i + 1]);
                        }
                        out[(c + i) / 2] = pack2(v.x, v.y, T());
                    }
                }
                if (tile_delta) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        remote_arrive(map_rank(smem_u32(&f_empty), 0));
                }
                if (__all_sync(0xffffffffu, valid)) {
#pragma unroll
                    for (int c = 0; c < kCols; c += kBoxCols) {
                        if (lane == 0)
                            box_free();
                        __syncwarp();
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            st_shared_v4(smem_u32(box) + sw64_off(lane, g), out[c / 2 + 4 * g], out[c / 2 + 4 * g + 1],
                                         out[c / 2 + 4 * g + 2], out[c / 2 + 4 * g + 3]);
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0 && o0 + c < p.a.d_out)
                            box_store(&p.map_y, box, o0 + c, row0);
                    }
                } else if (valid) {                  // the segments' last rows: what follows is not ours
                    T *y = static_cast<T *>(p.a.Y) + (int64_t)row * p.a.ldy + o0;
#pragma unroll
                    for (int c = 0; c < kCols; c += 8)
                        if (o0 + c < p.a.d_out)
                            *reinterpret_cast<uint4 *>(y + c) =
                                make_uint4(out[c / 2], out[c / 2 + 1], out[c / 2 + 2], out[c / 2 + 3]);
                }
            } else {
                if (!warp_wait(&acc_full[b], (t / NB) & 1, &abort_flag, p.a.err, p.wait_ns))
                    goto done;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < kCols; c += kBoxCols) {
                    uint32_t w[kBoxCols];
                    float sw[kBoxCols];
                    tmem_ld16s(acc + c, w);
                    load_sw(p, o0 + c, sw);
                    if (lane == 0)
                        box_free();
                    tmem_wait(w);
                    if (c + kBoxCols == kCols) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            remote_arrive(map_rank(smem_u32(&acc_empty[b]), 0));
                    }
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < kBoxCols; g += 16) {
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 v = scaled(w[g + i], w[g + i + 1], sx, sw[g + i], sw[g + i + 1]);
                            if constexpr (sizeof(T) == 4) {
                                x[i] = __float_as_uint(v.x);
                                x[i + 1] = __float_as_uint(v.y);
                            } else {
                                x[i / 2] = pack2(v.x, v.y, T());
                            }
                        }
                        constexpr int n = sizeof(T);         // 16-byte chunks of 16 outputs
#pragma unroll
                        for (int i = 0; i < n; ++i)
                            st_shared_v4(smem_u32(box) + sw128_off(lane, g / 16 * n + i), x[4 * i], x[4 * i + 1],
                                         x[4 * i + 2], x[4 * i + 3]);
                    }
                    fence_async_smem();
                    __syncwarp();
                    // (rows past N and outputs past d_out are clipped by the map)
                    if (lane == 0 && row0 < p.a.N && o0 + c < p.a.d_out)
                        box_store(&p.map_y, box, o0 + c, row0);
                }
            }
        }
    }
done:
    __syncwarp();
    box_done();                                      // y is written, the boxes are read
    // nothing may land in shared memory or TMEM, or be read by the pair's MMAs, after
    // either CTA lets go of them
    if (warp == 0 && rank == 0)
        drain_fills(full_bar, kStages, issued, p.a.err, p.wait_ns);
    if (warp == 1 && rank == 0 && lane == 0) {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(&mma_drain))
                     : "memory");
        const unsigned long long t0 = now_ns();
        while (!mbar_try_wait(&mma_drain, 0)) {
            if (now_ns() - t0 > p.wait_ns) {
                atomicOr(p.a.err, (uint32_t)LORA_ERR_TIMEOUT);
                break;
            }
        }
    }
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ------------------------------------------------------------------ few tokens
// k_i8_few, decode batches: the weight is what has to be read, so it takes the rows of the
// MMA (M = 128 output channels) and the tokens its columns (N = 16 .. 256).  The reduction
// is split over the CTAs of a cluster, which puts every SM to work on one weight; each CTA
// leaves its 32-bit partial sums in its shared memory and finishes a share of the tokens by
// reading the other CTAs' (integers: the order of the sum does not matter).  Weights do not
// come from the kernel before (which quantises the tokens), so their lines are requested
// into L2 ahead of the wait for it -- a prefetch only: the loads follow the wait, for that
// kernel may have written this very weight.
//
// With adapters (LORA) the base does not wait for the shrink in front of it: what that kernel
// waited for is all the base reads, so the product runs beside it, and only the finish waits
// for V.  Complete when the shrink let this grid start means written to L2, no more: this SM's
// L1 may hold lines that an earlier launch read (the scales of the call before, at the same
// address), so whatever is read ahead of this grid's own wait -- scales, segments, the pool's
// tables, B -- is read from L2 (__ldcg, TMA).  In the finish the cluster's tokens are cut into
// groups of eight; a warp adds to 8 tokens x 32 outputs the delta of each adapter among them, by
// mma.sync in registers (the adapter's B rows and the tokens' V straight from L2; columns of
// other adapters' tokens are not taken over, so that an infinity in B stays with its own
// tokens).  The delta is a few MFLOP: a tcgen05 product would need B in shared memory and a
// TMEM round trip for it.
constexpr int kFewThreads = 192;         // producer, MMA issuer, 4 warps that empty the accumulator
constexpr int kFewLoraThreads = 256;     // and two more for the finish (two CTAs of 128 registers a thread fill an SM)

struct __align__(16) FewTok {            // a token's adapter
    int64_t boff;
    int32_t a;
    int32_t r;                           // rank; 0: no delta, -1: outside the segments
};
struct __align__(16) FewScales {         // of the tile's outputs and tokens
    float w[128], x[128];
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT> struct FewCfg {
    static constexpr int stage = kAtom + NT * 128;
    // two CTAs to an SM up to 128 tokens
    static constexpr int stages = NT <= 32 ? 5 : (NT <= 64 ? 4 : (NT <= 128 ? 3 : 4));
    static constexpr int smem = stages * stage + 1024;
    static_assert(NT * 512 <= stages * stage, "the partial sums take the ring's place");
};

struct FewTc {
    I8Args a;
    CUtensorMap map_q;       // tokens, boxes 128 bytes x NT rows
    CUtensorMap map_w;       // weight, boxes 128 bytes x 128 rows
    int32_t split;           // CTAs of a cluster
    unsigned long long wait_ns;
    int32_t test_stall;
};

__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ int4 ld_remote_v4(uint32_t addr)
{
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ int ld_remote(uint32_t addr)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// The adapter of each of the tile's tokens and the scales of its tokens and outputs, by the four
// warps that empty the accumulator.  (Read from L2 by every finishing warp, the scales cost 256
// tokens in 16 segments, 4096 -> 4096, 25.7 us for 24.3.)
__device__ void few_tokens(const I8Args &a, FewTok *tok, FewScales &sc, int n0, int nv, int o0, int t0)
{
    for (int t = t0; t < nv; t += 128) {
        tok[t] = {0, -1, -1};
        sc.x[t] = __ldcg(a.Sx + n0 + t);
    }
    sc.w[t0] = o0 + t0 < a.d_out ? __ldcg(a.Sw + o0 + t0) : 0.f;
    __syncwarp();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    for (int k = t0; k < a.n_seg; k += 128) {        // (bad offsets mark anything: nothing is written then)
        const int lo = max(__ldcg(a.seg_off + k), n0) - n0, hi = min(__ldcg(a.seg_off + k + 1), n0 + nv) - n0;
        for (int t = lo; t < hi; ++t)
            tok[t].a = k;
    }
    __syncwarp();
    asm volatile("bar.sync 1, 128;" ::: "memory");
    for (int t = t0; t < nv; t += 128)
        if (tok[t].a >= 0) {
            const int32_t ad = __ldcg(a.seg_ad + tok[t].a);
            int32_t r = 0;
            int64_t ao = 0, bo = 0;
            // (the shrink reports a bad one)
            if (ad == -1 || !pool_adapter_ok<true>(a.pool, ad, &r, &ao, &bo))
                tok[t] = {0, -1, 0};
            else
                tok[t] = {bo, ad, r};
        }
}

// B rows o .. o + 3 at ranks k .. k + 7 and k + 32 .. k + 39 (zeros behind the last).
__device__ __forceinline__ void few_load_b(const I8Args &p, const FewTok &ad, int o, int k, uint4 (&b)[2][4])
{
    const __nv_bfloat16 *b_row = p.pool.B + ad.boff + (int64_t)o * ad.r + k;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[h][i] = make_uint4(0, 0, 0, 0);
            if (o < p.d_out && k + 32 * h < ad.r)
                b[h][i] = __ldcg(reinterpret_cast<const uint4 *>(b_row + i * ad.r + 32 * h));
        }
}

// Finishes 8 tokens t .. of the tile x 32 outputs from `ob`: the base from the cluster's sums
// at `part`, and the deltas.  The MMA's rows and reduction are numbered so that a thread has
// four outputs in a row (o ..) of two tokens (t + 2q, t + 2q + 1) and loads eight ranks at
// once: rows g, g + 8 of the first product are outputs 4g, 4g + 1, of the second 4g + 2,
// 4g + 3, and columns 2q, 2q + 1, 2q + 8, 2q + 9 of a pair of steps are ranks 8q .. 8q + 7.
// All but V is fetched before the wait for the shrink.
__device__ __forceinline__ void few_finish(const I8Args &p, const FewTok *tok, const FewScales &sc, uint32_t part, int split,
                                           int n0, int t, int t_end, int ob, int lane)
{
    const int g = lane >> 2, q = lane & 3, o = ob + 4 * g;
    const bool o_ok = o < p.d_out;
    const bool tok_ok = lane < 8 && t + lane < t_end && tok[min(t + lane, t_end - 1)].r > 0;
    const int my_ad = tok[min(t + (lane & 7), t_end - 1)].a;
    uint32_t left = __ballot_sync(0xffffffffu, tok_ok);
    uint4 b[2][4];
    if (left)
        few_load_b(p, tok[t + __ffs(left) - 1], o, 8 * q, b);
    float y[4][2] = {};
    if (o_ok) {
        const float4 sw4 = *reinterpret_cast<const float4 *>(&sc.w[o & 127]);
        const float sw[4] = {sw4.x, sw4.y, sw4.z, sw4.w};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (t + 2 * q + j < t_end) {
                const float sx = sc.x[t + 2 * q + j];
                int4 v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < split)
                        v[c] = ld_remote_v4(map_rank(part + (t + 2 * q + j) * 512 + (o & 127) * 4, c));
                int4 a = v[0];
#pragma unroll
                for (int c = 1; c < 8; ++c)
                    if (c < split) {
                        a.x += v[c].x;
                        a.y += v[c].y;
                        a.z += v[c].z;
                        a.w += v[c].w;
                    }
                y[0][j] = (float)a.x * (sx * sw[0]);
                y[1][j] = (float)a.y * (sx * sw[1]);
                y[2][j] = (float)a.z * (sx * sw[2]);
                y[3][j] = (float)a.w * (sx * sw[3]);
            }
    }
    pdl_wait();
    const bool write = __ldcg(&p.hdr->n_groups) != 0;
    const __nv_bfloat16 *v_row = p.Vb + (int64_t)(n0 + min(t + g, t_end - 1)) * p.ldvb + 8 * q;
    bool have_b = true;
    while (left) {
        const FewTok ad = tok[t + __ffs(left) - 1];
        const uint32_t same = __ballot_sync(0xffffffffu, tok_ok && my_ad == ad.a);
        left &= ~same;
        float d0[4] = {}, d1[4] = {};
        for (int k = 0; k < ad.r; k += 64) {
            uint4 vh[2] = {}, vl[2] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (k + 32 * h + 8 * q < ad.r) {
                    vh[h] = __ldcg(reinterpret_cast<const uint4 *>(v_row + k + 32 * h));
                    vl[h] = __ldcg(reinterpret_cast<const uint4 *>(v_row + p.kv + k + 32 * h));
                }
            if (!have_b)
                few_load_b(p, ad, o, k + 8 * q, b);
            have_b = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mma_bf16(d0, b[h][0].x, b[h][1].x, b[h][0].y, b[h][1].y, vh[h].x, vh[h].y);
                mma_bf16(d1, b[h][2].x, b[h][3].x, b[h][2].y, b[h][3].y, vh[h].x, vh[h].y);
                mma_bf16(d0, b[h][0].z, b[h][1].z, b[h][0].w, b[h][1].w, vh[h].z, vh[h].w);
                mma_bf16(d1, b[h][2].z, b[h][3].z, b[h][2].w, b[h][3].w, vh[h].z, vh[h].w);
                mma_bf16(d0, b[h][0].x, b[h][1].x, b[h][0].y, b[h][1].y, vl[h].x, vl[h].y);
                mma_bf16(d1, b[h][2].x, b[h][3].x, b[h][2].y, b[h][3].y, vl[h].x, vl[h].y);
                mma_bf16(d0, b[h][0].z, b[h][1].z, b[h][0].w, b[h][1].w, vl[h].z, vl[h].w);
                mma_bf16(d1, b[h][2].z, b[h][3].z, b[h][2].w, b[h][3].w, vl[h].z, vl[h].w);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if ((same >> (2 * q + j)) & 1) {
                y[0][j] += d0[j];
                y[1][j] += d0[2 + j];
                y[2][j] += d1[j];
                y[3][j] += d1[2 + j];
            }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int tj = t + 2 * q + j;
        if (o_ok && write && tj < t_end && tok[tj].r >= 0)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.Y) + (int64_t)(n0 + tj) * p.ldy + o) =
                make_uint2(pack2(y[0][j], y[1][j], __nv_bfloat16()), pack2(y[2][j], y[3][j], __nv_bfloat16()));
    }
}

template <int NT, class T, bool LORA>
__global__ void __launch_bounds__(LORA ? kFewLoraThreads : kFewThreads) k_i8_few(const __grid_constant__ FewTc p)
{
    using C = FewCfg<NT>;
    static_assert(!LORA || NT <= 128, "FewScales");
    constexpr int kStages = C::stages, kCols = NT < 32 ? 32 : NT;
    extern __shared__ __align__(1024) unsigned char sm_dyn[];
    // (every CTA of the cluster has its ring at the same offset: the launch gives all one base)
    unsigned char *sm = sm_dyn + ((1024 - (smem_u32(sm_dyn) & 1023)) & 1023);
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], acc_full, mma_drain;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ FewTok tok[LORA ? NT : 1];
    __shared__ std::conditional_t<LORA, FewScales, int> sc;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = p.split, rank = (int)cluster_rank();
    const int o0 = (blockIdx.x / split) * 128, n0 = blockIdx.y * NT;
    const int nv = min(NT, p.a.N - n0);
    const int n_kb = (p.a.d_in + kKB - 1) / kKB;
    const int k0 = rank * n_kb / split, k1 = (rank + 1) * n_kb / split;
    int issued = 0;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&mma_drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int k = k0; k < k1; ++k)
            tma_prefetch(&p.map_w, k * kKB, o0);
    }
    if (warp == 1)
        tmem_alloc(&tmem_base, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if constexpr (!LORA)
        pdl_wait();
    pdl_trigger();

    if (warp == 0) {
        if (lane == 0 && !p.test_stall) {
            const uint64_t pol_x = policy_evict_last(), pol_w = policy_evict_first();
            if constexpr (LORA)                      // (written by a kernel that no wait here names)
                asm volatile("fence.proxy.async;" ::: "memory");
            for (int k = k0; k < k1; ++k, ++issued) {
                const int s = issued % kStages;
                if (!mbar_wait(&empty_bar[s], ((issued / kStages) & 1) ^ 1, &abort_flag, p.a.err, p.wait_ns))
                    break;
                mbar_arrive_expect_tx(&full_bar[s], C::stage);
                tma_load_2d_hint(sm + s * C::stage, &p.map_w, &full_bar[s], k * kKB, o0, pol_w);
                tma_load_2d_hint(sm + s * C::stage + kAtom, &p.map_q, &full_bar[s], k * kKB, n0, pol_x);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_i8(128, NT);
            const uint64_t a0 = sw128_desc(smem_u32(sm)), b0 = sw128_desc(smem_u32(sm) + kAtom);
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int k = k0; k < k1; ++k) {
                if (!(ok = mbar_wait(&full_bar[s], ph, &abort_flag, p.a.err, p.wait_ns)))
                    break;
                tc_fence_after();
                const uint64_t at = (uint64_t)(s * (C::stage >> 4));
#pragma unroll
                for (int i = 0; i < kKB / 32; ++i)
                    mma_i8(tmem, a0 + at + i * 2, b0 + at + i * 2, idesc, (k > k0 || i > 0) ? 1u : 0u);
                tc_commit(&empty_bar[s]);
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (ok)
                tc_commit(&acc_full);
        }
    } else if (warp < 6) {
        // partial sums to shared memory as [token][128 outputs], in the ring's place: every
        // fill has been multiplied when the accumulator is full
        if constexpr (LORA)
            few_tokens(p.a, tok, sc, n0, nv, o0, tid - 64);
        const int q = warp & 3;
        if (warp_wait(&acc_full, 0, &abort_flag, p.a.err, p.wait_ns)) {
            tc_fence_after();
            int *part = reinterpret_cast<int *>(sm) + q * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < nv; c += 16) {
                uint32_t w[16];
                tmem_ld16_raw(tmem + ((uint32_t)(q * 32) << 16) + c, w);
                tmem_wait(w);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    part[(c + i) * 128] = (int)w[i];
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    if (warp == 0 && lane == 0)
        drain_fills(full_bar, kStages, issued, p.a.err, p.wait_ns);
    if (warp == 1 && lane == 0)
        drain_mma(&mma_drain, 0, p.a.err, p.wait_ns);
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
    __syncwarp();
    cluster_sync();
    // a CTA that gave up has no sums to offer: then no output of the tile is written
    bool whole = true;
    for (int r = 0; r < split; ++r)
        whole &= ld_remote(map_rank(smem_u32(&abort_flag), r)) == 0;
    const int per = (nv + split - 1) / split;
    const int o = o0 + lane * 4;
    if constexpr (LORA) {
        const int t_end = min(nv, (rank + 1) * per);
        if (whole)
            for (int u = warp; rank * per + (u >> 2) * 8 < t_end; u += kFewLoraThreads / 32)
                if (o0 + (u & 3) * 32 < p.a.d_out)
                    few_finish(p.a, tok, sc, smem_u32(sm), split, n0, rank * per + (u >> 2) * 8, t_end, o0 + (u & 3) * 32,
                               lane);
        pdl_wait();                                  // (who had nothing to finish, too: this kernel's
                                                     // end stands for the shrink's)
    } else if (whole && o < p.a.d_out) {
        const uint32_t mine = smem_u32(sm) + lane * 16;
        float sw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sw[i] = p.a.Sw[o + i];
        for (int t = rank * per + warp; t < min(nv, (rank + 1) * per); t += kFewThreads / 32) {
            int4 v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < split)
                    v[r] = ld_remote_v4(map_rank(mine + t * 512, r));
            const float sx = p.a.Sx[n0 + t];
            int4 a = v[0];
#pragma unroll
            for (int r = 1; r < 8; ++r)
                if (r < split) {
                    a.x += v[r].x;
                    a.y += v[r].y;
                    a.z += v[r].z;
                    a.w += v[r].w;
                }
            const float y0 = (float)a.x * (sx * sw[0]), y1 = (float)a.y * (sx * sw[1]);
            const float y2 = (float)a.z * (sx * sw[2]), y3 = (float)a.w * (sx * sw[3]);
            T *y = static_cast<T *>(p.a.Y) + (int64_t)(n0 + t) * p.a.ldy + o;
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float4 *>(y) = make_float4(y0, y1, y2, y3);
            else
                *reinterpret_cast<uint2 *>(y) = make_uint2(pack2(y0, y1, T()), pack2(y2, y3, T()));
        }
    }
    __syncwarp();
    cluster_sync();                                  // (its sums are read: a CTA may go)
}

// y of dtype: boxes of `bytes` (64 or 128, swizzled alike) x 32 rows
bool encode_y(CUtensorMap *m, void *Y, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, int bytes)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const int es = dtype == LORA_F32 ? 4 : 2;
    const CUtensorMapDataType t = dtype == LORA_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : dtype == LORA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * es};
    const cuuint32_t box[2] = {(cuuint32_t)(bytes / es), 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, t, 2, Y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row-major 8-bit matrix [rows, cols] with leading dimension ld: boxes of 128 bytes x
// box_rows rows, 128-byte swizzle, zeros outside the matrix.
bool encode_box8(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C, class T> cudaError_t launch_pair(const I8Args &a, cudaStream_t s, bool *ok)
{
    PairTc p = {};
    p.a = a;
    *ok = encode_box8(&p.map_q, a.Q, a.N, a.d_in, a.ldq, 128) && encode_box8(&p.map_w, a.W, a.d_out, a.d_in, a.ldw, C::BN / 2) &&
          encode_y(&p.map_y, a.Y, a.dtype, a.N, a.d_out, a.ldy, C::box_bytes);
    p.sw_vec = ((uintptr_t)a.Sw & 15) == 0;
    if (*ok && C::LORA) {
        *ok = encode_box(&p.map_v, a.Vb, a.N, 2 * (int64_t)a.kv, a.ldvb, 128);
        p.b_tma = encode_b_views(p.map_b, a.pool.B, a.pool.B_elems, C::BN / 2);
    }
    if (!*ok)
        return cudaSuccess;
    p.wait_ns = wait_bound_ns();
    p.test_stall = test_stall_mode();
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if ((e = cudaFuncSetAttribute(k_i8_pair<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem)) != cudaSuccess)
            return e;
        if (dev >= 0 && dev < 64)
            attr_set[dev] = true;
    }
    const int64_t units = ((int64_t)a.N + 255) / 256 * ((a.d_out + C::BN - 1) / C::BN);
    int clusters = sm_count() / 2;
    if (units < clusters)
        clusters = (int)units;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters);
    cfg.blockDim = dim3(C::threads);
    cfg.dynamicSmemBytes = C::smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_i8_pair<C, T>, p);
}

template <int NT, class T, bool LORA> cudaError_t launch_few(const I8Args &a, int split, cudaStream_t s, bool *ok)
{
    using C = FewCfg<NT>;
    FewTc p = {};
    p.a = a;
    p.split = split;
    *ok = encode_box8(&p.map_q, a.Q, a.N, a.d_in, a.ldq, NT) && encode_box8(&p.map_w, a.W, a.d_out, a.d_in, a.ldw, 128);
    if (!*ok)
        return cudaSuccess;
    p.wait_ns = wait_bound_ns();
    p.test_stall = test_stall_mode();
    static bool attr_set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        if ((e = cudaFuncSetAttribute(k_i8_few<NT, T, LORA>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem)) != cudaSuccess)
            return e;
        if (dev >= 0 && dev < 64)
            attr_set[dev] = true;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.d_out + 127) / 128 * split, (a.N + NT - 1) / NT);
    cfg.blockDim = dim3(LORA ? kFewLoraThreads : kFewThreads);
    cfg.dynamicSmemBytes = C::smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_i8_few<NT, T, LORA>, p);
}

// Microseconds of a call without adapters, by a model fitted to B200 timings over N = 1 ..
// 2048 and weights of 4096 x 1024 to 4096 x 14336 and 14336 x 4096, weights from HBM:
// * CTA pairs: 6 and 0.29 per k-block of every round of tiles over the 74 pairs of SMs;
// * few tokens: the ring's traffic at 85 bytes a nanosecond and SM, and 5.5 to 8 for launch,
//   first loads, the exchange of partial sums and the last stores.
// Measured on both sides (us, pairs / few): 1 x 4096 -> 4096 15.5 / 6.4; 256 x 4096 -> 4096
// 16.3 / 12.4; 256 x 4096 -> 14336 18.5 / 28; 512 x 4096 -> 4096 16.7 / 16.1; 1024 x 4096 ->
// 1024 16.0 / 11.9; 1024 x 4096 -> 4096 17.5 / 26.
double pair_us(const I8Args &a, int n_kb)
{
    const int64_t tiles = ((int64_t)a.N + 255) / 256 * ((a.d_out + 255) / 256);
    return 6.0 + (double)((tiles + 73) / 74) * n_kb * 0.29;
}

double few_us(const I8Args &a, int n_kb, int nt, int split)
{
    const int64_t ctas = (int64_t)((a.d_out + 127) / 128) * (((int64_t)a.N + nt - 1) / nt) * split;
    const int64_t slots = nt <= 128 ? 296 : 148;
    double load = (double)ctas / 148;                // CTAs an SM works through
    if (load < 1)
        load = 1;
    if (ctas > slots)
        load = (double)((ctas + slots - 1) / slots * slots) / 148;
    const int kb = (n_kb + split - 1) / split;
    return (nt <= 64 ? 5.5 : (nt <= 128 ? 6.5 : 8.1)) + load * kb * (16384 + nt * 128) / 85e3;
}

// The same with adapters, the shrink in front included (about 6 and d_in / 1500).
// * CTA pairs start behind it, and every tile adds its epilogue and each run of rows with one
//   adapter: 1.5 a run, 2.5 with ranks over 64, less from the seventh on; two thirds of it in
//   tiles of 128 outputs.
// * Few tokens multiply beside it where the CTAs of both find room, then finish in rounds of
//   eight warps: 1.1 a round, and 0.9 (ranks over 64: 1.1) for each adapter among eight tokens.
// Measured (us, pairs / few): 16 tokens in 4 segments, 4096 -> 4096 29 / 13.3, 14336 -> 4096
// 62 / 20.3; 256 in 16, 4096 -> 4096 38 / 24.5; 1024 in 16, 4096 -> 1024 34.4 / 23.6; 560 in
// 10, 8496 -> 6632 79 / 103; 1706 in 24, 3336 -> 3560 74 / 110.  Over 112 random shapes of 16
// to 2900 tokens the choice takes 2 % longer than the best of the forms that best_few() admits
// (tiles narrower than the tokens, which it does not, were not timed).
double shrink_us(const I8Args &a)
{
    return 6 + a.d_in / 1500.0;
}

bool narrow_pairs(const I8Args &a)
{
    return ((int64_t)a.N + 255) / 256 * ((a.d_out + 127) / 128) <= sm_count() / 2;
}

double pair_lora_us(const I8Args &a, int n_kb)
{
    double runs = 1 + 256.0 * a.n_seg / a.N;
    if (runs > a.n_seg)
        runs = a.n_seg;
    const double first = a.pool.max_rank <= 64 ? 1.5 : 2.5, more = a.pool.max_rank <= 64 ? 0.6 : 1.0;
    const double tile = 3 + (runs < 6 ? runs * first : 6 * first + (runs - 6) * more);
    const int64_t tiles = ((int64_t)a.N + 255) / 256 * ((a.d_out + 255) / 256);
    return shrink_us(a) + 2.5 + pair_us(a, n_kb) + (narrow_pairs(a) ? 0.65 * tile : (double)((tiles + 73) / 74) * tile);
}

double few_lora_us(const I8Args &a, int n_kb, int nt, int split)
{
    const int64_t ctas = (int64_t)((a.d_out + 127) / 128) * (((int64_t)a.N + nt - 1) / nt) * split;
    const int tokens = nt < a.N ? nt : a.N, groups = ((tokens + split - 1) / split + 7) / 8;
    const double runs = 1 + 8.0 * a.n_seg / a.N;
    const double finish = 2 + (groups * 4 + 7) / 8 * (1.1 + (a.pool.max_rank <= 64 ? 0.9 : 1.1) * (runs < 8 ? runs : 8));
    const double base = few_us(a, n_kb, nt, split), shrink = shrink_us(a);
    // (the shrink splits a tile over up to 8 CTAs of 8 of its k-blocks)
    const int64_t before = ((int64_t)a.N / 128 + a.n_seg) * (n_kb < 8 ? 1 : (n_kb < 32 ? n_kb / 4 : 8));
    const double beside = 3 + (base > shrink ? base + 0.25 * shrink : shrink + 0.25 * base) + finish;
    const double behind = 4.5 + 0.75 * shrink + base + (double)((ctas + 239) / 240) * finish;
    const double crowd = ctas > 240 ? 1 : (double)(ctas + before - 296) / 148;
    return crowd <= 0 ? beside : (crowd >= 1 ? behind : beside + crowd * (behind - beside));
}

// The few-token form that a model expects to be fastest, and its time.
struct FewChoice {
    int nt, split;
    double us;
};

FewChoice best_few(const I8Args &a, int n_kb, int max_nt, double (*model)(const I8Args &, int, int, int))
{
    FewChoice best = {0, 1, 1e30};
    for (int nt : {16, 32, 64, 128, 256}) {
        // (narrow tiles would read a large weight again and again -- over a small one, which they
        // would spread over more SMs, they are not measured; the model ends at some thousand tokens)
        if ((nt < 128 && nt < a.N) || nt > max_nt || a.N > 8192)
            continue;
        for (int split = 1; split <= 8 && (split == 1 || 2 * split <= n_kb); split *= 2) {
            const double us = model(a, n_kb, nt, split);
            if (us < best.us)
                best = {nt, split, us};
        }
        if (nt >= a.N)
            break;
    }
    return best;
}

template <class T, bool LORA> cudaError_t launch_few_nt(const I8Args &a, const FewChoice &c, cudaStream_t s, bool *ok)
{
    switch (c.nt) {
    case 16:
        return launch_few<16, T, LORA>(a, c.split, s, ok);
    case 32:
        return launch_few<32, T, LORA>(a, c.split, s, ok);
    case 64:
        return launch_few<64, T, LORA>(a, c.split, s, ok);
    case 256:
        if constexpr (!LORA)
            return launch_few<256, T, false>(a, c.split, s, ok);
    default:
        return launch_few<128, T, LORA>(a, c.split, s, ok);
    }
}

template <class T> cudaError_t launch_any(const I8Args &a, cudaStream_t s, bool *ok)
{
    const int n_kb = (a.d_in + kKB - 1) / kKB;
    const FewChoice few = best_few(a, n_kb, 256, few_us);
    return few.us < pair_us(a, n_kb) ? launch_few_nt<T, false>(a, few, s, ok)
                                     : launch_pair<PairCfg<false, 256>, T>(a, s, ok);
}

}  // namespace

cudaError_t launch_linear_i8(const I8Args &a, cudaStream_t s, bool *ok)
{
    if (a.seg_off) {
        const int n_kb = (a.d_in + kKB - 1) / kKB;
        // (256 tokens a CTA were never faster than 128: twice the finishing of one CTA)
        const FewChoice few = best_few(a, n_kb, 128, few_lora_us);
        if (few.us < pair_lora_us(a, n_kb))
            return launch_few_nt<__nv_bfloat16, true>(a, few, s, ok);
        // Tiles of 128 outputs where they still find a free pair of SMs each: the gathers and
        // the emptying of a tile halve (1535 tokens in 23 segments, 4096 -> 1024: 52 against 57 us
        // for the whole call), its loads do not.
        if (narrow_pairs(a))
            return launch_pair<PairCfg<true, 128>, __nv_bfloat16>(a, s, ok);
        return launch_pair<PairCfg<true, 256>, __nv_bfloat16>(a, s, ok);
    }
    return a.dtype == LORA_BF16 ? launch_any<__nv_bfloat16>(a, s, ok)
         : a.dtype == LORA_F16 ? launch_any<__half>(a, s, ok)
                               : launch_any<float>(a, s, ok);
}

}  // namespace lora
